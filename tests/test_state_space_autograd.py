"""What the differentiable selective scan keeps between its forward and its backward
call, without a GPU: the library's calls are stood in for by functions that record
their arguments and give tensors of the right shapes."""
import gc
import weakref

import pytest
import torch

from element_scan_recurrences_gb300 import autograd as ag
from element_scan_recurrences_gb300 import sequence

B, T, C, N = 2, 5, 4, 3


@pytest.fixture
def calls(monkeypatch):
    seen = []

    def forward(x, *_, checkpoints, **__):
        kept = torch.zeros(64, dtype=torch.uint8) if checkpoints else None
        seen.append(("forward", bool(checkpoints)))
        return x.detach().clone(), None, kept

    def backward(*args, checkpoints, **__):
        seen.append(("backward", checkpoints is not None))
        return tuple(None if t is None else torch.zeros_like(t) for t in args[:8]) + (None,)

    monkeypatch.setattr(sequence, "selective_scan", forward)
    monkeypatch.setattr(sequence, "selective_scan_backward", backward)
    return seen


def operands(leaf=True):
    x, delta = torch.zeros(B, T, C), torch.zeros(B, T, C)
    return x, delta, torch.zeros(C, N).requires_grad_(leaf), torch.zeros(B, T, 1, N), torch.zeros(B, T, 1, N)


def test_a_pass_that_will_have_a_backward_keeps_checkpoints(calls):
    ag.selective_scan(*operands())[0].sum().backward()
    assert calls == [("forward", True), ("backward", True)]


def test_no_checkpoints_where_none_are_wanted(calls):
    ag.selective_scan(*operands(), checkpoints=False)[0].sum().backward()
    assert calls == [("forward", False), ("backward", False)]


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_no_checkpoints_in_inference(calls, mode):
    """A trained layer's prompt: the parameters require a gradient, the call does not."""
    args = operands()
    with mode():
        ag.selective_scan(*args)
    ag.selective_scan(*operands(leaf=False))
    assert [c[1] for c in calls] == [False, False]


def test_checkpoints_are_saved_tensors(calls):
    """They pass by the hooks for saved tensors, as the operands do."""
    packed = []

    def pack(t):
        packed.append(t.dtype)
        return t

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        out, _ = ag.selective_scan(*operands())
    assert torch.uint8 in packed
    out.sum().backward()
    assert calls[-1] == ("backward", True)


def test_checkpoints_go_with_the_backward(calls):
    """They are let go of once the backward has run, however long its result lives."""
    class Held:
        def __init__(self, t):
            self.t = t

    held = []

    def pack(t):
        h = Held(t)
        if t.dtype == torch.uint8:
            held.append(weakref.ref(h))
        return h

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda h: h.t):
        out, _ = ag.selective_scan(*operands())
    assert len(held) == 1 and held[0]() is not None
    out.sum().backward()
    gc.collect()
    assert held[0]() is None
    with pytest.raises(RuntimeError):
        out.sum().backward()
