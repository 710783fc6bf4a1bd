"""The selective scan's gradients without channels: those of B and C are sums over no
channel at all, zeros wherever their elements lie."""
import pytest
import torch

import element_scan_recurrences_gb300 as es
from element_scan_recurrences_gb300 import binding, sequence

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    es.lib()


def dirty(elements, dtype):
    """Leaves memory of this size with NaNs in it to the allocator."""
    held = [torch.full((elements,), float("nan"), dtype=dtype, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    del held


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("groups,lengths", [(1, None), (3, [5, 0])])
def test_gradients_are_zeros(dtype, groups, lengths):
    B, T, N = 2, 5, 16
    rows, bc = torch.zeros(B, T, 0, dtype=dtype, device="cuda"), torch.ones(B, T, groups, N, dtype=dtype, device="cuda")
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    dirty(bc.numel(), dtype)
    g = es.selective_scan_backward(rows, rows, torch.zeros(0, N, device="cuda"), bc, bc, None, rows, None, rows, lengths=n)
    assert g[3].shape == g[4].shape == bc.shape
    assert torch.equal(g[3], torch.zeros_like(bc)) and torch.equal(g[4], torch.zeros_like(bc))
    assert g[0].numel() == g[1].numel() == g[2].numel() == g[6].numel() == 0
    leaves = [t.clone().requires_grad_(True) for t in (bc, bc)]
    dirty(bc.numel(), dtype)
    from element_scan_recurrences_gb300 import autograd as ag
    out, _ = ag.selective_scan(rows, rows, torch.zeros(0, N, device="cuda"), *leaves, lengths=n)
    out.backward(rows)
    for t in leaves:
        assert torch.equal(t.grad, torch.zeros_like(bc))


def test_strided_gradients_and_what_lies_between_them():
    B, T, G, N = 2, 5, 3, 6
    box = [torch.full((B, T, G, 2 * N), 7.0, device="cuda") for _ in range(2)]
    gb, gc = (t[..., :N] for t in box)
    at = lambda t: (t.data_ptr(), t.stride(0), t.stride(1), t.stride(2), G)  # noqa: E731
    bc = torch.ones(B, T, G, N, device="cuda")
    args = sequence._SCAN.pack(0, B, T, 0, N, G, 1, *(0,) * 12, *at(bc), *at(bc), *(0,) * 10)
    grads = sequence._SCAN_GRADS.pack(*(0,) * 12, *at(gb), *at(gc), *(0,) * 5)
    binding._check(es.lib().es_selective_scan_backward(args, grads, torch.cuda.current_stream().cuda_stream))
    for t in box:
        assert not t[..., :N].any() and bool((t[..., N:] == 7.0).all())
