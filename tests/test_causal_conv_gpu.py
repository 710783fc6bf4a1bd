"""The short causal convolution against the 64-bit oracle.

Tolerances, in units of 2^-24 of A (the sum of the absolute values of a
result's terms, the oracle's magnitude run): W products and sums, and 8 for the
activation; a gradient has twice that on its way, and the weights' sums one a
token: 4 W + 32 + B T.  A bf16 result is rounded once more, 2^-8 of its value.
"""
import numpy as np
import pytest
import torch

import element_scan_recurrences_gb300 as es
import oracle.state_space as S
from element_scan_recurrences_gb300 import autograd as ag

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
NAMES = ("gx", "gw", "gb", "ginitial")


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    es.lib()


def num(t):
    return None if t is None else t.double().cpu().numpy()


class Case:
    def __init__(self, dtype, B, T, C, W=4, wtype=None, bias=True, carry=True, lengths=None, act=True, seed=0):
        rng = np.random.default_rng(seed)
        n = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
        self.B, self.T, self.C, self.W, self.act = B, T, C, W, act
        wtype = wtype or dtype
        self.x, self.w, self.b = n(B, T, C).to(dtype), n(C, W).to(wtype), n(C).to(wtype) if bias else None
        self.init, self.gfin = (n(B, W - 1, C).to(dtype), n(B, W - 1, C).to(dtype)) if carry else (None, None)
        self.go = n(B, T, C).to(dtype)
        self.lengths = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")

    def kw(self):
        return dict(initial_state=self.init, lengths=self.lengths, activation=self.act)

    def okw(self):
        return dict(init=num(self.init), lengths=num(self.lengths), act=self.act)


def close(got, want, size, n, what):
    rounded = 2.0 ** -8 if got.dtype == BF16 else 0.0
    got = num(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    tol = rounded * np.abs(want) + 2.0 ** -24 * n * size + 1e-30
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of the tolerance, first at %s" % (
        what, bad.sum(), bad.size, float(np.nanmax(np.abs(got - want) / tol)), np.argwhere(bad)[0])


def check_forward(c, got=None):
    out, last = got or es.causal_conv(c.x, c.w, c.b, final_state=True, **c.kw())
    es.device_status()
    want, size = (S.causal_conv(num(c.x), num(c.w), num(c.b), **c.okw(), magnitude=m) for m in (False, True))
    close(out, want[0], size[0], 2 * c.W + 16, "out")
    assert np.array_equal(num(last), want[1])


def check_backward(c, got=None):
    got = got or es.causal_conv_backward(c.x, c.w, c.b, c.go, grad_final_state=c.gfin, **c.kw())
    es.device_status()
    args = (num(c.x), num(c.w), num(c.b), num(c.go))
    want, size = (S.causal_conv_backward(*args, gfin=num(c.gfin), **c.okw(), magnitude=m) for m in (False, True))
    for name, g, w, s, has in zip(NAMES, got, want, size, (True, True, c.b is not None, c.init is not None)):
        assert (g is not None) == has
        if has:
            close(g, w, s, 4 * c.W + 32 + c.B * c.T, name)


SHAPES = [(2, 37, 40, 4), (1, 1, 128, 4), (3, 2, 24, 4), (2, 70, 33, 3), (1, 33, 1030, 2), (2, 5, 16, 8), (1, 140, 8, 5), (2, 65, 24, 6),
          (1, 64, 7, 7)]


@pytest.mark.parametrize("dtype,wtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("shape", SHAPES)
def test_both_ways(dtype, wtype, shape):
    c = Case(dtype, *shape, wtype=wtype)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("bias,carry,act", [(False, False, False), (True, False, True), (False, True, True), (True, True, False)])
def test_options(bias, carry, act):
    c = Case(F32, 2, 70, 24, 4, None, bias, carry, [70, 33], act, seed=1)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("W", [2, 4, 8])
def test_lengths(dtype, W):
    """Rows without tokens, shorter than the taps, at the edges of runs; what lies past them is never read."""
    n = [0, 1, 2, 31, 64, 65, 129]
    c = Case(dtype, 7, 130, 16, W, lengths=n[:6] + [500], seed=2)
    n[6] = 130
    for t in (c.x, c.go):
        for b, m in enumerate(n):
            t[b, m:] = float("nan")
    got = es.causal_conv(c.x, c.w, c.b, final_state=True, **c.kw())
    grads = es.causal_conv_backward(c.x, c.w, c.b, c.go, grad_final_state=c.gfin, **c.kw())
    for t in (got[0], grads[0]):
        for b, m in enumerate(n):
            assert not t[b, m:].any()
    c.x.nan_to_num_(0.0)
    c.go.nan_to_num_(0.0)
    check_forward(c, got)
    check_backward(c, grads)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,C,W", [(1, 128, 4), (5, 40, 4), (3, 33, 2), (2, 8, 8)])
def test_step(dtype, B, C, W):
    c = Case(dtype, B, 1, C, W, seed=3)
    state = c.init.clone()
    out, new = es.causal_conv_step(c.x[:, 0], c.w, c.b, state)
    assert new is state
    check_forward(c, (out[:, None], state))
    other = torch.empty_like(state)
    out2, _ = es.causal_conv_step(c.x[:, 0], c.w, c.b, c.init, state_out=other)
    assert torch.equal(out, out2) and torch.equal(other, state)


def test_in_place_state_and_prompt_in_pieces():
    c = Case(BF16, 2, 150, 64, seed=4)
    whole, last = es.causal_conv(c.x, c.w, c.b, final_state=True, **c.kw())
    state, outs = c.init.clone(), []
    for a, b in ((0, 1), (1, 3), (3, 100), (100, 150)):
        o, s = es.causal_conv(c.x[:, a:b], c.w, c.b, initial_state=state, final_state=state)
        assert s is state
        outs.append(o)
    assert torch.equal(torch.cat(outs, 1), whole) and torch.equal(state, last)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_views(dtype):
    c = Case(dtype, 2, 70, 40, seed=5)
    want = es.causal_conv(c.x, c.w, c.b, final_state=True, **c.kw())
    gwant = es.causal_conv_backward(c.x, c.w, c.b, c.go, grad_final_state=c.gfin, **c.kw())

    def odd(t):
        box = torch.zeros(*t.shape[:-1], 2 * t.shape[-1] + 1, dtype=t.dtype, device="cuda")
        v = box[..., 1:1 + t.shape[-1]]
        v.copy_(t)
        return v

    def turned(t):
        return t.transpose(0, 1).contiguous().transpose(0, 1)

    for view in (odd, turned):
        got = es.causal_conv(view(c.x), c.w, c.b, final_state=True, out=view(torch.zeros_like(c.x)), **c.kw())
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        for x, y in zip(es.causal_conv_backward(view(c.x), c.w, c.b, view(c.go), grad_final_state=c.gfin, **c.kw()), gwant):
            assert torch.equal(x, y)


def test_empty():
    for B, T, C in ((0, 5, 8), (2, 0, 8), (2, 5, 0)):
        c = Case(F32, B, T, C, seed=6)
        out, last = es.causal_conv(c.x, c.w, c.b, final_state=True, **c.kw())
        assert out.shape == (B, T, C)
        if T == 0:
            assert torch.equal(last, c.init)
        gx, gw, gb, gi = es.causal_conv_backward(c.x, c.w, c.b, c.go, grad_final_state=c.gfin, **c.kw())
        if B * T == 0:
            assert not gw.any() and not gb.any()
        if T == 0:
            assert torch.equal(gi, c.gfin)


def test_autograd():
    c = Case(F32, 2, 70, 24, seed=7, lengths=[70, 2])
    leaves = [t.clone().requires_grad_(True) for t in (c.x, c.w, c.b, c.init)]
    out, last = ag.causal_conv(*leaves, lengths=c.lengths, final_state=True)
    torch.autograd.backward([out, last], [c.go, c.gfin])
    check_backward(c, [t.grad for t in leaves])


def test_captured():
    c, other = Case(BF16, 2, 100, 64, seed=8), Case(BF16, 2, 100, 64, seed=9)
    run = lambda: (es.causal_conv(c.x, c.w, c.b, final_state=True, **c.kw()) +  # noqa: E731
                   es.causal_conv_backward(c.x, c.w, c.b, c.go, grad_final_state=c.gfin, **c.kw()))
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for n in ("x", "w", "b", "init", "go", "gfin"):
        getattr(c, n).copy_(getattr(other, n))
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(got, run()):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_values_of_any_size(dtype):
    """Weights 0 and 1: s(x) for inputs up to the largest finite values, and its slope.  Some
    16 roundings and one to the result's type, 2^-20 and 2^-8 of it; a subnormal factor
    may be 0, under 2^-119 at |x| < 89."""
    rel, tiny = 2.0 ** -8 + 2.0 ** -20 if dtype == BF16 else 2.0 ** -20, 2.0 ** -119
    big = torch.finfo(dtype).max
    z = torch.tensor([-big, -1e30, -200.0, -89.0, -88.0, -87.0, -1.0, 0.0, 1.0, 88.0, 105.0, 200.0, 1e30, big], device="cuda").to(dtype)
    n = z.numel()
    x = z.view(1, 1, n).clone().requires_grad_()
    w = torch.tensor([0.0, 1.0], device="cuda").to(dtype).expand(n, 2).contiguous()
    out = ag.causal_conv(x, w)[0]
    out.backward(torch.ones_like(out))
    step = es.causal_conv_step(z.view(1, n), w, None, torch.zeros(1, 1, n, dtype=dtype, device="cuda"))[0]
    want, slope = S.silu(num(z)), S.slope(num(z))
    for got in (out.detach(), step):
        assert (np.abs(num(got).ravel() - want) <= rel * np.abs(want) + tiny).all(), got
    assert (np.abs(num(x.grad).ravel() - slope) <= rel * 2.0 + tiny).all(), x.grad


def test_refusals():
    c = Case(F32, 2, 10, 16, seed=10)

    def refused(kind, f):
        with pytest.raises(kind):
            f()

    refused(TypeError, lambda: es.causal_conv(c.x.half(), c.w, c.b))
    refused(TypeError, lambda: es.causal_conv(c.x, c.w.half(), c.b))
    refused(TypeError, lambda: es.causal_conv(c.x, c.w, c.b.bfloat16()))
    refused(es.EsError, lambda: es.causal_conv(c.x, c.w[:8], c.b))
    refused(es.EsError, lambda: es.causal_conv(c.x, c.w[:, :1].contiguous(), c.b))
    refused(es.EsError, lambda: es.causal_conv(c.x, torch.zeros(16, 9, device="cuda"), c.b))
    refused(es.EsError, lambda: es.causal_conv(c.x, torch.zeros(16, 0, device="cuda"), c.b))
    refused(es.EsError, lambda: es.causal_conv(c.x, c.w, c.b, out=c.x))
    refused(es.EsError, lambda: es.causal_conv(c.x[0], c.w, c.b))
    refused(es.EsError, lambda: es.causal_conv(c.x, c.w, c.b, initial_state=c.init[:, :2].contiguous()))
    refused(TypeError, lambda: es.causal_conv(c.x, c.w, c.b, initial_state=c.init.bfloat16()))
    refused(TypeError, lambda: es.causal_conv_step(c.x[:, 0], c.w, c.b, None))
    assert torch.equal(es.causal_conv(c.x, c.w, c.b)[0], es.causal_conv(c.x, c.w, c.b)[0])
