"""The group norm with a gate against the 64-bit oracle.

Tolerances, in units of 2^-24.  The mean is a sum of D terms in a tree of threads
(at most 16 in a row in one, 9 levels) and costs 32 of the largest value m; the
deviations from it are off by that, the square root and the reciprocal 4, the
weights 4, a gate 16: |error| <= 2^-24 (48 |n| + 32 m r) |w s| and the like, r
the reciprocal of the deviation.  Taken together here as 128 units of (1 + m r)
times the largest result of the row, twice that for a gradient, whose two sums
run over the same D terms; the weights' sums take B T more.  bf16 results are
rounded once more, 2^-8 of their value.
"""
import numpy as np
import pytest
import torch

import element_scan_recurrences_gb300 as es
import oracle.state_space as S
from element_scan_recurrences_gb300 import autograd as ag

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    es.lib()


def num(t):
    return None if t is None else t.double().cpu().numpy()


class Case:
    def __init__(self, dtype, B, T, H, D, wtype=None, weight=True, bias=True, gate=True, first=False, center=True, act=False, seed=0,
                 offset=0.5):
        rng = np.random.default_rng(seed)
        n = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
        wtype = wtype or dtype
        self.x = (n(B, T, H, D) + offset).to(dtype)
        self.w, self.b = (1 + 0.2 * n(H, D)).to(wtype) if weight else None, (0.3 * n(H, D)).to(wtype) if bias else None
        self.gate, self.go = n(B, T, H, D).to(dtype) if gate else None, n(B, T, H, D).to(dtype)
        self.kw = dict(gate_first=first, center=center, activation=act)
        self.okw = dict(first=first, center=center, act=act)

    def args(self):
        return self.x, self.w, self.b, self.gate


def close(got, want, size, what):
    rounded = 2.0 ** -8 if got.dtype == BF16 else 0.0
    got = num(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    tol = rounded * np.abs(want) + 2.0 ** -24 * size + 1e-30
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of the tolerance, first at %s" % (
        what, bad.sum(), bad.size, float(np.nanmax(np.abs(got - want) / tol)), np.argwhere(bad)[0])


def spread(c):
    """1 + m r of each row."""
    u = num(c.x) * S.silu(num(c.gate)) if c.kw["gate_first"] else num(c.x)
    v = u - u.mean(-1, keepdims=True) if c.kw["center"] else u
    return 1 + np.abs(u).max(-1, keepdims=True) / np.sqrt((v * v).mean(-1, keepdims=True) + 1e-5)


def top(x):
    return np.abs(x).max(-1, keepdims=True)


def check(c, out=None, grads=None):
    out = es.group_norm(*c.args(), **c.kw) if out is None else out
    grads = es.group_norm_backward(*c.args(), c.go, **c.kw) if grads is None else grads
    es.device_status()
    args = tuple(num(t) for t in c.args())
    want = S.group_norm(*args, **c.okw)
    r = spread(c)
    close(out, want, 128 * r * top(want), "out")
    gx, gw, gb, gg = S.group_norm_backward(*args, num(c.go), **c.okw)
    rows = c.x.shape[0] * c.x.shape[1]
    # the gradient of a row is what is left of its terms' two projections: their size is that of the gradient of n by r
    gy = np.abs(num(c.go)) * (1 if c.gate is None else 1 + np.abs(args[3])) * (1 if c.b is None else 1 + np.abs(args[2]))
    wide = 1 if c.w is None else np.abs(args[1]).max()
    u = args[0] * S.silu(args[3]) if c.kw["gate_first"] else args[0]
    v = u - u.mean(-1, keepdims=True) if c.kw["center"] else u
    inv = 1 / np.sqrt((v * v).mean(-1, keepdims=True) + 1e-5)
    n = np.abs(v) * inv
    close(grads[0], gx, 256 * r * inv * wide * top(gy * (1 + n)) * (top(args[3]) + 1 if c.kw["gate_first"] else 1), "gx")
    if c.w is not None:
        close(grads[1], gw, (rows + 256) * (gy * (r + n)).sum((0, 1)), "gw")
    if c.b is not None:
        close(grads[2], gb, (rows + 256) * (gy * r).sum((0, 1)), "gb")
    if c.gate is not None:
        size = top(gy) * (1 + top(n) * wide) * (1 + top(args[3])) * (inv * (1 + top(args[0])) * wide if c.kw["gate_first"] else 1)
        close(grads[3], gg, 256 * r * size, "ggate")
    assert [g is None for g in grads] == [False, c.w is None, c.b is None, c.gate is None]


SHAPES = [(2, 5, 3, 64), (1, 1, 16, 128), (1, 300, 16, 128), (2, 7, 2, 80), (1, 9, 1, 2560), (1, 3, 1, 8192), (2, 3, 40, 32), (1, 4, 3, 7), (1, 6, 2, 1000),
          (1, 3, 2, 129), (1, 2, 1, 2050), (1, 3, 1, 1), (2, 4, 1, 512), (1, 5, 300, 16), (1, 2, 1, 4100), (3, 3, 5, 255)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("first", [False, True])
def test_shapes(dtype, shape, first):
    check(Case(dtype, *shape, first=first, center=not first, bias=not first))


@pytest.mark.parametrize("kw", [dict(), dict(first=True), dict(center=False), dict(gate=False), dict(gate=False, act=True),
                                dict(gate=False, act=True, center=False), dict(weight=False), dict(bias=False),
                                dict(weight=False, bias=False, gate=False), dict(wtype=F32), dict(first=True, weight=False)])
def test_options(kw):
    check(Case(BF16, 2, 20, 4, 96, seed=1, **kw))
    check(Case(F32, 2, 20, 4, 96, seed=1, **{**kw, "wtype": BF16 if "wtype" in kw else None}))


def test_far_from_zero():
    """A mean far above the deviation: the variance is of the distances from it."""
    check(Case(F32, 2, 10, 2, 128, offset=1000.0, seed=2))


def test_constant_rows():
    """No deviation at all: n is 0, and the result the bias."""
    c = Case(F32, 1, 4, 2, 64, gate=False)
    c.x.fill_(3.0)
    assert torch.equal(es.group_norm(*c.args()), c.b.expand(1, 4, 2, 64))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_views(dtype):
    c = Case(dtype, 2, 30, 4, 64, seed=3)
    want, gwant = es.group_norm(*c.args()), es.group_norm_backward(*c.args(), c.go)

    def odd(t):
        box = torch.zeros(*t.shape[:-1], 2 * t.shape[-1] + 1, dtype=t.dtype, device="cuda")
        v = box[..., 1:1 + t.shape[-1]]
        v.copy_(t)
        return v

    def turned(t):
        return t.transpose(0, 2).contiguous().transpose(0, 2)

    got = es.group_norm(turned(c.x), c.w, c.b, turned(c.gate), out=turned(torch.zeros_like(c.x)))
    assert torch.equal(got, want)
    for x, y in zip(es.group_norm_backward(turned(c.x), c.w, c.b, turned(c.gate), turned(c.go)), gwant):
        assert torch.equal(x, y)
    # other widths of access sum in another order
    c.x, c.gate, c.go = odd(c.x), odd(c.gate), odd(c.go)
    check(c)


def test_repeats_and_captured():
    c, other = Case(BF16, 4, 200, 8, 128, seed=4), Case(BF16, 4, 200, 8, 128, seed=5)
    run = lambda: (es.group_norm(*c.args()),) + es.group_norm_backward(*c.args(), c.go)  # noqa: E731
    for x, y in zip(run(), run()):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for n in ("x", "w", "b", "gate", "go"):
        getattr(c, n).copy_(getattr(other, n))
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(got, run()):
        assert torch.equal(x, y)


def test_empty():
    for shape in ((0, 5, 2, 8), (2, 0, 2, 8), (2, 5, 0, 8)):
        c = Case(F32, *shape)
        assert es.group_norm(*c.args()).shape == shape
        _, gw, gb, _ = es.group_norm_backward(*c.args(), c.go)
        assert not gw.any() and not gb.any()


def test_autograd():
    c = Case(F32, 2, 20, 4, 64, seed=6)
    leaves = [t.clone().requires_grad_(True) for t in c.args()]
    out = ag.group_norm(*leaves)
    out.backward(c.go)
    check(c, out.detach(), [t.grad for t in leaves])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gates_of_any_size(dtype):
    """A row of ones by its mean square, 1 / sqrt(1 + eps), times s(z) for gates up to the
    largest finite values.  Some 16 roundings and one to the result's type, 2^-20 and
    2^-8 of it; a subnormal factor may be 0, under 2^-119 at |z| < 89."""
    rel, tiny = 2.0 ** -8 + 2.0 ** -20 if dtype == BF16 else 2.0 ** -20, 2.0 ** -119
    big = torch.finfo(dtype).max
    z = torch.tensor([-big, -1e30, -200.0, -89.0, -88.0, -87.0, -1.0, 0.0, 1.0, 88.0, 105.0, 200.0, 1e30, big, 0.5, -0.5], device="cuda").to(dtype)
    gate = z.view(1, 1, 1, -1).clone().requires_grad_()
    one = torch.ones_like(gate)
    out = ag.group_norm(one, gate=gate, center=False)
    out.backward(one)
    size = 1 / np.sqrt(1 + 1e-5)
    want, slope = size * S.silu(num(z)), size * S.slope(num(z))
    assert (np.abs(num(out.detach()).ravel() - want) <= rel * np.abs(want) + tiny).all(), out
    assert (np.abs(num(gate.grad).ravel() - slope) <= rel * 2.0 + tiny).all(), gate.grad


def test_refusals():
    c = Case(F32, 2, 10, 4, 16)

    def refused(kind, f):
        with pytest.raises(kind):
            f()

    refused(TypeError, lambda: es.group_norm(c.x.half()))
    refused(es.EsError, lambda: es.group_norm(c.x[0]))
    refused(es.EsError, lambda: es.group_norm(c.x, c.w[:2]))
    refused(TypeError, lambda: es.group_norm(c.x, c.w, c.b.bfloat16()))
    refused(es.EsError, lambda: es.group_norm(c.x, gate=c.gate[:, :5]))
    refused(es.EsError, lambda: es.group_norm(c.x, gate=c.gate, activation=True))
    refused(es.EsError, lambda: es.group_norm(c.x, gate_first=True))
    refused(es.EsError, lambda: es.group_norm(c.x, eps=-1.0))
    refused(es.EsError, lambda: es.group_norm(c.x, out=c.x))
    refused(es.EsError, lambda: es.group_norm(torch.zeros(1, 1, 1, 8200, device="cuda")))
    assert torch.equal(es.group_norm(c.x), es.group_norm(c.x))
