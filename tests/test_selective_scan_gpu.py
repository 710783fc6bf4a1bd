"""The selective scan against the 64-bit oracle: prompts, gradients, single
tokens.

Tolerances.  A is the result's sum with every factor by its absolute value (the
oracle's magnitude run); roundings are counted in units of 2^-24.  A step costs
8 (the exponential 4, its correction, the polynomial), a gate 8.  On its way
along the row a term passes one decay a token: the hardware's 2^x within 2^-22,
4 units, and a product, 1; the exponents' own roundings (two, and the step's 8)
are of their sum s, and what they cost, 10 s units of e^-s, is under 4.  Then N
terms are summed, and D x and the gate come: n = 5 T + N + 64, |error| <= 2^-24
n A.  A gradient's term has two such ways and is summed over up to C channels
and B T tokens: 10 T + N + C + B T + 128.  A bf16 result is rounded once more,
2^-8 of its value.
"""
import itertools

import numpy as np
import pytest
import torch

import element_scan_recurrences_gb300 as es
import oracle.state_space as S
from element_scan_recurrences_gb300 import autograd as ag

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
NAMES = ("gx", "gdelta", "gA", "gB", "gC", "gD", "ggate", "gbias", "ginitial")


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    es.lib()


def num(t):
    return None if t is None else t.double().cpu().numpy()


class Case:
    """Inputs on the GPU."""

    def __init__(self, dtype, B, T, C, N=16, G=1, gate=True, extra=True, carry=True, lengths=None, soft=True, seed=0):
        rng = np.random.default_rng(seed)
        n = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
        self.B, self.T, self.C, self.N, self.G = B, T, C, N, G
        self.x, self.B_, self.C_ = n(B, T, C).to(dtype), n(B, T, G, N).to(dtype), n(B, T, G, N).to(dtype)
        self.delta = (n(B, T, C) if soft else n(B, T, C).abs() * 0.3).to(dtype)
        self.A = -torch.from_numpy(rng.uniform(0.02, 4.0, (C, N)).astype(np.float32)).cuda()
        self.D, self.bias = (n(C), n(C) - 2) if extra else (None, None)
        if not soft and extra:
            self.bias = self.bias.abs() * 0.1
        self.gate = n(B, T, C).to(dtype) if gate else None
        self.init, self.gfin = (n(B, C, N), n(B, C, N)) if carry else (None, None)
        self.go = n(B, T, C).to(dtype)
        self.lengths = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.soft = soft

    @property
    def args(self):
        return (self.x, self.delta, self.A, self.B_, self.C_, self.D, self.gate, self.bias)

    @property
    def plain(self):
        return tuple(num(t) for t in self.args)

    def kw(self):
        return dict(softplus=self.soft, initial_state=self.init, lengths=self.lengths)

    def okw(self):
        return dict(soft=self.soft, init=num(self.init), lengths=num(self.lengths))


def close(got, want, size, n, what):
    rounded = 2.0 ** -8 if got.dtype == BF16 else 0.0
    got = num(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    tol = rounded * np.abs(want) + 2.0 ** -24 * n * size + 1e-30
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of the tolerance, first at %s" % (
        what, bad.sum(), bad.size, float(np.nanmax(np.abs(got - want) / tol)), np.argwhere(bad)[0])


def check_forward(c, got=None):
    out, state = (got or es.selective_scan(*c.args, final_state=True, **c.kw()))[:2]
    es.device_status()
    want, size = (S.selective_scan(*c.plain, **c.okw(), magnitude=m) for m in (False, True))
    n = 5 * c.T + c.N + 64
    close(out, want[0], size[0], n, "out")
    close(state, want[1], size[1], n, "state")


def check_backward(c, got=None, kept=None):
    if got is None:
        got = es.selective_scan_backward(*c.args, c.go, grad_final_state=c.gfin, checkpoints=kept, **c.kw())
    es.device_status()
    want, size = (S.selective_scan_backward(*c.plain, num(c.go), gfin=num(c.gfin), **c.okw(), magnitude=m) for m in (False, True))
    n = 10 * c.T + c.N + c.C + c.B * c.T + 128
    there = (True,) * 5 + (c.D is not None, c.gate is not None, c.bias is not None, c.init is not None)
    for name, g, w, s, has in zip(NAMES, got, want, size, there):
        assert (g is not None) == has, name
        if has:
            close(g, w, s, n, name)
    return got


SHAPES = [(2, 37, 40, 16, 1), (1, 1, 128, 16, 1), (3, 16, 130, 16, 2), (1, 50, 24, 5, 3), (2, 33, 48, 8, 1), (1, 40, 72, 32, 1),
          (2, 20, 33, 64, 1), (1, 17, 256, 12, 2), (1, 35, 20, 3, 2), (1, 100, 136, 16, 1)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(dtype, shape):
    check_forward(Case(dtype, *shape))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(dtype, shape):
    c = Case(dtype, *shape, seed=1)
    check_backward(c)


@pytest.mark.parametrize("gate,extra,carry,soft", list(itertools.product((True, False), repeat=4)))
def test_options(gate, extra, carry, soft):
    c = Case(F32, 2, 21, 24, 16, 1, gate, extra, carry, [21, 9], soft, seed=2)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_lengths(dtype):
    """Rows without tokens, with one, of whole tiles; what lies past them is never read."""
    c = Case(dtype, 5, 40, 36, 16, 1, lengths=[0, 1, 16, 39, 200], seed=3)
    for t in (c.x, c.delta, c.gate, c.go, c.B_, c.C_):
        for b, n in enumerate([0, 1, 16, 39, 40]):
            t[b, n:] = float("nan")
    out, state, kept = es.selective_scan(*c.args, final_state=True, checkpoints=True, **c.kw())
    grads = check_backward(c, kept=kept)
    for t in (out,) + tuple(grads[i] for i in (0, 1, 3, 4, 6)):
        for b, n in enumerate([0, 1, 16, 39, 40]):
            assert not t[b, n:].any()
    assert torch.equal(state[0], c.init[0])
    for t in (c.x, c.delta, c.gate, c.go, c.B_, c.C_):
        t.nan_to_num_(0.0)
    check_forward(c, (out, state))


@pytest.mark.parametrize("T,C,N", [(700, 32, 16), (1000, 16, 5), (333, 40, 64)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_segments(dtype, T, C, N):
    """Few channels and many tokens: the tokens are cut into segments."""
    c = Case(dtype, 2, T, C, N, 1, lengths=[T, T // 2 + 3], seed=4)
    check_forward(c)
    check_backward(c)


def test_segments_in_place():
    """The last state may take the first one's place, in one pass or in segments."""
    for T in (40, 900):
        c = Case(F32, 1, T, 16, seed=5)
        _, want, _ = es.selective_scan(*c.args, final_state=True, **c.kw())
        state = c.init.clone()
        kw = dict(c.kw(), initial_state=state)
        es.selective_scan(*c.args, final_state=state, **kw)
        assert torch.equal(state, want)


def test_checkpoints_are_what_the_backward_finds():
    c = Case(BF16, 2, 200, 64, seed=6, lengths=[200, 77])
    _, _, kept = es.selective_scan(*c.args, checkpoints=True, **c.kw())
    one = es.selective_scan_backward(*c.args, c.go, grad_final_state=c.gfin, checkpoints=kept, **c.kw())
    two = es.selective_scan_backward(*c.args, c.go, grad_final_state=c.gfin, **c.kw())
    for name, a, b in zip(NAMES, one, two):
        assert torch.equal(a, b), name


def test_results_repeat():
    c = Case(BF16, 3, 300, 192, 16, 2, seed=7)
    runs = [es.selective_scan_backward(*c.args, c.go, grad_final_state=c.gfin, **c.kw()) for _ in range(3)]
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,C,N,G", [(1, 128, 16, 1), (7, 40, 16, 2), (3, 24, 5, 1), (2, 33, 64, 1), (2, 9, 33, 3), (5, 64, 32, 1)])
def test_step(dtype, B, C, N, G):
    c = Case(dtype, B, 1, C, N, G, seed=8)
    state = c.init.clone()
    one = [None if t is None else t[:, 0] if t.dim() > 2 else t for t in c.args]
    out, new = es.selective_scan_step(*one, state)
    assert new is state
    check_forward(c, (out[:, None], state))
    keep, other = c.init.clone(), torch.empty_like(state)
    out2, new2 = es.selective_scan_step(*one, keep, state_out=other)
    assert torch.equal(keep, c.init) and torch.equal(new2, state) and torch.equal(out2, out)


def test_step_without_gate_and_extras():
    c = Case(F32, 3, 1, 20, 16, 1, gate=False, extra=False, soft=False, seed=9)
    one = [None if t is None else t[:, 0] if t.dim() > 2 else t for t in c.args]
    out, state = es.selective_scan_step(*one, c.init.clone(), softplus=False)
    check_forward(c, (out[:, None], state))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_views(dtype):
    """Operands as parts of projections' results, at odd addresses, rows in another order: the same results."""
    c = Case(dtype, 2, 50, 40, 16, 1, seed=10)
    want = es.selective_scan(*c.args, final_state=True, **c.kw())
    gwant = es.selective_scan_backward(*c.args, c.go, grad_final_state=c.gfin, **c.kw())

    def odd(t):          # one element off every alignment, twice the row
        box = torch.zeros(*t.shape[:-1], 2 * t.shape[-1] + 1, dtype=t.dtype, device="cuda")
        v = box[..., 1:1 + t.shape[-1]]
        v.copy_(t)
        return v

    def turned(t):       # tokens outermost
        return t.transpose(0, 1).contiguous().transpose(0, 1)

    for view in (odd, turned):
        a = [view(t) if t is not None and t.dim() > 2 else t for t in c.args]
        got = es.selective_scan(*a, final_state=True, out=view(torch.zeros_like(c.x)), **c.kw())
        for x, y in zip(got[:2], want[:2]):
            assert torch.equal(x, y)
        for x, y in zip(es.selective_scan_backward(*a, view(c.go), grad_final_state=c.gfin, **c.kw()), gwant):
            assert torch.equal(x, y)
    # B and C alone at odd addresses, then the rows alone
    for which in ((3, 4), (0, 1, 6)):
        a = [odd(t) if i in which else t for i, t in enumerate(c.args)]
        assert torch.equal(es.selective_scan(*a, **c.kw())[0], want[0])
        for x, y in zip(es.selective_scan_backward(*a, c.go, grad_final_state=c.gfin, **c.kw()), gwant):
            assert torch.equal(x, y)
    # states at addresses of 4 bytes
    box = torch.zeros(c.init.numel() + 1, device="cuda")
    init = box[1:].view_as(c.init)
    init.copy_(c.init)
    kw = dict(c.kw(), initial_state=init)
    assert torch.equal(es.selective_scan(*c.args, final_state=True, **kw)[1], want[1])
    assert torch.equal(es.selective_scan_backward(*c.args, c.go, grad_final_state=c.gfin, **kw)[8], gwant[8])


def test_empty():
    for B, T, C in ((0, 5, 8), (2, 0, 8), (2, 5, 0)):
        c = Case(F32, B, T, C, seed=11)
        out, state, _ = es.selective_scan(*c.args, final_state=True, **c.kw())
        assert out.shape == (B, T, C) and torch.equal(state, c.init)
        g = es.selective_scan_backward(*c.args, c.go, grad_final_state=c.gfin, **c.kw())
        assert torch.equal(g[8], c.gfin) and not g[2].any() and not g[5].any() and not g[7].any()


def test_strong_and_weak_steps():
    """Steps from 1e-6 to 30 and decays that reach zero."""
    c = Case(F32, 1, 60, 32, 16, seed=12)
    c.delta.copy_(torch.linspace(-14, 30, 60, device="cuda")[None, :, None] + c.delta)
    check_forward(c)
    check_backward(c)


def test_a_prompt_then_its_tokens():
    c = Case(F32, 2, 48, 40, seed=13)
    whole, last, _ = es.selective_scan(*c.args, final_state=True, **c.kw())
    cut = lambda a, b: [None if t is None else t[:, a:b] if t.dim() > 2 else t for t in c.args]  # noqa: E731
    out, state, _ = es.selective_scan(*cut(0, 30), initial_state=c.init, final_state=True)
    outs = [out]
    for t in range(30, 48):
        one = [None if v is None else v[:, 0] if v.dim() > 2 else v for v in cut(t, t + 1)]
        o, state = es.selective_scan_step(*one, state)
        outs.append(o[:, None])
    got = torch.cat(outs, 1)
    assert torch.allclose(got, whole, rtol=1e-5, atol=1e-5) and torch.allclose(state, last, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("keep", [True, False])
def test_autograd(keep):
    c = Case(F32, 2, 40, 24, seed=14)
    leaves = [None if t is None else t.clone().requires_grad_(True) for t in c.args + (c.init,)]
    out, state = ag.selective_scan(*leaves[:8], softplus=True, initial_state=leaves[8], final_state=True, checkpoints=keep)
    torch.autograd.backward([out, state], [c.go, c.gfin])
    check_backward(c, [t.grad for t in leaves])


def test_on_another_stream_and_captured():
    c = Case(BF16, 2, 300, 64, seed=15)
    run = lambda: es.selective_scan(*c.args, final_state=True, checkpoints=True, **c.kw())  # noqa: E731
    back = lambda: es.selective_scan_backward(*c.args, c.go, grad_final_state=c.gfin, **c.kw())  # noqa: E731
    want, gwant = run(), back()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = es.selective_scan(*c.args, final_state=True, stream=side, **c.kw())
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, ggot = run(), back()
    other = Case(BF16, 2, 300, 64, seed=16)
    for t, u in zip(c.args + (c.init, c.go, c.gfin), other.args + (other.init, other.go, other.gfin)):
        t.copy_(u)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(tuple(got) + tuple(ggot), tuple(run()) + tuple(back())):
        assert torch.equal(x, y)
    del want, gwant


def test_refusals():
    c = Case(F32, 2, 10, 16, seed=17)
    a = list(c.args)

    def refused(kind, f):
        with pytest.raises(kind):
            f()

    refused(TypeError, lambda: es.selective_scan(c.x.half(), *a[1:]))
    refused(TypeError, lambda: es.selective_scan(c.x.cpu(), *a[1:]))
    refused(TypeError, lambda: es.selective_scan(c.x, c.delta.bfloat16(), *a[2:]))
    refused(es.EsError, lambda: es.selective_scan(c.x, c.delta[:, :9], *a[2:]))
    refused(TypeError, lambda: es.selective_scan(*a[:2], c.A.bfloat16(), *a[3:]))
    refused(es.EsError, lambda: es.selective_scan(*a[:2], c.A[:8], *a[3:]))
    refused(es.EsError, lambda: es.selective_scan(*a[:3], c.B_.expand(2, 10, 3, 16), c.C_.expand(2, 10, 3, 16), *a[5:]))
    refused(es.EsError, lambda: es.selective_scan(*a, out=c.x))
    refused(es.EsError, lambda: es.selective_scan(*a, checkpoints=torch.empty(16, dtype=torch.uint8, device="cuda")))
    refused(es.EsError, lambda: es.selective_scan(c.x.transpose(1, 2).contiguous().transpose(1, 2), *a[1:]))
    refused(es.EsError, lambda: es.selective_scan(*a, initial_state=c.init[:, :, :8].contiguous()))
    refused(es.EsError, lambda: es.selective_scan_backward(*a, c.go[:1]))
    refused(TypeError, lambda: es.selective_scan(*a, lengths=torch.tensor([1, 2], device="cuda")))
    assert torch.equal(es.selective_scan(*a)[0], es.selective_scan(*a)[0])


SIZES = [-1e30, -200.0, -89.0, -88.0, -87.0, -1.0, 0.0, 1.0, 88.0, 105.0, 200.0, 1e30]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gates_and_steps_of_any_size(dtype):
    """Gates and steps up to the largest finite values, one state and token, y = 0.5: y
    times s(z), which is 0 far below 0 and z far above.  Some 16 roundings and one to
    the result's type: 2^-20 and 2^-8 of it; a subnormal factor may be 0, 2^-126 z at
    |z| < 89, under 2^-119."""
    rel, tiny = 2.0 ** -8 + 2.0 ** -20 if dtype == BF16 else 2.0 ** -20, 2.0 ** -119
    big = torch.finfo(dtype).max
    z = torch.tensor([-big] + SIZES + [big], device="cuda").to(dtype)
    n = z.numel()
    one, two = torch.ones(1, 1, n, dtype=dtype, device="cuda"), torch.ones(1, 1, 1, 1, dtype=dtype, device="cuda")
    a = torch.full((n, 1), -1.0, device="cuda")
    gate = z.view(1, 1, n)
    half = one * 0.5
    prompt = es.selective_scan(half, one, a, two, two, gate=gate, softplus=False)[0]
    state = torch.zeros(1, n, 1, device="cuda")
    step = es.selective_scan_step(half[0], one[0], a, two[0], two[0], None, gate[0], None, state, softplus=False)[0]
    want = 0.5 * S.silu(num(z))
    for out in (prompt, step):
        assert (np.abs(num(out).ravel() - want) <= rel * np.abs(want) + tiny).all(), out
    leaf = gate.clone().requires_grad_()
    ag.selective_scan(half, one, a, two, two, gate=leaf, softplus=False)[0].backward(one)
    want = 0.5 * S.slope(num(z))
    # the slope is a sum of terms no larger than 1 + |z| e^-|z|
    assert (np.abs(num(leaf.grad).ravel() - want) <= rel * 2.0 + tiny).all(), leaf.grad
    # steps: A = 0, so that the state is 2 softplus(delta); log 2 is of 3 roundings more
    d = torch.tensor([-1e30, -100.0, 0.0, 100.0, 1e30], device="cuda").view(1, 1, 5).to(dtype)
    x = torch.full_like(d, 2.0)
    out = num(es.selective_scan(x, d, torch.zeros(5, 1, device="cuda"), two, two)[0]).ravel()
    want = 2.0 * S.softplus(num(d)).ravel()
    assert (np.abs(out - want) <= rel * np.abs(want) + tiny).all(), out
