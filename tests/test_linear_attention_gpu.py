"""Linear attention with a decay for each head against the 64-bit oracle:
prompts, gradients, single tokens; both kernel paths.

Tolerances.  Every output is a sum of terms; A is the same sum over absolute
values (the oracle's magnitude run).  In f32, a term passes at most
n = dk + dv + 128 + 8 G + T / 8 roundings of 2^-24 (the sums over the widths
and a chunk, the decay's exponent with G the largest sum of a chunk's decays,
and one product and sum a chunk on the way along the sequence), so
|error| <= 2^-24 n A.  On the tensor cores an f32 factor goes in as a sum of
bf16 terms: two of them keep 2^-16 of it (outputs and the decays' gradient: at
most three such factors a term, 2^-14 A), three keep 2^-24 (states: 2^-20 A).
A bf16 result is rounded once more, 2^-8 of its value.
"""
import itertools

import numpy as np
import pytest
import torch

import element_scan_recurrences_gb300 as es
import oracle.attention as A

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    es.lib()


@pytest.fixture(autouse=True)
def paths():
    yield
    es.set_path_override("auto")
    es.device_status()


class Case:
    """Inputs on the GPU and the oracle's answers."""

    def __init__(self, dtype, B, T, heads, dk, dv, decay="token", carry=True, lengths=None, seed=0, fade=0.3):
        rng = np.random.default_rng(seed)
        hq, hk, hv, H = heads
        self.dtype, self.B, self.T, self.H, self.dk, self.dv = dtype, B, T, H, dk, dv

        def made(*shape):
            t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype).cuda()
            return t

        self.q, self.k, self.v = made(B, T, hq, dk), made(B, T, hk, dk), made(B, T, hv, dv)
        self.go = made(B, T, H, dv)
        f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
        self.init, self.gfin = (f(B, H, dk, dv), f(B, H, dk, dv)) if carry else (None, None)
        g = None
        if decay == "token":
            g = -rng.uniform(0, fade, (B, T, H)).astype(np.float32)
        elif decay == "head":
            g = -rng.uniform(0, fade, (H,)).astype(np.float32)
        self.g = None if g is None else torch.from_numpy(g).cuda()
        self.lengths = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.scale = dk ** -0.5
        self.n = dk + dv + 128 + 8 * 64 * fade + T / 8

    def numpy(self, t):
        return None if t is None else t.double().cpu().numpy()

    def args(self):
        return [self.numpy(x) for x in (self.q, self.k, self.v, self.g)]

    def kw(self):
        return dict(lengths=self.numpy(self.lengths), scale=self.scale, heads=self.H)


def close(got, want, size, n, what, f32=2.0 ** -14):
    """`size`: the magnitude A; `f32`: the share of A the splits may cost."""
    rounded = 2.0 ** -8 if got.dtype == BF16 else 0.0
    got = got.double().cpu().numpy()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    tol = rounded * np.abs(want) + (2.0 ** -24 * n + f32) * size + 1e-30
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of the tolerance" % (
        what, bad.sum(), bad.size, float(np.nanmax(np.abs(got - want) / tol)))


def check_forward(c, **over):
    split = c.dtype == BF16
    kw = dict(initial_state=c.init, lengths=c.lengths, scale=c.scale, final_state=True)
    kw.update(over)
    out, state = es.linear_attention(c.q, c.k, c.v, c.g, **kw)
    es.device_status()
    want, wstate = A.linear_attention(*c.args(), c.numpy(c.init), **c.kw())
    absolute = [np.abs(x) for x in c.args()[:3]]
    size, ssize = A.linear_attention(*absolute, c.args()[3], None if c.init is None else np.abs(c.numpy(c.init)), **c.kw())
    close(out, want, size, c.n, "out", 2.0 ** -14 if split else 0.0)
    close(state, wstate, ssize, c.n, "state", 2.0 ** -20 if split else 0.0)
    return out, state


def check_backward(c, got=None):
    split = c.dtype == BF16
    if got is None:
        got = es.linear_attention_backward(c.q, c.k, c.v, c.g, c.go, initial_state=c.init, grad_final_state=c.gfin,
                                           lengths=c.lengths, scale=c.scale)
    es.device_status()
    args = (*c.args(), c.numpy(c.go), c.numpy(c.init), c.numpy(c.gfin))
    want = A.linear_attention_backward(*args, **c.kw())
    size = A.linear_attention_backward(*args, magnitude=True, **c.kw())
    for i, name in enumerate(("gq", "gk", "gv", "gg", "gi")):
        if got[i] is not None:
            close(got[i], want[i], size[i], 2 * c.n, name, (2.0 ** -20 if name == "gi" else 2.0 ** -14) if split else 0.0)
    return got


SAME = (2, 2, 2, 2)
SHAPES = [
    # B, T, heads (q, k, v, H), dk, dv, decay, carry, lengths
    (1, 1, SAME, 64, 64, "token", True, None),
    (2, 2, SAME, 64, 64, "head", False, None),
    (2, 37, SAME, 64, 64, "token", True, [37, 5]),
    (3, 64, SAME, 128, 128, "token", True, [64, 0, 1]),
    (1, 65, SAME, 128, 128, None, True, None),
    (2, 130, SAME, 128, 64, "token", False, [129, 64]),
    (1, 200, SAME, 64, 128, "head", True, None),
    (1, 193, (1, 1, 4, 4), 128, 64, "token", True, None),
    (1, 96, (4, 2, 1, 4), 64, 64, "token", True, [95]),
    (2, 70, (1, 2, 4, 4), 64, 64, "head", True, None),
    (1, 131, SAME, 96, 80, "token", True, None),
    (1, 75, SAME, 8, 24, "token", True, None),
    (2, 67, SAME, 33, 17, "token", True, [66, 67]),
    (1, 40, (1, 1, 1, 3), 1, 1, "head", True, None),
    (1, 70, (2, 2, 2, 2), 256, 40, "token", True, None),
    (1, 1100, (1, 1, 1, 1), 64, 64, "token", True, None),
]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dx%d_%s_%dx%d_%s" % (s[0], s[1], "".join(map(str, s[2])), s[3], s[4], s[5]))
def test_against_the_oracle(shape, dtype):
    c = Case(dtype, *shape)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[5], SHAPES[8]], ids=str)
def test_the_direct_kernel_serves_bf16(shape):
    es.set_path_override("generic")
    c = Case(BF16, *shape)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_no_tokens(dtype):
    c = Case(dtype, 2, 0, SAME, 64, 64)
    out, state = es.linear_attention(c.q, c.k, c.v, c.g, initial_state=c.init, final_state=True)
    assert out.shape == (2, 0, 2, 64) and torch.equal(state, c.init)
    out, state = es.linear_attention(c.q, c.k, c.v, c.g, final_state=True)
    assert not state.any()
    grads = es.linear_attention_backward(c.q, c.k, c.v, c.g, c.go, initial_state=c.init, grad_final_state=c.gfin)
    assert torch.equal(grads[4], c.gfin)
    c = Case(dtype, 2, 0, SAME, 64, 64, decay="head")
    grads = es.linear_attention_backward(c.q, c.k, c.v, c.g, c.go)
    assert not grads[3].any()
    c = Case(dtype, 0, 5, SAME, 64, 64)
    assert es.linear_attention(c.q, c.k, c.v, c.g)[0].shape == (0, 5, 2, 64)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("low", [float("-inf"), float(np.finfo(np.float32).min), -200.0])
def test_tokens_that_start_afresh(dtype, low):
    """A decay of zero drops whatever was there, exactly, and costs the later sums no precision."""
    c = Case(dtype, 2, 150, SAME, 64, 64)
    for b, t, h in [(0, 0, 0), (0, 40, 1), (0, 63, 0), (0, 64, 0), (1, 10, 0), (1, 11, 0), (1, 149, 1), (1, 127, 1)]:
        c.g[b, t, h] = low
    check_forward(c)
    with np.errstate(invalid="ignore"):
        args = (*c.args(), c.numpy(c.go), c.numpy(c.init), c.numpy(c.gfin))
        got = es.linear_attention_backward(c.q, c.k, c.v, c.g, c.go, initial_state=c.init, grad_final_state=c.gfin,
                                           scale=c.scale)
        want = A.linear_attention_backward(*args, **c.kw())
        size = A.linear_attention_backward(*args, magnitude=True, **c.kw())
    for i, name in enumerate(("gq", "gk", "gv", "gg", "gi")):
        close(got[i], want[i], size[i], 2 * c.n, name, 2.0 ** -14 if dtype == BF16 else 0.0)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_nothing_is_read_past_the_lengths(dtype):
    """NaN and infinities in padded tokens reach no result, and padded results are zero."""
    c = Case(dtype, 3, 140, SAME, 64, 64, lengths=[139, 70, 0])
    clean = es.linear_attention(c.q, c.k, c.v, c.g, initial_state=c.init, lengths=c.lengths, final_state=True)
    cleang = es.linear_attention_backward(c.q, c.k, c.v, c.g, c.go, initial_state=c.init, grad_final_state=c.gfin,
                                          lengths=c.lengths)
    bad = itertools.cycle([float("nan"), float("inf"), float("-inf")])
    for b, n in enumerate([139, 70, 0]):
        for x in (c.q, c.k, c.v, c.g, c.go):
            x[b, n:] = next(bad)
    got = es.linear_attention(c.q, c.k, c.v, c.g, initial_state=c.init, lengths=c.lengths, final_state=True)
    grads = es.linear_attention_backward(c.q, c.k, c.v, c.g, c.go, initial_state=c.init, grad_final_state=c.gfin,
                                         lengths=c.lengths)
    for x, y in zip(clean + cleang, got + grads):
        assert torch.equal(x, y)
    for x in (got[0],) + grads[:4]:
        for b, n in enumerate([139, 70, 0]):
            assert not x[b, n:].any()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_views(dtype):
    """Parts of a fused projection, heads before tokens, a broadcast row, an
    odd offset, and results written into strided places: the same bits as
    dense operands (an operand the tensor cores cannot load goes to the
    direct kernel: within the tolerance)."""
    B, T, H, D = 2, 77, 4, 64
    gen = torch.Generator(device="cuda").manual_seed(0)
    qkv = torch.randn(B, T, 3 * H, D, generator=gen, device="cuda").to(dtype)
    q, k, v = qkv[:, :, :H], qkv[:, :, H:2 * H], qkv[:, :, 2 * H:]
    g = -torch.rand(B, H, T, generator=gen, device="cuda").transpose(1, 2) * 0.2
    want, wstate = es.linear_attention(q.contiguous(), k.contiguous(), v.contiguous(), g.contiguous(), final_state=True)
    got, state = es.linear_attention(q, k, v, g, final_state=True)
    assert torch.equal(got, want) and torch.equal(state, wstate)
    heads_first = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v)]
    room = torch.full((B, H, T + 2, D + 8), 7.0, dtype=dtype, device="cuda")
    place = room[:, :, 1:T + 1, :D].transpose(1, 2)
    got, _ = es.linear_attention(*heads_first, g, out=place)
    assert got is place and torch.equal(place, want)
    assert (room[:, :, 0] == 7).all() and (room[:, :, -1] == 7).all() and (room[..., D:] == 7).all()
    one = [x[:1].expand(B, T, H, D) for x in (q, k, v)]
    got, _ = es.linear_attention(*one, g[:1].expand(B, T, H))
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], want[0])
    odd = torch.empty(B * T * H * D + 1, dtype=dtype, device="cuda")[1:].view(B, T, H, D)
    odd.copy_(q)
    got, _ = es.linear_attention(odd, k, v, g)
    assert (got.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()
    grads = es.linear_attention_backward(q, k, v, g, want)
    dense = es.linear_attention_backward(q.contiguous(), k.contiguous(), v.contiguous(), g.contiguous(), want)
    for x, y in zip(grads[:4], dense[:4]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_the_same_bits_each_time_and_state_in_place(dtype):
    c = Case(dtype, 2, 300, (1, 1, 4, 4), 64, 64, decay="head")
    kw = dict(initial_state=c.init, scale=c.scale)
    first = es.linear_attention(c.q, c.k, c.v, c.g, final_state=True, **kw)
    grads = es.linear_attention_backward(c.q, c.k, c.v, c.g, c.go, grad_final_state=c.gfin, **kw)
    again = es.linear_attention_backward(c.q, c.k, c.v, c.g, c.go, grad_final_state=c.gfin, **kw)
    for x, y in zip(grads, again):
        assert torch.equal(x, y)
    place = c.init.clone()
    out, state = es.linear_attention(c.q, c.k, c.v, c.g, initial_state=place, scale=c.scale, final_state=place)
    assert state is place and torch.equal(place, first[1]) and torch.equal(out, first[0])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_a_sequence_in_pieces(dtype):
    """The state carried from piece to piece gives the whole sequence's results."""
    c = Case(dtype, 2, 210, SAME, 64, 64)
    state, outs = c.init, []
    for lo, hi in ((0, 1), (1, 100), (100, 164), (164, 210)):
        o, state = es.linear_attention(*(x[:, lo:hi] for x in (c.q, c.k, c.v, c.g)), initial_state=state, scale=c.scale,
                                       final_state=True)
        outs.append(o)
    want, wstate = A.linear_attention(*c.args(), c.numpy(c.init), **c.kw())
    size, ssize = A.linear_attention(*[np.abs(x) for x in c.args()[:3]], c.args()[3], np.abs(c.numpy(c.init)), **c.kw())
    split = dtype == BF16
    close(torch.cat(outs, 1), want, size, c.n, "out", 2.0 ** -14 if split else 0.0)
    close(state, wstate, ssize, c.n, "state", 2.0 ** -20 if split else 0.0)


STEPS = [
    # B, heads, dk, dv, decay
    (1, (16, 16, 16, 16), 128, 128, "token"),
    (3, (1, 2, 4, 4), 64, 64, "head"),
    (2, SAME, 96, 80, "token"),
    (5, SAME, 33, 17, None),
    (1, (1, 1, 1, 1), 1, 1, "token"),
    (2, SAME, 256, 256, "token"),
    (2, SAME, 7, 132, "head"),
]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", STEPS, ids=str)
def test_steps(shape, dtype):
    B, heads, dk, dv, decay = shape
    c = Case(dtype, B, 4, heads, dk, dv, decay)
    if decay == "token":
        c.g[0, 2] = float("-inf")
    want, wstate = A.linear_attention(*c.args(), c.numpy(c.init), **c.kw())
    size, ssize = A.linear_attention(*[np.abs(x) for x in c.args()[:3]], c.args()[3], np.abs(c.numpy(c.init)), **c.kw())
    state, other, outs = c.init.clone(), torch.empty_like(c.init), []
    for t in range(4):
        g = c.g[:, t] if decay == "token" else c.g
        if t % 2:       # in place
            o, s = es.linear_attention_step(c.q[:, t], c.k[:, t], c.v[:, t], g, state, scale=c.scale)
            assert s is state
        else:           # to another place, the old one kept
            before = state.clone()
            o, s = es.linear_attention_step(c.q[:, t], c.k[:, t], c.v[:, t], g, state, state_out=other, scale=c.scale)
            assert torch.equal(state, before)
            state, other = other, state
        outs.append(o)
    es.device_status()
    close(torch.stack(outs, 1), want, size, c.n, "out", 0.0)
    close(state, wstate, ssize, c.n, "state", 0.0)


def test_another_stream():
    c = Case(BF16, 2, 500, SAME, 128, 128)
    want = es.linear_attention(c.q, c.k, c.v, c.g, initial_state=c.init, final_state=True)
    wgrads = es.linear_attention_backward(c.q, c.k, c.v, c.g, c.go, initial_state=c.init)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = es.linear_attention(c.q, c.k, c.v, c.g, initial_state=c.init, final_state=True, stream=s)
    grads = es.linear_attention_backward(c.q, c.k, c.v, c.g, c.go, initial_state=c.init, stream=s.cuda_stream)
    s.synchronize()
    for x, y in zip(want + wgrads, got + grads):
        assert torch.equal(x, y)


@pytest.mark.parametrize("decay", ["token", "head", None])
def test_autograd(decay):
    from element_scan_recurrences_gb300.autograd import linear_attention
    c = Case(F32, 2, 70, (1, 1, 2, 2), 32, 16, decay, lengths=[70, 50])
    leaves = [x.clone().requires_grad_(True) for x in (c.q, c.k, c.v)]
    g = None if c.g is None else c.g.clone().requires_grad_(True)
    init = c.init.clone().requires_grad_(True)
    out, state = linear_attention(*leaves, g, init, c.lengths, c.scale, True)
    ((out * c.go).sum() + (state * c.gfin).sum()).backward()
    check_backward(c, tuple(x.grad for x in leaves) + (None if g is None else g.grad, init.grad))


def test_gradient_against_differences():
    """(L(x + d u) - L(x - d u)) / 2d against <gradient, u>, f32, L = <out, go>
    + <state, gfin>.  L is of third order along the line, so the difference is
    off by d^2 / 6 of its third derivative, bounded by the terms' sum S, and by
    the rounding of L, 2^-24 n S / d."""
    c = Case(F32, 2, 60, SAME, 32, 32, "token")
    x = [c.q, c.k, c.v, c.g, c.init]
    gen = torch.Generator(device="cuda").manual_seed(1)
    u = [torch.randn(y.shape, generator=gen, device="cuda") for y in x]
    grads = es.linear_attention_backward(*x[:4], c.go, initial_state=c.init, grad_final_state=c.gfin, scale=c.scale)

    def loss(s):
        y = [a + s * b for a, b in zip(x, u)]
        out, state = es.linear_attention(*y[:4], initial_state=y[4], scale=c.scale, final_state=True)
        return float((out.double() * c.go.double()).sum() + (state.double() * c.gfin.double()).sum())

    slope = sum(float((g.double() * b.double()).sum()) for g, b in zip(grads, u))
    sizes = A.linear_attention(*[np.abs(y) for y in c.args()[:3]], c.args()[3], np.abs(c.numpy(c.init)), **c.kw())
    S = float((sizes[0] * np.abs(c.numpy(c.go))).sum() + (sizes[1] * np.abs(c.numpy(c.gfin))).sum())
    d = 1e-2
    got = (loss(d) - loss(-d)) / (2 * d)
    root = np.sqrt(c.q.numel())     # random signs: the terms' sums grow as their root
    assert abs(got - slope) <= (d * d / 6 * 27 + 2.0 ** -24 * c.n / d) * S / root * 8, (got, slope, S / root)


def test_refusals():
    c = Case(BF16, 2, 10, SAME, 64, 64)
    status = {}

    def refused(code, *a, **k):
        with pytest.raises(es.EsError) as e:
            es.linear_attention(*a, **k)
        assert e.value.status == code, e.value
        status[code] = True

    refused(1, c.q, c.k[:, :5], c.v, c.g)
    refused(1, c.q, c.k, c.v, c.g[:, :, :1].expand(2, 10, 1))        # two operand heads, one head
    refused(1, c.q, c.k, c.v, torch.zeros(2, 10, 3, device="cuda"))
    refused(1, c.q, c.k, c.v, c.g, initial_state=torch.zeros(2, 2, 64, 63, device="cuda"))
    refused(1, c.q, c.k, c.v, c.g, lengths=torch.zeros(3, dtype=torch.int32, device="cuda"))
    refused(3, c.q, c.k, c.v, c.g, scale=0.0)
    refused(3, c.q, c.k, c.v, c.g, scale=float("nan"))
    refused(3, c.q, c.k, c.v, c.g, out=c.q)
    refused(3, c.q.transpose(2, 3), c.k.transpose(2, 3), c.v, c.g)
    wide = torch.zeros(1, 2, 1, 257, dtype=BF16, device="cuda")
    refused(4, wide, wide, wide)
    for bad in (dict(q=c.q.half()), dict(k=c.k.float()), dict(v=c.v.cpu()), dict(log_decay=c.g.double()),
                dict(lengths=torch.zeros(2, dtype=torch.int64, device="cuda")), dict(initial_state=c.init.to(BF16))):
        with pytest.raises(TypeError):
            es.linear_attention(**{**dict(q=c.q, k=c.k, v=c.v, log_decay=c.g), **bad})
    with pytest.raises(es.EsError):
        es.linear_attention_backward(c.q, c.k, c.v, c.g, c.go[:, :5])
    need = es.plan_linear_attention(c.q.shape, c.k.shape, c.v.shape, decay="token", backward=True)["workspace"]
    with pytest.raises(es.EsError) as e:
        es.linear_attention_backward(c.q, c.k, c.v, c.g, c.go, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
    with pytest.raises(TypeError):
        es.linear_attention_step(c.q[:, 0], c.k[:, 0], c.v[:, 0], c.g[:, 0], None)
    with pytest.raises(es.EsError):
        es.linear_attention_step(c.q[:, 0], c.k[:, 0], c.v[:, 0], c.g[:, 0], c.init[:1])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads", [(1, 1, 1, 1), (2, 1, 2, 2)], ids=str)
def test_long_rows_in_segments(heads, dtype):
    """Few heads and many tokens: the row is cut into segments (a workspace is
    asked for), with lengths that end in the first, a middle and the last of
    them, a carried state in place, and decays of zero at and near the cuts."""
    lengths = [1500, 64, 700]
    c = Case(dtype, 3, 1500, heads, 64, 64, lengths=lengths)
    assert es.plan_linear_attention(c.q.shape, c.k.shape, c.v.shape, "f32" if dtype == F32 else "bf16", decay="token",
                                    heads=heads[3])["workspace"] > 0
    c.g[0, 640, 0] = float("-inf")
    c.g[2, 512, 0] = float("-inf")
    out, state = check_forward(c)
    check_backward(c)
    place = c.init.clone()
    es.linear_attention(c.q, c.k, c.v, c.g, initial_state=place, lengths=c.lengths, scale=c.scale, final_state=place)
    assert torch.equal(place, state)
    c = Case(dtype, 1, 900, heads, 64, 64, decay="head", carry=False)
    check_forward(c)
    check_backward(c)
