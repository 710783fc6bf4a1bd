"""The norm of queries and keys with the position rotation against the 64-bit
oracle, forward and backward.

Tolerances.  With |u| <= sqrt(D) the unit row: the sum of squares over D
values, the root and the division cost (D / 2 + 6) roundings of 2^-24 of u, the
weight and the turn three more of at most |w| (|u_a| + |u_b|) <= 2 |w| sqrt(D);
backward the mean's sum over D more.  Weights' gradients add rows: 2^-24 times
the number of them and of the roundings of a term, on the sum of absolute
terms.  bf16 results are rounded once more, 2^-8 of their value.
"""
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


def made(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda()


def num(t):
    return None if t is None else t.double().cpu().numpy()


def close(got, want, size, what):
    rounded = 2.0 ** -8 if got.dtype == BF16 else 0.0
    got = num(got)
    assert got.shape == want.shape
    tol = rounded * np.abs(want) + 2.0 ** -24 * size + 1e-30
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g" % (what, bad.sum(), bad.size,
                                                            float(np.nanmax(np.abs(got - want) / tol)))


CASES = [
    # B, T, hq, hk, D, R, neighbours, weights
    (1, 1, 4, 4, 128, 128, False, "same"),
    (2, 5, 32, 8, 128, 128, False, "same"),
    (2, 7, 3, 1, 128, 64, False, "f32"),
    (2, 7, 3, 1, 128, 64, True, "f32"),
    (1, 33, 5, 2, 64, 64, True, "same"),
    (3, 11, 12, 12, 80, 32, True, "same"),
    (3, 11, 12, 12, 80, 32, False, "same"),
    (1, 9, 2, 2, 96, 96, False, None),
    (2, 3, 2, 1, 33, 12, False, "same"),
    (2, 3, 2, 1, 33, 32, True, "f32"),
    (1, 4, 1, 0, 7, 0, False, "same"),
    (1, 130, 2, 2, 256, 256, False, "same"),
    (1, 4, 2, 2, 1, 0, False, "same"),
    (1, 4, 2, 2, 8, 8, True, "same"),
    (1, 4, 2, 2, 40, 24, True, None),
    (1, 600, 9, 3, 16, 16, False, "same"),
]


def inputs(case, dtype, seed=0):
    B, T, hq, hk, D, R, neighbours, weights = case
    rng = np.random.default_rng(seed)
    q, k = made(rng, B, T, hq, D).to(dtype), made(rng, B, T, hk, D).to(dtype) if hk else None
    wd = {"same": dtype, "f32": F32, None: None}[weights]
    wq, wk = (made(rng, D).to(wd), made(rng, D).to(wd)) if weights else (None, None)
    if not hk:
        wk = None
    ang = rng.uniform(0, 6.3, (50, R // 2))
    cos, sin = (torch.from_numpy(f(ang).astype(np.float32)).cuda() if R else None for f in (np.cos, np.sin))
    pos = torch.from_numpy(rng.integers(-3, 60, (B, T))).cuda()
    gq, gk = made(rng, B, T, hq, D).to(dtype), made(rng, B, T, hk, D).to(dtype) if hk else None
    return q, k, wq, wk, cos, sin, pos, gq, gk, neighbours


def check(case, dtype, eps=1e-5, seed=0, got=None, pos32=False):
    q, k, wq, wk, cos, sin, pos, gq, gk, neighbours = inputs(case, dtype, seed)
    if pos32:
        pos = pos.to(torch.int32)
    kw = dict(positions=pos, eps=eps, neighbours=neighbours)
    outs = es.qk_norm_rotate(q, k, wq, wk, cos, sin, **kw)
    grads = es.qk_norm_rotate_backward(q, k, wq, wk, cos, sin, gq, gk, **kw)
    D = case[4]
    n = D / 2 + 16
    for i, (x, w, g) in enumerate(((q, wq, gq), (k, wk, gk))):
        if x is None:
            assert outs[i] is None and grads[i] is None and grads[2 + i] is None
            continue
        kwn = dict(positions=num(pos), eps=eps, neighbours=neighbours)
        if kwn["positions"] is not None:
            kwn["positions"] = kwn["positions"].astype(np.int64)
        want = A.norm_rotate(num(x), num(w), num(cos), num(sin), **kwn)
        gx, gw = A.norm_rotate_backward(num(x), num(w), num(cos), num(sin), num(g), **kwn)
        big = 1.0 if w is None else float(w.abs().max())
        root = np.sqrt((num(x) ** 2).mean(-1, keepdims=True) + eps)
        u = np.abs(num(x) / root)
        rows = u.max(-1, keepdims=True)
        close(outs[i], want, n * 2 * big * rows, "out")
        gmax = np.abs(num(g)).max(-1, keepdims=True)
        # w z and its share of u: each at most 2 |w| |g|max, the mean a sum of D of them times u
        size = (n + D) * (2 * big * gmax) * (1 + rows * rows) / root
        close(grads[i], gx, size, "gx")
        if w is not None:
            terms = (u * 2 * gmax).sum((0, 1, 2))
            close(grads[2 + i], gw, (n + 64 + np.sqrt(u[..., 0].size)) * terms, "gw")
    return outs, grads


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_the_oracle(case, dtype):
    check(case, dtype)


def test_default_positions_and_int32():
    check(CASES[1], BF16, pos32=True)
    q, k, wq, wk, cos, sin, _, _, _, nb = inputs((1, 60, 2, 2, 64, 64, False, "same"), F32)
    got = es.qk_norm_rotate(q, k, wq, wk, cos, sin)
    at = torch.arange(60, device="cuda")
    want = es.qk_norm_rotate(q, k, wq, wk, cos, sin, positions=at)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    far = es.qk_norm_rotate(q, k, wq, wk, cos, sin, positions=at + (1 << 40))     # clamped to the last row
    last = es.qk_norm_rotate(q, k, wq, wk, cos, sin, positions=torch.full_like(at, 49))
    assert torch.equal(far[0], last[0])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_views_and_in_place(dtype):
    B, T, hq, hk, D = 2, 9, 4, 2, 64
    q, k, wq, wk, cos, sin, pos, gq, gk, nb = inputs((B, T, hq, hk, D, D, False, "same"), dtype)
    kw = dict(positions=pos)
    want = es.qk_norm_rotate(q, k, wq, wk, cos, sin, **kw)
    fused = torch.cat([q, k, k], 2)
    fq, fk = fused[:, :, :hq], fused[:, :, hq:hq + hk]
    got = es.qk_norm_rotate(fq, fk, wq, wk, cos, sin, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    grads = es.qk_norm_rotate_backward(q, k, wq, wk, cos, sin, gq, gk, **kw)
    for x, y in zip(grads, es.qk_norm_rotate_backward(fq, fk, wq, wk, cos, sin, gq, gk, **kw)):
        assert torch.equal(x, y)
    kept = fused[:, :, hq + hk:].clone()
    es.qk_norm_rotate(fq, fk, wq, wk, cos, sin, q_out=fq, k_out=fk, **kw)          # in their own places
    assert torch.equal(fq, want[0]) and torch.equal(fk, want[1]) and torch.equal(fused[:, :, hq + hk:], kept)
    odd = torch.empty(q.numel() + 1, dtype=dtype, device="cuda")[1:].view(q.shape)
    odd.copy_(q)
    got = es.qk_norm_rotate(odd, k, wq, wk, cos, sin, **kw)
    assert (got[0].float() - want[0].float()).abs().max() <= 2.0 ** (-7 if dtype == BF16 else -18) * want[0].float().abs().max()
    hf = q.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(es.qk_norm_rotate(hf, k, wq, wk, cos, sin, **kw)[0], want[0])


def test_rows_of_zeros_and_no_rows():
    q = torch.zeros(1, 3, 2, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    out, none = es.qk_norm_rotate(q, None, w)
    assert none is None and not out.any()
    g = torch.ones_like(q)
    gq, _, gw, _ = es.qk_norm_rotate_backward(q, None, w, None, None, None, g, None, eps=1e-6)
    assert torch.isfinite(gq).all() and not gw.any()
    e = torch.zeros(0, 3, 2, 64, device="cuda")
    gq, _, gw, _ = es.qk_norm_rotate_backward(e, None, w, None, None, None, e, None)
    assert gq.shape == e.shape and not gw.any()


def test_the_same_bits_each_time_and_another_stream():
    q, k, wq, wk, cos, sin, pos, gq, gk, nb = inputs((2, 300, 8, 2, 128, 128, False, "same"), BF16)
    first = es.qk_norm_rotate_backward(q, k, wq, wk, cos, sin, gq, gk, positions=pos)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    again = es.qk_norm_rotate_backward(q, k, wq, wk, cos, sin, gq, gk, positions=pos, stream=s)
    s.synchronize()
    for x, y in zip(first, again):
        assert torch.equal(x, y)


def test_autograd_of_both_together():
    """Norm and rotation feeding linear attention, as a layer runs them, against the oracles' chain."""
    from element_scan_recurrences_gb300 import autograd as ag
    rng = np.random.default_rng(4)
    B, T, H, D = 2, 40, 2, 32
    q, k, v, go = (made(rng, B, T, H, D).requires_grad_(i < 3) for i in range(4))
    wq, wk = (made(rng, D).requires_grad_(True) for _ in range(2))
    g = (-torch.from_numpy(rng.uniform(0, 0.3, (B, T, H)).astype(np.float32)).cuda()).requires_grad_(True)
    ang = rng.uniform(0, 6.3, (T, D // 2))
    cos, sin = (torch.from_numpy(f(ang).astype(np.float32)).cuda() for f in (np.cos, np.sin))
    rq, rk = ag.qk_norm_rotate(q, k, wq, wk, cos, sin)
    out, _ = ag.linear_attention(rq, rk, v, g)
    (out * go).sum().backward()
    nq, nk = (A.norm_rotate(num(x.detach()), num(w.detach()), num(cos), num(sin)) for x, w in ((q, wq), (k, wk)))
    want = A.linear_attention_backward(nq, nk, num(v.detach()), num(g.detach()), num(go), scale=D ** -0.5)
    gq, gwq = A.norm_rotate_backward(num(q.detach()), num(wq.detach()), num(cos), num(sin), want[0])
    gk, gwk = A.norm_rotate_backward(num(k.detach()), num(wk.detach()), num(cos), num(sin), want[1])
    for x, y in ((q, gq), (k, gk), (v, want[2]), (g, want[3]), (wq, gwq), (wk, gwk)):
        # f32 sums of a few thousand terms of random signs: 2^-24 times their number's root, with room of 64
        assert np.abs(num(x.grad) - y).max() <= 2.0 ** -24 * 64 * 64 * np.abs(y).max()


def test_refusals():
    q, k, wq, wk, cos, sin, pos, gq, gk, nb = inputs((2, 5, 4, 2, 64, 64, False, "same"), BF16)

    def refused(code, *a, **kw):
        with pytest.raises(es.EsError) as e:
            es.qk_norm_rotate(*a, **kw)
        assert e.value.status == code, e.value

    refused(1, q, k[:, :3], wq, wk, cos, sin)
    refused(1, q, k, wq[:32], wk, cos, sin)
    refused(1, q, k, wq, wk, cos, sin, positions=pos[:, :2])
    wide = torch.zeros(4, 40, device="cuda")
    refused(1, q, k, wq, wk, wide, wide)                   # 80 values of 64
    refused(3, q, k, wq, wk, cos, sin, eps=-1.0)
    refused(3, q, k, wq, wk, cos, sin, q_out=torch.empty_like(q)[:, :1].expand_as(q))
    refused(3, q, q, wq, wk, cos, sin, k_out=q[:, :, :], q_out=q)
    huge = torch.zeros(1, 1, 1, 257, device="cuda")
    refused(4, huge, None)
    for bad in (dict(q=q.half()), dict(k=k.float()), dict(q_weight=wq.float()), dict(cos=cos.double()),
                dict(positions=pos.float()), dict(sin=None)):
        with pytest.raises((TypeError, es.EsError)):
            es.qk_norm_rotate(**{**dict(q=q, k=k, q_weight=wq, k_weight=wk, cos=cos, sin=sin), **bad})
