"""The decays' gradient over rows of several blocks (256 tokens each, between
kept states), held to its own size, and the results beside it.

Tolerances, relative to the whole tensor against 64 bits.  f32: a result is a
sum with some 150 roundings of 2^-24 in random directions, sqrt(150) = 12 of
them, 2^-20.  A token's decay gradient sums differences of such terms within a
block, and meets products of states at both of its ends; errors of one part in
n of the terms come out as up to 8 in n, and the terms are good to 2^-21: 2^-18.
bf16 results: their rounding, 2^-8; their decays' gradient is f32 and comes of
factors kept to 2^-17, eight times that: 2^-14.  A fixed decay's gradient adds
all tokens', whose signs cancel: its size may be an eighth of what random signs
leave, so eight times the token's tolerance, 2^-15 and 2^-11.  States: 2^-17 (two
roundings of 2^-24 a chunk).  Zeros, a block with its sign turned or without its
states, or a token of a row left out, are far outside all of these.
"""
import numpy as np
import pytest
import torch

import element_scan_recurrences_gb300 as es
import oracle.attention as A

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
SAME = (2, 2, 2, 2)
CASES = [
    # B, T, heads (q, k, v, H), dk, dv, decay, carry, lengths
    (1, 1100, (1, 1, 2, 2), 64, 64, "token", True, None),
    (2, 900, SAME, 64, 32, "token", False, [900, 300]),
    (2, 1030, (1, 2, 1, 2), 128, 64, "token", True, [513, 1030]),
    (2, 1300, (4, 4, 4, 4), 128, 128, "token", True, [1300, 1024]),
    (1, 2600, (1, 1, 1, 1), 32, 32, "token", True, None),
    (1, 1500, SAME, 64, 64, "head", True, None),
    (3, 600, SAME, 40, 24, "head", False, [600, 257, 0]),
    (2, 700, (1, 1, 4, 4), 64, 64, "head", False, None),
    (1, 520, SAME, 33, 17, "token", True, [515]),
]


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


def inputs(case, dtype, seed=0):
    B, T, (hq, hk, hv, H), dk, dv, decay, carry, lengths = case
    rng = np.random.default_rng(seed)
    made = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
    q, k, v, go = made(B, T, hq, dk).to(dtype), made(B, T, hk, dk).to(dtype), made(B, T, hv, dv).to(dtype), made(B, T, H, dv).to(dtype)
    g = torch.from_numpy(-rng.uniform(0, 0.1, (B, T, H) if decay == "token" else H).astype(np.float32)).cuda()
    init, gfin = (made(B, H, dk, dv), made(B, H, dk, dv)) if carry else (None, None)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    return q, k, v, g, go, init, gfin, n


def numpy(t):
    return None if t is None else t.double().cpu().numpy()


def far(x, y):
    return np.linalg.norm(numpy(x) - y) / np.linalg.norm(y)


def check(case, dtype):
    q, k, v, g, go, init, gfin, n = inputs(case, dtype)
    scale = case[3] ** -0.5
    kw = dict(lengths=numpy(n), scale=scale, heads=case[2][3])
    out, fin = es.linear_attention(q, k, v, g, initial_state=init, lengths=n, scale=scale, final_state=True)
    grads = es.linear_attention_backward(q, k, v, g, go, initial_state=init, grad_final_state=gfin, lengths=n, scale=scale)
    es.device_status()
    want = A.linear_attention(*map(numpy, (q, k, v, g, init)), **kw)
    want += A.linear_attention_backward(*map(numpy, (q, k, v, g, go, init, gfin)), **kw)
    token = 2.0 ** -18 if dtype == F32 else 2.0 ** -14
    tol = dict.fromkeys(("out", "gq", "gk", "gv"), 2.0 ** -20 if dtype == F32 else 2.0 ** -8)
    tol.update(state=2.0 ** -17, gi=2.0 ** -17, gg=token if case[5] == "token" else 8 * token)
    off = {name: far(x, y) for name, x, y in zip(("out", "state", "gq", "gk", "gv", "gg", "gi"), (out, fin, *grads), want)
           if x is not None}
    assert all(off[name] <= tol[name] for name in off), {name: "%.1e of %.1e" % (off[name], tol[name]) for name in off}
    for b, length in enumerate(case[7] or []):
        if case[5] == "token":
            assert not grads[3][b, length:].any()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_gradients_over_several_blocks(case, dtype):
    check(case, dtype)


@pytest.mark.parametrize("case", [CASES[1], CASES[5]], ids=str)
def test_the_direct_kernel_with_bf16(case):
    es.set_path_override("generic")
    check(case, BF16)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", [(1, 600, SAME, 32, 32, "token", True, [520]), (2, 600, SAME, 32, 32, "head", False, None)], ids=str)
def test_decay_gradient_against_differences(case, dtype):
    """<gradient, u> against the difference of the 64-bit loss <out, go> +
    <state, gfin> along u: the gradient's tolerance times the sizes, and the
    difference's own error, d^2 / 6 times a third derivative of at most 10^4
    times the slope's size (memories of 20 tokens, cubed)."""
    q, k, v, g, go, init, gfin, n = inputs(case, dtype, seed=7)
    scale = case[3] ** -0.5
    grads = es.linear_attention_backward(q, k, v, g, go, initial_state=init, grad_final_state=gfin, lengths=n, scale=scale)
    gg = numpy(grads[3])
    u = np.random.default_rng(8).standard_normal(gg.shape)
    goz = numpy(go).copy()
    for b, length in enumerate(case[7] or []):
        goz[b, length:] = 0

    def loss(s):
        out, fin = A.linear_attention(*map(numpy, (q, k, v)), numpy(g) + s * u, numpy(init), lengths=numpy(n), scale=scale, heads=2)
        return float((out * goz).sum()) + (0.0 if gfin is None else float((fin * numpy(gfin)).sum()))

    d = 1e-4
    size = np.linalg.norm(gg) * np.linalg.norm(u)
    tol = (2.0 ** -18 if dtype == F32 else 2.0 ** -14) * (1 if case[5] == "token" else 8) + d * d / 6 * 1e4
    assert abs((loss(d) - loss(-d)) / (2 * d) - float((gg * u).sum())) <= tol * size
