"""Tokens that forget strongly among tokens that hardly do: decays of e^-20 to
e^-100, which leave nothing of what was before but are no zeros in f32.  The
sum of a chunk's log decays passes 1000 while the weights that count lie
between tokens a few hundredths apart; what the sum loses there may not reach
them.

Tolerances, relative to the whole tensor against 64 bits; none grows with the
decays.  f32: a result is a sum with some 150 roundings of 2^-24 in random
directions, sqrt(150) = 12 of them, 2^-20.  The decays' gradient sums
differences of such terms over a block; errors of one part in n of the terms
come out as up to 8 in n of this gradient (the same sums with random errors of
that size put in), and the terms are good to 2^-21: 2^-18.  bf16 results: their
rounding, 2^-8.  Their decays' gradient is f32 and comes of factors kept to
2^-17, eight times that: 2^-14.  A state is rounded twice a chunk: 2^-18.
Each value may be off by 2^-126 besides, f32's smallest normal number: the first
state's gradient after a first token of -100 is 1e-43.
"""
import numpy as np
import pytest
import torch

import element_scan_recurrences_gb300 as es
import oracle.attention as A

pytestmark = pytest.mark.gpu

B, T, H, D = 1, 200, 2, 64


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    es.lib()


def decays(strong, pattern, rng):
    """Half of the tokens at random, or 24 of every 32 in a row."""
    which = rng.random((B, T, H)) < 0.5 if pattern == "random" else np.broadcast_to(np.arange(T)[None, :, None] % 32 < 24, (B, T, H))
    return np.where(which, strong, -0.04 * rng.random((B, T, H))).astype(np.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("strong,pattern", [(-20.0, "random"), (-60.0, "random"), (-100.0, "random"), (-100.0, "row")], ids=str)
def test_small_decays_after_strong_ones(strong, pattern, dtype):
    rng = np.random.default_rng(3)
    made = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
    q, k, v, go = (made(B, T, H, D).to(dtype) for _ in range(4))
    init, gfin = made(B, H, D, D), made(B, H, D, D)
    g = torch.from_numpy(decays(strong, pattern, rng)).cuda()
    scale = D ** -0.5
    out, fin = es.linear_attention(q, k, v, g, initial_state=init, scale=scale, final_state=True)
    grads = es.linear_attention_backward(q, k, v, g, go, initial_state=init, grad_final_state=gfin, scale=scale)
    es.device_status()
    num = [x.double().cpu().numpy() for x in (q, k, v, g, go, init, gfin)]
    want = A.linear_attention(*num[:4], num[5], scale=scale) + A.linear_attention_backward(*num, scale=scale)
    far = {}
    for name, x, y in zip(("out", "state", "gq", "gk", "gv", "gg", "gi"), (out, fin, *grads), want):
        off = np.maximum(np.abs(x.double().cpu().numpy() - y) - 2.0 ** -126, 0.0)
        far[name] = np.linalg.norm(off) / np.linalg.norm(y)
    if dtype == torch.float32:
        tol = dict.fromkeys(far, 2.0 ** -20)
        tol["gg"] = 2.0 ** -18
    else:
        tol = dict.fromkeys(far, 2.0 ** -8)
        tol.update(state=2.0 ** -18, gi=2.0 ** -18, gg=2.0 ** -14)
    assert all(far[n] <= tol[n] for n in far), {n: "%.1e of %.1e" % (far[n], tol[n]) for n in far}
