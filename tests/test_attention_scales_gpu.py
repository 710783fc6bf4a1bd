"""Linear attention at scales far from one.  The states that a call takes and
gives are the ones that it computes with, so no scale's reciprocal is needed
and none of them leaves f32's range while the results are in it.

Tolerances, relative to the whole tensor against 64 bits: bf16 results 2^-8
(their rounding); their f32 companions and f32 results 2^-18 (as many roundings
of 2^-24 as in a plain call, random in direction), bf16 inputs' decay gradient
2^-14 (factors kept to 2^-17, eight times that).  Each value may be off by
2^-126 besides, f32's smallest normal number.
"""
import numpy as np
import pytest
import torch

import element_scan_recurrences_gb300 as es
import oracle.attention as A

pytestmark = pytest.mark.gpu

B, T, H, D = 1, 130, 2, 64


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    es.lib()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e-39, 1e-38, -0.3, 1e30])
def test_scale(scale, dtype):
    rng = np.random.default_rng(5)
    made = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
    q, k, v, go = (made(B, T, H, D).to(dtype) for _ in range(4))
    init, gfin = made(B, H, D, D), 100 * made(B, H, D, D)
    g = torch.from_numpy(-rng.uniform(0, 0.02, (B, T, H)).astype(np.float32)).cuda()
    out, fin = es.linear_attention(q, k, v, g, initial_state=init, scale=scale, final_state=True)
    grads = es.linear_attention_backward(q, k, v, g, go, initial_state=init, grad_final_state=gfin, scale=scale)
    es.device_status()
    num = [x.double().cpu().numpy() for x in (q, k, v, g, go, init, gfin)]
    s = float(np.float32(scale))
    want = A.linear_attention(*num[:4], num[5], scale=s) + A.linear_attention_backward(*num, scale=s)
    for name, x, y in zip(("out", "state", "gq", "gk", "gv", "gg", "gi"), (out, fin, *grads), want):
        off = np.maximum(np.abs(x.double().cpu().numpy() - y) - 2.0 ** -126, 0.0)
        tol = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -14 if name == "gg" and dtype == torch.bfloat16 else 2.0 ** -18
        # (a tensor of numbers that f32 hardly holds is held by the floor alone)
        assert np.linalg.norm(off) <= tol * np.linalg.norm(y), (name, np.linalg.norm(off) / np.linalg.norm(y))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_a_state_s_gradient_goes_through_unchanged(dtype):
    """No decay, nothing written: the first state's gradient is the last one's, bit for bit, at any scale."""
    z = torch.zeros(1, 100, 2, D, dtype=dtype, device="cuda")
    gfin = torch.randn(1, 2, D, D, device="cuda")
    for scale in (0.3, 1e-3, 7.0):
        grads = es.linear_attention_backward(z, z, z, None, z, initial_state=torch.zeros_like(gfin), grad_final_state=gfin, scale=scale)
        assert torch.equal(grads[4], gfin)
    es.device_status()
