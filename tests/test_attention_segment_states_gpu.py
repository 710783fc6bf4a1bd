"""Linear attention in segments of several chunks on the tensor cores: each
segment's own state is gathered with two chunks in turn, by warps of which
those past the value columns (values narrower than 128) have nothing to do and
run ahead.  Decays so mild that every segment's first tokens live on the
states of the segments before.

Tolerances, relative to the whole tensor: a bf16 result is rounded by 2^-9 to
2^-8 of itself, all else (factors kept to 2^-16) is far below: 2^-8.  A state is
rounded by 2^-24 at most twice a chunk on its way (its decay, its sum), 47
chunks: 2^-17.
"""
import numpy as np
import pytest
import torch

import element_scan_recurrences_gb300 as es
import oracle.attention as A

pytestmark = pytest.mark.gpu

B, T, H = 2, 3000, 4
LENGTHS = [3000, 1700]       # of the forward call


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    es.lib()


def near(got, want, tol, what):
    got = got.double().cpu().numpy()
    far = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert far <= tol, "%s: %.2e of the whole" % (what, far)


@pytest.mark.parametrize("widths", [(64, 64), (128, 64), (64, 8), (64, 96), (96, 80), (64, 128)], ids=str)
def test_states_of_several_chunks(widths):
    dk, dv = widths
    rng = np.random.default_rng(dk + dv)
    made = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
    q, k, v, go = made(B, T, H, dk).bfloat16(), made(B, T, H, dk).bfloat16(), made(B, T, H, dv).bfloat16(), made(B, T, H, dv).bfloat16()
    init, gfin = made(B, H, dk, dv), made(B, H, dk, dv)
    g = torch.from_numpy(-rng.uniform(0, 0.01, (B, T, H)).astype(np.float32)).cuda()
    n = torch.tensor(LENGTHS, dtype=torch.int32, device="cuda")
    # segments of several chunks, both ways
    for backward, runs in ((False, 1), (True, 3)):
        plan = es.plan_linear_attention(q.shape, k.shape, v.shape, decay="token" if not backward else None, heads=H,
                                        lengths=not backward, state=True, backward=backward)
        segments = plan["workspace"] // (4 * runs * B * H * dk * dv)
        assert plan["path"] == "tensor" and 2 <= segments <= 47 // 2
    scale = dk ** -0.5
    out, fin = es.linear_attention(q, k, v, g, initial_state=init, lengths=n, scale=scale, final_state=True)
    grads = es.linear_attention_backward(q, k, v, g, go, initial_state=init, grad_final_state=gfin, scale=scale,
                                         decay_grad=False)
    es.device_status()
    num = [x.double().cpu().numpy() for x in (q, k, v, g, go, init, gfin)]
    wout, wfin = A.linear_attention(*num[:4], num[5], lengths=LENGTHS, scale=scale)
    near(out, wout, 2.0 ** -8, "out")
    near(fin, wfin, 2.0 ** -17, "state")
    want = A.linear_attention_backward(*num, scale=scale)
    for i, (name, tol) in enumerate((("gq", 2.0 ** -8), ("gk", 2.0 ** -8), ("gv", 2.0 ** -8), ("gg", None), ("gi", 2.0 ** -17))):
        if tol is not None:
            near(grads[i], want[i], tol, name)
    # the same bits each time
    for _ in range(3):
        again, _ = es.linear_attention(q, k, v, g, initial_state=init, lengths=n, scale=scale, final_state=True)
        assert torch.equal(again, out)
        more = es.linear_attention_backward(q, k, v, g, go, initial_state=init, grad_final_state=gfin, scale=scale,
                                            decay_grad=False)
        assert all(torch.equal(x, y) for x, y in zip((*more[:3], more[4]), (*grads[:3], grads[4])))
