"""The sequence operators together as a layer trains and serves with them
(examples/sequence_layer.py), bounded waits in the tensor-core pipeline, and
offsets that pass 32 bits."""
import os
import sys

import numpy as np
import pytest
import torch

import element_scan_recurrences_gb300 as es
import oracle.attention as A

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def restore():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    es.set_drop_tile(-1)
    es.set_wait_limit_ns(2_000_000_000)
    es.set_path_override("auto")


def test_layer_learns_and_serves():
    """The loss of a repetition falls from that of guessing (ln 32 = 3.5) to
    under half of it, and single tokens predict what the whole sequence
    predicts: both round q, k, v and the results to bf16 (2^-8), so logits of
    256 terms agree to 2^-5 of the largest."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import sequence_layer
    losses, far, right = sequence_layer.main(150)
    assert losses[0] > 3.0 and losses[-1] < 0.5 * losses[0], (losses[0], losses[-1])
    assert far <= 2.0 ** -5, far
    assert right > 0.5


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("T", [200, 3000])
def test_a_tile_that_never_arrives(backward, T):
    """The pipeline gives up after the wait limit, reports it, and the next
    call is right (T = 3000 with two heads runs in segments of one chunk)."""
    rng = np.random.default_rng(0)
    q, k, v, go = (torch.from_numpy(rng.standard_normal((1, T, 2, 64)).astype(np.float32)).bfloat16().cuda() for _ in range(4))
    g = -torch.rand(1, T, 2, device="cuda") * 0.2

    def run():
        if backward:
            return es.linear_attention_backward(q, k, v, g, go)
        return es.linear_attention(q, k, v, g, final_state=True)

    want = run()
    es.device_status()
    es.set_wait_limit_ns(20_000_000)
    es.set_drop_tile(0)
    run()
    with pytest.raises(es.EsError) as e:
        es.device_status()
    assert e.value.status == 6
    es.device_status()
    es.set_drop_tile(-1)
    es.set_wait_limit_ns(2_000_000_000)
    got = run()
    es.device_status()
    for x, y in zip(got, want):
        assert (x is None and y is None) or torch.equal(x, y)


@pytest.mark.parametrize("path", ["auto", "generic"])
def test_offsets_past_32_bits_attention(path):
    """More than 2^32 bytes (and 2^31 elements) an operand.  The decays leave
    nothing of tokens 512 back (e^-256), so the last tokens are those of a
    short sequence."""
    es.set_path_override(path)
    T, H, D = 64 * 2100, 256, 64
    gen = torch.Generator(device="cuda").manual_seed(0)
    q, k, v = (torch.empty(1, T, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    assert q.numel() > 2 ** 31
    for x in (q, k, v):
        x.normal_(generator=gen)
    g = torch.full((1, T, H), -0.5, device="cuda")
    out, state = es.linear_attention(q, k, v, g, final_state=True)
    near = slice(T - 1024, T)
    wout, wstate = es.linear_attention(q[:, near].contiguous(), k[:, near].contiguous(), v[:, near].contiguous(),
                                       g[:, near].contiguous(), final_state=True)
    es.device_status()
    # the same chunks in the same order: what differs is at most e^-256 of the sums
    assert torch.equal(out[:, T - 512:], wout[:, 512:])
    assert (state - wstate).abs().max() <= 2.0 ** -20 * wstate.abs().max()
    for h in (0, 255):
        args = [x[:, T - 64:, h:h + 1].double().cpu().numpy() for x in (q, k, v)]
        want, _ = A.linear_attention(*args, np.full((1, 64, 1), -0.5), scale=D ** -0.5)
        # the 32 tokens left out before these leave e^-16 of the sums at the last 32
        got = out[:, T - 32:, h:h + 1].double().cpu().numpy()
        assert np.abs(got - want[:, 32:]).max() <= 2.0 ** -6 * np.abs(want).max()


def test_offsets_past_32_bits_rotation():
    T, H, D = 70000, 256, 128
    q = torch.empty(1, T, H, D, dtype=torch.bfloat16, device="cuda").normal_()
    assert q.numel() > 2 ** 31
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    ang = torch.rand(128, D // 2, device="cuda") * 6
    cos, sin = ang.cos(), ang.sin()
    pos = torch.randint(0, 128, (1, T), device="cuda")
    got, _ = es.qk_norm_rotate(q, None, w, None, cos, sin, positions=pos)
    gx, _, gw, _ = es.qk_norm_rotate_backward(q, None, w, None, cos, sin, got, None, positions=pos)
    last = slice(T - 40, T)
    want, _ = es.qk_norm_rotate(q[:, last].contiguous(), None, w, None, cos, sin, positions=pos[:, last].contiguous())
    wx, _, _, _ = es.qk_norm_rotate_backward(q[:, last].contiguous(), None, w, None, cos, sin, want, None,
                                             positions=pos[:, last].contiguous())
    assert torch.equal(got[:, last], want) and torch.equal(gx[:, last], wx)
