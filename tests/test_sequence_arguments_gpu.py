"""Arguments of the sequence-layer operators at the edge of what they take."""
import numpy as np
import pytest
import torch

import element_scan_recurrences_gb300 as es

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    es.lib()


def test_flags_without_a_truth_value():
    """The object's own exception comes through."""
    x, many = torch.zeros(1, 4, 2, 64, device="cuda"), np.array([1, 2])
    for call in (lambda: es.linear_attention(x, x, x, final_state=many),
                 lambda: es.linear_attention_backward(x, x, x, None, x, decay_grad=many),
                 lambda: es.qk_norm_rotate(x, x, neighbours=many)):
        with pytest.raises(ValueError):
            call()
    assert es.linear_attention(x, x, x, final_state=1)[1].shape == (1, 2, 64, 64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_weights_of_no_heads_get_zeros(dtype):
    """Keys (or queries) without heads: their weight's gradient is a sum of nothing."""
    x, none = torch.randn(2, 5, 3, 64, device="cuda").to(dtype), torch.zeros(2, 5, 0, 64, dtype=dtype, device="cuda")
    w, u = torch.rand(64, device="cuda").to(dtype), torch.rand(64, device="cuda").to(dtype)
    want = es.qk_norm_rotate_backward(x, None, w, None, None, None, x, None)
    got = es.qk_norm_rotate_backward(x, none, w, u, None, None, x, none)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2]) and got[1].shape == none.shape and not got[3].any()
    got = es.qk_norm_rotate_backward(none, x, u, w, None, None, none, x)
    assert torch.equal(got[1], want[0]) and torch.equal(got[3], want[2]) and not got[2].any()
    got = es.qk_norm_rotate_backward(none, none, u, w, None, None, none, none)
    assert not got[2].any() and not got[3].any()
    es.device_status()
