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
