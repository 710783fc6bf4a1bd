"""The selective scan without channels through the C ABI, without a GPU: the gradients
of b and c have elements all the same, and are checked like other results."""
import pytest

import element_scan_recurrences_gb300 as es

NONE = (2, 100, 0)


@pytest.fixture(scope="module", autouse=True)
def built():
    from element_scan_recurrences_gb300 import build
    build.build()


def test_plans():
    for backward in (False, True):
        p = es.plan_selective_scan(NONE, 16, groups=3, backward=backward)
        assert (p["elements"], p["path"], p["workspace"], p["checkpoints"]) == (0, "empty", 0, 0)


@pytest.mark.parametrize("kw,code", [
    (dict(ptrs={"grad_b": 0}), 3), (dict(ptrs={"grad_c": (90 << 44) + 1}), 3),
    (dict(strides={"grad_b": (1600, 0, 16)}), 3), (dict(strides={"grad_c": (0, 16, 16)}), 3),
    (dict(ptrs={"grad_b": 90 << 44, "grad_c": (90 << 44) + 64}), 3),          # over one another
    (dict(groups=1 << 31), 4), (dict(groups=1 << 32), 4), (dict(shape=(1 << 20, 1 << 20, 0), groups=1 << 8), 4),
])
def test_refusals(kw, code):
    with pytest.raises(es.EsError) as e:
        es.plan_selective_scan(**{**dict(shape=NONE, states=16, backward=True), **kw})
    assert e.value.status == code, e.value
