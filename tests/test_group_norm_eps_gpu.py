"""The group norm's gradients at an eps of zero and others, on rows that do not fill a
block: a team of threads without a row of its own adds nothing to the weights' sums.

Tolerances as in test_group_norm_gpu.py, with the eps of the call."""
import numpy as np
import pytest
import torch

import element_scan_recurrences_gb300 as es
import oracle.state_space as S
from test_group_norm_gpu import BF16, F32, Case, close, num, top

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    es.lib()


def check(c, eps):
    out, grads = es.group_norm(*c.args(), eps=eps, **c.kw), es.group_norm_backward(*c.args(), c.go, eps=eps, **c.kw)
    es.device_status()
    x, w, b, z = args = tuple(num(t) for t in c.args())
    first = c.kw["gate_first"]
    u = x * S.silu(z) if first else x
    v = u - u.mean(-1, keepdims=True) if c.kw["center"] else u
    inv = 1 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    r, n, wide = 1 + top(u) * inv, np.abs(v) * inv, np.abs(w).max()
    want = S.group_norm(*args, **c.okw, eps=eps)
    close(out, want, 128 * r * top(want), "out")
    gx, gw, gb, gz = S.group_norm_backward(*args, num(c.go), **c.okw, eps=eps)
    rows = c.x.shape[0] * c.x.shape[1]
    gy = np.abs(num(c.go)) * (1 if z is None else 1 + np.abs(z)) * (1 + np.abs(b))
    close(grads[0], gx, 256 * r * inv * wide * top(gy * (1 + n)) * (top(z) + 1 if first else 1), "gx")
    close(grads[1], gw, (rows + 256) * (gy * (r + n)).sum((0, 1)), "gw")
    close(grads[2], gb, (rows + 256) * (gy * r).sum((0, 1)), "gb")
    if z is not None:
        close(grads[3], gz, 256 * r * top(gy) * (1 + top(n) * wide) * (1 + top(z)) * (inv * (1 + top(x)) * wide if first else 1), "ggate")


OPTIONS = [dict(), dict(first=True), dict(center=False), dict(first=True, center=False), dict(gate=False), dict(gate=False, act=True),
           dict(gate=False, act=True, center=False)]


# 1e-50 is 0 in f32
@pytest.mark.parametrize("eps", [0.0, 1e-50, 0.25])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kw", OPTIONS, ids=str)
def test_rows_that_do_not_fill_a_block(eps, dtype, kw):
    for shape in ((1, 3, 1, 64), (1, 1, 1, 128), (2, 7, 3, 80), (1, 33, 2, 33), (1, 3, 2, 1000)):
        check(Case(dtype, *shape, seed=20, **kw), eps)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_that_end_in_a_later_turn(dtype):
    """Teams that had rows and have none in the last turn, beside teams that never had one."""
    for T in (40, 9000, 20011):
        check(Case(dtype, 1, T, 1, 64, seed=21), 0.0)
