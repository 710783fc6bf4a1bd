"""Tokens masked by a step of nothing: delta = -inf gives log(1 + e^-inf) = 0, so the
state stays as it is and no gradient passes; a NaN is not hidden by it."""
import numpy as np
import pytest
import torch

import element_scan_recurrences_gb300 as es
import oracle.state_space as S
from test_selective_scan_gpu import BF16, F32, Case, check_backward, check_forward, num

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    es.lib()


def masked(dtype, B, T, C, N, bias=True):
    c = Case(dtype, B, T, C, N, seed=30, extra=bias)
    gen = torch.Generator(device="cuda").manual_seed(30)
    off = torch.rand(B, T, generator=gen, device="cuda") < 0.4
    off[0, :17] = True                                   # a whole tile from the first token on
    off[-1, -3:] = True
    c.delta[off] = float("-inf")
    return c, off


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,C,N", [(2, 41, 40, 16), (2, 30, 9, 5), (2, 700, 32, 16)])
@pytest.mark.parametrize("bias", [True, False])
def test_prompt_and_gradients(dtype, B, T, C, N, bias):
    c, off = masked(dtype, B, T, C, N, bias)
    check_forward(c)
    g = check_backward(c)
    assert not g[1][off].any()                           # the steps' own gradients
    assert not g[3][off].any()                           # what enters the state there is nothing of B


def test_every_token_masked():
    """No step anywhere: the last state is the first, bit for bit, as its gradient."""
    c = Case(F32, 2, 40, 24, seed=31)
    c.delta.fill_(float("-inf"))
    assert torch.equal(es.selective_scan(*c.args, final_state=True, **c.kw())[1], c.init)
    g = es.selective_scan_backward(*c.args, torch.zeros_like(c.go), grad_final_state=c.gfin, **c.kw())
    assert torch.equal(g[8], c.gfin) and not g[2].any() and not g[7].any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_single_token(dtype):
    c = Case(dtype, 3, 1, 40, 16, seed=32)
    c.delta[1] = float("-inf")
    state = c.init.clone()
    one = [None if t is None else t[:, 0] if t.dim() > 2 else t for t in c.args]
    out, _ = es.selective_scan_step(*one, state)
    check_forward(c, (out[:, None], state))
    assert torch.equal(state[1], c.init[1])


def test_nan_and_far_steps():
    d = torch.tensor([float("nan"), float("-inf"), -3e38, -104.0, -95.0, 3e38], device="cuda").view(1, 1, -1)
    one, two = torch.ones_like(d), torch.ones(1, 1, 1, 1, device="cuda")
    zero = torch.zeros(d.numel(), 1, device="cuda")
    out = num(es.selective_scan(one, d, zero, two, two)[0]).ravel()
    state = torch.zeros(1, d.numel(), 1, device="cuda")
    single = num(es.selective_scan_step(one[0], d[0], zero, two[0], two[0], None, None, None, state)[0]).ravel()
    want = S.softplus(num(d)).ravel()
    for got in (out, single):
        assert np.isnan(got[0]) and got[1] == 0.0
        # results under 2^-126 may be 0
        assert (np.abs(got[1:] - want[1:]) <= 2.0 ** -22 * want[1:] + 2.0 ** -126).all(), got
