"""How far the selective scan's states, results and gradients drift from 64 bits over
rows that remember hundreds of tokens, and how precise its functions are.

In units of 2^-24 of the value.  The hardware's 2^q is off by 0.7 at random (root mean
square) and low in the mean, by 0.24 about q = -0.0047; the kernels put that mean back.  A
state that loses a fraction 1 / M a token keeps the errors of about M of them: the random
ones, with the rounding of the state's own sum (0.41), add up to sqrt((0.7^2 + 0.41^2) M /
2), what is left of the mean to M times it.  With steps of 1 to 1.3 and decays q = -0.0041
to -0.0054 a token M is some 300, the random part 10 units, and a mean left 0.05 of a unit
off 15; exponents, steps and factors round some 6 times.  So 2 x 10 + 15 + 6, here 42
units, holds for the whole tensor (root of the sum of squares) where all values have one
sign.  The mean left in is 72, one put back by 0.37 whatever q is 40 beside the 10.  In a
gradient with respect to A both the state and its gradient have it: 84 units."""
import numpy as np
import pytest
import torch

import element_scan_recurrences_gb300 as es
import oracle.state_space as S

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
UNIT = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    es.lib()


def num(t):
    return t.double().cpu().numpy()


def far(got, want):
    """Units of 2^-24 between two tensors, relative, whole."""
    return float(np.linalg.norm((num(got) - want).ravel()) / np.linalg.norm(want.ravel()) / UNIT)


def weak(dtype, T, C=64, N=16, B=1, seed=0):
    """x, delta, A, B, C and gradients of positive values; steps of 1 to 1.3 with e^(d A) from 1 - 1/353 to 1 - 1/266."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    u = lambda lo, hi, *s: lo + (hi - lo) * torch.rand(s, generator=gen, device="cuda")  # noqa: E731
    x, delta, go = u(0.5, 1.5, B, T, C).to(dtype), u(1.0, 1.3, B, T, C).to(dtype), u(0.5, 1.5, B, T, C).to(dtype)
    b, c = u(0.5, 1.5, B, T, 1, N).to(dtype), u(0.5, 1.5, B, T, 1, N).to(dtype)
    a = -u(0.00284, 0.0029, C, N)
    assert float(a.max()) * np.log2(np.e) * 1.0 < -2.0 ** -8      # every decay below the size where the mean is another
    return (x, delta, a, b, c, None, None, None), go


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_long_prompt(dtype):
    args, go = weak(dtype, 2048)
    out, state, _ = es.selective_scan(*args, softplus=False, final_state=True)
    grads = es.selective_scan_backward(*args, go, softplus=False)
    es.device_status()
    plain = [None if t is None else num(t) for t in args]
    want_out, want = S.selective_scan(*plain, soft=False)
    assert far(state, want) <= 42
    g = S.selective_scan_backward(*plain, num(go), soft=False)
    assert far(grads[2], g[2]) <= 84, "grad_A"
    if dtype == F32:
        for i, name in ((0, "grad_x"), (3, "grad_B"), (4, "grad_C")):
            assert far(grads[i], g[i]) <= 42, name
        assert far(out, want_out) <= 42


def in_tiles(args, state):
    """The prompt a tile of 16 tokens at a time, the state carried: no segments."""
    for t in range(0, args[0].shape[1], 16):
        cut = [v[:, t:t + 16] if v is not None and v.dim() > 2 else v for v in args]
        es.selective_scan(*cut, softplus=False, initial_state=state, final_state=state)
    return state


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N", [16, 5])
def test_a_prompt_in_tiles(dtype, N):
    args, _ = weak(dtype, 2048, C=40, N=N, B=2, seed=1)
    state = in_tiles(args, torch.zeros(2, 40, N, device="cuda"))
    want = S.selective_scan(*(None if v is None else num(v) for v in args), soft=False)[1]
    assert far(state, want) <= 42


def tokens(args, state):
    """... and one by one."""
    x, delta, a, b, c = args[:5]
    for t in range(x.shape[1]):
        es.selective_scan_step(x[:, t], delta[:, t], a, b[:, t], c[:, t], None, None, None, state, softplus=False)
    return state


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N", [16, 5])
def test_single_tokens(dtype, N):
    """Served token by token, a state is as near 64 bits as a prompt's.  Where the steps of
    each tile are alike they are the same bits (the same sums in the same order)."""
    args, _ = weak(dtype, 2048, C=40, N=N, B=2, seed=1)
    state = tokens(args, torch.zeros(2, 40, N, device="cuda"))
    want = S.selective_scan(*(None if v is None else num(v) for v in args), soft=False)[1]
    assert far(state, want) <= 42
    alike = args[1][:, ::16].repeat_interleave(16, 1)
    args = (args[0], alike) + args[2:]
    assert torch.equal(tokens(args, torch.zeros(2, 40, N, device="cuda")), in_tiles(args, torch.zeros(2, 40, N, device="cuda")))


def test_no_decay_keeps_every_bit():
    """A = 0: states are the sums of their inputs, here whole numbers, exactly, however
    long the row, on the prompt's way and token by token; the tokens that a block past a
    row's end still takes leave a state as it is."""
    T, C, N = 4099, 8, 4
    one = torch.ones(1, T, C, device="cuda")
    two = torch.ones(1, T, 1, N, device="cuda")
    zero = torch.zeros(C, N, device="cuda")
    out, state, _ = es.selective_scan(one, one, zero, two, two, softplus=False, final_state=True)
    assert torch.equal(state, torch.full((1, C, N), float(T), device="cuda"))
    assert torch.equal(out[0, :, 0], N * torch.arange(1, T + 1, device="cuda").float())
    step = torch.full((1, C, N), 2.0 ** 22, device="cuda")
    for t in range(64):
        es.selective_scan_step(one[:, 0], one[:, 0], zero, two[:, 0], two[:, 0], None, None, None, step, softplus=False)
    assert torch.equal(step, torch.full_like(step, 2.0 ** 22 + 64))
    # one live token and seven that take no step
    weak_a = torch.full((C, N), -2.0 ** -8, device="cuda")
    first = torch.rand(1, C, N, device="cuda")
    alone = es.selective_scan(one[:, :1], one[:, :1], weak_a, two[:, :1], two[:, :1], softplus=False, initial_state=first, final_state=True)[1]
    token = first.clone()
    es.selective_scan_step(one[:, 0], one[:, 0], weak_a, two[:, 0], two[:, 0], None, None, None, token, softplus=False)
    assert torch.equal(alone, token)


def test_steps_and_gates_pointwise():
    """log(1 + e^x) and z / (1 + e^-z) over a dense range, one state and one token.  Where
    it counts, log(1 + e^x) is the exponential (2^-22) times a polynomial (1.3e-7, 2.2
    units), with three roundings: 4 + 2.2 + 3 units, here 10.  The gate is an exponential
    (4), a sum, a reciprocal (2^-23, 2) and three products: 4 + 0.5 + 2 + 1.5, here 9.  An
    exponent rounded without its correction costs up to 40 units of e^-80."""
    n = 1 << 16
    x = torch.linspace(-85.0, 40.0, n, device="cuda").view(1, 1, n)
    one, two = torch.ones_like(x), torch.ones(1, 1, 1, 1, device="cuda")
    zero = torch.zeros(n, 1, device="cuda")
    steps = num(es.selective_scan(one, x, zero, two, two)[0]).ravel()
    token = torch.zeros(1, n, 1, device="cuda")
    single = num(es.selective_scan_step(one[0], x[0], zero, two[0], two[0], None, None, None, token)[0]).ravel()
    want = S.softplus(num(x)).ravel()
    for got in (steps, single):
        assert (np.abs(got - want) <= 10 * UNIT * want).all(), float(np.max(np.abs(got - want) / want) / UNIT)
    gates = num(es.selective_scan(one, one, zero, two, two, gate=x, softplus=False)[0]).ravel()
    token.zero_()
    single = num(es.selective_scan_step(one[0], one[0], zero, two[0], two[0], None, x[0], None, token, softplus=False)[0]).ravel()
    want = S.silu(num(x)).ravel()
    for got in (gates, single):
        assert (np.abs(got - want) <= 9 * UNIT * np.abs(want)).all()
