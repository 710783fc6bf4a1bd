"""The state-space oracle against differences of its own forward functions and
against hand-made cases (no GPU)."""
import numpy as np
import pytest

import oracle.state_space as S


def differences(f, args, at, h=1e-6):
    """Central differences of the scalar f(*args) with respect to args[at]."""
    x = args[at]
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        for s in (1, -1):
            y = x.copy()
            y[i] += s * h
            out[i] += s * f(*args[:at], y, *args[at + 1:]) / (2 * h)
    return out


def matches(got, want):
    np.testing.assert_allclose(got, want, rtol=2e-6, atol=2e-7 * max(1.0, np.abs(want).max()))


@pytest.mark.parametrize("act,lengths", [(True, None), (False, [3, 1])])
def test_conv_gradients(act, lengths):
    rng = np.random.default_rng(0)
    x, w, b, init = rng.standard_normal((2, 5, 3)), rng.standard_normal((3, 4)), rng.standard_normal(3), rng.standard_normal((2, 3, 3))
    go, gs = rng.standard_normal(x.shape), rng.standard_normal(init.shape)

    def loss(x, w, b, init):
        out, last = S.causal_conv(x, w, b, init, lengths, act)
        return (out * go).sum() + (last * gs).sum()

    got = S.causal_conv_backward(x, w, b, go, init, gs, lengths, act)
    for i, g in enumerate(got):
        matches(g, differences(loss, (x, w, b, init), i))


@pytest.mark.parametrize("soft,lengths,gated", [(True, None, True), (False, [4, 2], True), (True, [1, 4], False)])
def test_scan_gradients(soft, lengths, gated):
    rng = np.random.default_rng(1)
    B, T, C, N, G = 2, 4, 4, 3, 2
    n = rng.standard_normal
    args = [n((B, T, C)), n((B, T, C)) * 0.3 + (0 if soft else 0.5), -np.abs(n((C, N))), n((B, T, G, N)), n((B, T, G, N)), n(C),
            n((B, T, C)), n(C) * 0.1, n((B, C, N))]
    go, gs = n((B, T, C)), n((B, C, N))

    def loss(x, delta, A, Bm, Cm, D, gate, bias, init):
        out, last = S.selective_scan(x, delta, A, Bm, Cm, D, gate if gated else None, bias, soft, init, lengths)
        return (out * go).sum() + (last * gs).sum()

    got = S.selective_scan_backward(*args[:6], args[6] if gated else None, args[7], go, soft, args[8], gs, lengths)
    for i, g in enumerate(got):
        matches(g, differences(loss, args, i))


@pytest.mark.parametrize("first,center,act", [(False, True, False), (True, False, False), (True, True, False), (False, False, True),
                                              (False, True, True)])
def test_norm_gradients(first, center, act):
    rng = np.random.default_rng(2)
    n = rng.standard_normal
    args = [n((2, 3, 2, 5)), n((2, 5)), n((2, 5)), n((2, 3, 2, 5))]
    go = n(args[0].shape)

    def loss(x, w, b, gate):
        return (S.group_norm(x, w, b, None if act else gate, first, center, act) * go).sum()

    got = S.group_norm_backward(*args[:3], None if act else args[3], go, first, center, act)
    for i, g in enumerate(got):
        if g is not None:
            matches(g, differences(loss, args, i))


def test_scan_by_hand():
    """One channel, one state: h = e^-d h + d x b, twice."""
    out, last = S.selective_scan([[[2.0], [4.0]]], [[[1.0], [0.5]]], [[-1.0]], [[[[1.0]], [[3.0]]]], [[[[1.0]], [[10.0]]]], soft=False)
    h = 2.0
    h2 = np.exp(-0.5) * h + 0.5 * 4 * 3
    np.testing.assert_allclose(out.ravel(), [2.0, 10 * h2])
    np.testing.assert_allclose(last.ravel(), [h2])


def test_conv_by_hand():
    out, last = S.causal_conv([[[1.0], [2.0], [3.0]]], [[10.0, 1.0]], [0.5], [[[7.0]]], act=False)
    np.testing.assert_allclose(out.ravel(), [71.5, 12.5, 23.5])
    np.testing.assert_allclose(last.ravel(), [3.0])
    # a row shorter than the taps keeps carried inputs
    _, last = S.causal_conv(np.ones((1, 3, 1)), np.ones((1, 4)), None, np.arange(3.0).reshape(1, 3, 1), lengths=[1])
    np.testing.assert_allclose(last.ravel(), [1, 2, 1])
