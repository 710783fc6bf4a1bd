"""The 64-bit oracle of linear attention and of the query/key norm with
rotation: hand-worked values, and its gradients against central differences
(no GPU)."""
import numpy as np
import pytest

import oracle.attention as A


def test_hand_worked_two_tokens():
    q = np.array([1.0, 2.0]).reshape(1, 2, 1, 1)
    k = np.array([3.0, 4.0]).reshape(1, 2, 1, 1)
    v = np.array([5.0, 6.0]).reshape(1, 2, 1, 1)
    g = np.log(np.array([0.5, 0.25])).reshape(1, 2, 1)
    out, state = A.linear_attention(q, k, v, g, np.full((1, 1, 1, 1), 8.0), scale=0.5)
    # h = 0.5 * 8 + 15 = 19, then 0.25 * 19 + 24 = 28.75
    assert np.allclose(out.reshape(-1), [9.5, 28.75]) and np.allclose(state, 28.75)
    out, state = A.linear_attention(q, k, v, g, np.full((1, 1, 1, 1), 8.0), lengths=[1], scale=0.5)
    assert np.allclose(out.reshape(-1), [9.5, 0.0]) and np.allclose(state, 19.0)


def test_a_token_that_starts_afresh():
    rng = np.random.default_rng(0)
    q, k, v = (rng.standard_normal((1, 5, 2, 3)) for _ in range(3))
    g = -rng.uniform(0, 1, (1, 5, 2))
    g[0, 3] = -np.inf
    out, state = A.linear_attention(q, k, v, g, rng.standard_normal((1, 2, 3, 3)))
    late, last = A.linear_attention(q[:, 3:], k[:, 3:], v[:, 3:], g[:, 3:], None)
    assert np.allclose(out[:, 3:], late) and np.allclose(state, last)


@pytest.mark.parametrize("per_head,heads", [(False, (2, 2, 2)), (True, (4, 2, 1)), (False, (1, 4, 2))])
def test_gradients_against_differences(per_head, heads):
    rng = np.random.default_rng(1)
    B, T, H, dk, dv = 2, 6, max(heads), 3, 4
    x = {"q": rng.standard_normal((B, T, heads[0], dk)), "k": rng.standard_normal((B, T, heads[1], dk)),
         "v": rng.standard_normal((B, T, heads[2], dv)),
         "g": -rng.uniform(0, 1, (H,) if per_head else (B, T, H)), "i": rng.standard_normal((B, H, dk, dv))}
    go, gf = rng.standard_normal((B, T, H, dv)), rng.standard_normal((B, H, dk, dv))
    lengths = [T, 4]

    def loss(x):
        o, s = A.linear_attention(x["q"], x["k"], x["v"], x["g"], x["i"], lengths, 0.7)
        return float((o * go).sum() + (s * gf).sum())

    got = dict(zip(("q", "k", "v", "g", "i"), A.linear_attention_backward(x["q"], x["k"], x["v"], x["g"], go, x["i"], gf,
                                                                         lengths, 0.7)))
    for n in x:
        for at in [tuple(rng.integers(0, s) for s in x[n].shape) for _ in range(12)]:
            d = 1e-5
            up, down = ({m: y.copy() for m, y in x.items()} for _ in range(2))
            up[n][at] += d
            down[n][at] -= d
            # central differences: error of order d^2 and 1e-16 / d
            assert abs((loss(up) - loss(down)) / (2 * d) - got[n][at]) < 1e-6 * (1 + abs(got[n][at])), (n, at)


@pytest.mark.parametrize("neighbours", [False, True])
def test_norm_rotate_gradients_against_differences(neighbours):
    rng = np.random.default_rng(2)
    B, T, H, D, R = 2, 3, 2, 6, 4
    x, w, go = rng.standard_normal((B, T, H, D)), rng.standard_normal(D), rng.standard_normal((B, T, H, D))
    ang = rng.uniform(0, 6, (5, R // 2))
    pos = rng.integers(-2, 9, (B, T))
    f = lambda x, w: float((A.norm_rotate(x, w, np.cos(ang), np.sin(ang), pos, 1e-3, neighbours) * go).sum())  # noqa: E731
    gx, gw = A.norm_rotate_backward(x, w, np.cos(ang), np.sin(ang), go, pos, 1e-3, neighbours)
    d = 1e-5
    for _ in range(20):
        at, c = tuple(rng.integers(0, s) for s in x.shape), int(rng.integers(0, D))
        e, u = np.zeros_like(x), np.zeros_like(w)
        e[at], u[c] = d, d
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * d) - gx[at]) < 1e-6 * (1 + abs(gx[at]))
        assert abs((f(x, w + u) - f(x, w - u)) / (2 * d) - gw[c]) < 1e-6 * (1 + abs(gw[c]))


def test_rotation_keeps_length_and_undoes():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((1, 4, 1, 8))
    ang = rng.uniform(0, 6, (4, 4))
    y = A.norm_rotate(x, None, np.cos(ang), np.sin(ang), eps=0.0)
    assert np.allclose((y * y).mean(-1), 1.0)
    back = A.norm_rotate(y, None, np.cos(ang), -np.sin(ang), eps=0.0)
    assert np.allclose(back, x / np.sqrt((x * x).mean(-1, keepdims=True)))
