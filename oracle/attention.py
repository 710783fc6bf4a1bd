"""CPU oracle of linear attention with a decay for each head and of the
query/key norm with rotation: plain loops over tokens in 64 bits (numpy), from
the definitions, with the gradients from the recurrences run backwards.  Test
infrastructure; the library never imports it.

``magnitude=True`` runs the same sums over absolute values: what a rounding
error of one part in n of each term can add up to.
"""
from __future__ import annotations

import numpy as np


def _expand(x, H):
    """[B, T, heads, D] -> [B, T, H, D], head h reading operand head h // (H / heads)."""
    return np.repeat(x, H // x.shape[2], axis=2)


def _fold(x, heads):
    B, T, H, D = x.shape
    return x.reshape(B, T, heads, H // heads, D).sum(3)


def linear_attention(q, k, v, g, initial=None, lengths=None, scale=1.0, heads=None):
    """(out [B, T, H, Dv], last state [B, H, Dk, Dv]) in 64 bits; ``g`` [B, T, H], [H] or None."""
    B, T = q.shape[:2]
    H = heads if heads is not None else (max(q.shape[2], k.shape[2], v.shape[2]) if g is None else g.shape[-1])
    q, k, v = (_expand(np.asarray(x, np.float64), H) for x in (q, k, v))
    g = np.broadcast_to(np.zeros(H) if g is None else np.asarray(g, np.float64), (B, T, H))
    state = np.zeros((B, H, q.shape[3], v.shape[3])) if initial is None else np.asarray(initial, np.float64).copy()
    out = np.zeros((B, T, H, v.shape[3]))
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        for t in range(n):
            for h in range(H):
                fade = np.exp(g[b, t, h])
                state[b, h] = (0.0 if fade == 0.0 else fade * state[b, h]) + np.outer(k[b, t, h], v[b, t, h])
                out[b, t, h] = scale * (q[b, t, h] @ state[b, h])
    return out, state


def linear_attention_backward(q, k, v, g, grad_out, initial=None, grad_final=None, lengths=None, scale=1.0, heads=None,
                              magnitude=False):
    """(grad_q, grad_k, grad_v, grad_g, grad_initial) in 64 bits.  With
    ``magnitude`` the inputs are taken by absolute value and grad_g is a bound
    of the terms the library's sum of differences takes."""
    if magnitude:
        q, k, v, grad_out = (np.abs(x) for x in (q, k, v, grad_out))
        initial = None if initial is None else np.abs(initial)
        grad_final = None if grad_final is None else np.abs(grad_final)
        scale = abs(scale)
    B, T = q.shape[:2]
    H = heads if heads is not None else (max(q.shape[2], k.shape[2], v.shape[2]) if g is None else g.shape[-1])
    hq, hk, hv = q.shape[2], k.shape[2], v.shape[2]
    q, k, v = (_expand(np.asarray(x, np.float64), H) for x in (q, k, v))
    go = np.asarray(grad_out, np.float64)
    per_head = g is not None and np.ndim(g) == 1
    g = np.broadcast_to(np.zeros(H) if g is None else np.asarray(g, np.float64), (B, T, H))
    dk, dv = q.shape[3], v.shape[3]
    gq, gk, gv, gg = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros((B, T, H))
    gi = np.zeros((B, H, dk, dv))
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        for h in range(H):
            state = np.zeros((dk, dv)) if initial is None else np.asarray(initial[b, h], np.float64)
            states = [state]
            fades = np.exp(g[b, :, h])
            for t in range(n):
                state = (0.0 if fades[t] == 0.0 else fades[t] * state) + np.outer(k[b, t, h], v[b, t, h])
                states.append(state)
            gs = np.zeros((dk, dv)) if grad_final is None else np.asarray(grad_final[b, h], np.float64).copy()
            ends = float((gs * state).sum())
            for t in range(n - 1, -1, -1):
                gq[b, t, h] = scale * (states[t + 1] @ go[b, t, h])
                gs = gs + scale * np.outer(q[b, t, h], go[b, t, h])
                gk[b, t, h] = gs @ v[b, t, h]
                gv[b, t, h] = k[b, t, h] @ gs
                gg[b, t, h] = fades[t] * float((gs * np.where(np.isfinite(states[t]), states[t], 0.0)).sum())
                gs = np.zeros_like(gs) if fades[t] == 0.0 else gs * fades[t]
            if magnitude:
                run = ends
                for t in range(n - 1, -1, -1):
                    run += q[b, t, h] @ gq[b, t, h] + k[b, t, h] @ gk[b, t, h]
                    gg[b, t, h] = run
            gi[b, h] = gs
    if per_head:
        gg = gg.sum((0, 1))
    return _fold(gq, hq), _fold(gk, hk), _fold(gv, hv), gg, gi


def _turn(y, cos, sin, neighbours, sign):
    R = 2 * cos.shape[-1]
    z = y.copy()
    a, b = (y[..., 0:R:2], y[..., 1:R:2]) if neighbours else (y[..., :R // 2], y[..., R // 2:R])
    na, nb = a * cos - sign * b * sin, b * cos + sign * a * sin
    if neighbours:
        z[..., 0:R:2], z[..., 1:R:2] = na, nb
    else:
        z[..., :R // 2], z[..., R // 2:R] = na, nb
    return z


def _angles(x, cos, sin, positions):
    B, T = x.shape[:2]
    pos = np.broadcast_to(np.arange(T) if positions is None else np.asarray(positions), (B, T))
    pos = np.clip(pos, 0, cos.shape[0] - 1)
    return np.asarray(cos, np.float64)[pos][:, :, None], np.asarray(sin, np.float64)[pos][:, :, None]


def norm_rotate(x, w, cos, sin, positions=None, eps=1e-6, neighbours=False):
    """Norm and rotation of one operand [B, T, heads, D] in 64 bits."""
    x = np.asarray(x, np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if w is not None:
        y = y * np.asarray(w, np.float64)
    if cos is None:
        return y
    return _turn(y, *_angles(x, cos, sin, positions), neighbours, 1.0)


def norm_rotate_backward(x, w, cos, sin, grad, positions=None, eps=1e-6, neighbours=False):
    """(gradient of x, gradient of w) in 64 bits."""
    x, z = np.asarray(x, np.float64), np.asarray(grad, np.float64)
    if cos is not None:
        z = _turn(z, *_angles(x, cos, sin, positions), neighbours, -1.0)
    root = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = x / root
    zw = z if w is None else z * np.asarray(w, np.float64)
    return (zw - u * (zw * u).mean(-1, keepdims=True)) / root, (z * u).sum((0, 1, 2))
