"""CPU oracle of the state-space layer's operators in 64 bits (numpy): the short
causal convolution, the selective scan and the gated group norm, from the
definitions token by token, with the gradients from the recurrences run
backwards.  Test infrastructure; the library never imports it.

``magnitude=True`` takes every factor by its absolute value: what a rounding
error of one part in n of each term can add up to.
"""
from __future__ import annotations

import numpy as np


def wide(x):
    return None if x is None else np.asarray(x, np.float64)


def logistic(z):
    return np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))


def silu(z):
    return z * logistic(z)


def slope(z):
    """The derivative of silu."""
    s = logistic(z)
    return s + z * s * (1 - s)


def _lengths(lengths, B, T):
    return np.full(B, T) if lengths is None else np.clip(np.asarray(lengths, np.int64), 0, T)


# ---------------------------------------------------------------------------
# convolution

def _conv_rows(x, init, taps, n):
    """The inputs from the first carried one to token n - 1, row by row."""
    B, _, C = x.shape
    init = np.zeros((B, taps - 1, C)) if init is None else wide(init)
    return [np.concatenate([init[b], x[b, :n[b]]], 0) for b in range(B)]


def causal_conv(x, w, bias=None, init=None, lengths=None, act=True, magnitude=False):
    """(out [B, T, C], the last inputs [B, taps - 1, C])."""
    x, w, bias = wide(x), wide(w), wide(bias)
    B, T, C = x.shape
    taps, n = w.shape[1], _lengths(lengths, B, T)
    out, last = np.zeros((B, T, C)), np.zeros((B, taps - 1, C))
    for b, row in enumerate(_conv_rows(x, init, taps, n)):
        for t in range(n[b]):
            terms = row[t:t + taps].T * w
            p = terms.sum(1) + (0 if bias is None else bias)
            if magnitude:
                size = np.abs(terms).sum(1) + (0 if bias is None else np.abs(bias))
                # silu's slope is at most 1.1, its own roundings are of its value
                out[b, t] = size * 1.1 + np.abs(silu(p)) if act else size
            else:
                out[b, t] = silu(p) if act else p
        last[b] = row[len(row) - (taps - 1):]
    return out, last


def causal_conv_backward(x, w, bias, go, init=None, gfin=None, lengths=None, act=True, magnitude=False):
    """(grad_x, grad_w, grad_bias, grad_init); with `magnitude` bounds of their terms."""
    x, w, bias, go = wide(x), wide(w), wide(bias), wide(go)
    B, T, C = x.shape
    taps, n = w.shape[1], _lengths(lengths, B, T)
    gx, gw, gb, gi = np.zeros_like(x), np.zeros_like(w), np.zeros(C), np.zeros((B, taps - 1, C))
    for b, row in enumerate(_conv_rows(x, init, taps, n)):
        grow = np.zeros_like(row)
        for t in range(n[b]):
            terms = row[t:t + taps].T * w
            p = terms.sum(1) + (0 if bias is None else bias)
            if magnitude:
                size = np.abs(terms).sum(1) + (0 if bias is None else np.abs(bias))
                # the slope's own slope is at most 1/2
                gp = np.abs(go[b, t]) * (0.5 * size + np.abs(slope(p)) + 1 if act else 1)
                grow[t:t + taps] += gp * np.abs(w).T
                gw += gp[:, None] * np.abs(row[t:t + taps]).T
            else:
                gp = go[b, t] * (slope(p) if act else 1)
                grow[t:t + taps] += gp * w.T
                gw += gp[:, None] * row[t:t + taps].T
            gb += gp
        if gfin is not None:
            g = wide(gfin[b])
            grow[len(row) - (taps - 1):] += np.abs(g) if magnitude else g
        gi[b], gx[b, :n[b]] = grow[:taps - 1], grow[taps - 1:]
    return gx, gw, gb, gi


# ---------------------------------------------------------------------------
# selective scan

def _spread(m, C):
    """[groups, N] -> [C, N]: each channel's group."""
    return np.repeat(m, C // m.shape[0], axis=0)


def _fold(m, groups):
    return m.reshape(groups, m.shape[0] // groups, m.shape[1]).sum(1)


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def selective_scan(x, delta, A, Bm, Cm, D=None, gate=None, bias=None, soft=True, init=None, lengths=None, magnitude=False):
    """(out [B, T, C], last state [B, C, N])."""
    x, delta, A, Bm, Cm, D, gate, bias = (wide(v) for v in (x, delta, A, Bm, Cm, D, gate, bias))
    B, T, C = x.shape
    n = _lengths(lengths, B, T)
    state = np.zeros((B, C, A.shape[1])) if init is None else wide(init).copy()
    if magnitude:
        x, Bm, Cm, state = np.abs(x), np.abs(Bm), np.abs(Cm), np.abs(state)
        D = None if D is None else np.abs(D)
    out = np.zeros((B, T, C))
    for b in range(B):
        for t in range(n[b]):
            d = delta[b, t] + (0 if bias is None else bias)
            d = softplus(d) if soft else d
            fade = np.exp(d[:, None] * A)
            state[b] = np.where(fade == 0, 0, fade * state[b]) + ((np.abs(d) if magnitude else d) * x[b, t])[:, None] * _spread(Bm[b, t], C)
            y = (state[b] * _spread(Cm[b, t], C)).sum(1) + (0 if D is None else D * x[b, t])
            if gate is not None:
                y = y * (np.abs(silu(gate[b, t])) if magnitude else silu(gate[b, t]))
            out[b, t] = y
    return out, state


def selective_scan_backward(x, delta, A, Bm, Cm, D, gate, bias, go, soft=True, init=None, gfin=None, lengths=None,
                            magnitude=False):
    """(gx, gdelta, gA, gB, gC, gD, ggate, gbias, ginit)."""
    x, delta, A, Bm, Cm, D, gate, bias, go = (wide(v) for v in (x, delta, A, Bm, Cm, D, gate, bias, go))
    B, T, C = x.shape
    N, groups, n = A.shape[1], Bm.shape[2], _lengths(lengths, B, T)
    m = np.abs if magnitude else (lambda v: v)
    first = np.zeros((B, C, N)) if init is None else m(wide(init))
    x, Bm, Cm, go = m(x), m(Bm), m(Cm), m(go)
    skip = np.zeros(C) if D is None else m(D)
    gx, gdelta, ggate = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
    gA, gD, gbias = np.zeros_like(A), np.zeros(C), np.zeros(C)
    gB, gC = np.zeros_like(Bm), np.zeros_like(Cm)
    ginit = np.zeros((B, C, N)) if gfin is None else m(wide(gfin)).copy()
    for b in range(B):
        raw = delta[b] + (0 if bias is None else bias)
        d = softplus(raw) if soft else raw
        states = [first[b]]
        for t in range(n[b]):
            states.append(np.exp(d[t][:, None] * A) * states[-1] + (m(d[t]) * x[b, t])[:, None] * _spread(Bm[b, t], C))
        dh = ginit[b]
        for t in range(n[b] - 1, -1, -1):
            bm, cm, g = _spread(Bm[b, t], C), _spread(Cm[b, t], C), go[b, t]
            if gate is not None:
                y = (states[t + 1] * cm).sum(1) + skip * x[b, t]
                # in the magnitude run the slope's roundings are of its terms: at most 1 + |z| of them
                ggate[b, t] = g * y * (1 + np.abs(gate[b, t]) if magnitude else slope(gate[b, t]))
                g = g * m(silu(gate[b, t]))
            gC[b, t] = _fold(g[:, None] * states[t + 1], groups)
            gD += g * x[b, t]
            dh = dh + g[:, None] * cm
            gB[b, t] = _fold(dh * (m(d[t]) * x[b, t])[:, None], groups)
            of_b = (dh * bm).sum(1)
            gx[b, t] = of_b * m(d[t]) + g * skip
            fade = np.exp(d[t][:, None] * A)
            u = dh * fade * states[t]
            gA += u * m(d[t])[:, None]
            gd = (u * m(A)).sum(1) + of_b * x[b, t]
            gdelta[b, t] = gd * logistic(raw[t]) if soft else gd
            gbias += gdelta[b, t]
            dh = dh * fade
        ginit[b] = dh
    return gx, gdelta, gA, gB, gC, gD, ggate, gbias, ginit


# ---------------------------------------------------------------------------
# group norm

def group_norm(x, w=None, bias=None, gate=None, first=False, center=True, act=False, eps=1e-5):
    x, w, bias, gate = wide(x), wide(w), wide(bias), wide(gate)
    u = x * silu(gate) if first else x
    u = u - u.mean(-1, keepdims=True) if center else u
    y = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps) * (1 if w is None else w) + (0 if bias is None else bias)
    if gate is not None and not first:
        return y * silu(gate)
    return silu(y) if act else y


def group_norm_backward(x, w, bias, gate, go, first=False, center=True, act=False, eps=1e-5):
    """(gx, gw, gbias, ggate)."""
    x, w, bias, gate, go = wide(x), wide(w), wide(bias), wide(gate), wide(go)
    u = x * silu(gate) if first else x
    u = u - u.mean(-1, keepdims=True) if center else u
    size = np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    n = u / size
    w1 = np.ones(x.shape[-2:]) if w is None else w
    y = n * w1 + (0 if bias is None else bias)
    gy, ggate = go, None
    if gate is not None and not first:
        ggate, gy = go * y * slope(gate), go * silu(gate)
    elif act:
        gy = go * slope(y)
    gw, gb = (gy * n).sum((0, 1)), gy.sum((0, 1))
    gn = gy * w1
    gu = (gn - n * (gn * n).mean(-1, keepdims=True)) / size
    if center:
        gu = gu - gn.mean(-1, keepdims=True) / size
    if first:
        return gu * silu(gate), gw, gb, gu * x * slope(gate)
    return gu, gw, gb, ggate
