"""The sequence-layer operators: linear attention with a decay for each head
(chunked for prompts and training, recurrent for single tokens) and the norm
of queries and keys with the position rotation; the short causal convolution,
the selective scan (each for prompts, training and single tokens) and the group
norm with a gate.

Thin wrappers like ``binding``'s (``include/es.h`` holds the contract): tensors
are CUDA tensors in float32 or bfloat16, any strides with an innermost stride
of 1; calls are asynchronous on ``stream`` (a ``torch.cuda.Stream`` or a
handle; default: PyTorch's current stream of the tensors' device); results and
workspaces that are not passed in are allocated by PyTorch on that stream.
Every refusal is an ``EsError`` with the library's message, or a ``TypeError``
for a tensor of the wrong kind.  There is no CPU fallback.

The marshalling is native (``csrc/torch/es_torch.cpp``, built beside
libes.so): in Python it would take several times as long as a single token's
kernel.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import struct
import threading
from typing import Optional, Union

import torch

from . import binding
from . import build as _build
from .binding import EsError, LibraryMissing, PATHS, _check

# The structs of include/es.h, in its order: every field is 64 bits wide (for the plans, which take no tensors)
_ATTN = struct.Struct("6qd20q5q5q")
_ATTN_GRADS = struct.Struct("20q3q")
_ROTATE = struct.Struct("7qd20q4q5q2q")
_ROTATE_GRADS = struct.Struct("10q2q")
_CONV = struct.Struct("7q6q7q")
_CONV_GRADS = struct.Struct("6q4q")
_SCAN = struct.Struct("7q12q10q10q")
_SCAN_GRADS = struct.Struct("12q10q5q")
_NORM = struct.Struct("8qd15q4q")
_NORM_GRADS = struct.Struct("15q2q")

_lock = threading.Lock()
_native_module = None


def _native():
    """The marshalling module (loaded on first use)."""
    global _native_module
    if _native_module is None:
        with _lock:
            if _native_module is None:
                if not os.path.exists(_build.TORCH_LIB):
                    raise LibraryMissing("es_torch.so is not built (%s); run __graft_entry__.build() first" % _build.TORCH_LIB)
                binding.lib()
                loader = importlib.machinery.ExtensionFileLoader("es_torch", _build.TORCH_LIB)
                m = importlib.util.module_from_spec(importlib.util.spec_from_loader("es_torch", loader))
                loader.exec_module(m)
                m.set_error(EsError)
                _native_module = m
    return _native_module


def linear_attention(q, k, v, log_decay=None, initial_state=None, lengths=None, scale: Optional[float] = None,
                     final_state: Union[bool, torch.Tensor] = False, out=None, workspace=None, stream=None):
    """Linear attention over whole sequences: for each batch row and head

        h[t] = exp(g[t]) * h[t-1] + k[t] v[t]^T,    out[t] = scale * q[t] h[t]

    q [B, T, Hq, Dk], k [B, T, Hk, Dk], v [B, T, Hv, Dv]; ``log_decay`` g (f32)
    [B, T, H], or [H] for one fixed value a head, or None; each of Hq, Hk, Hv
    divides H (the largest of them without decays).  ``initial_state`` f32
    [B, H, Dk, Dv]; ``lengths`` int32 [B]: tokens past a row's length are not
    read and give zeros.  ``scale`` defaults to Dk ** -0.5.  Returns (out
    [B, T, H, Dv], the last state or None); ``final_state`` is True, or the
    tensor to write it to (which may be ``initial_state``).
    """
    return (_native_module or _native()).linear_attention(q, k, v, log_decay, initial_state, lengths, scale, final_state, out,
                                                          workspace, stream)


def linear_attention_backward(q, k, v, log_decay, grad_out, initial_state=None, grad_final_state=None, lengths=None,
                              scale: Optional[float] = None, decay_grad: bool = True, workspace=None, stream=None):
    """Gradients of ``linear_attention``: (grad_q, grad_k, grad_v,
    grad_log_decay or None, grad_initial_state or None).

    ``grad_out`` [B, T, H, Dv] in q's dtype, ``grad_final_state`` f32 or None.
    Shared operand heads get the sum over the heads that read them, a fixed
    decay the sum over batch and tokens.  ``decay_grad`` False leaves the
    decays' gradient out (and its cost).
    """
    return (_native_module or _native()).linear_attention_backward(q, k, v, log_decay, grad_out, initial_state,
                                                                   grad_final_state, lengths, scale, decay_grad, workspace,
                                                                   stream)


def linear_attention_step(q, k, v, log_decay, state, state_out=None, scale: Optional[float] = None, out=None, stream=None):
    """One token of each batch row: q [B, Hq, Dk], k [B, Hk, Dk], v [B, Hv,
    Dv], ``log_decay`` [B, H] or [H] or None, ``state`` f32 [B, H, Dk, Dv].
    Returns (out [B, H, Dv], the new state): ``state`` itself, updated in
    place, unless ``state_out`` is given."""
    return (_native_module or _native()).linear_attention_step(q, k, v, log_decay, state, state_out, scale, out, stream)


def _stand_in(shape, k):
    """(data, strides, heads) of a dense view at a stand-in address."""
    b, t, h, d = shape
    return ((k + 1) << 44, t * h * d, h * d, d, h)


def plan_linear_attention(q_shape, k_shape, v_shape, dtype="bf16", decay=None, heads=None, lengths=False, state=False,
                          backward=False, scale=1.0, strides=None, ptrs=None) -> dict:
    """Validate and plan a call without a GPU (pure host logic).  ``decay``:
    "token", "head" or None; ``heads``: H (default: the largest); ``ptrs`` and
    ``strides`` ({"q": ...}) replace the dense stand-ins of q, k, v, out."""
    B, T = q_shape[:2]
    dk, dv = q_shape[3], v_shape[3]
    H = max(q_shape[2], k_shape[2], v_shape[2]) if heads is None else heads
    shapes = {"q": q_shape, "k": k_shape, "v": v_shape, "out": (B, T, H, dv)}
    views = {}
    for i, n in enumerate(("q", "k", "v", "out")):
        f = list(_stand_in(shapes[n], i))
        if ptrs and n in ptrs:
            f[0] = ptrs[n]
        if strides and n in strides:
            f[1:4] = strides[n]
        views[n] = f
    g = {None: (0, 0, 0, 0, 0), "token": (5 << 44, T * H, H, 1, 0), "head": (5 << 44, 0, 0, 1, 1)}[decay]
    args = _ATTN.pack({"f32": 0, "bf16": 1}.get(dtype, 9), B, T, H, dk, dv, scale, *views["q"], *views["k"], *views["v"],
                      *views["out"], *g, (6 << 44) if lengths else 0, (7 << 44) if state else 0, (8 << 44) if state else 0,
                      0, 0)
    grads = None
    if backward:
        grads = _ATTN_GRADS.pack(*_stand_in((B, T, H, dv), 9), *_stand_in(q_shape, 10), *_stand_in(k_shape, 11),
                                 *_stand_in(v_shape, 12), (14 << 44) if state else 0, (15 << 44) if decay else 0,
                                 (16 << 44) if state else 0)
    info, n = binding.PlanInfo(), ctypes.c_size_t()
    L = binding.lib()
    _check(L.es_plan_linear_attention(args, grads, ctypes.byref(info)))
    _check(L.es_linear_attention_workspace(args, grads, ctypes.byref(n)))
    return {"O": info.O, "T": info.T, "J": info.J, "W": info.W, "elements": info.elements, "path": PATHS[info.path],
            "workspace": n.value}


def qk_norm_rotate(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, eps: float = 1e-6,
                   neighbours: bool = False, q_out=None, k_out=None, stream=None):
    """Norm of each head's query and key, then the position rotation, in one
    pass: x / sqrt(mean(x^2) + eps) * w, with pairs of the first R values
    turned by the angles of the token's position.

    q [B, T, Hq, D], k [B, T, Hk, D] or None; weights [D] (float32 or bfloat16)
    or None; ``cos``, ``sin`` f32 [rows, R / 2] (None: no rotation);
    ``positions`` int32 or int64 [B, T] or [T] (None: 0, 1, ...), clamped to
    the tables.  ``neighbours``: values 2i and 2i+1 pair, else i and i + R/2.
    Returns (q, k) results, new tensors unless ``q_out`` / ``k_out`` are given
    (they may be q and k themselves)."""
    return (_native_module or _native()).qk_norm_rotate(q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours, q_out,
                                                        k_out, stream)


def qk_norm_rotate_backward(q, k, q_weight, k_weight, cos, sin, grad_q_out, grad_k_out, positions=None,
                            eps: float = 1e-6, neighbours: bool = False, workspace=None, stream=None):
    """Gradients of ``qk_norm_rotate``: (grad_q, grad_k, grad_q_weight,
    grad_k_weight), None where there is no operand."""
    return (_native_module or _native()).qk_norm_rotate_backward(q, k, q_weight, k_weight, cos, sin, positions, eps,
                                                                 neighbours, grad_q_out, grad_k_out, workspace, stream)


def causal_conv(x, weight, bias=None, initial_state=None, lengths=None, activation: bool = True,
                final_state: Union[bool, torch.Tensor] = False, out=None, stream=None):
    """The short causal convolution of each channel:

        p[t] = bias + sum_j weight[:, j] * x[t - W + 1 + j],    out = p / (1 + exp(-p))

    (or p, without ``activation``).  x [B, T, C]; ``weight`` [C, W], W 2..8, and
    ``bias`` [C] in one dtype; ``initial_state`` [B, W - 1, C] in x's dtype: the
    inputs before the first token, oldest first (None: zeros); ``lengths`` int32
    [B]: tokens past a row's length are not read and give zeros.  Returns (out,
    the last W - 1 inputs or None); ``final_state`` is True, or the tensor to
    write them to (which may be ``initial_state``).
    """
    return (_native_module or _native()).causal_conv(x, weight, bias, initial_state, lengths, activation, final_state, out, stream)


def causal_conv_backward(x, weight, bias, grad_out, initial_state=None, grad_final_state=None, lengths=None,
                         activation: bool = True, workspace=None, stream=None):
    """Gradients of ``causal_conv``: (grad_x, grad_weight, grad_bias or None,
    grad_initial_state or None)."""
    return (_native_module or _native()).causal_conv_backward(x, weight, bias, grad_out, initial_state, grad_final_state,
                                                              lengths, activation, workspace, stream)


def causal_conv_step(x, weight, bias, state, state_out=None, activation: bool = True, out=None, stream=None):
    """One token of each batch row: x [B, C], ``state`` [B, W - 1, C].  Returns
    (out [B, C], the new state): ``state`` itself, updated in place, unless
    ``state_out`` is given."""
    return (_native_module or _native()).causal_conv_step(x, weight, bias, state, state_out, activation, out, stream)


def selective_scan(x, delta, A, B, C, D=None, gate=None, delta_bias=None, softplus: bool = True, initial_state=None,
                   lengths=None, final_state: Union[bool, torch.Tensor] = False,
                   checkpoints: Union[bool, torch.Tensor] = False, out=None, workspace=None, stream=None):
    """The selective state-space scan: for each channel c, with N states,

        d[t] = log(1 + exp(delta[t] + delta_bias))
        h[t] = exp(d[t] * A[c]) * h[t-1] + d[t] * x[t] * B[t]
        out[t] = (C[t] . h[t] + D[c] * x[t]) * gate[t] / (1 + exp(-gate[t]))

    (d the sum itself without ``softplus``, with it 0 for a delta of -inf; no
    last factor without ``gate``).  x, delta, gate [B, T, channels]; A
    [channels, N] f32, N 1..64, meant to be negative; B, C [B, T, groups, N],
    the groups dividing the channels; D, ``delta_bias`` f32 [channels];
    ``initial_state`` f32 [B, channels, N]; ``lengths`` int32 [B]: tokens past a
    row's length are not read and give zeros.  Returns (out, the last state or
    None, checkpoints or None).
    ``final_state`` is True, or the tensor to write it to (which may be
    ``initial_state``); ``checkpoints`` likewise: states on the way, which
    ``selective_scan_backward`` of the same operands takes.
    """
    return (_native_module or _native()).selective_scan(x, delta, A, B, C, D, gate, delta_bias, softplus, initial_state,
                                                        lengths, final_state, checkpoints, out, workspace, stream)


def selective_scan_backward(x, delta, A, B, C, D, gate, delta_bias, grad_out, softplus: bool = True, initial_state=None,
                            grad_final_state=None, lengths=None, checkpoints=None, workspace=None, stream=None):
    """Gradients of ``selective_scan``: (grad_x, grad_delta, grad_A, grad_B,
    grad_C, grad_D, grad_gate, grad_delta_bias, grad_initial_state), None where
    there is no operand.  Without ``checkpoints`` the states on the way are
    found again first."""
    return (_native_module or _native()).selective_scan_backward(x, delta, A, B, C, D, gate, delta_bias, grad_out, softplus,
                                                                 initial_state, grad_final_state, lengths, checkpoints,
                                                                 workspace, stream)


def selective_scan_step(x, delta, A, B, C, D, gate, delta_bias, state, softplus: bool = True, state_out=None, out=None,
                        stream=None):
    """One token of each batch row: x, delta, gate [B, channels], B, C [B,
    groups, N], ``state`` f32 [B, channels, N].  Returns (out [B, channels], the
    new state): ``state`` itself, updated in place, unless ``state_out`` is
    given."""
    return (_native_module or _native()).selective_scan_step(x, delta, A, B, C, D, gate, delta_bias, state, softplus,
                                                             state_out, out, stream)


def group_norm(x, weight=None, bias=None, gate=None, gate_first: bool = False, center: bool = True, activation: bool = False,
               eps: float = 1e-5, out=None, stream=None):
    """The norm of each group (head) of a token's channels, with a gate: for x
    [B, T, H, D], s(z) = z / (1 + exp(-z)),

        (u - mean(u)) / sqrt(var(u) + eps) * weight + bias,   u = x

    times s(gate), or with ``gate_first`` for u = x * s(gate); without
    ``center`` u / sqrt(mean(u^2) + eps).  ``weight``, ``bias`` [H, D] in one
    dtype, or None; without a gate, ``activation`` makes y into s(y).  D
    1..8192."""
    return (_native_module or _native()).group_norm(x, weight, bias, gate, gate_first, center, activation, eps, out, stream)[0]


def group_norm_backward(x, weight, bias, gate, grad_out, gate_first: bool = False, center: bool = True,
                        activation: bool = False, eps: float = 1e-5, workspace=None, stream=None):
    """Gradients of ``group_norm``: (grad_x, grad_weight, grad_bias,
    grad_gate), None where there is no operand."""
    return (_native_module or _native()).group_norm_backward(x, weight, bias, gate, gate_first, center, activation, eps,
                                                             grad_out, workspace, stream)


_DTYPES = {"f32": 0, "bf16": 1}


def _planned(op: str, args: bytes, grads: Optional[bytes]) -> dict:
    info, n = binding.PlanInfo(), ctypes.c_size_t()
    L = binding.lib()
    _check(getattr(L, "es_plan_" + op)(args, grads, ctypes.byref(info)))
    _check(getattr(L, "es_%s_workspace" % op)(args, grads, ctypes.byref(n)))
    return {"O": info.O, "T": info.T, "J": info.J, "W": info.W, "elements": info.elements, "path": PATHS[info.path],
            "workspace": n.value}


class _Places:
    """Stand-in addresses and dense views of a plan's operands; ``ptrs`` and
    ``strides`` (by name) replace them."""

    def __init__(self, ptrs, strides):
        self.ptrs, self.strides, self.count = ptrs or {}, strides or {}, 0

    def at(self, name, there=True):
        self.count += 1
        return self.ptrs.get(name, self.count << 44 if there else 0)

    def rows(self, name, shape, there=True):
        b, t, c = shape
        return (self.at(name, there),) + tuple(self.strides.get(name, (t * c, c)))

    def heads(self, name, shape, there=True):
        b, t, h, d = shape
        return (self.at(name, there),) + tuple(self.strides.get(name, (t * h * d, h * d, d))) + (h,)


def plan_causal_conv(shape, taps: int, dtype="bf16", weight_dtype=None, bias=True, lengths=False, state=False, backward=False,
                     ptrs=None, strides=None) -> dict:
    """Validate and plan a call without a GPU (pure host logic): x's ``shape``
    [B, T, C]; ``ptrs`` and ``strides`` ({"x": ...}) replace dense stand-ins."""
    p = _Places(ptrs, strides)
    b, t, c = shape
    args = _CONV.pack(_DTYPES.get(dtype, 9), _DTYPES.get(weight_dtype or dtype, 9), b, t, c, taps, 1, *p.rows("x", shape),
                      *p.rows("out", shape), p.at("weight"), p.at("bias", bias), p.at("lengths", lengths),
                      p.at("initial_state", state), p.at("final_state", state and not backward), p.at("workspace", False),
                      1 << 50)
    grads = None
    if backward:
        grads = _CONV_GRADS.pack(*p.rows("grad_out", shape), *p.rows("grad_x", shape), p.at("grad_weight"),
                                 p.at("grad_bias", bias), p.at("grad_final_state", state), p.at("grad_initial_state", state))
    return _planned("causal_conv", args, grads)


def plan_selective_scan(shape, states: int, groups: int = 1, dtype="bf16", gate=True, skip=True, delta_bias=True, lengths=False,
                        state=False, checkpoints=False, backward=False, ptrs=None, strides=None) -> dict:
    """Validate and plan a call without a GPU, as ``plan_causal_conv``; the
    result also holds the bytes of its "checkpoints"."""
    p = _Places(ptrs, strides)
    b, t, c = shape
    bc = (b, t, groups, states)
    args = _SCAN.pack(_DTYPES.get(dtype, 9), b, t, c, states, groups, 1, *p.rows("x", shape), *p.rows("delta", shape),
                      *p.rows("gate", shape, gate), *p.rows("out", shape), *p.heads("b", bc), *p.heads("c", bc), p.at("a"),
                      p.at("skip", skip), p.at("delta_bias", delta_bias), p.at("lengths", lengths), p.at("initial_state", state),
                      p.at("final_state", state and not backward), p.at("checkpoints", checkpoints), 1 << 50,
                      p.at("workspace", False), 1 << 50)
    grads = None
    if backward:
        grads = _SCAN_GRADS.pack(*p.rows("grad_out", shape), *p.rows("grad_x", shape), *p.rows("grad_delta", shape),
                                 *p.rows("grad_gate", shape, gate), *p.heads("grad_b", bc), *p.heads("grad_c", bc),
                                 p.at("grad_a"), p.at("grad_skip", skip), p.at("grad_delta_bias", delta_bias),
                                 p.at("grad_final_state", state), p.at("grad_initial_state", state))
    plan = _planned("selective_scan", args, grads)
    n = ctypes.c_size_t()
    _check(binding.lib().es_selective_scan_checkpoints(args, ctypes.byref(n)))
    plan["checkpoints"] = n.value
    return plan


def plan_group_norm(shape, dtype="bf16", weight_dtype=None, weight=True, bias=True, gate=True, gate_first=False, center=True,
                    activation=False, eps=1e-5, backward=False, ptrs=None, strides=None) -> dict:
    """Validate and plan a call without a GPU, as ``plan_causal_conv``: x's
    ``shape`` is [B, T, H, D]."""
    p = _Places(ptrs, strides)
    b, t, h, d = shape
    args = _NORM.pack(_DTYPES.get(dtype, 9), _DTYPES.get(weight_dtype or dtype, 9), b, t, d, center, gate_first, activation, eps,
                      *p.heads("x", shape), *p.heads("gate", shape, gate), *p.heads("out", shape), p.at("weight", weight),
                      p.at("bias", bias), p.at("workspace", False), 1 << 50)
    grads = None
    if backward:
        grads = _NORM_GRADS.pack(*p.heads("grad_out", shape), *p.heads("grad_x", shape), *p.heads("grad_gate", shape, gate),
                                 p.at("grad_weight", weight), p.at("grad_bias", bias))
    return _planned("group_norm", args, grads)
