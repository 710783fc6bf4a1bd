"""The sequence-layer operators: linear attention with a decay for each head
(chunked for prompts and training, recurrent for single tokens) and the norm
of queries and keys with the position rotation.

A thin marshalling layer over libes.so like ``binding`` (``include/es.h``
holds the contract): tensors are CUDA tensors in float32 or bfloat16, any
strides with an innermost stride of 1; calls are asynchronous on ``stream``
(default: PyTorch's current stream of the tensors' device); results and
workspaces that are not passed in are allocated by PyTorch on that stream.
Every refusal is an ``EsError`` with the library's message, or a ``TypeError``
for a tensor of the wrong kind.  There is no CPU fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import struct
from typing import Optional, Union

import torch

from . import binding
from .binding import EsError, PATHS, _check

_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
# es_linear_attention_args, es_linear_attention_grads, es_qk_norm_rotate_args,
# es_qk_norm_rotate_grads: every field is 64 bits wide
_ATTN = struct.Struct("6qd20q5q5q")
_ATTN_GRADS = struct.Struct("20q3q")
_ROTATE = struct.Struct("7qd20q4q5q2q")
_ROTATE_GRADS = struct.Struct("10q2q")


def _view(t, name, dtype, dev, rank):
    """(data, stride_b, stride_t, stride_h, heads) of a [B, T, heads, dim] or [B, heads, dim] tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype is not dtype or t.get_device() != dev:
        raise TypeError("%s must be a %s tensor on cuda:%d (got %s on %s)" % (name, dtype, dev, t.dtype, t.device))
    s, n = t.stride(), t.shape
    if len(s) != rank:
        raise EsError(1, "E-DIM-001 %s has rank %d, not %d" % (name, len(s), rank))
    if s[-1] != 1 and n[-1] > 1 and t.numel():
        raise EsError(3, "the last axis of %s has stride %d; it must be 1" % (name, s[-1]))
    if rank == 3:
        return (t.data_ptr(), s[0], 0, s[1], n[1])
    return (t.data_ptr(), s[0], s[1], s[2], n[2])


def _plain(t, name, dtype, dev, shape):
    """Address of a dense tensor of one dtype and shape (0 for None)."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise TypeError("%s must be a contiguous %s tensor on cuda:%d" % (name, dtype, dev))
    if t.shape != shape:
        raise EsError(1, "E-DIM-001 %s has shape %s, not %s" % (name, list(t.shape), list(shape)))
    return t.data_ptr()


_raw_stream = torch._C._cuda_getCurrentRawStream       # the current stream's handle, without a Stream object


class _On:
    """The device and stream of a call that names one, or that is not on the
    current device: ``with _On(dev, stream) as handle``.  What is allocated
    inside belongs to that stream."""

    __slots__ = ("dev", "stream", "stack")

    def __init__(self, dev, stream):
        self.dev, self.stream, self.stack = dev, stream, contextlib.ExitStack()

    def __enter__(self):
        self.stack.enter_context(torch.cuda.device(self.dev))
        if self.stream is not None:
            s = self.stream
            if isinstance(s, int):
                s = torch.cuda.ExternalStream(s, device=self.dev)
            self.stack.enter_context(torch.cuda.stream(s))
        return _raw_stream(self.dev)

    def __exit__(self, *exc):
        return self.stack.__exit__(*exc)


def _here(dev, stream):
    """Whether a call runs on the current device and stream, as most do."""
    return stream is None and dev == torch.cuda.current_device()


def _operands(q, k, v, log_decay, step):
    """Check q, k, v and the decays; (dtype, dev, B, T, H, dk, dv, views, decay fields)."""
    if not isinstance(q, torch.Tensor) or q.dtype not in _DTYPES or not q.is_cuda:
        raise TypeError("q must be a float32 or bfloat16 CUDA tensor")
    dtype, dev, rank = q.dtype, q.get_device(), 3 if step else 4
    qv, kv, vv = _view(q, "q", dtype, dev, rank), _view(k, "k", dtype, dev, rank), _view(v, "v", dtype, dev, rank)
    n, nk, nv = q.shape, k.shape, v.shape
    B, T, dk = n[0], 1 if step else n[1], n[-1]
    if nk[0] != B or nv[0] != B or nk[-1] != dk or (not step and (nk[1] != T or nv[1] != T)):
        raise EsError(1, "E-DIM-001 q %s, k %s and v %s do not fit" % (list(n), list(nk), list(nv)))
    H = max(qv[4], kv[4], vv[4])
    decay = (0, 0, 0, 0, 0)
    if log_decay is not None:
        if not isinstance(log_decay, torch.Tensor) or log_decay.dtype is not torch.float32 or log_decay.get_device() != dev:
            raise TypeError("log_decay must be a float32 tensor on cuda:%d" % dev)
        s, m = log_decay.stride(), log_decay.shape
        if len(m) == 1:
            H = m[0]
            decay = (log_decay.data_ptr(), 0, 0, s[0], 1)
        elif len(m) == rank - 1 and m[0] == B and (step or m[1] == T):
            H = m[-1]
            decay = (log_decay.data_ptr(), s[0], 0 if step else s[1], s[-1], 0)
        else:
            raise EsError(1, "E-DIM-001 log_decay %s fits neither %s nor one value a head"
                          % (list(m), list(n[:rank - 2]) + [H]))
    return dtype, dev, B, T, H, dk, nv[-1], (qv, kv, vv), decay


def _pack(dtype, B, T, H, dk, dv, scale, views, out, decay, lengths, init, fin, ws=0, nbytes=0):
    if scale is None:
        scale = dk ** -0.5
    return _ATTN.pack(_DTYPES[dtype], B, T, H, dk, dv, scale, *views[0], *views[1], *views[2], *out, *decay, lengths,
                      init, fin, ws, nbytes)


def _workspace(fn, args, grads, workspace, dev):
    """(tensor or None, arguments with the workspace a call needs)."""
    n = ctypes.c_size_t()
    _check(fn(args, grads, ctypes.byref(n)))
    if workspace is None:
        if n.value == 0:
            return None, args
        workspace = torch.empty(n.value, dtype=torch.uint8, device=dev)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous tensor on cuda:%d" % dev)
    return workspace, args[:-16] + _TAIL.pack(workspace.data_ptr(), workspace.numel() * workspace.element_size())


_TAIL = struct.Struct("2q")


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
    if isinstance(q, torch.Tensor) and q.is_cuda and not _here(q.get_device(), stream):
        with _On(q.get_device(), stream):
            return linear_attention(q, k, v, log_decay, initial_state, lengths, scale, final_state, out, workspace)
    dtype, dev, B, T, H, dk, dv, views, decay = _operands(q, k, v, log_decay, False)
    lens = _plain(lengths, "lengths", torch.int32, dev, (B,))
    shape = (B, H, dk, dv)
    init = _plain(initial_state, "initial_state", torch.float32, dev, shape)
    if out is None:
        out = q.new_empty((B, T, H, dv))
        ov = (out.data_ptr(), T * H * dv, H * dv, dv, H)
    else:
        ov = _view(out, "out", dtype, dev, 4)
        if out.shape != (B, T, H, dv):
            raise EsError(1, "E-DIM-001 out has shape %s, not %s" % (list(out.shape), [B, T, H, dv]))
    fin, finp = None, 0
    if isinstance(final_state, torch.Tensor):
        fin, finp = final_state, _plain(final_state, "final_state", torch.float32, dev, shape)
    elif final_state:
        fin = q.new_empty(shape, dtype=torch.float32)
        finp = fin.data_ptr()
    args = _pack(dtype, B, T, H, dk, dv, scale, views, ov, decay, lens, init, finp)
    L = binding.lib()
    # only long sequences with few heads are cut into segments, which take a workspace
    # (the library refuses a call that needs one and has none)
    if workspace is not None or (T > 384 and B * H <= 76):
        workspace, args = _workspace(L.es_linear_attention_workspace, args, None, workspace, dev)
    _check(L.es_linear_attention(args, _raw_stream(dev)))
    return out, fin


def linear_attention_backward(q, k, v, log_decay, grad_out, initial_state=None, grad_final_state=None, lengths=None,
                              scale: Optional[float] = None, decay_grad: bool = True, workspace=None, stream=None):
    """Gradients of ``linear_attention``: (grad_q, grad_k, grad_v,
    grad_log_decay or None, grad_initial_state or None).

    ``grad_out`` [B, T, H, Dv] in q's dtype, ``grad_final_state`` f32 or None.
    Shared operand heads get the sum over the heads that read them, a fixed
    decay the sum over batch and tokens.  ``decay_grad`` False leaves the
    decays' gradient out (and its cost).
    """
    if isinstance(q, torch.Tensor) and q.is_cuda and not _here(q.get_device(), stream):
        with _On(q.get_device(), stream):
            return linear_attention_backward(q, k, v, log_decay, grad_out, initial_state, grad_final_state, lengths, scale,
                                             decay_grad, workspace)
    dtype, dev, B, T, H, dk, dv, views, decay = _operands(q, k, v, log_decay, False)
    shape = (B, H, dk, dv)
    lens = _plain(lengths, "lengths", torch.int32, dev, (B,))
    init = _plain(initial_state, "initial_state", torch.float32, dev, shape)
    gfin = _plain(grad_final_state, "grad_final_state", torch.float32, dev, shape)
    gov = _view(grad_out, "grad_out", dtype, dev, 4)
    if grad_out.shape != (B, T, H, dv):
        raise EsError(1, "E-DIM-001 grad_out has shape %s, not %s" % (list(grad_out.shape), [B, T, H, dv]))
    L = binding.lib()
    gq, gk, gv = q.new_empty(q.shape), q.new_empty(k.shape), q.new_empty(v.shape)
    gg = q.new_empty(log_decay.shape, dtype=torch.float32) if log_decay is not None and decay_grad else None
    gi = q.new_empty(shape, dtype=torch.float32) if initial_state is not None else None
    args = _pack(dtype, B, T, H, dk, dv, scale, views, (0, 0, 0, 0, 0), decay, lens, init, 0)
    hq, hk, hv = views[0][4], views[1][4], views[2][4]
    grads = _ATTN_GRADS.pack(*gov, gq.data_ptr(), T * hq * dk, hq * dk, dk, hq, gk.data_ptr(), T * hk * dk, hk * dk, dk, hk,
                             gv.data_ptr(), T * hv * dv, hv * dv, dv, hv, gfin, 0 if gg is None else gg.data_ptr(),
                             0 if gi is None else gi.data_ptr())
    workspace, args = _workspace(L.es_linear_attention_workspace, args, grads, workspace, dev)
    _check(L.es_linear_attention_backward(args, grads, _raw_stream(dev)))
    return gq, gk, gv, gg, gi


def linear_attention_step(q, k, v, log_decay, state, state_out=None, scale: Optional[float] = None, out=None, stream=None):
    """One token of each batch row: q [B, Hq, Dk], k [B, Hk, Dk], v [B, Hv,
    Dv], ``log_decay`` [B, H] or [H] or None, ``state`` f32 [B, H, Dk, Dv].
    Returns (out [B, H, Dv], the new state): ``state`` itself, updated in
    place, unless ``state_out`` is given."""
    if isinstance(q, torch.Tensor) and q.is_cuda and not _here(q.get_device(), stream):
        with _On(q.get_device(), stream):
            return linear_attention_step(q, k, v, log_decay, state, state_out, scale, out)
    dtype, dev, B, _, H, dk, dv, views, decay = _operands(q, k, v, log_decay, True)
    shape = (B, H, dk, dv)
    if state is None:
        raise TypeError("state must be a float32 tensor")
    init = _plain(state, "state", torch.float32, dev, shape)
    if state_out is None:
        state_out, fin = state, init
    else:
        fin = _plain(state_out, "state_out", torch.float32, dev, shape)
    if out is None:
        out = q.new_empty((B, H, dv))
        ov = (out.data_ptr(), H * dv, 0, dv, H)
    else:
        ov = _view(out, "out", dtype, dev, 3)
        if out.shape != (B, H, dv):
            raise EsError(1, "E-DIM-001 out has shape %s, not %s" % (list(out.shape), [B, H, dv]))
    args = _pack(dtype, B, 1, H, dk, dv, scale, views, ov, decay, 0, init, fin)
    _check(binding.lib().es_linear_attention_step(args, _raw_stream(dev)))
    return out, state_out


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


_WDTYPES = {None: 0, torch.float32: 0, torch.bfloat16: 1}


def _rotate_args(q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours):
    if not isinstance(q, torch.Tensor) or q.dtype not in _DTYPES or not q.is_cuda:
        raise TypeError("q must be a float32 or bfloat16 CUDA tensor")
    dtype, dev = q.dtype, q.get_device()
    qv = _view(q, "q", dtype, dev, 4)
    B, T, d = q.shape[0], q.shape[1], q.shape[3]
    kv = (0, 0, 0, 0, 0)
    if k is not None:
        kv = _view(k, "k", dtype, dev, 4)
        if k.shape[:2] != q.shape[:2] or k.shape[3] != d:
            raise EsError(1, "E-DIM-001 q %s and k %s do not fit" % (list(q.shape), list(k.shape)))
    wdtype = None
    for w in (q_weight, k_weight):
        if w is not None:
            if not isinstance(w, torch.Tensor) or w.dtype not in _DTYPES or wdtype not in (None, w.dtype):
                raise TypeError("q_weight and k_weight must be tensors of one dtype, float32 or bfloat16")
            wdtype = w.dtype
    wq = _plain(q_weight, "q_weight", wdtype, dev, (d,))
    wk = _plain(k_weight, "k_weight", wdtype, dev, (d,))
    turned, rows, cp, sp = 0, 0, 0, 0
    if cos is not None:
        if not isinstance(cos, torch.Tensor) or cos.dim() != 2:
            raise TypeError("cos must be a [rows, turned / 2] float32 tensor")
        rows, turned = cos.shape[0], 2 * cos.shape[1]
        cp = _plain(cos, "cos", torch.float32, dev, cos.shape)
        sp = _plain(sin, "sin", torch.float32, dev, cos.shape)
    elif sin is not None:
        raise TypeError("sin without cos")
    pos = (0, 0, 0, 0)
    if positions is not None:
        if not isinstance(positions, torch.Tensor) or positions.dtype not in (torch.int32, torch.int64) or positions.get_device() != dev:
            raise TypeError("positions must be an int32 or int64 tensor on cuda:%d" % dev)
        s = positions.stride()
        if positions.shape == (B, T):
            pos = (positions.data_ptr(), int(positions.dtype == torch.int64), s[0], s[1])
        elif positions.shape == (T,):
            pos = (positions.data_ptr(), int(positions.dtype == torch.int64), 0, s[0])
        else:
            raise EsError(1, "E-DIM-001 positions %s fits neither %s nor %s" % (list(positions.shape), [B, T], [T]))
    head = (_DTYPES[dtype], _WDTYPES[wdtype], B, T, d, turned, int(bool(neighbours)), eps)
    tail = (wq, wk, cp, sp, rows, *pos)
    return dtype, dev, head, qv, kv, tail, wdtype


def _result(t, like, name, dtype, dev):
    """A result's tensor (a new dense one unless given) and its view."""
    if t is None:
        t = like.new_empty(like.shape)
        _, T, h, d = like.shape
        return t, (t.data_ptr(), T * h * d, h * d, d, h)
    if t.shape != like.shape:
        raise EsError(1, "E-DIM-001 %s has shape %s, not %s" % (name, list(t.shape), list(like.shape)))
    return t, _view(t, name, dtype, dev, 4)


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
    if isinstance(q, torch.Tensor) and q.is_cuda and not _here(q.get_device(), stream):
        with _On(q.get_device(), stream):
            return qk_norm_rotate(q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours, q_out, k_out)
    dtype, dev, head, qv, kv, tail, _ = _rotate_args(q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours)
    q_out, qov = _result(q_out, q, "q_out", dtype, dev)
    kov = kv
    if k is not None:
        k_out, kov = _result(k_out, k, "k_out", dtype, dev)
    args = _ROTATE.pack(*head, *qv, *kv, *qov, *kov, *tail, 0, 0)
    _check(binding.lib().es_qk_norm_rotate(args, _raw_stream(dev)))
    return q_out, k_out


def qk_norm_rotate_backward(q, k, q_weight, k_weight, cos, sin, grad_q_out, grad_k_out, positions=None,
                            eps: float = 1e-6, neighbours: bool = False, workspace=None, stream=None):
    """Gradients of ``qk_norm_rotate``: (grad_q, grad_k, grad_q_weight,
    grad_k_weight), None where there is no operand."""
    if isinstance(q, torch.Tensor) and q.is_cuda and not _here(q.get_device(), stream):
        with _On(q.get_device(), stream):
            return qk_norm_rotate_backward(q, k, q_weight, k_weight, cos, sin, grad_q_out, grad_k_out, positions, eps,
                                           neighbours, workspace)
    dtype, dev, head, qv, kv, tail, wdtype = _rotate_args(q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours)
    gqv, gkv = _view(grad_q_out, "grad_q_out", dtype, dev, 4), kv
    pairs = [(q, grad_q_out, "grad_q_out")]
    if k is not None:
        gkv = _view(grad_k_out, "grad_k_out", dtype, dev, 4)
        pairs.append((k, grad_k_out, "grad_k_out"))
    for x, g, name in pairs:
        if g.shape != x.shape:
            raise EsError(1, "E-DIM-001 %s has shape %s, not %s" % (name, list(g.shape), list(x.shape)))
    L = binding.lib()
    gq, gqo = _result(None, q, "grad_q", dtype, dev)
    gk, gko = _result(None, k, "grad_k", dtype, dev) if k is not None else (None, kv)
    gwq = torch.empty_like(q_weight) if q_weight is not None else None
    gwk = torch.empty_like(k_weight) if k_weight is not None and k is not None else None
    args = _ROTATE.pack(*head, *qv, *kv, *gqo, *gko, *tail, 0, 0)
    grads = _ROTATE_GRADS.pack(*gqv, *gkv, 0 if gwq is None else gwq.data_ptr(), 0 if gwk is None else gwk.data_ptr())
    workspace, args = _workspace(L.es_qk_norm_rotate_workspace, args, grads, workspace, dev)
    _check(L.es_qk_norm_rotate_backward(args, grads, _raw_stream(dev)))
    return gq, gk, gwq, gwk
