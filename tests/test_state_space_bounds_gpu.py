"""Guard regions around every buffer of the state-space operators, through the C
ABI: results, states, checkpoints, gradients, workspaces and inputs are views into
larger allocations whose margins hold a sentinel.  After each call no margin has
changed, every result was written everywhere, no input changed, and the results are
those of the same call on plain buffers, bit for bit.  Ordinary in-bounds calls all
of them: channels, states and lengths that end inside tiles, segments, groups."""
import ctypes

import numpy as np
import pytest
import torch

import element_scan_recurrences_gb300 as es
from element_scan_recurrences_gb300 import binding, sequence
from test_sequence_bounds_gpu import BF16, F32, I32, U8, address, guarded, heads, need, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    es.lib()


def rows(t):
    return (0, 0, 0) if t is None else (t.data_ptr(), t.stride(0), t.stride(1))


def kind(dtype):
    return 1 if dtype == BF16 else 0


def maker(seed=0):
    rng = np.random.default_rng(seed)
    return lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()


def stand_in(inputs, outputs):
    return {**inputs, **{name: torch.empty(s, dtype=t, device="cuda") for name, (s, t) in outputs.items()}}


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", [(2, 77, 40, 4, [77, 10]), (1, 131, 1032, 3, None), (3, 5, 33, 8, [0, 1, 5]), (1, 300, 8, 2, None),
                                  (2, 1, 24, 5, None)], ids=str)
def test_conv(case, dtype):
    B, T, C, W, lengths = case
    made = maker()
    n = None if lengths is None else torch.tensor(lengths, dtype=I32, device="cuda")
    inputs = dict(x=made(B, T, C).to(dtype), w=made(C, W).to(dtype), b=made(C).to(dtype), init=made(B, W - 1, C).to(dtype), lengths=n)

    def pack(x, ws, out=None, fin=None):
        return sequence._CONV.pack(kind(dtype), kind(dtype), B, T, C, W, 1, *rows(x["x"]), *rows(out), address(x["w"]), address(x["b"]),
                                   address(x.get("lengths")), address(x["init"]), address(fin), address(ws), 0 if ws is None else ws.numel())

    guarded(inputs, dict(out=((B, T, C), dtype), fin=((B, W - 1, C), dtype)),
            lambda x, ws: run("es_causal_conv", pack(x, ws, x["out"], x["fin"])), 0, "forward")
    if T == 1:
        step = {k: v for k, v in inputs.items() if k != "lengths"}
        guarded(step, dict(out=((B, T, C), dtype), fin=((B, W - 1, C), dtype)),
                lambda x, ws: run("es_causal_conv_step", pack(x, ws, x["out"], x["fin"])), 0, "step")
    inputs.update(go=made(B, T, C).to(dtype), gfin=made(B, W - 1, C).to(dtype))
    outputs = dict(gx=((B, T, C), dtype), gw=((C, W), dtype), gb=((C,), dtype), gi=((B, W - 1, C), dtype))

    def grads(x):
        return sequence._CONV_GRADS.pack(*rows(x["go"]), *rows(x["gx"]), address(x["gw"]), address(x["gb"]), address(x["gfin"]),
                                         address(x["gi"]))

    s = stand_in(inputs, outputs)
    bytes_ = need("es_causal_conv_workspace", pack(s, None), grads(s))
    guarded(inputs, outputs, lambda x, ws: run("es_causal_conv_backward", pack(x, ws), grads(x)), bytes_, "backward")


SCANS = [(2, 77, 40, 16, 1, [77, 10]), (1, 35, 136, 16, 2, None), (3, 20, 33, 5, 3, [0, 20, 1]), (1, 50, 300, 8, 1, None),
         (1, 40, 72, 32, 1, [39]), (2, 33, 20, 64, 2, None), (1, 900, 24, 16, 1, [700]), (2, 1, 40, 16, 2, None), (2, 1, 9, 33, 1, None)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", SCANS, ids=str)
def test_scan(case, dtype):
    B, T, C, N, G, lengths = case
    made = maker(1)
    n = None if lengths is None else torch.tensor(lengths, dtype=I32, device="cuda")
    inputs = dict(x=made(B, T, C).to(dtype), delta=made(B, T, C).to(dtype), gate=made(B, T, C).to(dtype), b=made(B, T, G, N).to(dtype),
                  c=made(B, T, G, N).to(dtype), a=-made(C, N).abs(), skip=made(C), bias=made(C), lengths=n, init=made(B, C, N))

    def pack(x, ws, out=None, fin=None, kept=None):
        return sequence._SCAN.pack(kind(dtype), B, T, C, N, G, 1, *rows(x["x"]), *rows(x["delta"]), *rows(x["gate"]), *rows(out),
                                   *heads(x["b"]), *heads(x["c"]), address(x["a"]), address(x["skip"]), address(x["bias"]),
                                   address(x.get("lengths")), address(x["init"]), address(fin), address(kept),
                                   0 if kept is None else kept.numel(), address(ws), 0 if ws is None else ws.numel())

    kept_bytes = need_checkpoints(pack(inputs, None, made(B, T, C).to(dtype), made(B, C, N)))
    outputs = dict(out=((B, T, C), dtype), fin=((B, C, N), F32))
    s = stand_in(inputs, outputs)
    bytes_ = need("es_selective_scan_workspace", pack(s, None, s["out"], s["fin"]), None)
    guarded(inputs, outputs, lambda x, ws: run("es_selective_scan", pack(x, ws, x["out"], x["fin"])), bytes_, "forward")
    kept = torch.zeros(kept_bytes, dtype=U8, device="cuda")
    if lengths is None:      # every state on the way is written
        guarded(inputs, dict(outputs, kept=((kept_bytes // 4,), F32)),
                lambda x, ws: run("es_selective_scan", pack(x, ws, x["out"], x["fin"], x["kept"].view(U8))), bytes_, "with checkpoints")
    ws = torch.empty(max(bytes_, 1), dtype=U8, device="cuda")
    run("es_selective_scan", pack(s, ws, s["out"], s["fin"], kept))
    if T == 1:
        step = {k: v for k, v in inputs.items() if k != "lengths"}
        guarded(step, outputs, lambda x, ws: run("es_selective_scan_step", pack(x, ws, x["out"], x["fin"])), 0, "step")
    inputs.update(go=made(B, T, C).to(dtype), gfin=made(B, C, N))
    outputs = dict(gx=((B, T, C), dtype), gdelta=((B, T, C), dtype), ggate=((B, T, C), dtype), gb=((B, T, G, N), dtype),
                   gc=((B, T, G, N), dtype), ga=((C, N), F32), gskip=((C,), F32), gbias=((C,), F32), gi=((B, C, N), F32))

    def grads(x):
        return sequence._SCAN_GRADS.pack(*rows(x["go"]), *rows(x["gx"]), *rows(x["gdelta"]), *rows(x["ggate"]), *heads(x["gb"]),
                                         *heads(x["gc"]), address(x["ga"]), address(x["gskip"]), address(x["gbias"]), address(x["gfin"]),
                                         address(x["gi"]))

    for given in (False, True):
        ins = dict(inputs, kept=kept) if given else inputs
        s = stand_in(ins, outputs)
        bytes_ = need("es_selective_scan_workspace", pack(s, None, kept=s.get("kept")), grads(s))
        guarded(ins, outputs, lambda x, ws: run("es_selective_scan_backward", pack(x, ws, kept=x.get("kept")), grads(x)), bytes_,
                "backward with checkpoints" if given else "backward")


def need_checkpoints(args):
    n = ctypes.c_size_t()
    binding._check(binding.lib().es_selective_scan_checkpoints(args, ctypes.byref(n)))
    return n.value


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("first", [0, 1])
@pytest.mark.parametrize("case", [(2, 37, 5, 128), (1, 30, 3, 80), (1, 3, 1, 2560), (2, 11, 3, 33), (1, 4, 1, 8191), (1, 700, 16, 64)], ids=str)
def test_norm(case, first, dtype):
    B, T, H, D = case
    made = maker(2)
    inputs = dict(x=made(B, T, H, D).to(dtype), gate=made(B, T, H, D).to(dtype), w=made(H, D).to(dtype), b=made(H, D).to(dtype))

    def pack(x, ws, out=None):
        return sequence._NORM.pack(kind(dtype), kind(dtype), B, T, D, 1, first, 0, 1e-5, *heads(x["x"]), *heads(x["gate"]), *heads(out),
                                   address(x["w"]), address(x["b"]), address(ws), 0 if ws is None else ws.numel())

    guarded(inputs, dict(out=((B, T, H, D), dtype)), lambda x, ws: run("es_group_norm", pack(x, ws, x["out"])), 0, "forward")
    inputs.update(go=made(B, T, H, D).to(dtype))
    outputs = dict(gx=((B, T, H, D), dtype), ggate=((B, T, H, D), dtype), gw=((H, D), dtype), gb=((H, D), dtype))

    def grads(x):
        return sequence._NORM_GRADS.pack(*heads(x["go"]), *heads(x["gx"]), *heads(x["ggate"]), address(x["gw"]), address(x["gb"]))

    s = stand_in(inputs, outputs)
    bytes_ = need("es_group_norm_workspace", pack(s, None), grads(s))
    guarded(inputs, outputs, lambda x, ws: run("es_group_norm_backward", pack(x, ws), grads(x)), bytes_, "backward")
