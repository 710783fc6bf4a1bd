"""Guard regions around every buffer of the sequence-layer operators, through
the C ABI: results, states, gradients, workspaces and inputs are views into
larger allocations whose margins hold a sentinel.  After each call no margin
has changed, every result was written everywhere, no input changed, and the
results are those of the same call on plain buffers, bit for bit.  Ordinary
in-bounds calls all of them: widths and lengths that end inside tiles, both
kernel paths, segments, shared heads."""
import ctypes
import math

import numpy as np
import pytest
import torch

import element_scan_recurrences_gb300 as es
from element_scan_recurrences_gb300 import binding, sequence

pytestmark = pytest.mark.gpu

F32, BF16, U8, I32 = torch.float32, torch.bfloat16, torch.uint8, torch.int32
# patterns no kernel produces (NaNs of the two floating types), and the integers they are compared as
SENTINEL = {F32: (torch.int32, 0x7FA5A5A5), BF16: (torch.int16, 0x7FA5), U8: (torch.uint8, 0xA5), I32: (torch.int32, 0x7FA5A5A5)}
PAD = 4096                 # elements on each side (keeps every alignment)


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    es.lib()
    yield
    es.set_path_override("auto")


class Guarded:
    def __init__(self, shape, dtype):
        self.n = math.prod(shape)
        self.buf = torch.empty(self.n + 2 * PAD, dtype=dtype, device="cuda")
        kind, self.sentinel = SENTINEL[dtype]
        self.bits = self.buf.view(kind)
        self.bits.fill_(self.sentinel)
        self.t = self.buf[PAD:PAD + self.n].view(tuple(shape))

    def check(self, what, written):
        changed = int((self.bits[:PAD] != self.sentinel).sum()), int((self.bits[PAD + self.n:] != self.sentinel).sum())
        assert changed == (0, 0), "%s: %d elements before and %d after it were written" % ((what,) + changed)
        if written:
            left = int((self.bits[PAD:PAD + self.n] == self.sentinel).sum())
            assert left == 0, "%s: %d of %d positions were never written" % (what, left, self.n)


def guarded(inputs, outputs, call, ws_bytes, what):
    """`call(tensors, workspace)`: inputs by name (tensors or None), outputs by name as (shape, dtype)."""
    boxes = {}
    for name, x in inputs.items():
        if x is not None:
            boxes[name] = Guarded(x.shape, x.dtype)
            boxes[name].t.copy_(x)
    for name, (shape, dtype) in outputs.items():
        boxes[name] = Guarded(shape, dtype)
    ws = Guarded((ws_bytes,), U8) if ws_bytes else None
    call({n: b.t for n, b in boxes.items()}, None if ws is None else ws.t)
    es.device_status()
    for name, box in boxes.items():
        box.check("%s %s" % (what, name), name in outputs)
        if name in inputs:
            assert torch.equal(box.t, inputs[name]), "%s: %s changed" % (what, name)
    if ws is not None:
        ws.check(what + " workspace", False)
    plain = {n: x.clone() for n, x in inputs.items() if x is not None}
    plain.update({n: torch.empty(shape, dtype=dtype, device="cuda") for n, (shape, dtype) in outputs.items()})
    call(plain, torch.empty(ws_bytes, dtype=U8, device="cuda") if ws_bytes else None)
    es.device_status()
    for name in outputs:
        kind = SENTINEL[outputs[name][1]][0]
        assert torch.equal(boxes[name].t.contiguous().view(kind), plain[name].view(kind)), "%s: %s differs" % (what, name)


def address(t):
    return 0 if t is None else t.data_ptr()


def heads(t):
    if t is None:
        return (0, 0, 0, 0, 0)
    return (t.data_ptr(), *t.stride()[:3], t.shape[2])


def run(name, args, *rest):
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    binding._check(getattr(binding.lib(), name)(args, *rest, stream))


def need(name, args, grads):
    n = ctypes.c_size_t()
    binding._check(getattr(binding.lib(), name)(args, grads, ctypes.byref(n)))
    return n.value


ATTENTION = [
    # path, dtype, B, T, heads, dk, dv, decay, lengths
    ("tensor", BF16, 2, 77, (2, 2, 2, 2), 64, 64, "token", [77, 10]),
    ("tensor", BF16, 1, 131, (1, 2, 4, 4), 96, 80, "head", None),
    ("tensor", BF16, 2, 1500, (1, 1, 2, 2), 128, 128, "token", [1500, 70]),
    ("tensor", BF16, 2, 1500, (2, 2, 2, 2), 64, 8, None, [3, 1500]),
    ("generic", BF16, 2, 77, (2, 2, 2, 2), 33, 17, "token", [76, 0]),
    ("generic", BF16, 1, 1000, (1, 1, 2, 2), 64, 72, "token", None),
    ("generic", F32, 2, 70, (2, 1, 2, 2), 256, 40, "head", [70, 33]),
    ("generic", F32, 2, 900, (1, 1, 2, 2), 64, 64, "token", [900, 40]),
]


@pytest.mark.parametrize("case", ATTENTION, ids=str)
def test_attention(case):
    path, dtype, B, T, (hq, hk, hv, H), dk, dv, decay, lengths = case
    rng = np.random.default_rng(0)
    made = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
    q, k, v, go = (made(B, T, h, d).to(dtype) for h, d in ((hq, dk), (hk, dk), (hv, dv), (H, dv)))
    g = None if decay is None else torch.from_numpy(-rng.uniform(0, 0.2, (B, T, H) if decay == "token" else (H,)).astype(np.float32)).cuda()
    n = None if lengths is None else torch.tensor(lengths, dtype=I32, device="cuda")
    inputs = dict(q=q, k=k, v=v, g=g, init=made(B, H, dk, dv), lengths=n)

    def pack(x, ws, out=None, fin=None):
        x = dict.fromkeys(("g", "lengths"), None) | x
        decays = (0, 0, 0, 0, 0) if x["g"] is None else (address(x["g"]), T * H, H, 1, 0) if decay == "token" else (address(x["g"]), 0, 0, 1, 1)
        return sequence._ATTN.pack(1 if dtype == BF16 else 0, B, T, H, dk, dv, dk ** -0.5, *heads(x["q"]), *heads(x["k"]), *heads(x["v"]),
                                   *heads(out), *decays, address(x["lengths"]), address(x["init"]), address(fin), address(ws),
                                   0 if ws is None else ws.numel())

    es.set_path_override(path)
    some = made(B, T, H, dv).to(dtype)
    bytes_ = need("es_linear_attention_workspace", pack(inputs, None, some, made(B, H, dk, dv)), None)
    guarded(inputs, dict(out=((B, T, H, dv), dtype), fin=((B, H, dk, dv), F32)),
            lambda x, ws: run("es_linear_attention", pack(x, ws, x["out"], x["fin"])), bytes_, "forward")

    inputs.update(go=go, gfin=made(B, H, dk, dv))
    for wants in ((True, False) if g is not None else (False,)):
        outputs = dict(gq=(q.shape, dtype), gk=(k.shape, dtype), gv=(v.shape, dtype), gi=((B, H, dk, dv), F32))
        if wants:
            outputs["gg"] = (g.shape, F32)

        def grads(x):
            return sequence._ATTN_GRADS.pack(*heads(x["go"]), *heads(x["gq"]), *heads(x["gk"]), *heads(x["gv"]), address(x["gfin"]),
                                             address(x.get("gg")), address(x["gi"]))

        stand_in = {**inputs, **{name: torch.empty(s, dtype=t, device="cuda") for name, (s, t) in outputs.items()}}
        bytes_ = need("es_linear_attention_workspace", pack(stand_in, None), grads(stand_in))
        guarded(inputs, outputs, lambda x, ws: run("es_linear_attention_backward", pack(x, ws), grads(x)), bytes_,
                "backward %s the decays'" % ("with" if wants else "without"))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("widths", [(64, 64), (128, 100), (7, 33), (256, 1)], ids=str)
def test_step(widths, dtype):
    dk, dv = widths
    B, H = 3, 4
    made = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    inputs = dict(q=made(B, 1, 2, dk).to(dtype), k=made(B, 1, 1, dk).to(dtype), v=made(B, 1, H, dv).to(dtype), g=-made(B, 1, H).abs(),
                  state=made(B, H, dk, dv))

    def call(x, ws):
        run("es_linear_attention_step",
            sequence._ATTN.pack(1 if dtype == BF16 else 0, B, 1, H, dk, dv, 0.3, *heads(x["q"]), *heads(x["k"]), *heads(x["v"]),
                                *heads(x["out"]), address(x["g"]), H, 0, 1, 0, 0, address(x["state"]), address(x["next"]), 0, 0))

    guarded(inputs, dict(out=((B, 1, H, dv), dtype), next=((B, H, dk, dv), F32)), call, 0, "step")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("neighbours", [0, 1])
@pytest.mark.parametrize("case", [(2, 37, 5, 3, 128, 128), (1, 300, 8, 2, 80, 32), (3, 1, 1, 0, 64, 0), (2, 11, 3, 3, 33, 6), (1, 9, 2, 1, 255, 254)],
                         ids=str)
def test_rotation(case, neighbours, dtype):
    B, T, hq, hk, D, turned = case
    made = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    rows = 50
    pos = torch.randint(-3, rows + 3, (B, T), device="cuda").to(I32)
    inputs = dict(q=made(B, T, hq, D).to(dtype), k=made(B, T, hk, D).to(dtype) if hk else None, wq=made(D).to(dtype),
                  wk=made(D).to(dtype) if hk else None, cos=made(rows, turned // 2) if turned else None,
                  sin=made(rows, turned // 2) if turned else None, pos=pos)
    kind = 1 if dtype == BF16 else 0

    def pack(x, ws, qo, ko):
        x = dict.fromkeys(inputs, None) | x
        return sequence._ROTATE.pack(kind, kind, B, T, D, turned, neighbours, 1e-6, *heads(x["q"]), *heads(x["k"]), *heads(qo), *heads(ko),
                                     address(x["wq"]), address(x["wk"]), address(x["cos"]), address(x["sin"]), rows, address(x["pos"]), 0, T, 1,
                                     address(ws), 0 if ws is None else ws.numel())

    def shapes(*names):
        out = {names[0]: ((B, T, hq, D), dtype)}
        if hk:
            out[names[1]] = ((B, T, hk, D), dtype)
        return out

    guarded(inputs, shapes("qo", "ko"), lambda x, ws: run("es_qk_norm_rotate", pack(x, ws, x["qo"], x.get("ko"))), 0, "rotation")

    inputs.update(gqo=made(B, T, hq, D).to(dtype), gko=made(B, T, hk, D).to(dtype) if hk else None)
    outputs = shapes("gq", "gk")
    outputs["gwq"] = ((D,), dtype)
    if hk:
        outputs["gwk"] = ((D,), dtype)

    def grads(x):
        return sequence._ROTATE_GRADS.pack(*heads(x["gqo"]), *heads(x.get("gko")), address(x["gwq"]), address(x.get("gwk")))

    stand_in = {**inputs, **{name: torch.empty(s, dtype=t, device="cuda") for name, (s, t) in outputs.items()}}
    bytes_ = need("es_qk_norm_rotate_workspace", pack(stand_in, None, stand_in["gq"], stand_in.get("gk")), grads(stand_in))
    assert bytes_ > 0
    guarded(inputs, outputs, lambda x, ws: run("es_qk_norm_rotate_backward", pack(x, ws, x["gq"], x.get("gk")), grads(x)), bytes_,
            "rotation backward")
