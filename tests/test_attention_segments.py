"""How linear attention shares a row's chunks out among segments
(csrc/es_segments.h, compiled here for the host: every case on the CPU), and
rows of very different lengths in segments on the GPU."""
import ctypes
import itertools
import os
import subprocess

import numpy as np
import pytest
import torch

import element_scan_recurrences_gb300 as es

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "element_scan_recurrences_gb300", "csrc")


class Part(ctypes.Structure):
    _fields_ = [("c0", ctypes.c_int), ("c1", ctypes.c_int), ("last", ctypes.c_int), ("begins", ctypes.c_bool),
                ("ends", ctypes.c_bool), ("entry", ctypes.c_int)]


@pytest.fixture(scope="module")
def part(tmp_path_factory):
    at = tmp_path_factory.mktemp("segments")
    src = at / "s.cpp"
    src.write_text('#include "es_segments.h"\nextern "C" void part(int s, int n, int each, int chunks, bool r, es::SegmentPart* p) '
                   '{ *p = es::segment_part(s, n, each, chunks, r); }\n')
    lib = str(at / "s.so")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", lib], check=True)
    f = ctypes.CDLL(lib).part
    f.argtypes = [ctypes.c_int] * 4 + [ctypes.c_bool, ctypes.POINTER(Part)]

    def call(*a):
        p = Part()
        f(*a, ctypes.byref(p))
        return p
    return call


@pytest.mark.parametrize("reverse", [False, True])
def test_every_segment_takes_a_state_that_is_there(part, reverse):
    """Calls of 1..20 chunks in every number of segments, rows of every length:
    the segments cover the row's chunks once, the run begins and ends once, and
    a segment takes the state its predecessor along the run left (a place that
    the pass before wrote), the first state where it begins, none past the row."""
    for most, each in itertools.product(range(1, 21), range(1, 21)):
        n = -(-most // each)
        for chunks in range(most + 1):
            parts = [part(s, n, each, chunks, reverse) for s in range(n)]
            covered = [c for p in parts for c in range(p.c0, p.c1)]
            assert covered == list(range(chunks))
            last = max(0, -(-chunks // each) - 1)
            assert [s for s in range(n) if parts[s].begins] == [last if reverse else 0]
            assert [s for s in range(n) if parts[s].ends] == [0 if reverse else last]
            for s, p in enumerate(parts):
                assert p.last == last
                if n == 1 or s > last:
                    assert p.entry == -1
                elif p.begins:
                    assert p.entry == (0 if reverse else last)
                else:
                    before = s + 1 if reverse else s - 1
                    assert p.entry == before and 0 <= before <= last


def test_a_short_row_s_last_segment_reads_nothing(part):
    """2 x 8192 tokens x 2 heads of 96 and 80 in 12 segments of 11 chunks: the
    row of 64 tokens has one chunk, and the place after the last segment's
    would lie behind a workspace that holds the states alone."""
    from element_scan_recurrences_gb300 import build
    build.build()
    plan = es.plan_linear_attention((2, 8192, 2, 96), (2, 8192, 2, 96), (2, 8192, 2, 80), lengths=True, backward=True)
    runs, rows, n, each, state = 3, 4, 12, 11, 4 * 96 * 80
    assert plan["path"] == "tensor" and plan["workspace"] == runs * rows * n * state + 768
    assert runs * rows * n * state < plan["workspace"] < (runs * rows * n + 1) * state
    p = part(n - 1, n, each, 1, True)
    assert p.c1 <= p.c0 and p.entry == -1 and not p.begins and not p.ends


@pytest.mark.gpu
@pytest.mark.parametrize("decay", ["token", "head", None])
def test_short_rows_beside_long_ones_without_the_decays_gradient(decay):
    """The same call on the GPU, no decays' gradient, the workspace just as
    large as asked for: each row's results are the bits of the row by itself
    at its own length, and nothing around the workspace changes."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gen = torch.Generator(device="cuda").manual_seed(0)
    made = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    B, T, H, lengths = 2, 8192, 2, [8192, 64]
    q, k = made(B, T, H, 96).bfloat16(), made(B, T, H, 96).bfloat16()
    v, go = made(B, T, H, 80).bfloat16(), made(B, T, H, 80).bfloat16()
    g = {"token": lambda: -torch.rand(B, T, H, generator=gen, device="cuda") * 0.2,
         "head": lambda: -torch.rand(H, generator=gen, device="cuda") * 0.2, None: lambda: None}[decay]()
    init, gfin = made(B, H, 96, 80), made(B, H, 96, 80)
    need = es.plan_linear_attention(q.shape, k.shape, v.shape, decay=decay, heads=H, lengths=True, state=True)["workspace"]
    grad_need = 3 * 4 * 12 * 4 * 96 * 80 + 768
    room = torch.full((grad_need + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = room[4096:4096 + grad_need]
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, fin = es.linear_attention(q, k, v, g, initial_state=init, lengths=n, final_state=True,
                                   workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    grads = es.linear_attention_backward(q, k, v, g, go, initial_state=init, grad_final_state=gfin, lengths=n,
                                         decay_grad=False, workspace=ws)
    es.device_status()
    assert (room[:4096] == 0xA5).all() and (room[4096 + grad_need:] == 0xA5).all()
    assert grads[3] is None
    # the short row by itself is one chunk, without segments
    one = [x[1:, :64] for x in (q, k, v)]
    g1 = g[1:, :64] if decay == "token" else g
    wout, wfin = es.linear_attention(*one, g1, initial_state=init[1:], final_state=True)
    wgrads = es.linear_attention_backward(*one, g1, go[1:, :64], initial_state=init[1:], grad_final_state=gfin[1:],
                                          decay_grad=False)
    assert torch.equal(out[1:, :64], wout) and not out[1, 64:].any() and torch.equal(fin[1:], wfin)
    for x, y in zip(grads[:3], wgrads[:3]):
        assert torch.equal(x[1:, :64], y) and not x[1, 64:].any()
    assert torch.equal(grads[4][1:], wgrads[4])
    # and the long one the bits it has without its neighbour's length
    fout, ffin = es.linear_attention(q, k, v, g, initial_state=init, final_state=True)
    fgrads = es.linear_attention_backward(q, k, v, g, go, initial_state=init, grad_final_state=gfin, decay_grad=False)
    assert torch.equal(out[0], fout[0]) and torch.equal(fin[0], ffin[0])
    for x, y in zip((*grads[:3], grads[4]), (*fgrads[:3], fgrads[4])):
        assert torch.equal(x[0], y[0])
    es.device_status()
    assert np.isfinite(out.float().cpu().numpy()).all()
