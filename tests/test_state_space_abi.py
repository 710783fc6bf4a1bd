"""The short causal convolution, the selective scan and the gated group norm
through the C ABI without a GPU: plans, workspaces and refusals."""
import os
import subprocess

import pytest

import element_scan_recurrences_gb300 as es
from element_scan_recurrences_gb300 import sequence

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
X = (2, 100, 64)
FAR = 1 << 44          # where a plan's first stand-in operand (x) lies


@pytest.fixture(scope="module", autouse=True)
def built():
    from element_scan_recurrences_gb300 import build
    build.build()


def test_packed_structs_have_the_header_s_sizes(tmp_path):
    names = ("es_causal_conv_args", "es_causal_conv_grads", "es_selective_scan_args", "es_selective_scan_grads",
             "es_group_norm_args", "es_group_norm_grads")
    src = tmp_path / "s.c"
    src.write_text('#include "es.h"\n#include <stdio.h>\nint main(void) { printf("%s", %s); return 0; }\n' % (
        " ".join(["%zu"] * len(names)), ", ".join("sizeof(%s)" % n for n in names)))
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    sizes = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(s) for s in sizes] == [x.size for x in (sequence._CONV, sequence._CONV_GRADS, sequence._SCAN, sequence._SCAN_GRADS,
                                                        sequence._NORM, sequence._NORM_GRADS)]


def test_plans():
    p = es.plan_causal_conv(X, 4, state=True, lengths=True)
    assert (p["O"], p["T"], p["J"], p["W"], p["elements"], p["path"], p["workspace"]) == (2, 100, 64, 4, 12800, "generic", 0)
    p = es.plan_causal_conv(X, 4, backward=True)
    # a row of partial sums for each run of tokens
    assert p["workspace"] % (4 * 64 * 5) == 0 and p["workspace"] > 0
    p = es.plan_selective_scan(X, 16)
    assert (p["O"], p["T"], p["J"], p["W"], p["checkpoints"]) == (2, 100, 64, 16, 7 * 2 * 64 * 16 * 4)
    assert es.plan_selective_scan((0, 100, 64), 16)["path"] == "empty"
    p = es.plan_group_norm((2, 100, 4, 64))
    assert (p["O"], p["T"], p["J"], p["W"], p["workspace"]) == (2, 100, 4, 64, 0)
    assert es.plan_group_norm((2, 100, 4, 64), backward=True)["workspace"] > 0
    assert es.plan_group_norm((2, 100, 4, 64), backward=True, weight=False, bias=False)["workspace"] == 0


def test_few_channels_and_many_tokens_are_cut_into_segments():
    assert es.plan_selective_scan((1, 65536, 64), 16)["workspace"] > 0          # the segments' own states
    assert es.plan_selective_scan((8, 4096, 4096), 16)["workspace"] == 0        # channels enough for the GPU
    assert es.plan_selective_scan((1, 16, 64), 16)["workspace"] == 0            # one chunk


def test_checkpoints_save_the_backward_s_workspace():
    shape = (2, 1000, 512)
    kept = es.plan_selective_scan(shape, 16)["checkpoints"]
    given, found = (es.plan_selective_scan(shape, 16, backward=True, checkpoints=c)["workspace"] for c in (True, False))
    assert found - given >= kept


def test_in_place_states_and_fused_operands():
    for plan, args in ((es.plan_causal_conv, (X, 4)), (es.plan_selective_scan, (X, 16))):
        plan(*args, state=True, ptrs={"initial_state": 99 << 44, "final_state": 99 << 44})
    # x and the gate as halves of one tensor, B and C of another
    es.plan_selective_scan(X, 16, ptrs={"gate": FAR + 64 * 2, "c": (5 << 44) + 32, "b": 5 << 44},
                           strides={"x": (12800, 128), "gate": (12800, 128), "b": (3200, 32, 16), "c": (3200, 32, 16)})


@pytest.mark.parametrize("kw,code", [
    (dict(dtype="f16"), 2), (dict(weight_dtype="f16"), 2),
    (dict(taps=1), 4), (dict(taps=9), 4), (dict(taps=0), 4),
    (dict(shape=(-1, 5, 8)), 1), (dict(shape=(1 << 30, 1 << 20, 8)), 4), (dict(shape=(1, 1 << 31, 8)), 4),
    (dict(ptrs={"x": 0}), 3), (dict(ptrs={"weight": 0}), 3), (dict(ptrs={"x": FAR + 1}), 3), (dict(ptrs={"bias": FAR * 9 + 1}), 3),
    (dict(ptrs={"out": FAR + 128}), 3),                               # over x
    (dict(ptrs={"final_state": FAR + 128}, state=True), 3),
    (dict(ptrs={"initial_state": 99 << 44, "final_state": (99 << 44) + 2}, state=True), 3),     # half in its place
    (dict(ptrs={"workspace": FAR + 256}, backward=True), 3),
    (dict(strides={"x": (-1, 64)}), 3), (dict(strides={"out": (6400, 0)}), 3), (dict(strides={"x": (1 << 62, 64)}), 4),
])
def test_conv_refusals(kw, code):
    with pytest.raises(es.EsError) as e:
        es.plan_causal_conv(**{**dict(shape=X, taps=4), **kw})
    assert e.value.status == code, e.value


@pytest.mark.parametrize("kw,code", [
    (dict(dtype="f16"), 2),
    (dict(states=0), 4), (dict(states=65), 4),
    (dict(groups=3), 1), (dict(groups=0), 1),
    (dict(shape=(-1, 5, 64)), 1), (dict(shape=(1 << 30, 1 << 20, 64)), 4),
    (dict(ptrs={"a": 0}), 3), (dict(ptrs={"a": FAR * 70 + 2}), 3), (dict(ptrs={"delta": 0}), 3),
    (dict(ptrs={"out": FAR}), 3),                                     # over x
    (dict(ptrs={"checkpoints": FAR}, checkpoints=True), 3), (dict(ptrs={"checkpoints": (90 << 44) + 4}, checkpoints=True), 3),
    (dict(ptrs={"workspace": FAR}, backward=True), 3),
    (dict(ptrs={"grad_gate": 0}, backward=True), 3), (dict(ptrs={"grad_skip": 90 << 44}, skip=False, backward=True), 3),
    (dict(ptrs={"grad_delta_bias": 90 << 44}, delta_bias=False, backward=True), 3),
    (dict(ptrs={"grad_b": FAR}, backward=True), 3),
    (dict(strides={"b": (1600, 16, -1)}), 3), (dict(strides={"grad_c": (1600, 0, 16)}, backward=True), 3),
])
def test_scan_refusals(kw, code):
    with pytest.raises(es.EsError) as e:
        es.plan_selective_scan(**{**dict(shape=X, states=16), **kw})
    assert e.value.status == code, e.value


@pytest.mark.parametrize("kw,code", [
    (dict(dtype="f16"), 2), (dict(weight_dtype="f16"), 2),
    (dict(shape=(2, 100, 4, 0)), 4), (dict(shape=(2, 100, 4, 8193)), 4), (dict(shape=(2, 100, 65536, 8)), 4),
    (dict(shape=(-2, 100, 4, 64)), 1),
    (dict(eps=-1.0), 3), (dict(eps=float("nan")), 3), (dict(eps=float("inf")), 3),
    (dict(activation=True), 3), (dict(gate=False, gate_first=True), 3),
    (dict(ptrs={"x": 0}), 3), (dict(ptrs={"weight": FAR * 70 + 1}), 3), (dict(ptrs={"out": FAR}), 3),
    (dict(ptrs={"workspace": FAR}, backward=True), 3), (dict(ptrs={"grad_gate": 0}, backward=True), 3),
    (dict(ptrs={"grad_weight": 90 << 44}, weight=False, backward=True), 3),
    (dict(strides={"out": (25600, 256, 32)}), 3),                     # groups that share addresses
])
def test_norm_refusals(kw, code):
    with pytest.raises(es.EsError) as e:
        es.plan_group_norm(**{**dict(shape=(2, 100, 4, 64)), **kw})
    assert e.value.status == code, e.value
