"""Linear attention and the query/key norm with rotation through the C ABI
without a GPU: plans, workspaces and refusals."""
import ctypes
import os
import subprocess

import pytest

import element_scan_recurrences_gb300 as es
from element_scan_recurrences_gb300 import binding, sequence

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
Q = (2, 100, 8, 64)


@pytest.fixture(scope="module", autouse=True)
def built():
    from element_scan_recurrences_gb300 import build
    build.build()


@pytest.fixture(autouse=True)
def restore():
    yield
    es.set_path_override("auto")


def test_packed_structs_have_the_header_s_sizes(tmp_path):
    src = tmp_path / "s.c"
    src.write_text('#include "es.h"\n#include <stdio.h>\nint main(void) { printf("%zu %zu %zu %zu", '
                   'sizeof(es_linear_attention_args), sizeof(es_linear_attention_grads), '
                   'sizeof(es_qk_norm_rotate_args), sizeof(es_qk_norm_rotate_grads)); return 0; }\n')
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    sizes = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(s) for s in sizes] == [x.size for x in (sequence._ATTN, sequence._ATTN_GRADS, sequence._ROTATE,
                                                        sequence._ROTATE_GRADS)]


def test_plans():
    p = es.plan_linear_attention(Q, Q, Q, decay="token")
    assert (p["O"], p["T"], p["J"], p["W"]) == (2, 100, 8, 4096) and p["elements"] == 2 * 100 * 8 * 64
    assert es.plan_linear_attention(Q, Q, Q, dtype="f32")["path"] == "generic"
    assert es.plan_linear_attention((2, 100, 8, 33), (2, 100, 8, 33), Q)["path"] == "generic"
    assert es.plan_linear_attention((0, 100, 8, 64), (0, 100, 8, 64), (0, 100, 8, 64))["path"] == "empty"
    es.set_path_override("generic")
    assert es.plan_linear_attention(Q, Q, Q)["path"] == "generic"
    es.set_path_override("lane_tma")
    with pytest.raises(es.EsError) as e:
        es.plan_linear_attention(Q, Q, Q)
    assert e.value.status == 4


def test_backward_workspace_grows_with_what_is_asked():
    es.set_path_override("generic")
    plain = es.plan_linear_attention(Q, Q, Q, decay=None, backward=True)["workspace"]
    decay = es.plan_linear_attention(Q, Q, Q, decay="token", backward=True)["workspace"]
    shared = es.plan_linear_attention((2, 100, 2, 64), Q, Q, decay=None, backward=True)["workspace"]
    assert plain == 0 and decay > 0 and shared >= 4 * 2 * 100 * 8 * 64


@pytest.mark.parametrize("kw,code", [
    (dict(q_shape=(2, 100, 3, 64)), 1),                            # 3 heads of 8
    (dict(dtype="f16"), 2),
    (dict(scale=0.0), 3), (dict(scale=float("inf")), 3), (dict(scale=float("nan")), 3), (dict(scale=1e-60), 3),
    (dict(q_shape=(2, 100, 8, 257), k_shape=(2, 100, 8, 257)), 4),
    (dict(ptrs={"out": (1 << 44) + 64}), 3),                       # out over q
    (dict(ptrs={"q": 0}), 3), (dict(ptrs={"k": (2 << 44) + 1}), 3),
    (dict(strides={"v": (-1, 512, 64)}), 3),
    (dict(strides={"out": (0, 512, 64)}), 3),
    (dict(strides={"out": (51200, 512, 32)}), 3),                  # heads of out share addresses
    (dict(strides={"q": (1 << 62, 512, 64)}), 4),
    (dict(q_shape=(1 << 20, 100, 1 << 12, 64), k_shape=(1 << 20, 100, 1 << 12, 64), v_shape=(1 << 20, 100, 1 << 12, 64)), 4),
    (dict(q_shape=(1, 1 << 32, 1, 64), k_shape=(1, 1 << 32, 1, 64), v_shape=(1, 1 << 32, 1, 64)), 4),
])
def test_refusals(kw, code):
    with pytest.raises(es.EsError) as e:
        es.plan_linear_attention(**{**dict(q_shape=Q, k_shape=Q, v_shape=Q, decay="token"), **kw})
    assert e.value.status == code, e.value


def rotate(dtype=1, wdtype=1, B=2, T=5, D=64, turned=64, nb=0, eps=1e-6, q=None, k=None, qo=None, ko=None, w=(5 << 44, 6 << 44),
           tables=(7 << 44, 8 << 44), rows=50, pos=(0, 0, 0, 0), grads=None):
    view = lambda i, h: ((i + 1) << 44, T * h * D, h * D, D, h)  # noqa: E731
    args = sequence._ROTATE.pack(dtype, wdtype, B, T, D, turned, nb, eps, *(q or view(0, 4)), *(k or view(1, 2)),
                                 *(qo or view(2, 4)), *(ko or view(3, 2)), *w, *tables, rows, *pos, 0, 0)
    g = None
    if grads:
        g = sequence._ROTATE_GRADS.pack(*view(10, 4), *view(11, 2), 20 << 44, 21 << 44)
    info, n, L = binding.PlanInfo(), ctypes.c_size_t(), binding.lib()
    binding._check(L.es_plan_qk_norm_rotate(args, g, ctypes.byref(info)))
    binding._check(L.es_qk_norm_rotate_workspace(args, g, ctypes.byref(n)))
    return info, n.value


def test_rotate_plans():
    info, n = rotate()
    assert (info.O, info.T, info.J, info.W, info.path) == (2, 5, 6, 64, 2) and n == 0
    assert rotate(grads=True)[1] > 0
    assert rotate(B=0)[0].path == 1
    # in place, and beside one another in one tensor
    one = 1 << 44
    q, k = (one, 5 * 6 * 64, 6 * 64, 64, 4), (one + 4 * 64 * 2, 5 * 6 * 64, 6 * 64, 64, 2)
    rotate(q=q, k=k, qo=q, ko=k)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), 2), (dict(wdtype=-1), 2),
    (dict(turned=3), 1), (dict(turned=66), 1), (dict(turned=-2), 1),
    (dict(D=300, turned=64), 4),
    (dict(eps=-1.0), 3), (dict(eps=float("nan")), 3),
    (dict(rows=0), 1), (dict(tables=(0, 8 << 44)), 3), (dict(tables=((7 << 44) + 2, 8 << 44)), 3),
    (dict(q=(0, 1280, 256, 64, 4)), 3),
    (dict(qo=((1 << 44) + 64, 1280, 256, 64, 4)), 3),              # over q, shifted
    (dict(qo=(3 << 44, 1280, 256, 64, 3)), 1),
    (dict(qo=(3 << 44, 0, 256, 64, 4)), 3),
    (dict(ko=(3 << 44, 640, 128, 64, 2)), 3),                      # both results in one place
    (dict(w=((5 << 44) + 1, 0)), 3),
])
def test_rotate_refusals(kw, code):
    with pytest.raises(es.EsError) as e:
        rotate(**kw)
    assert e.value.status == code, e.value


def test_a_workspace_over_an_operand_is_refused():
    """The backward's workspace begins in q, in a gradient; the rotation's in its gradient of q."""
    es.set_path_override("generic")
    B, T, H, D = Q
    view = lambda i: ((i + 1) << 44, T * H * D, H * D, D, H)  # noqa: E731
    for at in ((1 << 44) + 256, (11 << 44) + 4096):
        args = sequence._ATTN.pack(1, B, T, H, D, D, 1.0, *view(0), *view(1), *view(2), *view(3), 5 << 44, T * H, H, 1, 0, 0, 0, 0,
                                   at, 1 << 40)
        grads = sequence._ATTN_GRADS.pack(*view(9), *view(10), *view(11), *view(12), 0, 15 << 44, 0)
        with pytest.raises(es.EsError) as e:
            binding._check(binding.lib().es_plan_linear_attention(args, grads, None))
        assert e.value.status == 3 and "workspace" in e.value.message
    args = sequence._ROTATE.pack(1, 1, 2, 5, 64, 64, 0, 1e-6, *((1 << 44, 1280, 256, 64, 4)), *((2 << 44, 640, 128, 64, 2)),
                                 *((3 << 44, 1280, 256, 64, 4)), *((4 << 44, 640, 128, 64, 2)), 5 << 44, 6 << 44, 7 << 44, 8 << 44,
                                 50, 0, 0, 0, 0, (3 << 44) + 16, 1 << 30)
    grads = sequence._ROTATE_GRADS.pack(*((10 << 44, 1280, 256, 64, 4)), *((11 << 44, 640, 128, 64, 2)), 20 << 44, 21 << 44)
    with pytest.raises(es.EsError) as e:
        binding._check(binding.lib().es_plan_qk_norm_rotate(args, grads, None))
    assert e.value.status == 3 and "workspace" in e.value.message
