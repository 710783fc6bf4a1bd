"""The norm with rotation in the place of its operands: views that share no
element are taken whatever the strides of axes with one entry, and those that
do are refused."""
import itertools

import pytest
import torch

import element_scan_recurrences_gb300 as es
from element_scan_recurrences_gb300 import binding, sequence

SIZE = 2
HQ, HK, D = 8, 4, 64


@pytest.fixture(scope="module", autouse=True)
def built():
    from element_scan_recurrences_gb300 import build
    build.build()


def plan(B, T, q, k):
    """In place: q and k (first element, batch, token and head stride) are their own results."""
    q, k = ((1 << 44) + SIZE * q[0], *q[1:], HQ), ((1 << 44) + SIZE * k[0], *k[1:], HK)
    args = sequence._ROTATE.pack(1, 1, B, T, D, D, 0, 1e-6, *q, *k, *q, *k, 0, 0, 7 << 44, 8 << 44, 50, 0, 0, 0, 0, 0, 0)
    binding._check(binding.lib().es_plan_qk_norm_rotate(args, None, None))


ROW = (HQ + 2 * HK) * D
AT = HQ * D
GOOD = {
    "fused": (2, 5, (0, 5 * ROW, ROW, D), (AT, 5 * ROW, ROW, D)),
    "one token, its axis made last": (3, 1, (0, ROW, HQ * D, D), (AT, ROW, HK * D, D)),
    "one token, odd strides": (3, 1, (0, ROW, 1, D), (AT, ROW, 7, D)),
    "one row": (1, 5, (0, 3, ROW, D), (AT, 11, ROW, D)),
    "one row and token": (1, 1, (0, 0, 0, D), (AT, 1, 2, D)),
    "tokens first": (2, 5, (0, ROW, 2 * ROW, D), (AT, ROW, 2 * ROW, D)),
    "keys before queries": (3, 1, (HK * D, ROW, HQ * D, D), (0, ROW, HK * D, D)),
}
BAD = {
    "one token, rows into the next": (3, 1, (0, AT, HQ * D, D), (AT, AT, HK * D, D)),
    "one token, shifted": (3, 1, (0, ROW, 1, D), (AT - D, ROW, 1, D)),
    "one row, rows into the next": (1, 5, (0, 0, AT + D, D), (AT, 0, AT + D, D)),
    "one row and token, shifted": (1, 1, (0, 0, 0, D), (AT - 8, 0, 0, D)),
    "tokens first, rows into the next": (2, 5, (0, AT, 2 * AT, D), (AT, AT, 2 * AT, D)),
    "rows of both axes interleaved": (2, 5, (0, 2 * ROW, ROW, D), (AT, 2 * ROW, ROW, D)),
}


def elements(B, T, x, heads):
    return [x[0] + b * x[1] + t * x[2] + h * x[3] + i for b, t, h, i in itertools.product(range(B), range(T), range(heads), range(D))]


@pytest.mark.parametrize("name", GOOD)
def test_apart(name):
    B, T, q, k = GOOD[name]
    at = elements(B, T, q, HQ) + elements(B, T, k, HK)
    assert len(set(at)) == len(at)
    plan(B, T, q, k)


@pytest.mark.parametrize("name", BAD)
def test_overlapping(name):
    B, T, q, k = BAD[name]
    at = elements(B, T, q, HQ) + elements(B, T, k, HK)
    assert len(set(at)) < len(at)
    with pytest.raises(es.EsError) as e:
        plan(B, T, q, k)
    assert e.value.status == 3, e.value


@pytest.mark.gpu
def test_decoding_in_place():
    """Queries and keys of one step, cut from a fused projection of all rows: in place as by themselves."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qkv = torch.randn(5, 24, 64, device="cuda").bfloat16()
    ang = torch.rand(50, 32, device="cuda") * 6
    w = torch.rand(64, device="cuda").bfloat16()
    pos = torch.tensor([[3], [0], [49], [7], [7]], dtype=torch.int32, device="cuda")
    q, k = qkv[:, :8].unsqueeze(1), qkv[:, 8:16].unsqueeze(1)
    want = es.qk_norm_rotate(q.contiguous(), k.contiguous(), w, w, ang.cos(), ang.sin(), positions=pos)
    rest = qkv[:, 16:].clone()
    got = es.qk_norm_rotate(q, k, w, w, ang.cos(), ang.sin(), positions=pos, q_out=q, k_out=k)
    es.device_status()
    assert got[0] is q and got[1] is k
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, 16:], rest)
