"""The state-space operators together as a layer trains and serves with them
(examples/state_space_layer.py), captured and replayed, and offsets that pass 32
bits."""
import os
import sys

import numpy as np
import pytest
import torch

import element_scan_recurrences_gb300 as es
import oracle.state_space as S
from element_scan_recurrences_gb300 import autograd as ag

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    es.lib()


def test_the_example_runs_and_serves():
    """Single tokens predict what the whole sequence predicts: x, the steps, the
    selections and the results are rounded to bf16 on both ways (2^-8 each, some ten
    roundings in a row), in the same places, so the logits agree to 2^-5."""
    import state_space_layer
    losses, far, _ = state_space_layer.main(5)
    assert len(losses) == 5 and all(np.isfinite(losses))
    assert far <= 2.0 ** -5, far


def pieces(dtype, B=2, T=45, C=32, N=16, G=4, W=4):
    gen = torch.Generator(device="cuda").manual_seed(0)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    return dict(xz=n(B, T, 2 * C).to(dtype), w=(n(C, W) / 2).to(dtype), b=(0.1 * n(C)).to(dtype), delta=n(B, T, C).to(dtype),
                A=-(n(C, N).abs() + 0.1), B=n(B, T, 1, N).to(dtype), C=n(B, T, 1, N).to(dtype), D=n(C), bias=n(C) - 2,
                nw=(1 + 0.1 * n(G, C // G)).to(dtype), nb=(0.1 * n(G, C // G)).to(dtype), go=n(B, T, G, C // G).to(dtype)), G


def layer(p, G, lengths=None):
    x, z = p["xz"].split(p["w"].shape[0], -1)
    x, _ = ag.causal_conv(x, p["w"], p["b"], lengths=lengths)
    y, _ = ag.selective_scan(x, p["delta"], p["A"], p["B"], p["C"], p["D"], None, p["bias"], lengths=lengths)
    return ag.group_norm(y.unflatten(-1, (G, -1)), p["nw"], p["nb"], z.unflatten(-1, (G, -1)))


def test_a_layer_against_the_oracle():
    """Convolution, scan and norm in a row, forwards and backwards in f32, against the
    oracle's in 64 bits.  Each operator is off by less than 1e-5 of its terms' sums
    (their own tests); the norm divides by deviations of about 1, and the scan's
    gradients sum 45 tokens: 1e-3 of the largest value holds for all."""
    p, G = pieces(torch.float32)
    names = [k for k in p if k != "go"]
    leaves = {k: p[k].clone().requires_grad_(True) for k in names}
    out = layer(leaves, G)
    out.backward(p["go"])
    q = {k: v.double().cpu().numpy() for k, v in p.items()}
    C = q["w"].shape[0]
    x0, z = q["xz"][..., :C], q["xz"][..., C:]
    x1, _ = S.causal_conv(x0, q["w"], q["b"])
    y, _ = S.selective_scan(x1, q["delta"], q["A"], q["B"], q["C"], q["D"], None, q["bias"])
    cut = lambda v: v.reshape(*v.shape[:2], G, -1)  # noqa: E731
    want = S.group_norm(cut(y), q["nw"], q["nb"], cut(z))
    gy, gnw, gnb, gz = S.group_norm_backward(cut(y), q["nw"], q["nb"], cut(z), q["go"])
    g = S.selective_scan_backward(x1, q["delta"], q["A"], q["B"], q["C"], q["D"], None, q["bias"], gy.reshape(y.shape))
    gx, gw, gb, _ = S.causal_conv_backward(x0, q["w"], q["b"], g[0])
    grads = dict(xz=np.concatenate([gx, gz.reshape(y.shape)], -1), w=gw, b=gb, delta=g[1], A=g[2], B=g[3], C=g[4], D=g[5], bias=g[7],
                 nw=gnw, nb=gnb)
    for name, got, ref in [("out", out, want)] + [(k, leaves[k].grad, grads[k]) for k in names]:
        err = np.abs(got.detach().double().cpu().numpy() - ref).max() / np.abs(ref).max()
        assert err <= 1e-3, (name, err)


def test_padding_changes_nothing():
    """A row's results are the same bits however far its batch is padded."""
    p, G = pieces(torch.bfloat16)
    args = [p[k] for k in ("delta", "A", "B", "C", "D")]
    x = p["xz"][..., :32]
    whole, state, _ = es.selective_scan(x, *args, None, p["bias"], final_state=True, lengths=torch.tensor([19, 45], dtype=torch.int32, device="cuda"))
    cut = [v[:1, :19] if v.dim() > 2 else v for v in args]
    alone, one, _ = es.selective_scan(x[:1, :19], *cut, None, p["bias"], final_state=True)
    assert torch.equal(whole[:1, :19], alone) and torch.equal(state[:1], one)
    o, s = es.causal_conv(x, p["w"], p["b"], final_state=True, lengths=torch.tensor([19, 45], dtype=torch.int32, device="cuda"))
    o1, s1 = es.causal_conv(x[:1, :19], p["w"], p["b"], final_state=True)
    assert torch.equal(o[:1, :19], o1) and torch.equal(s[:1], s1)


def test_a_captured_layer_with_gradients():
    """A training pass of the three operators in one graph, through the entry points
    that autograd calls, replayed on other inputs."""
    p, G = pieces(torch.bfloat16)
    x, z = p["xz"].split(32, -1)
    cut = lambda v: v.unflatten(-1, (G, -1))  # noqa: E731

    def run():
        x1, _ = es.causal_conv(x, p["w"], p["b"])
        args = (x1, p["delta"], p["A"], p["B"], p["C"], p["D"], None, p["bias"])
        y, _, kept = es.selective_scan(*args, checkpoints=True)
        out = es.group_norm(cut(y), p["nw"], p["nb"], cut(z))
        g = es.group_norm_backward(cut(y), p["nw"], p["nb"], cut(z), p["go"])
        gs = es.selective_scan_backward(*args, g[0].flatten(2), checkpoints=kept)
        return (out,) + g + tuple(t for t in gs if t is not None) + es.causal_conv_backward(x, p["w"], p["b"], gs[0])[:3]

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    p["xz"].normal_()
    p["go"].normal_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, run()):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Two rows more than 2^31 elements apart: the second row's results are those of a small call."""
    C, T, N, gap = 32, 40, 16, (1 << 31) + 64
    gen = torch.Generator(device="cuda").manual_seed(1)
    made = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731

    def far(t):          # [2, ...]: the second row far behind the first
        box = torch.empty(gap + t[0].numel(), dtype=t.dtype, device="cuda")
        v = box.as_strided(t.shape, (gap,) + t[0].stride())
        v.copy_(t)
        return v

    x, delta, go = made(2, T, C), made(2, T, C), made(2, T, C)
    b, c = made(2, T, 1, N), made(2, T, 1, N)
    a, w = -torch.rand(C, N, generator=gen, device="cuda"), made(C, 4)
    xf, df, gf = far(x), far(delta), far(go)
    out = far(torch.zeros_like(x))
    got = es.selective_scan(xf, df, a, b, c, out=out)[0]
    assert torch.equal(got, es.selective_scan(x, delta, a, b, c)[0])
    for p, q in zip(es.selective_scan_backward(xf, df, a, b, c, None, None, None, gf),
                    es.selective_scan_backward(x, delta, a, b, c, None, None, None, go)):
        assert p is q is None or torch.equal(p, q)
    assert torch.equal(es.causal_conv(xf, w, out=out)[0], es.causal_conv(x, w)[0])
    for p, q in zip(es.causal_conv_backward(xf, w, None, gf), es.causal_conv_backward(x, w, None, go)):
        assert p is q is None or torch.equal(p, q)
    cut = lambda t: t.unflatten(-1, (2, -1))  # noqa: E731
    assert torch.equal(es.group_norm(cut(xf), out=cut(out)), es.group_norm(cut(x)))
    assert torch.equal(es.group_norm_backward(cut(xf), None, None, None, cut(gf))[0],
                       es.group_norm_backward(cut(x), None, None, None, cut(go))[0])


def test_long_checkpoints():
    """Checkpoints of more than 2^32 bytes: the last token's gradients are those of the last tokens alone."""
    B, T, C, N = 1, 16 * 4100, 4096, 64
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(B, T, C, generator=gen, device="cuda", dtype=torch.bfloat16)
    delta = torch.full((B, T, C), 2.0, device="cuda", dtype=torch.bfloat16)          # steps of 2.1: e^-2.1 a token and more
    a = -(1 + torch.rand(C, N, generator=gen, device="cuda"))
    b, c = (torch.randn(B, T, 1, N, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    out, last, kept = es.selective_scan(x, delta, a, b, c, final_state=True, checkpoints=True)
    assert kept.numel() > 1 << 32
    g = es.selective_scan_backward(x, delta, a, b, c, None, None, None, out, checkpoints=kept)
    # 64 tokens back nothing is left (e^-134)
    cut = lambda t: t[:, -128:]  # noqa: E731
    o2, l2, _ = es.selective_scan(cut(x), cut(delta), a, cut(b), cut(c), final_state=True)
    g2 = es.selective_scan_backward(cut(x), cut(delta), a, cut(b), cut(c), None, None, None, o2)
    # a state is a sum in which each token's rounding fades with the token: 2^-20 of its size of about 2
    assert torch.allclose(last, l2, rtol=2.0 ** -20, atol=2.0 ** -19)
    assert torch.allclose(out[:, -64:].float(), o2[:, -64:].float(), rtol=2.0 ** -7, atol=2.0 ** -7)
    for i in (0, 1, 3, 4):
        assert torch.allclose(g[i][:, -64:].float(), g2[i][:, -64:].float(), rtol=2.0 ** -7, atol=2.0 ** -7), i


def test_autograd_in_a_graph():
    """Forward and backward of the layer through autograd in one graph, replayed on
    other inputs.  (No eager graph of the same leaves may live meanwhile: PyTorch's
    own nodes of the leaves then wait on the stream it was made on.)"""
    p, G = pieces(torch.float32)
    leaves = {k: p[k].requires_grad_(True) for k in p if k != "go"}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            torch.autograd.grad(layer(leaves, G), list(leaves.values()), p["go"])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(leaves, G)
        got = torch.autograd.grad(out, list(leaves.values()), p["go"])
    with torch.no_grad():
        p["xz"].normal_()
        p["delta"].normal_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, torch.autograd.grad(layer(leaves, G), list(leaves.values()), p["go"])):
        assert torch.equal(a, b)


def test_calls_on_two_streams():
    """Two calls at once, each with its own results: those of one after the other."""
    sides = [torch.cuda.Stream() for _ in range(2)]
    cases = []
    for seed in range(2):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
        x, delta, go, b, c = n(2, 600, 256), n(2, 600, 256), n(2, 600, 256), n(2, 600, 1, 16), n(2, 600, 1, 16)
        a = -torch.rand(256, 16, generator=gen, device="cuda") - 0.1
        cases.append(((x, delta, a, b, c, None, None, None), go))

    def run(case):
        args, go = case
        out, _, kept = es.selective_scan(*args, checkpoints=True)
        return (out,) + tuple(t for t in es.selective_scan_backward(*args, go, checkpoints=kept) if t is not None)

    want = [run(c) for c in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(sides):
            with torch.cuda.stream(s):
                got[i] = run(cases[i])
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        for p, q in zip(x, y):
            assert torch.equal(p, q)
