"""Workloads of the state-space layer's operators: the short causal convolution,
the selective scan, and the group norm with a gate.

``listed()`` and ``draw()`` give cases, ``prepare()`` the tensors a program has
in hand, ``run()`` one pass: with ``own`` the library's entry points, without
it the operators' plain form in 32-bit torch operations.  ``exact()`` gives
the same outputs from the definitions in 64 bits.

Convolution, for each channel (s the logistic function, tokens before the first
those of the carried state):

    p[t] = bias + sum_j w[j] x[t - W + 1 + j],   out[t] = p[t] s(p[t])

Selective scan, for each channel, state h of N values (B, C of its group):

    d[t] = log(1 + exp(delta[t] + bias))
    h[t, n] = exp(d[t] A[n]) h[t-1, n] + d[t] x[t] B[t, n]
    out[t] = (sum_n C[t, n] h[t, n] + D x[t]) * gate[t] s(gate[t])

Group norm, for each group of a token's channels: (x - mean) / sqrt(var + eps)
* w + b, times gate s(gate); or, for `first`, x gate s(gate) / sqrt(mean
square + eps) * w.
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases

def _conv(name, op, dtype, b, t, c, w, ragged=False, carry=False):
    """`op` conv, conv_train or conv_step; `w` taps; `ragged`: the rows of the
    batch have lengths of their own; `carry`: a state comes in and goes out
    (and its gradient the other way)."""
    return {"name": name, "op": op, "dtype": dtype, "b": b, "t": t, "c": c, "w": w, "ragged": ragged, "carry": carry}


def _scan(name, op, dtype, b, t, c, n=16, groups=1, gate=True, ragged=False, carry=False):
    """`op` scan, scan_train or scan_step; `c` channels with `n` states each,
    B and C shared by the channels of one of `groups` groups."""
    return {"name": name, "op": op, "dtype": dtype, "b": b, "t": t, "c": c, "n": n, "groups": groups, "gate": gate,
            "ragged": ragged, "carry": carry}


def _norm(name, op, dtype, b, t, h, d, first=False):
    """`op` norm or norm_train; `h` groups of `d` channels; `first`: the gate
    comes before the norm, which is without mean and bias."""
    return {"name": name, "op": op, "dtype": dtype, "b": b, "t": t, "h": h, "d": d, "first": first}


def listed():
    return [
        # a short question to an interactive model: latency
        _scan("scan_prompt_short", "scan", "bf16", 1, 37, 2048, carry=True),
        # a batch of prompts of different lengths, padded to the longest
        _scan("scan_prompt_batch", "scan", "bf16", 8, 2048, 4096, ragged=True, carry=True),
        # one long document: few channels for the machine, many tokens
        _scan("scan_prompt_long", "scan", "bf16", 1, 65536, 2048, carry=True),
        # a training step's layer
        _scan("scan_train", "scan_train", "bf16", 4, 2048, 4096),
        # the framework's own type, an odd length, an uncommon width in groups, states carried between windows
        _scan("scan_train_f32", "scan_train", "f32", 2, 501, 744, groups=3, carry=True),
        # one token of each of many conversations: the states' bandwidth
        _scan("scan_step", "scan_step", "bf16", 256, 1, 4096),
        # a batch of prompts of different lengths
        _conv("conv_prompt", "conv", "bf16", 8, 2048, 4096, 4, ragged=True, carry=True),
        # a training step's layer, both directions
        _conv("conv_train", "conv_train", "bf16", 4, 2047, 4096, 4),
        # one token of each of some conversations: latency
        _conv("conv_step", "conv_step", "bf16", 64, 1, 4096, 4),
        # the heads' outputs of a prompt, normed one by one and gated
        _norm("norm_prompt", "norm", "bf16", 1, 16384, 16, 128),
        # a training step's layer, both directions
        _norm("norm_train", "norm_train", "bf16", 4, 4096, 16, 128),
        # one wide group, the gate before the norm, in the framework's own type, an odd length
        _norm("norm_train_f32", "norm_train", "f32", 2, 777, 1, 2560, first=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_train", "scan_train", "scan_step", "conv", "conv_train", "conv_step", "norm",
                     "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    wide = 1 if dtype == "bf16" else 2
    ragged, carry = rng.random() < 0.4, rng.random() < 0.5
    if op.startswith("norm"):
        h = rng.choice([1, 1, 2, 8, 12, 16])
        d = rng.choice([64, 80, 96, 128, 256]) if h > 2 else 8 * _log(rng, 16, 768)
        b = _log(rng, 1, 64)
        t = _log(rng, 1, max(1, min(32768, (1 << 25) // (b * h * d * wide))))
        c = _norm("", op, dtype, b, t, h, d, rng.random() < 0.4)
    elif op.startswith("conv"):
        ch = 8 * _log(rng, 16, 1024) if rng.random() < 0.8 else _log(rng, 100, 4000)
        w = rng.choice([2, 3, 4, 4, 4])
        b = _log(rng, 1, 64)
        most = (1 << 26) // wide // (2 if op == "conv_train" else 1)
        t = 1 if op == "conv_step" else _log(rng, 1, max(1, min(32768, most // (b * ch))))
        c = _conv("", op, dtype, b, t, ch, w, ragged and t > 1, carry)
    else:
        groups = rng.choice([1, 1, 1, 2, 4])
        ch = groups * (8 * _log(rng, 8, 640 // groups) if rng.random() < 0.8 else _log(rng, 30, 1500))
        n = rng.choice([16, 16, 16, 16, 8, 12, 32, 64])
        gate = rng.random() < 0.7
        if op == "scan_step":
            b = _log(rng, 2, max(2, min(512, (1 << 24) // (ch * n))))
            c = _scan("", op, dtype, b, 1, ch, n, groups, gate)
        else:
            b = _log(rng, 1, 16)
            most = (1 << 30 if op == "scan" else 1 << 28) // wide // max(n, 16)
            t = _log(rng, 1, max(1, min(32768, most // (b * ch))))
            c = _scan("", op, dtype, b, t, ch, n, groups, gate, ragged and t > 1, carry)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    dtype = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEVICE)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=DEVICE)

    op, b, t, s = case["op"], case["b"], case["t"], {"case": dict(case)}
    train = op.endswith("_train")
    lead = (b,) if op.endswith("_step") else (b, t)
    if op.startswith("norm"):
        h, d = case["h"], case["d"]
        s["x"], s["gate"] = normal(b, t, h, d).to(dtype), normal(b, t, h, d).to(dtype)
        s["w"] = (1 + 0.1 * normal(h, d)).to(dtype)
        s["b"] = None if case["first"] else (0.1 * normal(h, d)).to(dtype)
        if train:
            s["go"] = normal(b, t, h, d).to(dtype)
        return s
    s["lengths"] = None
    if case["ragged"]:
        s["lengths"] = torch.randint(max(1, t // 4), t + 1, (b,), generator=gen, device=DEVICE).to(torch.int32)
    c = case["c"]
    if op.startswith("conv"):
        # half of a fused projection's result: a view of rows twice as long
        s["x"] = normal(*lead, 2 * c).to(dtype)[..., :c]
        s["w"], s["b"] = (normal(c, case["w"]) / math.sqrt(case["w"])).to(dtype), (0.1 * normal(c)).to(dtype)
        carry = case["carry"] or op == "conv_step"
        s["state"] = normal(b, case["w"] - 1, c).to(dtype) if carry else None
        if op == "conv_step":
            s["next"] = torch.empty_like(s["state"])
        if train:
            s["go"] = normal(b, t, c).to(dtype)
            s["gstate"] = normal(b, case["w"] - 1, c).to(dtype) if carry else None
        return s
    n, groups = case["n"], case["groups"]
    x = normal(*lead, c)
    s["x"] = (x * torch.sigmoid(x)).to(dtype)
    s["delta"] = (0.7 * normal(*lead, c)).to(dtype)
    s["A"] = -(1 + torch.arange(n, device=DEVICE, dtype=torch.float32)) * (0.8 + 0.4 * uniform(c, n))
    # B and C lie in one projection's result
    bc = normal(*lead, 2, groups, n).to(dtype)
    s["B"], s["C"] = bc.select(-3, 0), bc.select(-3, 1)
    s["D"] = 1 + 0.1 * normal(c)
    s["gate"] = normal(*lead, c).to(dtype) if case["gate"] else None
    # steps from a thousandth to a tenth
    first = torch.exp(uniform(c) * math.log(100.0) + math.log(1e-3))
    s["bias"] = first + torch.log(-torch.expm1(-first))
    carry = case["carry"] or op == "scan_step"
    s["state"] = normal(b, c, n) if carry else None
    if op == "scan_step":
        s["next"] = torch.empty_like(s["state"])
    if train:
        s["go"] = normal(b, t, c).to(dtype)
        s["gstate"] = normal(b, c, n) if carry else None
    return s


# ---------------------------------------------------------------------------
# one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"conv": _own_conv, "conv_train": _own_conv_train, "conv_step": _own_conv_step, "scan": _own_scan,
                "scan_train": _own_scan_train, "scan_step": _own_scan_step, "norm": _own_norm,
                "norm_train": _own_norm_train}[op](s)
    return {"conv": _plain_conv, "conv_train": _plain_conv_train, "conv_step": _plain_conv_step, "scan": _plain_scan,
            "scan_train": _plain_scan_train, "scan_step": _plain_scan_step, "norm": _plain_norm,
            "norm_train": _plain_norm_train}[op](s)


def _es():
    import element_scan_recurrences_gb300 as es
    return es


def _own_conv(s):
    o, state = _es().causal_conv(s["x"], s["w"], s["b"], initial_state=s["state"], lengths=s["lengths"], final_state=True)
    return {"o": o, "state": state}


def _own_conv_train(s):
    es, carry = _es(), s["state"] is not None
    kw = dict(initial_state=s["state"], lengths=s["lengths"])
    o, state = es.causal_conv(s["x"], s["w"], s["b"], final_state=carry, **kw)
    gx, gw, gb, gi = es.causal_conv_backward(s["x"], s["w"], s["b"], s["go"], grad_final_state=s["gstate"], **kw)
    out = {"o": o, "gx": gx, "gw": gw, "gb": gb}
    if carry:
        out.update(state=state, ginitial=gi)
    return out


def _own_conv_step(s):
    o, state = _es().causal_conv_step(s["x"], s["w"], s["b"], s["state"], state_out=s["next"])
    return {"o": o, "state": state}


def _own_scan(s):
    o, state, _ = _es().selective_scan(s["x"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["gate"], s["bias"],
                                       initial_state=s["state"], lengths=s["lengths"], final_state=True)
    return {"o": o, "state": state}


def _own_scan_train(s):
    es, carry = _es(), s["state"] is not None
    args = (s["x"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["gate"], s["bias"])
    kw = dict(initial_state=s["state"], lengths=s["lengths"])
    o, state, kept = es.selective_scan(*args, final_state=carry, checkpoints=True, **kw)
    gx, gdelta, ga, gb, gc, gd, ggate, gbias, gi = es.selective_scan_backward(
        *args, s["go"], grad_final_state=s["gstate"], checkpoints=kept, **kw)
    out = {"o": o, "gx": gx, "gdelta": gdelta, "gA": ga, "gB": gb, "gC": gc, "gD": gd, "gbias": gbias}
    if s["gate"] is not None:
        out["ggate"] = ggate
    if carry:
        out.update(state=state, ginitial=gi)
    return out


def _own_scan_step(s):
    o, state = _es().selective_scan_step(s["x"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["gate"], s["bias"],
                                         s["state"], state_out=s["next"])
    return {"o": o, "state": state}


def _own_norm(s):
    first = s["case"]["first"]
    return {"o": _es().group_norm(s["x"], s["w"], s["b"], s["gate"], gate_first=first, center=not first, eps=EPS)}


def _own_norm_train(s):
    es, first = _es(), s["case"]["first"]
    kw = dict(gate_first=first, center=not first, eps=EPS)
    o = es.group_norm(s["x"], s["w"], s["b"], s["gate"], **kw)
    gx, gw, gb, ggate = es.group_norm_backward(s["x"], s["w"], s["b"], s["gate"], s["go"], **kw)
    out = {"o": o, "gx": gx, "gw": gw, "ggate": ggate}
    if not first:
        out["gb"] = gb
    return out


# the plain forms

def _silu(x):
    return x / (1 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _live(s, lengths, t):
    """[B, T, 1] truth values, or None where every token counts."""
    if lengths is None:
        return None
    return (torch.arange(t, device=s.device)[None] < lengths[:, None])[..., None]


def _conv32(x, w, b, state, lengths):
    """out [B, T, C] in 32 bits and the last W - 1 inputs."""
    n, t, c = x.shape
    taps = w.shape[1]
    if state is None:
        state = torch.zeros(n, taps - 1, c, device=x.device)
    live = _live(x, lengths, t)
    if live is not None:
        x = torch.where(live, x, 0.0)
    row = torch.cat([state, x], 1)
    p = b
    for j in range(taps):
        p = p + w[:, j] * row[:, j:j + t]
    o = _silu(p)
    if live is None:
        return o, row[:, t:]
    at = lengths.long()[:, None] + torch.arange(taps - 1, device=x.device)
    return torch.where(live, o, 0.0), row[torch.arange(n, device=x.device)[:, None], at]


def _plain_conv(s):
    dtype = s["x"].dtype
    state = None if s["state"] is None else s["state"].float()
    o, state = _conv32(s["x"].float(), s["w"].float(), s["b"].float(), state, s["lengths"])
    return {"o": o.to(dtype), "state": state.to(dtype).contiguous()}


def _plain_conv_train(s):
    dtype, carry = s["x"].dtype, s["state"] is not None
    names = ["x", "w", "b"] + (["state"] if carry else [])
    leaves = [s[n].float().detach().requires_grad_(True) for n in names]
    with torch.enable_grad():
        o, state = _conv32(*leaves[:3], leaves[3] if carry else None, s["lengths"])
        outs, gouts = ([o, state], [s["go"].float(), s["gstate"].float()]) if carry else ([o], [s["go"].float()])
        grads = torch.autograd.grad(outs, leaves, gouts)
    out = {"o": o, "gx": grads[0], "gw": grads[1], "gb": grads[2]}
    if carry:
        out.update(state=state, ginitial=grads[3])
    return {n: x.detach().to(dtype).contiguous() for n, x in out.items()}


def _plain_conv_step(s):
    row = torch.cat([s["state"], s["x"][:, None]], 1)
    s["next"].copy_(row[:, 1:])
    p = s["b"].float() + (row.float() * s["w"].float().t()).sum(1)
    return {"o": _silu(p).to(s["x"].dtype), "state": s["next"]}


def _spread(x, c):
    """[..., groups, N] -> [..., C, N]: each channel's group."""
    return x.repeat_interleave(c // x.shape[-2], dim=-2)


def _scan32(x, delta, a, bm, cm, d, gate, bias, state, lengths):
    """out [B, T, C] in 32 bits and the last state: all spans of tokens at
    once from zero, the states between spans, then what each token sees of the
    state that enters its span."""
    n, t, c = x.shape
    live = _live(x, lengths, t)
    step = _softplus(delta + bias)
    if live is not None:
        step, xin = torch.where(live, step, 0.0), torch.where(live, x, 0.0)
        bm, cm = torch.where(live[..., None], bm, 0.0), torch.where(live[..., None], cm, 0.0)
    else:
        xin = x
    span = max(1, int(math.sqrt(t)))
    spans = -(-t // span)

    def cut(v):       # [B, T, ...] -> a list of [B, spans, ...], one for each place in a span
        v = torch.nn.functional.pad(v, (0, 0) * (v.dim() - 2) + (0, spans * span - t))
        return v.reshape(n, spans, span, *v.shape[2:]).unbind(2)

    steps, adds, bs, cs = cut(step), cut(step * xin), cut(bm), cut(cm)
    h = torch.zeros(n, spans, c, a.shape[1], device=x.device)
    ys, since, sums = [], torch.zeros(n, spans, c, device=x.device), []
    for i in range(span):
        h = torch.exp(steps[i][..., None] * a) * h + adds[i][..., None] * _spread(bs[i], c)
        ys.append((h * _spread(cs[i], c)).sum(-1))
        since = since + steps[i]
        sums.append(since)
    enter = []
    state = torch.zeros(n, c, a.shape[1], device=x.device) if state is None else state
    for j in range(spans):
        enter.append(state)
        state = torch.exp(since[:, j, :, None] * a) * state + h[:, j]
    enter = torch.stack(enter, 1)
    ys = [y + (torch.exp(q[..., None] * a) * enter * _spread(m, c)).sum(-1) for y, q, m in zip(ys, sums, cs)]
    y = torch.stack(ys, 2).reshape(n, spans * span, c)[:, :t] + d * xin
    if gate is not None:
        y = y * _silu(gate)
    if live is not None:
        y = torch.where(live, y, 0.0)
    return y, state


def _plain_scan(s):
    f = [None if s[k] is None else s[k].float() for k in ("x", "delta", "A", "B", "C", "D", "gate", "bias", "state")]
    o, state = _scan32(*f, s["lengths"])
    return {"o": o.to(s["x"].dtype), "state": state.contiguous()}


def _plain_scan_train(s):
    dtype, carry, gated = s["x"].dtype, s["state"] is not None, s["gate"] is not None
    names = ["x", "delta", "A", "B", "C", "D"] + (["gate"] if gated else []) + ["bias"] + (["state"] if carry else [])
    leaf = {k: s[k].float().detach().requires_grad_(True) for k in names}
    with torch.enable_grad():
        o, state = _scan32(*(leaf.get(k) for k in ("x", "delta", "A", "B", "C", "D", "gate", "bias", "state")), s["lengths"])
        outs, gouts = ([o, state], [s["go"].float(), s["gstate"]]) if carry else ([o], [s["go"].float()])
        grads = dict(zip(names, torch.autograd.grad(outs, list(leaf.values()), gouts)))
    out = {"o": o.to(dtype)}
    for k in names:
        out["ginitial" if k == "state" else "g" + k] = grads[k].to(s[k].dtype)
    if carry:
        out["state"] = state
    return {k: v.detach().contiguous() for k, v in out.items()}


def _plain_scan_step(s):
    c = s["case"]["c"]
    x, delta, bm, cm = (s[k].float() for k in ("x", "delta", "B", "C"))
    d = _softplus(delta + s["bias"])
    s["next"].copy_(torch.exp(d[..., None] * s["A"]) * s["state"] + (d * x)[..., None] * _spread(bm, c))
    y = (s["next"] * _spread(cm, c)).sum(-1) + s["D"] * x
    if s["gate"] is not None:
        y = y * _silu(s["gate"].float())
    return {"o": y.to(s["x"].dtype), "state": s["next"]}


def _norm32(x, w, b, gate, first):
    if first:
        x = x * _silu(gate)
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    x = x - x.mean(-1, keepdim=True)
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w + b) * _silu(gate)


def _plain_norm(s):
    b = None if s["b"] is None else s["b"].float()
    o = _norm32(s["x"].float(), s["w"].float(), b, s["gate"].float(), s["case"]["first"])
    return {"o": o.to(s["x"].dtype)}


def _plain_norm_train(s):
    dtype, first = s["x"].dtype, s["case"]["first"]
    names = ["x", "w", "gate"] + ([] if first else ["b"])
    leaf = {k: s[k].float().detach().requires_grad_(True) for k in names}
    with torch.enable_grad():
        o = _norm32(leaf["x"], leaf["w"], leaf.get("b"), leaf["gate"], first)
        grads = torch.autograd.grad([o], list(leaf.values()), [s["go"].float()])
    out = {"o": o.detach().to(dtype)}
    out.update({"g" + k: g.to(dtype).contiguous() for k, g in zip(names, grads)})
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    op, tokens = case["op"], case["b"] * case["t"]
    if op.startswith("norm"):
        one, weights = tokens * case["h"] * case["d"], (1 if case["first"] else 2) * case["h"] * case["d"]
        if op == "norm":
            return {"bytes": (3 * one + weights) * size, "flops": 14 * one}
        return {"bytes": (6 * one + 2 * weights) * size, "flops": 40 * one}
    c, b = case["c"], case["b"]
    one = tokens * c
    if op.startswith("conv"):
        w = case["w"]
        state, weights = b * (w - 1) * c, c * (w + 1)
        if op == "conv_train":
            return {"bytes": (4 * one + 2 * weights + (4 * state if case["carry"] else 0)) * size,
                    "flops": (6 * w + 14) * one}
        states = 2 if case["carry"] or op == "conv_step" else 1
        return {"bytes": (2 * one + weights + states * state) * size, "flops": (2 * w + 4) * one}
    n, gate = case["n"], 1 if case["gate"] else 0
    bc, weights, state = 2 * tokens * case["groups"] * n * size, 4 * c * (n + 2), 4 * b * c * n
    if op == "scan_train":
        # x, delta, gate, B, C, out's gradient once; out and the gradients once
        return {"bytes": (6 + 2 * gate) * one * size + 2 * (bc + weights) + (4 * state if case["carry"] else 0),
                "flops": (27 * n + 40) * one}
    states = 2 if case["carry"] or op == "scan_step" else 1
    return {"bytes": (3 + gate) * one * size + bc + weights + states * state, "flops": (7 * n + 20) * one}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(s, case)
    if case["op"].startswith("conv"):
        return _exact_conv(s, case)
    return _exact_scan(s, case)


def _s64(x):
    return torch.sigmoid(x)


def _alive(s, b, t):
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((b,), t, device=DEVICE)
    return n, (torch.arange(t, device=DEVICE)[None] < n[:, None]).double()[..., None]


def _exact_conv(s, case):
    b, t, c, taps, op = case["b"], case["t"], case["c"], case["w"], case["op"]
    w, bias = s["w"].double(), s["b"].double()
    if op == "conv_step":
        p = bias + s["x"].double() * w[:, -1]
        for j in range(taps - 1):
            p = p + s["state"][:, j].double() * w[:, j]
        return {"o": p * _s64(p), "state": torch.cat([s["state"][:, 1:], s["x"][:, None]], 1).double()}
    n, live = _alive(s, b, t)
    x = torch.where(live > 0, s["x"].double(), 0.0)
    before = torch.zeros(b, taps - 1, c, dtype=torch.float64, device=DEVICE) if s["state"] is None else s["state"].double()

    def moved(k):         # the inputs k tokens earlier
        return x if k == 0 else torch.cat([before[:, max(0, taps - 1 - k):taps - 1 - k + t], x[:, :max(0, t - k)]], 1)

    p = bias.expand(b, t, c).clone()
    for k in range(taps):
        p += moved(k) * w[:, taps - 1 - k]
    q = _s64(p)
    out = {"o": p * q * live}
    last = torch.empty_like(before)
    for i in range(b):
        m = int(n[i])
        row = torch.cat([before[i], x[i, :m]], 0)
        last[i] = row[row.shape[0] - taps + 1:]
    if op == "conv":
        out["state"] = last
        return out
    gp = s["go"].double() * live * (q + p * q * (1 - q))
    gx = torch.zeros_like(x)
    gi = torch.zeros_like(before)
    gw = torch.empty_like(w)
    for k in range(taps):
        tap = w[:, taps - 1 - k]
        gw[:, taps - 1 - k] = (gp * moved(k)).sum((0, 1))
        gx[:, :max(0, t - k)] += gp[:, k:] * tap
        for i in range(min(k, t)):          # token i reads the carried input k - i before the first
            gi[:, taps - 1 - k + i] += gp[:, i] * tap
    if s["gstate"] is not None:
        for i in range(b):
            m = int(n[i])
            whole = torch.cat([gi[i], gx[i, :m]], 0)
            whole[whole.shape[0] - taps + 1:] += s["gstate"][i].double()
            gi[i], gx[i, :m] = whole[:taps - 1], whole[taps - 1:]
    out.update(gx=gx * live, gw=gw, gb=gp.sum((0, 1)))
    if case["carry"]:
        out.update(state=last, ginitial=gi)
    return out


def _exact_scan(s, case):
    """Token by token; the gradients from the recurrence run backwards."""
    b, t, c, n, groups, op = (case[k] for k in ("b", "t", "c", "n", "groups", "op"))
    train, step = op == "scan_train", op == "scan_step"
    if t * (4 if train else 1) * max(120e-6, b * c * n * 8 * 10 / 5e12) > 15:
        return None
    if train and b * t * c * n * 8 > 30e9:
        return None

    def tokens(x):        # [T][B, ...]
        return (x[:, None] if step else x).double().unbind(1)

    def spread(x):        # [B, groups, N] -> [B, C, N]
        return x[:, :, None].expand(b, groups, c // groups, n).reshape(b, c, n)

    _, live = _alive(s, b, t) if not step else (None, torch.ones(b, 1, 1, dtype=torch.float64, device=DEVICE))
    a, skip, bias = s["A"].double(), s["D"].double(), s["bias"].double()
    raw, x = [v + bias for v in tokens(s["delta"])], tokens(s["x"])
    bm, cm = tokens(s["B"]), tokens(s["C"])
    gate = None if s["gate"] is None else tokens(s["gate"])
    state = torch.zeros(b, c, n, dtype=torch.float64, device=DEVICE) if s["state"] is None else s["state"].double()
    o, kept = torch.empty(b, t, c, dtype=torch.float64, device=DEVICE), []
    ds = []
    for i in range(t):
        on = live[:, i]
        d = torch.logaddexp(raw[i], torch.zeros_like(raw[i])) * on
        if train:
            kept.append(state)
            ds.append(d)
        state = torch.exp(d[..., None] * a) * state + (d * x[i])[..., None] * spread(bm[i])
        y = torch.einsum("bcn,bcn->bc", state, spread(cm[i])) + skip * x[i]
        if gate is not None:
            y = y * gate[i] * _s64(gate[i])
        o[:, i] = y * on
    if not train:
        return {"o": o[:, 0] if step else o, "state": state}
    go = tokens(s["go"])
    gs = torch.zeros_like(state) if s["gstate"] is None else s["gstate"].double()
    gx, gdelta, ggate = torch.zeros_like(o), torch.zeros_like(o), torch.zeros_like(o)
    gb = torch.zeros(b, t, groups, n, dtype=torch.float64, device=DEVICE)
    gc, ga, gd = torch.zeros_like(gb), torch.zeros_like(a), torch.zeros_like(skip)
    after = state
    for i in range(t - 1, -1, -1):
        on, d, before = live[:, i], ds[i], kept[i]
        g = go[i] * on
        if gate is not None:
            z, q = gate[i], _s64(gate[i])
            y = torch.einsum("bcn,bcn->bc", after, spread(cm[i])) + skip * x[i]
            ggate[:, i] = g * y * (q + z * q * (1 - q))
            g = g * z * q
        gc[:, i] = (after * g[..., None]).reshape(b, groups, c // groups, n).sum(2)
        gd += (g * x[i]).sum(0)
        gs = gs + g[..., None] * spread(cm[i])
        gb[:, i] = (gs * (d * x[i])[..., None]).reshape(b, groups, c // groups, n).sum(2)
        of_b = (gs * spread(bm[i])).sum(-1)
        gx[:, i] = (of_b * d + g * skip) * on
        fade = torch.exp(d[..., None] * a)
        through = gs * fade * before
        ga += (through * d[..., None]).sum(0)
        gdelta[:, i] = ((through * a).sum(-1) + of_b * x[i]) * _s64(raw[i]) * on
        gs = gs * fade
        after = before
    out = {"o": o, "gx": gx, "gdelta": gdelta, "gA": ga, "gB": gb, "gC": gc, "gD": gd, "gbias": gdelta.sum((0, 1))}
    if gate is not None:
        out["ggate"] = ggate
    if case["carry"]:
        out.update(state=state, ginitial=gs)
    return out


def _exact_norm(s, case):
    x, w, z, first = s["x"].double(), s["w"].double(), s["gate"].double(), case["first"]
    q = _s64(z)
    u = x * z * q if first else x - x.sum(-1, keepdim=True) / case["d"]
    size = ((u * u).sum(-1, keepdim=True) / case["d"] + EPS).sqrt()
    unit = u / size
    y = unit * w if first else unit * w + s["b"].double()
    out = {"o": y if first else y * z * q}
    if case["op"] == "norm":
        return out
    g = s["go"].double()
    slope = q + z * q * (1 - q)
    gy = g if first else g * z * q
    out["gw"] = (gy * unit).sum((0, 1))
    gu = gy * w
    gu = (gu - unit * (gu * unit).sum(-1, keepdim=True) / case["d"]) / size
    if first:
        out.update(gx=gu * z * q, ggate=gu * x * slope)
    else:
        out.update(gx=gu - gu.sum(-1, keepdim=True) / case["d"], ggate=g * y * slope, gb=gy.sum((0, 1)))
    return out
