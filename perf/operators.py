"""Workloads of the sequence-layer operators: linear attention with a decay for
each head, and the norm of queries and keys with the position rotation.

``listed()`` and ``draw()`` give cases, ``prepare()`` the tensors a program has
in hand, ``run()`` one pass: with ``own`` the library's entry points, without
it the operators' plain form in 32-bit torch operations.  ``exact()`` gives
the same outputs from the definitions in 64 bits.

Linear attention, for each head, state h of Dk x Dv values:

    h[t] = exp(g[t]) * h[t-1] + k[t] v[t]^T,   o[t] = scale * q[t] h[t]

Norm and rotation, for each head of q and k: x / sqrt(mean(x^2) + eps) * w,
then pairs of the first R values turned by the angles of the token's position.
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases

def _attend(name, op, dtype, b, t, h, dk, dv, hq=None, hk=None, hv=None, decay="token", ragged=False, carry=True):
    """`op` prompt, train or step; `decay` "token" (a value for every token and
    head, as a learned gate gives) or "head" (one fixed value a head);
    `ragged`: the rows of the batch have lengths of their own; `carry`: a
    state comes in and goes out (and its gradient the other way)."""
    return {"name": name, "op": op, "dtype": dtype, "b": b, "t": t, "h": h, "hq": hq or h, "hk": hk or h,
            "hv": hv or h, "dk": dk, "dv": dv, "decay": decay, "ragged": ragged, "carry": carry}


def _rotate(name, op, dtype, b, t, hq, hk, d, turned, neighbours=False):
    """`op` rotate or rotate_train; `turned`: how many of the d values turn;
    `neighbours`: pairs are neighbours, not halves."""
    return {"name": name, "op": op, "dtype": dtype, "b": b, "t": t, "hq": hq, "hk": hk, "d": d, "turned": turned,
            "neighbours": neighbours}


def listed():
    return [
        # a short question to an interactive model: latency
        _attend("prompt_short", "prompt", "bf16", 1, 37, 16, 64, 64),
        # a batch of prompts of different lengths, padded to the longest
        _attend("prompt_batch", "prompt", "bf16", 8, 2048, 16, 128, 128, ragged=True),
        # one long document, fixed decays
        _attend("prompt_long", "prompt", "bf16", 1, 65536, 16, 128, 128, decay="head"),
        # a small research model in the framework's own type, an odd length
        _attend("train_small_f32", "train", "f32", 2, 501, 8, 64, 64, decay="head", carry=True),
        # a training step's layer, queries and keys shared by four heads, values narrower than the keys
        _attend("train_shared", "train", "bf16", 4, 2047, 16, 128, 64, hq=4, hk=4, carry=False),
        # a training step's layer at full width
        _attend("train_wide", "train", "bf16", 8, 4096, 16, 128, 128, carry=False),
        # one token of one conversation: latency
        _attend("step_one", "step", "bf16", 1, 1, 16, 128, 128),
        # one token of each of many conversations: the states' bandwidth
        _attend("step_many", "step", "bf16", 256, 1, 16, 128, 128),
        # the queries and keys of one decoding step
        _rotate("rotate_tokens", "rotate", "bf16", 32, 1, 32, 8, 128, 128),
        # the queries and keys of a prompt, fewer key heads than query heads
        _rotate("rotate_prompt", "rotate", "bf16", 1, 16384, 32, 8, 128, 128),
        # a training step's layer, a part of each head turned, both directions
        _rotate("rotate_train", "rotate_train", "bf16", 4, 4096, 16, 16, 128, 64),
        # the framework's own type, neighbouring pairs, an odd length and an uncommon width
        _rotate("rotate_train_f32", "rotate_train", "f32", 2, 777, 12, 12, 80, 32, neighbours=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "train", "train", "step", "rotate", "rotate_train"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    size = 2 if dtype == "bf16" else 4
    if op in ("rotate", "rotate_train"):
        hq = rng.choice([4, 8, 12, 16, 32])
        hk = rng.choice([hq, max(1, hq // 4)])
        d = rng.choice([64, 80, 96, 128, 128])
        turned = rng.choice([d, d, 32])
        b = _log(rng, 1, 64)
        t = _log(rng, 1, max(1, min(32768, (1 << 27) // (b * (hq + hk) * d * size))))
        c = _rotate("", op, dtype, b, t, hq, hk, d, turned, rng.random() < 0.3)
    else:
        dk, dv = rng.choice([(64, 64), (128, 128), (128, 64), (64, 128), (96, 96), (80, 80)])
        h = rng.choice([2, 4, 8, 12, 16, 24, 32])
        few = h if h % 4 else h // 4
        hq, hk, hv = rng.choice([(h, h, h), (h, h, h), (few, few, h), (h, few, few)])
        decay = rng.choice(["token", "head"])
        carry = rng.random() < 0.5
        if op == "step":
            b = _log(rng, 2, min(512, 4096 // h))
            c = _attend("", op, dtype, b, 1, h, dk, dv, hq, hk, hv, decay)
        else:
            most = (1 << 26) // (2 if dtype == "f32" else 1) // (2 if op == "train" else 1)   # b*t*h*d
            b = _log(rng, 1, 16)
            t = _log(rng, 1, max(1, min(32768, most // (b * h * max(dk, dv)))))
            c = _attend("", op, dtype, b, t, h, dk, dv, hq, hk, hv, decay, rng.random() < 0.5, carry)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs

def _scale(case):
    return 1.0 / math.sqrt(case["dk"])


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    dtype = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEVICE)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=DEVICE)

    b, t, s = case["b"], case["t"], {"case": dict(case)}
    if case["op"] in ("rotate", "rotate_train"):
        d, r = case["d"], case["turned"]
        # q and k as a fused projection leaves them: views of one tensor
        qkv = normal(b, t, case["hq"] + case["hk"], d).to(dtype)
        s["q"], s["k"] = qkv[:, :, :case["hq"]], qkv[:, :, case["hq"]:]
        s["wq"], s["wk"] = (1 + 0.1 * normal(d)).to(dtype), (1 + 0.1 * normal(d)).to(dtype)
        rows = max(2 * t, 4096)
        angle = torch.arange(rows, device=DEVICE, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(r // 2, device=DEVICE, dtype=torch.float64) * 2 / r)
        s["cos"], s["sin"] = angle.cos().float().contiguous(), angle.sin().float().contiguous()
        # every row of the batch begins at a position of its own
        first = torch.randint(0, rows - t + 1, (b, 1), generator=gen, device=DEVICE)
        s["positions"] = (first + torch.arange(t, device=DEVICE)[None]).to(torch.int32).contiguous()
        if case["op"] == "rotate_train":
            s["gq"], s["gk"] = normal(b, t, case["hq"], d).to(dtype), normal(b, t, case["hk"], d).to(dtype)
        return s
    h, dk, dv = case["h"], case["dk"], case["dv"]
    lead = (b,) if case["op"] == "step" else (b, t)
    s["q"] = normal(*lead, case["hq"], dk).to(dtype)
    s["k"] = normal(*lead, case["hk"], dk).to(dtype)
    s["v"] = normal(*lead, case["hv"], dv).to(dtype)
    if case["decay"] == "head":      # memories from a few tokens to some hundreds
        s["g"] = -torch.exp2(-1.0 - 7.0 * torch.arange(h, device=DEVICE, dtype=torch.float32) / h) * (
            0.5 + uniform(h))
    else:                            # a learned gate: mostly near one, now and then a forgetting token
        s["g"] = -torch.exp(normal(*lead, h) * 1.5 - 3.5)
    s["lengths"] = None
    if case["ragged"]:
        s["lengths"] = torch.randint(t // 4, t + 1, (b,), generator=gen, device=DEVICE).to(torch.int32)
    carry = case["carry"] or case["op"] == "step"
    s["state"] = normal(b, h, dk, dv) if carry else None
    if case["op"] == "step":
        s["next"] = torch.empty_like(s["state"])
    if case["op"] == "train":
        s["go"] = normal(b, t, h, dv).to(dtype)
        s["gstate"] = normal(b, h, dk, dv) if carry else None
    return s


# ---------------------------------------------------------------------------
# one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        return {"prompt": _own_prompt, "train": _own_train, "step": _own_step, "rotate": _own_rotate,
                "rotate_train": _own_rotate_train}[op](s, case)
    return {"prompt": _plain_prompt, "train": _plain_train, "step": _plain_step, "rotate": _plain_rotate,
            "rotate_train": _plain_rotate_train}[op](s, case)


def _es():
    import element_scan_recurrences_gb300 as es
    return es


def _own_prompt(s, case):
    o, state = _es().linear_attention(s["q"], s["k"], s["v"], s["g"], initial_state=s["state"], lengths=s["lengths"],
                                      scale=_scale(case), final_state=True)
    return {"o": o, "state": state}


def _own_train(s, case):
    es = _es()
    kw = dict(initial_state=s["state"], lengths=s["lengths"], scale=_scale(case))
    o, state = es.linear_attention(s["q"], s["k"], s["v"], s["g"], final_state=case["carry"], **kw)
    gq, gk, gv, gg, gi = es.linear_attention_backward(s["q"], s["k"], s["v"], s["g"], s["go"],
                                                      grad_final_state=s["gstate"], **kw)
    out = {"o": o, "gq": gq, "gk": gk, "gv": gv, "gg": gg}
    if case["carry"]:
        out.update(state=state, ginitial=gi)
    return out


def _own_step(s, case):
    o, state = _es().linear_attention_step(s["q"], s["k"], s["v"], s["g"], s["state"], state_out=s["next"],
                                           scale=_scale(case))
    return {"o": o, "state": state}


def _own_rotate(s, case):
    q, k = _es().qk_norm_rotate(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], positions=s["positions"],
                                eps=EPS, neighbours=case["neighbours"])
    return {"q": q, "k": k}


def _own_rotate_train(s, case):
    es = _es()
    kw = dict(positions=s["positions"], eps=EPS, neighbours=case["neighbours"])
    q, k = es.qk_norm_rotate(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], **kw)
    gq, gk, gwq, gwk = es.qk_norm_rotate_backward(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["gq"],
                                                  s["gk"], **kw)
    return {"q": q, "k": k, "gq": gq, "gk": gk, "gwq": gwq, "gwk": gwk}


# the plain forms

CHUNK = 64


def _spread(x, h):
    """[B, T, heads, D] in 32 bits, [B, h, T, D] for the heads that read it."""
    x = x.float().transpose(1, 2)
    return x if x.shape[1] == h else x.repeat_interleave(h // x.shape[1], dim=1)


def _sums(x):
    """[..., n] -> [..., n, n]: the sum of x over (j, i] at [i, j], -inf above the diagonal."""
    n = x.shape[-1]
    rows = x[..., :, None].expand(*x.shape, n)
    below = torch.ones(n, n, dtype=torch.bool, device=x.device).tril(-1)
    keep = torch.ones(n, n, dtype=torch.bool, device=x.device).tril()
    return torch.where(below, rows, 0.0).cumsum(-2).masked_fill(~keep, float("-inf"))


def _plain_attention(q, k, v, g, state, lengths, scale, h):
    """o [B, T, H, Dv] and the last state in 32 bits, in chunks of tokens."""
    b, t = q.shape[:2]
    q, k, v = _spread(q, h), _spread(k, h), _spread(v, h)
    g = g.float().expand(b, t, h).transpose(1, 2)
    if lengths is not None:
        there = (torch.arange(t, device=q.device)[None] < lengths[:, None])[:, None]       # [B, 1, T]
        k = torch.where(there[..., None], k, 0.0)
        v = torch.where(there[..., None], v, 0.0)
        g = torch.where(there, g, 0.0)
    n = -(-t // CHUNK)
    pad = n * CHUNK - t
    if pad:
        q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, pad)) for x in (q, k, v))
        g = torch.nn.functional.pad(g, (0, pad))
    q, k, v = (x.reshape(b, h, n, CHUNK, x.shape[-1]) for x in (q, k, v))
    g = g.reshape(b, h, n, CHUNK)
    inside = (q @ k.transpose(-1, -2)) * _sums(g).exp() @ v
    whole = g.sum(-1)                                                                      # [B, H, n]
    after = (whole[..., None] - g.cumsum(-1)).clamp(max=0.0).exp()
    add = (k * after[..., None]).transpose(-1, -2) @ v                                     # [B, H, n, Dk, Dv]
    first = torch.zeros_like(add[:, :, :1]) if state is None else state.float()[:, :, None]
    terms = torch.cat([first, add], 2)
    steps = _sums(torch.nn.functional.pad(whole, (1, 0))).exp()                            # [B, H, n + 1, n + 1]
    states = (steps @ terms.flatten(-2)).reshape(terms.shape)
    across = (q * g.cumsum(-1).exp()[..., None]) @ states[:, :, :-1]
    o = ((inside + across) * scale).reshape(b, h, n * CHUNK, -1)[:, :, :t].transpose(1, 2)
    if lengths is not None:
        o = torch.where(there[:, 0, :, None, None], o, 0.0)
    return o, states[:, :, -1]


def _plain_prompt(s, case):
    o, state = _plain_attention(s["q"], s["k"], s["v"], s["g"], s["state"], s["lengths"], _scale(case), case["h"])
    return {"o": o.to(s["q"].dtype).contiguous(), "state": state.contiguous()}


def _plain_train(s, case):
    dtype = s["q"].dtype
    leaves = [x.float().detach().requires_grad_(True) for x in (s["q"], s["k"], s["v"], s["g"])]
    if case["carry"]:
        leaves.append(s["state"].detach().clone().requires_grad_(True))
    with torch.enable_grad():
        o, state = _plain_attention(*leaves[:4], leaves[4] if case["carry"] else None, s["lengths"], _scale(case),
                                    case["h"])
        outs, gouts = ([o, state], [s["go"].float(), s["gstate"]]) if case["carry"] else ([o], [s["go"].float()])
        grads = torch.autograd.grad(outs, leaves, gouts)
    out = {"o": o.detach().to(dtype).contiguous(), "gq": grads[0].to(dtype), "gk": grads[1].to(dtype),
           "gv": grads[2].to(dtype), "gg": grads[3]}
    if case["carry"]:
        out.update(state=state.detach().contiguous(), ginitial=grads[4])
    return {name: x.contiguous() for name, x in out.items()}


def _plain_step(s, case):
    h = case["h"]
    q, k, v = (x.float().repeat_interleave(h // x.shape[1], dim=1) for x in (s["q"], s["k"], s["v"]))
    s["next"].copy_(s["state"] * s["g"].expand(q.shape[0], h).exp()[..., None, None] + k[..., :, None] * v[..., None, :])
    o = (q[..., None, :] @ s["next"])[..., 0, :] * _scale(case)
    return {"o": o.to(s["q"].dtype), "state": s["next"]}


def _plain_turn(x, w, s, case):
    r = case["turned"]
    at = s["positions"].long()
    cos, sin = s["cos"][at][:, :, None], s["sin"][at][:, :, None]
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    if case["neighbours"]:
        x1, x2 = x[..., 0:r:2], x[..., 1:r:2]
    else:
        x1, x2 = x[..., :r // 2], x[..., r // 2:r]
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    y = torch.stack([y1, y2], -1).flatten(-2) if case["neighbours"] else torch.cat([y1, y2], -1)
    return torch.cat([y, x[..., r:]], -1)


def _plain_rotate(s, case):
    dtype = s["q"].dtype
    return {"q": _plain_turn(s["q"], s["wq"], s, case).to(dtype), "k": _plain_turn(s["k"], s["wk"], s, case).to(dtype)}


def _plain_rotate_train(s, case):
    dtype = s["q"].dtype
    leaves = [x.float().detach().requires_grad_(True) for x in (s["q"], s["k"], s["wq"], s["wk"])]
    with torch.enable_grad():
        q, k = _plain_turn(leaves[0], leaves[2], s, case), _plain_turn(leaves[1], leaves[3], s, case)
        grads = torch.autograd.grad([q, k], leaves, [s["gq"].float(), s["gk"].float()])
    return {name: x.detach().to(dtype).contiguous() for name, x in zip(("q", "k", "gq", "gk", "gwq", "gwk"),
                                                                       (q, k) + tuple(grads))}


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    b, t = case["b"], case["t"]
    if case["op"] in ("rotate", "rotate_train"):
        d, heads = case["d"], case["hq"] + case["hk"]
        one = b * t * heads * d
        tables = b * t * (4 + 8 * (case["turned"] // 2)) + 2 * d * size
        if case["op"] == "rotate":
            return {"bytes": 2 * one * size + tables, "flops": 7 * one}
        return {"bytes": 5 * one * size + tables + 2 * d * size, "flops": 22 * one}
    h, dk, dv = case["h"], case["dk"], case["dv"]
    tokens = b * t
    inputs = tokens * (case["hq"] * dk + case["hk"] * dk + case["hv"] * dv) * size
    out = tokens * h * dv * size
    decay = 4 * (h if case["decay"] == "head" else tokens * h)
    state = 4 * b * h * dk * dv
    if case["op"] == "step":
        return {"bytes": inputs + out + decay + 2 * state, "flops": 5 * tokens * h * dk * dv}
    if case["op"] == "prompt":
        return {"bytes": inputs + out + decay + (2 if case["carry"] else 1) * state, "flops": 4 * tokens * h * dk * dv}
    # forward and backward of one layer: the inputs are read and their gradients written once, as are o and its gradient
    return {"bytes": 2 * (inputs + out + decay) + (4 * state if case["carry"] else 0),
            "flops": 14 * tokens * h * dk * dv}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rotate", "rotate_train"):
        return _exact_rotate(s, case)
    if case["op"] == "step":
        s = dict(s, **{n: s[n][:, None] for n in ("q", "k", "v")})
        s["g"] = s["g"] if case["decay"] == "head" else s["g"][:, None]
    return _exact_attention(s, case)


def _exact_attention(s, case):
    """Token by token; the gradients from the recurrence run backwards."""
    b, t, h, dk, dv = (case[n] for n in ("b", "t", "h", "dk", "dv"))
    scale, train = _scale(case), case["op"] == "train"
    steps = t * (2 if train else 1)
    if steps * max(60e-6, b * h * dk * dv * 8 * 12 / 5e12) > 15:
        return None

    def wide(x):      # [B, T, heads, D] -> one head for each reader
        x = x.double()
        return x[:, :, :, None].expand(b, t, x.shape[2], h // x.shape[2], x.shape[3]).reshape(b, t, h, x.shape[3])

    q, k, v = wide(s["q"]), wide(s["k"]), wide(s["v"])
    fade = torch.exp(s["g"].double()).expand(b, t, h)
    length = s["lengths"] if s["lengths"] is not None else torch.full((b,), t, device=DEVICE, dtype=torch.int32)
    live = (torch.arange(t, device=DEVICE)[None] < length[:, None]).double()                  # [B, T]
    k, v, q = (x * live[:, :, None, None] for x in (k, v, q))
    fade = torch.where(live[:, :, None] > 0, fade, 1.0)
    state = torch.zeros(b, h, dk, dv, dtype=torch.float64, device=DEVICE) if s["state"] is None else s["state"].double()
    o = torch.empty(b, t, h, dv, dtype=torch.float64, device=DEVICE)
    if train:
        go = s["go"].double() * live[:, :, None, None]
        gq = torch.empty_like(q)
    for i in range(t):
        state = state * fade[:, i, :, None, None]
        state += torch.einsum("bhi,bhj->bhij", k[:, i], v[:, i])
        o[:, i] = torch.einsum("bhi,bhij->bhj", q[:, i], state)
        if train:
            gq[:, i] = torch.einsum("bhj,bhij->bhi", go[:, i], state)
    o *= scale
    if case["op"] == "step":
        return {"o": o[:, 0], "state": state}
    if not train:
        return {"o": o, "state": state}
    gq *= scale
    gs = torch.zeros_like(state) if s["gstate"] is None else s["gstate"].double()
    # what the log-decay of the last token sees of the last state
    tail = (gs * state).sum((-1, -2))
    gk, gv = torch.empty_like(k), torch.empty_like(v)
    for i in range(t - 1, -1, -1):
        gs = gs + torch.einsum("bhi,bhj->bhij", q[:, i] * scale, go[:, i])
        gk[:, i] = torch.einsum("bhij,bhj->bhi", gs, v[:, i])
        gv[:, i] = torch.einsum("bhij,bhi->bhj", gs, k[:, i])
        gs = gs * fade[:, i, :, None, None]
    # exp(g[t]) <gs[t], h[t-1]>, summed from the end: each token adds what it reads of the state less what it wrote
    gg = ((q * gq).sum(-1) - (k * gk).sum(-1)).flip(1).cumsum(1).flip(1) + tail[:, None]
    dead = live[:, :, None, None]
    gg = gg * live[:, :, None]
    gq, gk, gv = gq * dead, gk * dead, gv * dead
    if case["decay"] == "head":
        gg = gg.sum((0, 1))

    def fold(x, heads):
        return x.reshape(b, t, heads, h // heads, x.shape[-1]).sum(3)

    out = {"o": o, "gq": fold(gq, case["hq"]), "gk": fold(gk, case["hk"]), "gv": fold(gv, case["hv"]), "gg": gg}
    if case["carry"]:
        out.update(state=state, ginitial=gs)
    return out


def _exact_rotate(s, case):
    """Each pair as a complex number, turned by a product."""
    r, d = case["turned"], case["d"]
    turn = torch.complex(s["cos"].double(), s["sin"].double())[s["positions"].long()][:, :, None]     # [B, T, 1, r/2]

    def pairs(x):
        if case["neighbours"]:
            return torch.view_as_complex(x[..., :r].reshape(*x.shape[:-1], r // 2, 2).contiguous())
        return torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous())

    def values(z, rest):
        y = torch.view_as_real(z).flatten(-2) if case["neighbours"] else torch.cat([z.real, z.imag], -1)
        return torch.cat([y, rest], -1)

    out = {}
    for n in ("q", "k"):
        x, w = s[n].double(), s["w" + n].double()
        size = ((x * x).sum(-1, keepdim=True) / d + EPS).sqrt()
        unit = x / size
        y = unit * w
        out[n] = values(pairs(y) * turn, y[..., r:])
        if case["op"] == "rotate_train":
            g = s["g" + n].double()
            back = values(pairs(g) * turn.conj(), g[..., r:])
            gu = back * w
            out["gw" + n] = (back * unit).sum((0, 1, 2))
            out["g" + n] = (gu - unit * (gu * unit).sum(-1, keepdim=True) / d) / size
    names = ("q", "k") if case["op"] == "rotate" else ("q", "k", "gq", "gk", "gwq", "gwk")
    return {n: out[n] for n in names}
