"""Workloads of the selective-layer operators: the short causal convolution, the
selective state space scan and gradient clipping.

Each case is one call, or one forward and its backward, as a program calls it.
`run` computes it in plain elementary torch operations (own = False) or with
the framework's kernels (own = True); `exact` computes it from the definition in
64 bits.

The layer these operators serve: a projection gives every token its heads'
inputs x, the shared B and C and a step size dt per head.  x, B and C pass
together through a causal depthwise convolution of a few taps and a SiLU, then
drive one linear recurrence per head,

    S_t = exp(dt_t A) S_{t-1} + dt_t B_t x_t^T        S [N, P]
    y_t = S_t^T C_t + D x_t

whose state is all that a prompt leaves behind for the tokens after it.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_CHUNK = 64


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # Nine prompts of very different lengths packed end to end, one of them
        # empty and one of a single token, each going on from a cached tail.
        {"name": "conv_prompts", "kind": "conv", "mode": "prompt", "type": "bf16", "channels": 2304, "taps": 4,
         "lengths": "1731,64,0,517,1,2048,255,803,96", "bias": True, "silu": True, "state": True},
        # A training step's convolution over a full batch of long sequences.
        {"name": "conv_train", "kind": "conv", "mode": "train", "type": "bf16", "channels": 4352, "taps": 4,
         "batch": 4, "length": 4096, "bias": True, "silu": True, "state": False},
        # The same in fp32 at sizes that fill no tile, without bias or SiLU.
        {"name": "conv_train_f32_odd", "kind": "conv", "mode": "train", "type": "f32", "channels": 776, "taps": 3,
         "batch": 3, "length": 1021, "bias": False, "silu": False, "state": True},
        # One new token for each of 16 running sequences: latency counts.
        {"name": "conv_token", "kind": "conv", "mode": "token", "type": "bf16", "channels": 2304, "taps": 4,
         "batch": 16, "bias": True, "silu": True, "state": True},
        # The packed prompts' scan; the final states start the decoding.
        {"name": "ssm_prompts", "kind": "ssm", "mode": "prompt", "type": "bf16", "heads": 32, "width": 64,
         "groups": 1, "states": 128, "lengths": "1731,64,0,517,1,2048,255,803,96", "state": True},
        # One long prompt alone: the work has to be found along its length.
        {"name": "ssm_long_prompt", "kind": "ssm", "mode": "prompt", "type": "bf16", "heads": 24, "width": 64,
         "groups": 8, "states": 64, "batch": 1, "length": 32768, "state": False},
        # A training step's scan over a full batch of long sequences.
        {"name": "ssm_train", "kind": "ssm", "mode": "train", "type": "bf16", "heads": 32, "width": 64,
         "groups": 1, "states": 128, "batch": 4, "length": 4096, "state": False},
        # The same in fp32 at odd sizes, between two slices of a longer sequence.
        {"name": "ssm_train_f32_odd", "kind": "ssm", "mode": "train", "type": "f32", "heads": 10, "width": 40,
         "groups": 2, "states": 24, "batch": 3, "length": 333, "state": True},
        # One token of a few running sequences: latency counts.
        {"name": "ssm_token", "kind": "ssm", "mode": "token", "type": "bf16", "heads": 24, "width": 64,
         "groups": 1, "states": 64, "batch": 2, "state": True},
        # One token of many running sequences: the states' bytes count.
        {"name": "ssm_token_batch", "kind": "ssm", "mode": "token", "type": "bf16", "heads": 32, "width": 64,
         "groups": 1, "states": 128, "batch": 256, "state": True},
        # The temporal scan's three weight gradients and a few small ones.
        {"name": "clip_few", "kind": "clip", "tensors": 14, "largest": 1 << 17, "types": "f32", "layout": 5},
        # A model's worth of gradients, large and tiny, in two types.
        {"name": "clip_many", "kind": "clip", "tensors": 60, "largest": 100_000_000, "types": "both", "layout": 6},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _ragged(rng, total):
    out = []
    while total > 0 and len(out) < 12:
        n = min(total, _log(rng, 1, 4096)) if rng.random() > 0.1 else 0
        out.append(n)
        total -= n
    return ",".join(str(n) for n in out) if sum(out) else "1"


def draw(rng):
    kind = rng.choice(["conv", "conv", "ssm", "ssm", "ssm", "clip"])
    if kind == "clip":
        return _fit({"kind": "clip", "tensors": _log(rng, 1, 62), "largest": _log(rng, 1, 20_000_000),
                "types": rng.choice(["f32", "bf16", "both"]), "layout": rng.randrange(1 << 30)})
    mode = rng.choice(["prompt", "train", "token"])
    case = {"kind": kind, "mode": mode, "type": rng.choice(["bf16", "bf16", "f32"])}
    if mode == "token":
        case["batch"] = _log(rng, 1, 256)
    elif mode == "prompt" and rng.random() < 0.5:
        case["lengths"] = _ragged(rng, _log(rng, 1, 16384))
    else:
        case["batch"], case["length"] = _log(rng, 1, 8), _log(rng, 1, 4096)
    case["state"] = mode == "token" or rng.random() < 0.5
    if kind == "conv":
        case.update(channels=_log(rng, 8, 2200), taps=rng.choice([2, 3, 4]), bias=rng.random() < 0.7,
                    silu=rng.random() < 0.7)
        if case["type"] == "bf16" and rng.random() < 0.6:
            case["channels"] = -(-case["channels"] // 8) * 8
        return _fit(case)
    groups = rng.choice([1, 1, 2, 3, 8])
    case.update(groups=groups, heads=groups * rng.randint(1, max(1, 24 // groups)),
                width=8 * _log(rng, 1, 16), states=8 * _log(rng, 1, 16))
    return _fit(case)


def _fit(case):
    """Shortens a drawn case until it needs no more than the largest listed one of its kind."""
    peers = [work(c) for c in listed() if c["kind"] == case["kind"]]
    most = {k: max(w[k] for w in peers) for k in ("bytes", "flops")}
    while any(work(case)[k] > most[k] for k in most):
        if case["kind"] == "clip":
            case["largest"] //= 2
        elif "lengths" in case:
            case["lengths"] = ",".join(str(n // 2) for n in _lengths(case))
        elif case.get("length", 1) > 1:
            case["length"] //= 2
        else:
            case["batch"] //= 2
    return case


def _lengths(case):
    return [int(v) for v in case["lengths"].split(",")] if "lengths" in case else None


def _tokens(case):
    return sum(_lengths(case)) if "lengths" in case else case["batch"] * case.get("length", 1)


def _clip_sizes(case):
    rng = random.Random(case["layout"])
    sizes = [256 * 16] * 3 if case["tensors"] >= 8 and case["largest"] >= 4096 else []
    while len(sizes) < case["tensors"] - 1:
        sizes.append(_log(rng, 1, case["largest"]))
    return sizes[: case["tensors"] - 1] + [case["largest"]]


def _clip_type(case, i):
    return {"f32": torch.float32, "bf16": torch.bfloat16}.get(
        case["types"], torch.bfloat16 if i % 3 else torch.float32)


# ----------------------------------------------------------------- the inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(shape, generator=gen, device="cuda")

    if case["kind"] == "clip":
        grads = [(normal(n) * float(10.0 ** ((i % 5) - 3))).to(_clip_type(case, i))
                 for i, n in enumerate(_clip_sizes(case))]
        return {"case": case, "grads": grads, "out": [torch.empty_like(g) for g in grads], "max_norm": 1.0}

    st = {"case": case}
    typ = _TYPES[case["type"]]
    lengths = _lengths(case)
    if lengths is not None:
        lead, rows = (sum(lengths),), len(lengths)
        ends = [0]
        for n in lengths:
            ends.append(ends[-1] + n)
        st["ends"] = ends
        st["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    elif case["mode"] == "token":
        lead = (case["batch"],)
        rows = case["batch"]
    else:
        lead = (case["batch"], case["length"])
        rows = case["batch"]

    if case["kind"] == "conv":
        c, w = case["channels"], case["taps"]
        st["x"] = normal(*lead, c).to(typ)
        st["weight"] = uniform(-1, 1, c, w) / math.sqrt(w)
        st["bias"] = uniform(-1, 1, c) / math.sqrt(w) if case["bias"] else None
        st["state"] = normal(rows, w - 1, c).to(typ) if case["state"] else None
        if case["mode"] == "train":
            st["d_y"] = normal(*lead, c).to(typ)
            st["d_final"] = normal(rows, w - 1, c).to(typ) if case["state"] else None
        elif case["mode"] == "token":
            st["new_state"] = torch.empty_like(st["state"])
        return st

    h, p, g, n = case["heads"], case["width"], case["groups"], case["states"]

    def silu(v):
        return v / (1 + torch.exp(-v))

    # x, B and C are slices of the convolution's one output, as in the layer
    mixed = silu(normal(*lead, h * p + 2 * g * n)).to(typ)
    st["x"] = mixed[..., : h * p].unflatten(-1, (h, p))
    st["B"] = mixed[..., h * p: h * p + g * n].unflatten(-1, (g, n))
    st["C"] = mixed[..., h * p + g * n:].unflatten(-1, (g, n))
    st["dt"] = normal(*lead, h).to(typ)
    st["A"] = -uniform(1, 16, h)
    step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), h))
    st["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus(dt_bias) = step
    st["D"] = 1 + 0.1 * normal(h)
    st["state"] = 0.3 * normal(rows, h, n, p) if case["state"] else None
    if case["mode"] == "train":
        st["d_y"] = normal(*lead, h, p).to(typ)
        st["d_final"] = 0.1 * normal(rows, h, n, p) if case["state"] else None
    elif case["mode"] == "token":
        st["new_state"] = torch.empty_like(st["state"])
    return st


# -------------------------------------------------------------------- the run
def run(st):
    case = st["case"]
    if own:
        return _OWN[case["kind"]](st)
    return _PLAIN[case["kind"]](st)


def _own_conv(st):
    import bwd_mamba2_scan_amd as m2

    case = st["case"]
    if case["mode"] == "token":
        y = m2.conv_step(st["x"], st["weight"], st["state"], st["bias"], silu=case["silu"],
                         new_state=st["new_state"])
        return y, st["new_state"]
    y, final = m2.conv_fwd(st["x"], st["weight"], st["bias"], silu=case["silu"], initial_state=st["state"],
                           offsets=st.get("offsets"), want_final_state=True)
    if case["mode"] == "prompt":
        return y, final
    g = m2.conv_bwd(st["x"], st["weight"], st["d_y"], st["bias"], silu=case["silu"], initial_state=st["state"],
                    d_final_state=st["d_final"])
    return y, final, g["d_x"], g["d_weight"], g.get("d_bias"), g.get("d_initial_state")


def _own_ssm(st):
    import bwd_mamba2_scan_amd as m2

    case = st["case"]
    args = (st["x"], st["dt"], st["A"], st["B"], st["C"])
    kw = {"D": st["D"], "dt_bias": st["dt_bias"], "softplus": True}
    if case["mode"] == "token":
        y = m2.ssm_step(*args, st["state"], new_state=st["new_state"], **kw)
        return y, st["new_state"]
    y, final = m2.ssm_fwd(*args, initial_state=st["state"], offsets=st.get("offsets"), want_final_state=True, **kw)
    if case["mode"] == "prompt":
        return y, final
    g = m2.ssm_bwd(*args, st["d_y"], initial_state=st["state"], d_final_state=st["d_final"], **kw)
    return (y, final, g["d_x"], g["d_dt"], g["d_A"], g["d_B"], g["d_C"], g["d_D"], g["d_dt_bias"],
            g.get("d_initial_state"))


def _own_clip(st):
    import bwd_mamba2_scan_amd as m2

    norm = m2.clip_grads(st["grads"], st["max_norm"], out=st["out"])
    return norm, st["out"]


_OWN = {"conv": _own_conv, "ssm": _own_ssm, "clip": _own_clip}


# ------------------------------------------------------------- the plain form
def _plain_conv_rows(x, weight, bias, state, silu):
    """x [rows, length, C], state [rows, W - 1, C] -> y, the last W - 1 inputs."""
    taps = weight.shape[1]
    length = x.shape[1]
    padded = torch.cat([state, x], dim=1)
    acc = torch.zeros_like(x)
    for k in range(taps):
        acc = acc + padded[:, k: k + length] * weight[:, k]
    if bias is not None:
        acc = acc + bias
    y = acc / (1 + torch.exp(-acc)) if silu else acc
    return y, padded[:, length:]


def _plain_conv(st):
    case = st["case"]
    typ = st["x"].dtype
    train = case["mode"] == "train"
    taps, c = case["taps"], case["channels"]
    x = st["x"].float()
    rows = len(_lengths(case)) if "lengths" in case else case["batch"]
    state = (st["state"].float() if st["state"] is not None
             else torch.zeros(rows, taps - 1, c, device=x.device))
    weight, bias = st["weight"], st["bias"]
    if "lengths" in case:
        parts = [_plain_conv_rows(x[a:b].unsqueeze(0), weight, bias, state[i: i + 1], case["silu"])
                 for i, (a, b) in enumerate(zip(st["ends"], st["ends"][1:]))]
        return (torch.cat([p[0][0] for p in parts]).to(typ), torch.cat([p[1] for p in parts]).to(typ))
    if case["mode"] == "token":
        y, final = _plain_conv_rows(x.unsqueeze(1), weight, bias, state, case["silu"])
        return y[:, 0].to(typ), final.to(typ)
    if not train:
        y, final = _plain_conv_rows(x, weight, bias, state, case["silu"])
        return y.to(typ), final.to(typ)
    leaves = [v.detach().requires_grad_() for v in (x, weight, state)]
    if bias is not None:
        leaves.append(bias.detach().requires_grad_())
    with torch.enable_grad():
        y, final = _plain_conv_rows(leaves[0], leaves[1], leaves[3] if bias is not None else None, leaves[2],
                                    case["silu"])
        outs, ups = [y], [st["d_y"].float()]
        if st["d_final"] is not None:
            outs.append(final)
            ups.append(st["d_final"].float())
        g = torch.autograd.grad(outs, leaves, ups)
    return (y.detach().to(typ), final.detach().to(typ), g[0].to(typ), g[1], g[3] if bias is not None else None,
            g[2].to(typ) if st["state"] is not None else None)


def _plain_ssm_rows(x, dt, A, B, C, D, dt_bias, state):
    """The scan in chunks: products inside a chunk, the state passed between them.

    x [rows, length, H, P], dt [rows, length, H], B and C [rows, length, G, N],
    state [rows, H, N, P] -> y, final state.
    """
    rows, length, heads, width = x.shape
    groups, n = B.shape[2:]
    q = _CHUNK
    chunks = -(-length // q)
    pad = chunks * q - length
    dt = torch.logaddexp(dt + dt_bias, torch.zeros((), device=x.device))

    def cut(v):  # [rows, length, K, ...] -> [rows, chunks, K, q, ...]
        if pad:
            v = torch.cat([v, torch.zeros(rows, pad, *v.shape[2:], dtype=v.dtype, device=v.device)], dim=1)
        return v.reshape(rows, chunks, q, *v.shape[2:]).transpose(2, 3)

    def heads_of(v):  # groups to heads
        return v.repeat_interleave(heads // groups, dim=2)

    # log decays summed in 64 bits: their differences reach far below them
    cum = cut((dt * A).double()).cumsum(-1)                       # [rows, chunks, H, q]
    tri = torch.ones(q, q, dtype=torch.bool, device=x.device).tril()
    inner = (cum.unsqueeze(-1) - cum.unsqueeze(-2)).masked_fill(~tri, -math.inf)
    u = cut(x * dt.unsqueeze(-1))                                 # [rows, chunks, H, q, P]
    bc, cc = cut(B), cut(C)
    scores = heads_of(cc @ bc.transpose(-1, -2).contiguous()) * torch.exp(inner).float()
    y = scores @ u
    to_end = torch.exp(cum[..., -1:] - cum).float().unsqueeze(-1)
    adds = (heads_of(bc) * to_end).transpose(-1, -2).contiguous() @ u      # [rows, chunks, H, N, P]
    carry = torch.exp(cum[..., -1]).float()[..., None, None]
    starts = []
    for i in range(chunks):
        starts.append(state)
        state = state * carry[:, i] + adds[:, i]
    y = y + torch.exp(cum).float().unsqueeze(-1) * (heads_of(cc) @ torch.stack(starts, 1))
    y = y.transpose(2, 3).reshape(rows, chunks * q, heads, width)[:, :length]
    return y + D[:, None] * x, state


def _plain_ssm_token(x, dt, A, B, C, D, dt_bias, state):
    heads = x.shape[1]
    dt = torch.logaddexp(dt + dt_bias, torch.zeros((), device=x.device))
    b = B.repeat_interleave(heads // B.shape[1], dim=1)
    c = C.repeat_interleave(heads // C.shape[1], dim=1)
    state = state * torch.exp(dt * A)[..., None, None] + b.unsqueeze(-1) * (dt.unsqueeze(-1) * x).unsqueeze(-2)
    return (state * c.unsqueeze(-1)).sum(-2) + D[:, None] * x, state


def _plain_ssm(st):
    case = st["case"]
    typ = st["x"].dtype
    x, dt, B, C = (st[k].float() for k in ("x", "dt", "B", "C"))
    A, D, bias = st["A"], st["D"], st["dt_bias"]
    rows = len(_lengths(case)) if "lengths" in case else case["batch"]
    state = (st["state"] if st["state"] is not None
             else torch.zeros(rows, case["heads"], case["states"], case["width"], device=x.device))
    if case["mode"] == "token":
        y, new = _plain_ssm_token(x, dt, A, B, C, D, bias, state)
        return y.to(typ), new
    if "lengths" in case:
        ys, finals = [], []
        for i, (a, b) in enumerate(zip(st["ends"], st["ends"][1:])):
            if a == b:
                finals.append(state[i: i + 1])
                continue
            y, f = _plain_ssm_rows(*(v[a:b].unsqueeze(0) for v in (x, dt)), A,
                                   *(v[a:b].unsqueeze(0) for v in (B, C)), D, bias, state[i: i + 1])
            ys.append(y[0].to(typ))
            finals.append(f)
        return torch.cat(ys), torch.cat(finals)
    if case["mode"] == "prompt":
        y, final = _plain_ssm_rows(x, dt, A, B, C, D, bias, state)
        return y.to(typ), final
    leaves = [v.detach().requires_grad_() for v in (x, dt, A, B, C, D, bias, state)]
    with torch.enable_grad():
        y, final = _plain_ssm_rows(*leaves)
        outs, ups = [y], [st["d_y"].float()]
        if st["d_final"] is not None:
            outs.append(final)
            ups.append(st["d_final"])
        g = torch.autograd.grad(outs, leaves, ups)
    return (y.detach().to(typ), final.detach(), g[0].to(typ), g[1].to(typ), g[2], g[3].to(typ), g[4].to(typ), g[5],
            g[6], g[7] if st["state"] is not None else None)


def _plain_clip(st):
    total = torch.zeros((), dtype=torch.float64, device=st["grads"][0].device)
    for g in st["grads"]:
        v = g.float()
        total = total + (v * v).sum(dtype=torch.float64)
    norm = torch.sqrt(total).float()
    factor = torch.clamp(st["max_norm"] / (norm + 1e-6), max=1.0)
    return norm, [(g.float() * factor).to(g.dtype) for g in st["grads"]]


_PLAIN = {"conv": _plain_conv, "ssm": _plain_ssm, "clip": _plain_clip}


# --------------------------------------------------------------------- the work
def work(case):
    if case["kind"] == "clip":
        sizes = _clip_sizes(case)
        nbytes = sum(2 * n * _clip_type(case, i).itemsize for i, n in enumerate(sizes)) + 4
        return {"bytes": nbytes, "flops": 3 * sum(sizes)}
    e = 2 if case["type"] == "bf16" else 4
    tokens = _tokens(case)
    rows = len(_lengths(case)) if "lengths" in case else case["batch"]
    train = case["mode"] == "train"
    if case["kind"] == "conv":
        c, w = case["channels"], case["taps"]
        tails = rows * (w - 1) * c * e
        nbytes = 2 * tokens * c * e + (w + 1) * c * 4 + tails * (2 if case["state"] else 1)
        flops = tokens * c * (2 * w + 4)
        if train:  # reads x and d_y, writes d_x and the weights' gradients
            nbytes += 2 * tokens * c * e + (w + 1) * c * 4 + (2 * tails if case["state"] else 0)
            flops += tokens * c * (6 * w + 10)
        return {"bytes": nbytes, "flops": flops}
    h, p, g, n = case["heads"], case["width"], case["groups"], case["states"]
    states = rows * h * n * p * 4
    mixed = tokens * (h * p + 2 * g * n + h) * e  # x, B, C and dt
    nbytes = mixed + tokens * h * p * e + states * (2 if case["state"] else 1) + 3 * h * 4
    # per token and head: S = a S + B u^T (3 N P), y = S^T C (2 N P)
    flops = tokens * h * 5 * n * p
    if train:
        # reads d_y, writes the gradients of x, B, C and dt
        nbytes += tokens * h * p * e + mixed + 3 * h * 4 + (2 * states if case["state"] else 0)
        # G = a G + C d_y^T and S again (3 N P each); G^T B, G u, S d_y, <G, S> (2 N P each)
        flops += tokens * h * 14 * n * p
    return {"bytes": nbytes, "flops": flops}


# ----------------------------------------------------------- the definition
def exact(case, seed):
    st = prepare(case, seed)
    with torch.no_grad():
        return {"conv": _exact_conv, "ssm": _exact_ssm, "clip": _exact_clip}[case["kind"]](st)


def _exact_clip(st):
    square = sum(torch.dot(g.double(), g.double()) for g in st["grads"])
    norm = square ** 0.5
    scale = min(1.0, st["max_norm"] / (float(norm) + 1e-6))
    return norm, [g.double() * scale for g in st["grads"]]


def _spans(st):
    """(row index, slice of the token axis as [1, length, ...]) of every sequence."""
    case = st["case"]
    if "lengths" in case:
        return [(i, lambda v, a=a, b=b: v[a:b].unsqueeze(0)) for i, (a, b) in enumerate(zip(st["ends"], st["ends"][1:]))]
    if case["mode"] == "token":
        return [(slice(None), lambda v: v.unsqueeze(1))]
    return [(slice(None), lambda v: v)]


def _exact_conv(st):
    case = st["case"]
    w = st["weight"].double()
    c, taps = w.shape
    ys, finals, grads = [], [], None
    for row, take in _spans(st):
        x = take(st["x"]).double()
        rows, length = x.shape[:2]
        tail = torch.zeros(rows, taps - 1, c, dtype=torch.float64, device=x.device)
        if st["state"] is not None:
            tail = st["state"][row].double().reshape(rows, taps - 1, c)
        source = torch.cat([tail, x], 1)
        # index of the input that tap k of output t multiplies
        idx = torch.arange(length, device=x.device)[:, None] + torch.arange(taps, device=x.device)
        pre = torch.zeros_like(x) if st["bias"] is None else st["bias"].double().expand_as(x).clone()
        for k in range(taps):
            pre += w[:, k] * source[:, idx[:, k]]
        gate = torch.sigmoid(pre) if case["silu"] else None
        ys.append(pre * gate if case["silu"] else pre)
        finals.append(source[:, source.shape[1] - (taps - 1):])
        if case["mode"] == "train":
            d = st["d_y"].double()
            if case["silu"]:
                d = d * (gate + pre * gate * (1 - gate))
            d_source = torch.zeros_like(source)
            if st["d_final"] is not None:
                d_source[:, source.shape[1] - (taps - 1):] += st["d_final"].double()
            d_w = torch.zeros_like(w)
            for k in range(taps):
                d_source[:, k: k + length] += d * w[:, k]
                d_w[:, k] = (d * source[:, k: k + length]).sum((0, 1))
            grads = (d_source[:, taps - 1:], d_w, d.sum((0, 1)) if st["bias"] is not None else None,
                     d_source[:, : taps - 1] if st["state"] is not None else None)
    if "lengths" in case:
        return torch.cat([y[0] for y in ys]), torch.cat(finals)
    if case["mode"] == "token":
        return ys[0][:, 0], finals[0]
    return (ys[0], finals[0]) + (grads or ())


def _exact_ssm(st):
    case = st["case"]
    ratio = case["heads"] // case["groups"]
    A, D, bias = st["A"].double(), st["D"].double(), st["dt_bias"].double()
    ys, finals = [], []
    for row, take in _spans(st):
        x, raw = take(st["x"]).double(), take(st["dt"]).double() + bias
        rows, length = x.shape[:2]
        dt = torch.where(raw > 40, raw, torch.log1p(torch.exp(torch.clamp(raw, max=40))))
        b, c = (take(st[k]).double().repeat_interleave(ratio, 2) for k in ("B", "C"))
        start = torch.zeros(rows, case["heads"], case["states"], case["width"], dtype=torch.float64, device=x.device)
        if st["state"] is not None:
            start = st["state"][row].double().reshape(start.shape)

        def advance(s, t):
            return (torch.exp(A * dt[:, t])[..., None, None] * s
                    + b[:, t].unsqueeze(-1) * (dt[:, t].unsqueeze(-1) * x[:, t]).unsqueeze(-2))

        s = start
        y = torch.empty_like(x)
        marks = []
        for t in range(length):
            if case["mode"] == "train" and t % _CHUNK == 0:
                marks.append(s)
            s = advance(s, t)
            y[:, t] = (s * c[:, t].unsqueeze(-1)).sum(-2) + D[:, None] * x[:, t]
        ys.append(y)
        finals.append(s)
        if case["mode"] == "train":
            return (y, s) + _exact_ssm_grads(st, x, raw, dt, b, c, marks, advance, ratio)
    if "lengths" in case:
        return torch.cat([y[0] for y in ys]), torch.cat(finals)
    if case["mode"] == "token":
        return ys[0][:, 0], finals[0]
    return ys[0], finals[0]


def _exact_ssm_grads(st, x, raw, dt, b, c, marks, advance, ratio):
    """The reverse recurrence: G_t = C_t d_y_t^T + a_{t+1} G_{t+1} is the gradient of S_t."""
    A, D = st["A"].double(), st["D"].double()
    d_y = st["d_y"].double()
    rows, length, heads, width = x.shape
    d_x, d_dt = torch.empty_like(x), torch.empty_like(dt)
    d_b, d_c = torch.empty_like(b), torch.empty_like(c)
    d_A = torch.zeros_like(A)
    g = torch.zeros_like(marks[0]) if st["d_final"] is None else st["d_final"].double().clone()
    for block in range(len(marks) - 1, -1, -1):
        lo, hi = block * _CHUNK, min(length, (block + 1) * _CHUNK)
        states = [marks[block]]
        for t in range(lo, hi):
            states.append(advance(states[-1], t))
        for t in range(hi - 1, lo - 1, -1):
            g = g + c[:, t].unsqueeze(-1) * d_y[:, t].unsqueeze(-2)
            d_c[:, t] = (states[t - lo + 1] * d_y[:, t].unsqueeze(-2)).sum(-1)
            gb = (g * b[:, t].unsqueeze(-1)).sum(-2)
            d_x[:, t] = dt[:, t].unsqueeze(-1) * gb + D[:, None] * d_y[:, t]
            d_b[:, t] = (g * (dt[:, t].unsqueeze(-1) * x[:, t]).unsqueeze(-2)).sum(-1)
            decay = torch.exp(A * dt[:, t])[..., None, None]
            d_log = (g * states[t - lo]).sum((-1, -2)) * decay[..., 0, 0]
            d_dt[:, t] = (gb * x[:, t]).sum(-1) + A * d_log
            d_A += (dt[:, t] * d_log).sum(0)
            g = decay * g
    d_raw = d_dt * torch.sigmoid(raw)
    groups = heads // ratio
    fold = (rows, length, groups, ratio, b.shape[-1])
    return (d_x, d_raw, d_A, d_b.reshape(fold).sum(3), d_c.reshape(fold).sum(3), (d_y * x).sum((0, 1, 3)),
            d_raw.sum((0, 1)), g if st["state"] is not None else None)
