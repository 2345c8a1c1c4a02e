"""Workloads of the gated delta rule and of the group norm beside it.

Each case is one call, or one forward and its backward, as a program calls it.
`run` computes it in plain elementary torch operations (own = False) or with
the framework's kernels (own = True); `exact` computes it from the definition in
64 bits.

The layer these operators serve: queries, keys and values come out of the short
causal convolution; queries and keys are brought to length one per head (a group
norm without a mean), and drive a recurrence per head whose state is corrected
towards each new value instead of only being added to,

    S' = e^g_t S_{t-1}                                  S [K, V]
    S_t = S' + k_t (beta_t (v_t - S'^T k_t))^T
    y_t = scale S_t^T q_t

and whose results pass through a group norm, one group a head, that a gate
multiplies.
"""
from __future__ import annotations

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_CHUNK = 64


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # Nine prompts of very different lengths packed end to end, one of them
        # empty and one of a single token; the final states start the decoding.
        {"name": "delta_prompts", "kind": "delta", "mode": "prompt", "type": "bf16", "gates": "f32", "heads": 32,
         "width": 128, "groups": 16, "states": 128, "lengths": "1731,64,0,517,1,2048,255,803,96", "state": True},
        # One long prompt alone: the work has to be found along its length.
        {"name": "delta_long_prompt", "kind": "delta", "mode": "prompt", "type": "bf16", "gates": "bf16", "heads": 24,
         "width": 64, "groups": 8, "states": 64, "batch": 1, "length": 32768, "state": False},
        # A training step over a full batch of long sequences.
        {"name": "delta_train", "kind": "delta", "mode": "train", "type": "bf16", "gates": "f32", "heads": 32,
         "width": 128, "groups": 16, "states": 128, "batch": 4, "length": 4096, "state": False},
        # The same in fp32 at odd sizes, between two slices of a longer sequence.
        {"name": "delta_train_f32_odd", "kind": "delta", "mode": "train", "type": "f32", "gates": "f32", "heads": 10,
         "width": 40, "groups": 2, "states": 24, "batch": 3, "length": 333, "state": True},
        # One token of a few running sequences: latency counts.
        {"name": "delta_token", "kind": "delta", "mode": "token", "type": "bf16", "gates": "f32", "heads": 24,
         "width": 64, "groups": 24, "states": 64, "batch": 2, "state": True},
        # One token of many running sequences: the states' bytes count.
        {"name": "delta_token_batch", "kind": "delta", "mode": "token", "type": "bf16", "gates": "f32", "heads": 32,
         "width": 64, "groups": 16, "states": 128, "batch": 256, "state": True},
        # A training step's norm behind the recurrence: one group a head, one
        # weight for all heads, the gate's SiLU on the result.
        {"name": "norm_train", "kind": "norm", "mode": "train", "type": "bf16", "groups": 32, "width": 128,
         "batch": 4, "length": 4096, "centered": False, "weight": "group", "bias": False, "form": "gated"},
        # The norm of packed prompts, the gate in front of it, one wide group.
        {"name": "norm_prompts", "kind": "norm", "mode": "prompt", "type": "bf16", "groups": 1, "width": 2048,
         "batch": 1, "length": 5515, "centered": False, "weight": "channel", "bias": False, "form": "gate_first"},
        # Mean, bias and SiLU in fp32 over groups that fill no vector, training.
        {"name": "norm_train_f32_odd", "kind": "norm", "mode": "train", "type": "f32", "groups": 8, "width": 97,
         "batch": 3, "length": 1021, "centered": True, "weight": "channel", "bias": True, "form": "silu"},
        # Keys of one token of 16 running sequences: latency counts.
        {"name": "norm_token", "kind": "norm", "mode": "token", "type": "bf16", "groups": 16, "width": 128,
         "batch": 16, "length": 1, "centered": False, "weight": "group", "bias": False, "form": "plain"},
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
    kind = rng.choice(["delta", "delta", "norm"])
    mode = rng.choice(["prompt", "train", "token"])
    case = {"kind": kind, "mode": mode, "type": rng.choice(["bf16", "bf16", "f32"])}
    if kind == "norm":
        case["batch"] = 1 if mode == "prompt" else _log(rng, 1, 256 if mode == "token" else 8)
        case["length"] = 1 if mode == "token" else _log(rng, 1, 8192 if mode == "prompt" else 4096)
        case["width"] = _log(rng, 8, 4096)
        if rng.random() < 0.6:
            case["width"] = -(-case["width"] // 8) * 8
        case["groups"] = _log(rng, 1, max(1, min(64, 16384 // case["width"])))
        case.update(centered=rng.random() < 0.4, weight=rng.choice(["channel", "group", "none"]),
                    form=rng.choice(["plain", "silu", "gated", "gate_first"]))
        case["bias"] = case["weight"] != "none" and rng.random() < 0.4
        return _fit(case)
    if mode == "token":
        case["batch"] = _log(rng, 1, 256)
    elif mode == "prompt" and rng.random() < 0.5:
        case["lengths"] = _ragged(rng, _log(rng, 1, 16384))
    else:
        case["batch"], case["length"] = _log(rng, 1, 8), _log(rng, 1, 4096)
    case["state"] = mode == "token" or rng.random() < 0.5
    case["gates"] = "f32" if case["type"] == "f32" else rng.choice(["f32", "bf16"])
    groups = rng.choice([1, 2, 3, 8, 16])
    case.update(groups=groups, heads=groups * rng.randint(1, max(1, 24 // groups)),
                width=8 * _log(rng, 1, 16), states=8 * _log(rng, 1, 16))
    return _fit(case)


def _fit(case):
    """Shortens a drawn case until it needs no more than the largest listed one of its kind."""
    peers = [work(c) for c in listed() if c["kind"] == case["kind"]]
    most = {k: max(w[k] for w in peers) for k in ("bytes", "flops")}
    while any(work(case)[k] > most[k] for k in most):
        if "lengths" in case:
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


# ----------------------------------------------------------------- the inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(shape, generator=gen, device="cuda")

    def silu(v):
        return v / (1 + torch.exp(-v))

    st = {"case": case}
    typ = _TYPES[case["type"]]
    if case["kind"] == "norm":
        lead = (case["batch"],) if case["mode"] == "token" else (case["batch"], case["length"])
        channels = case["groups"] * case["width"]
        # heads of different sizes, as a recurrence leaves them
        size = torch.exp(uniform(-1, 1, case["groups"])).repeat_interleave(case["width"])
        st["x"] = (normal(*lead, channels) * size + (0.3 if case["centered"] else 0.0)).to(typ)
        n = {"channel": channels, "group": case["width"], "none": 0}[case["weight"]]
        st["weight"] = 1 + 0.2 * normal(n) if n else None
        st["bias"] = 0.2 * normal(n) if case["bias"] else None
        # the gate is a slice of the projection that also gave x
        st["gate"] = (normal(*lead, channels + 64).to(typ)[..., 64:]
                      if case["form"] in ("gated", "gate_first") else None)
        if case["mode"] == "train":
            st["d_y"] = normal(*lead, channels).to(typ)
        return st

    lengths = _lengths(case)
    if lengths is not None:
        lead, rows = (sum(lengths),), len(lengths)
        ends = [0]
        for n in lengths:
            ends.append(ends[-1] + n)
        st["ends"] = ends
        st["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    else:
        lead = (case["batch"],) if case["mode"] == "token" else (case["batch"], case["length"])
        rows = case["batch"]
    h, p, g, n = case["heads"], case["width"], case["groups"], case["states"]

    def unit(v):
        return v / torch.sqrt((v * v).sum(-1, keepdim=True) + 1e-6)

    # v is a slice of the convolution's output; q and k went through their norm
    mixed = silu(normal(*lead, 2 * g * n + h * p))
    st["q"] = unit(mixed[..., : g * n].unflatten(-1, (g, n))).to(typ)
    st["k"] = unit(mixed[..., g * n: 2 * g * n].unflatten(-1, (g, n))).to(typ)
    st["v"] = mixed.to(typ)[..., 2 * g * n:].unflatten(-1, (h, p))
    # log decays -A softplus(a + bias), as a trained layer's
    rate, step = uniform(1, 16, h), torch.exp(uniform(math.log(1e-3), math.log(1e-1), h))
    a = normal(*lead, h) + step + torch.log(-torch.expm1(-step))
    st["g"] = (-rate * torch.logaddexp(a, torch.zeros((), device="cuda"))).to(_TYPES[case["gates"]])
    st["beta"] = (1 / (1 + torch.exp(-normal(*lead, h)))).to(_TYPES[case["gates"]])
    st["state"] = 0.3 * normal(rows, h, n, p) if case["state"] else None
    if case["mode"] == "train":
        st["d_y"] = normal(*lead, h, p).to(typ)
        st["d_final"] = 0.1 * normal(rows, h, n, p) if case["state"] else None
    elif case["mode"] == "token":
        st["new_state"] = torch.empty_like(st["state"])
    return st


# -------------------------------------------------------------------- the run
def run(st):
    if own:
        return _own_delta(st) if st["case"]["kind"] == "delta" else _own_norm(st)
    return _plain_delta(st) if st["case"]["kind"] == "delta" else _plain_norm(st)


def _own_delta(st):
    import bwd_mamba2_scan_amd as m2

    case = st["case"]
    args = (st["q"], st["k"], st["v"], st["g"], st["beta"])
    if case["mode"] == "token":
        y = m2.delta_step(*args, st["state"], new_state=st["new_state"])
        return y, st["new_state"]
    y, final = m2.delta_fwd(*args, initial_state=st["state"], offsets=st.get("offsets"), want_final_state=True)
    if case["mode"] == "prompt":
        return y, final
    g = m2.delta_bwd(*args, st["d_y"], initial_state=st["state"], d_final_state=st["d_final"])
    return y, final, g["d_q"], g["d_k"], g["d_v"], g["d_g"], g["d_beta"], g["d_initial_state"]


def _own_norm(st):
    import bwd_mamba2_scan_amd as m2

    case = st["case"]
    kw = {"groups": case["groups"], "gate": st["gate"], "gate_first": case["form"] == "gate_first",
          "silu": case["form"] == "silu", "centered": case["centered"]}
    y = m2.group_norm_fwd(st["x"], st["weight"], st["bias"], **kw)
    if case["mode"] != "train":
        return y
    g = m2.group_norm_bwd(st["x"], st["d_y"], st["weight"], st["bias"], **kw)
    return y, g["d_x"], g["d_weight"], g["d_bias"], g["d_gate"]


# ------------------------------------------------------------- the plain form
def _plain_delta_rows(q, k, v, g, beta, scale, state):
    """The recurrence in chunks: inside a chunk a triangular system, the state passed between them.

    q, k [rows, length, G, K], v [rows, length, H, V], g, beta [rows, length, H],
    state [rows, H, K, V] -> y, final state.  With c the sums of g from the
    chunk's start, T_ij = beta_i e^(c_i - c_j) k_i.k_j (j < i) and
    M = (1 + T)^-1, the chunk's corrections are
    U = M (beta V) - M (beta e^c K) S.
    """
    rows, length, groups, n = q.shape
    heads, width = v.shape[2:]
    size = _CHUNK
    chunks = -(-length // size)

    def cut(x):  # [rows, length, *, ...] -> [rows, chunks, *, size, ...]
        pad = x.new_zeros(rows, chunks * size - length, *x.shape[2:])
        return torch.cat([x, pad], dim=1).reshape(rows, chunks, size, *x.shape[2:]).transpose(2, 3)

    def of_heads(x):
        return x.repeat_interleave(heads // groups, dim=2)

    # log decays summed in 64 bits: their differences reach far below them
    cum = cut(g.double()).cumsum(-1)                                       # [rows, chunks, H, size]
    lower = torch.ones(size, size, dtype=torch.bool, device=q.device).tril()
    decay = torch.exp((cum.unsqueeze(-1) - cum.unsqueeze(-2)).masked_fill(~lower, -math.inf)).float()
    from_start = torch.exp(cum).float().unsqueeze(-1)
    to_end = torch.exp(cum[..., -1:] - cum).float().unsqueeze(-1)
    carry = torch.exp(cum[..., -1]).float()[..., None, None]
    qc, kc, vc, b = cut(q), cut(k), cut(v), cut(beta).unsqueeze(-1)
    kt = kc.transpose(-1, -2).contiguous()
    t = of_heads(kc @ kt) * decay * b * lower.tril(-1)
    p = of_heads(qc @ kt) * decay
    qh, kh = of_heads(qc), of_heads(kc)
    # the inverse by halves: blocks of 1, 2, 4, .. on the diagonal are already inverted
    i = torch.arange(size, device=q.device)
    m = torch.eye(size, device=q.device).expand_as(t)
    for s in (1, 2, 4, 8, 16, 32):
        same = (i // (2 * s)).unsqueeze(-1) == i // (2 * s)
        half = ((i // s) % 2 == 1).unsqueeze(-1) & ((i // s) % 2 == 0)
        m = m - m @ (t * (same & half)) @ m
    own_part, of_state = m @ (b * vc), m @ (b * from_start * kh)
    writes = (kh * to_end).transpose(-1, -2).contiguous()
    starts, parts = [], []
    for c in range(chunks):
        starts.append(state)
        u = own_part[:, c] - of_state[:, c] @ state
        parts.append(u)
        state = carry[:, c] * state + writes[:, c] @ u
    y = scale * ((from_start * qh) @ torch.stack(starts, 1) + p @ torch.stack(parts, 1))
    return y.transpose(2, 3).reshape(rows, chunks * size, heads, width)[:, :length], state


def _plain_delta(st):
    case = st["case"]
    typ, gates = st["v"].dtype, st["g"].dtype
    scale = case["states"] ** -0.5
    q, k, v, g, beta = (st[n].float() for n in ("q", "k", "v", "g", "beta"))
    rows = len(_lengths(case)) if "lengths" in case else case["batch"]
    state = (st["state"] if st["state"] is not None
             else torch.zeros(rows, case["heads"], case["states"], case["width"], device=q.device))
    if case["mode"] == "token":
        ratio = case["heads"] // case["groups"]
        q, k = q.repeat_interleave(ratio, 1), k.repeat_interleave(ratio, 1)
        state = state * torch.exp(g)[..., None, None]
        u = beta.unsqueeze(-1) * (v - (state * k.unsqueeze(-1)).sum(-2))
        state = state + k.unsqueeze(-1) * u.unsqueeze(-2)
        return (scale * (state * q.unsqueeze(-1)).sum(-2)).to(typ), state
    if "lengths" in case:
        ys, finals = [], []
        for i, (a, b) in enumerate(zip(st["ends"], st["ends"][1:])):
            if a == b:
                finals.append(state[i: i + 1])
                continue
            y, f = _plain_delta_rows(*(x[a:b].unsqueeze(0) for x in (q, k, v, g, beta)), scale, state[i: i + 1])
            ys.append(y[0].to(typ))
            finals.append(f)
        return torch.cat(ys), torch.cat(finals)
    if case["mode"] == "prompt":
        y, final = _plain_delta_rows(q, k, v, g, beta, scale, state)
        return y.to(typ), final
    leaves = [x.detach().requires_grad_() for x in (q, k, v, g, beta, state)]
    with torch.enable_grad():
        y, final = _plain_delta_rows(*leaves[:5], scale, leaves[5])
        outs, ups = [y], [st["d_y"].float()]
        if st["d_final"] is not None:
            outs.append(final)
            ups.append(st["d_final"])
        d = torch.autograd.grad(outs, leaves, ups)
    return (y.detach().to(typ), final.detach(), d[0].to(typ), d[1].to(typ), d[2].to(typ), d[3].to(gates),
            d[4].to(gates), d[5] if st["state"] is not None else None)


def _plain_norm_of(case, x, weight, bias, gate):
    groups = case["groups"]
    swish = gate / (1 + torch.exp(-gate)) if gate is not None else None
    if case["form"] == "gate_first":
        x = x * swish
    x = x.unflatten(-1, (groups, case["width"]))
    if case["centered"]:
        x = x - x.mean(-1, keepdim=True)
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5)
    if case["weight"] == "group":
        x = x * weight if bias is None else x * weight + bias
    x = x.flatten(-2)
    if case["weight"] == "channel":
        x = x * weight if bias is None else x * weight + bias
    if case["form"] == "silu":
        x = x / (1 + torch.exp(-x))
    return x * swish if case["form"] == "gated" else x


def _plain_norm(st):
    case = st["case"]
    typ = st["x"].dtype
    x = st["x"].float()
    gate = st["gate"].float() if st["gate"] is not None else None
    weight, bias = st["weight"], st["bias"]
    if case["mode"] != "train":
        return _plain_norm_of(case, x, weight, bias, gate).to(typ)
    x, weight, bias, gate = (None if t is None else t.detach().requires_grad_() for t in (x, weight, bias, gate))
    with torch.enable_grad():
        y = _plain_norm_of(case, x, weight, bias, gate)
        leaves = [t for t in (x, weight, bias, gate) if t is not None]
        grads = list(torch.autograd.grad(y, leaves, st["d_y"].float()))
    d_x = grads.pop(0).to(typ)
    d_weight = grads.pop(0) if weight is not None else None
    d_bias = grads.pop(0) if bias is not None else None
    return y.detach().to(typ), d_x, d_weight, d_bias, grads.pop(0).to(typ) if gate is not None else None


# --------------------------------------------------------------------- the work
def work(case):
    e = 2 if case["type"] == "bf16" else 4
    tokens = _tokens(case)
    train = case["mode"] == "train"
    if case["kind"] == "norm":
        channels = case["groups"] * case["width"]
        gate = case["form"] in ("gated", "gate_first")
        n = {"channel": channels, "group": case["width"], "none": 0}[case["weight"]] * (2 if case["bias"] else 1)
        act = case["form"] != "plain"
        nbytes = tokens * channels * e * (2 + gate) + n * 4
        flops = tokens * channels * (5 + 4 * act)
        if train:  # reads x, the gate and d_y, writes d_x, the gate's and the parameters' gradients
            nbytes += tokens * channels * e * (1 + 1 + gate) + n * 4
            flops += tokens * channels * (14 + 8 * act)
        return {"bytes": nbytes, "flops": flops}
    h, p, g, n = case["heads"], case["width"], case["groups"], case["states"]
    rows = len(_lengths(case)) if "lengths" in case else case["batch"]
    eg = 2 if case["gates"] == "bf16" else 4
    states = rows * h * n * p * 4
    ins = tokens * ((2 * g * n + h * p) * e + 2 * h * eg)
    nbytes = ins + tokens * h * p * e + states * (2 if case["state"] else 1)
    # per token and head: S^T k, a S + k u^T and S^T q: 2, 3 and 2 N P
    flops = tokens * h * 7 * n * p
    if train:
        # reads d_y, writes the inputs' gradients
        nbytes += tokens * h * p * e + ins + (2 * states if case["state"] else 0)
        # S again (5 N P); G += q d_y^T, G^T k, G - k d^T, their decay; S d_y, G u, S d, <G, S>
        flops += tokens * h * 19 * n * p
    return {"bytes": nbytes, "flops": flops}


# ----------------------------------------------------------- the definition
def exact(case, seed):
    st = prepare(case, seed)
    with torch.no_grad():
        return _exact_delta(st) if case["kind"] == "delta" else _exact_norm(st)


def _exact_delta(st):
    """Token by token from the recurrence, and its reverse for the gradients."""
    case = st["case"]
    ratio, scale = case["heads"] // case["groups"], case["states"] ** -0.5
    if "lengths" in case:
        pieces = [(i, [st[n][a:b].double().unsqueeze(0) for n in ("q", "k", "v", "g", "beta")])
                  for i, (a, b) in enumerate(zip(st["ends"], st["ends"][1:]))]
    else:
        token = case["mode"] == "token"
        pieces = [(slice(None), [st[n].double().unsqueeze(1) if token else st[n].double()
                                 for n in ("q", "k", "v", "g", "beta")])]
    ys, finals = [], []
    for which, (q, k, v, g, beta) in pieces:
        q, k = q.repeat_interleave(ratio, 2), k.repeat_interleave(ratio, 2)
        rows, length = v.shape[:2]
        s = torch.zeros(rows, case["heads"], case["states"], case["width"], dtype=torch.float64, device=v.device)
        if st["state"] is not None:
            s = st["state"][which].double().reshape(s.shape)
        fade = torch.exp(g)[..., None, None]

        def move(s, t):
            kept = fade[:, t] * s
            miss = v[:, t] - (kept * k[:, t].unsqueeze(-1)).sum(-2)
            return kept, miss, kept + k[:, t].unsqueeze(-1) * (beta[:, t].unsqueeze(-1) * miss).unsqueeze(-2)

        y = torch.empty_like(v)
        marks = []
        for t in range(length):
            if case["mode"] == "train" and t % _CHUNK == 0:
                marks.append(s)
            s = move(s, t)[2]
            y[:, t] = scale * (s * q[:, t].unsqueeze(-1)).sum(-2)
        ys.append(y)
        finals.append(s)
        if case["mode"] == "train":
            return (y, s) + _exact_delta_grads(st, q, k, v, g, beta, scale, ratio, marks, move)
    if "lengths" in case:
        return torch.cat([y[0] for y in ys]), torch.cat(finals)
    return (ys[0][:, 0] if case["mode"] == "token" else ys[0]), finals[0]


def _exact_delta_grads(st, q, k, v, g, beta, scale, ratio, marks, move):
    d_y = st["d_y"].double()
    d_q, d_k, d_v = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    d_g, d_beta = torch.empty_like(g), torch.empty_like(beta)
    d_s = torch.zeros_like(marks[0]) if st["d_final"] is None else st["d_final"].double()
    for block in range(len(marks) - 1, -1, -1):
        first, behind = block * _CHUNK, min(v.shape[1], (block + 1) * _CHUNK)
        states = [marks[block]]
        for t in range(first, behind):
            states.append(move(states[-1], t)[2])
        for t in range(behind - 1, first - 1, -1):
            kept, miss, _ = move(states[t - first], t)
            d_q[:, t] = scale * (states[t - first + 1] * d_y[:, t].unsqueeze(-2)).sum(-1)
            d_s = d_s + scale * q[:, t].unsqueeze(-1) * d_y[:, t].unsqueeze(-2)
            d_u = (d_s * k[:, t].unsqueeze(-1)).sum(-2)
            d_beta[:, t] = (d_u * miss).sum(-1)
            d_v[:, t] = beta[:, t].unsqueeze(-1) * d_u
            d_k[:, t] = ((d_s * (beta[:, t].unsqueeze(-1) * miss).unsqueeze(-2)).sum(-1)
                         - (kept * d_v[:, t].unsqueeze(-2)).sum(-1))
            d_s = d_s - k[:, t].unsqueeze(-1) * d_v[:, t].unsqueeze(-2)
            d_g[:, t] = (d_s * kept).sum((-1, -2))
            d_s = torch.exp(g[:, t])[..., None, None] * d_s
    shared = (*q.shape[:2], q.shape[2] // ratio, ratio, q.shape[3])
    return (d_q.reshape(shared).sum(3), d_k.reshape(shared).sum(3), d_v, d_g, d_beta,
            d_s if st["state"] is not None else None)


def _exact_norm(st):
    case = st["case"]
    groups, width = case["groups"], case["width"]

    def split(t):
        return t.double().reshape(-1, groups, width)

    def parameter(t, without):
        if t is None:
            return torch.full((groups, width), without, dtype=torch.float64, device=st["x"].device)
        return t.double().reshape(-1, width).expand(groups, width)

    x, w, b = split(st["x"]), parameter(st["weight"], 1.0), parameter(st["bias"], 0.0)
    z = split(st["gate"]) if st["gate"] is not None else None
    sz = torch.sigmoid(z) if z is not None else None
    h = x * (z * sz) if case["form"] == "gate_first" else x
    centre = h.mean(-1, keepdim=True) if case["centered"] else 0.0
    r = ((h - centre).square().mean(-1, keepdim=True) + 1e-5) ** -0.5
    n = (h - centre) * r
    o = n * w + b
    so = torch.sigmoid(o)
    y = {"plain": lambda: o, "gate_first": lambda: o, "silu": lambda: o * so, "gated": lambda: o * z * sz}[case["form"]]()
    y = y.reshape(st["x"].shape)
    if case["mode"] != "train":
        return y
    d = split(st["d_y"])
    d_gate = None
    if case["form"] == "silu":
        d = d * so * (1 + o * (1 - so))
    elif case["form"] == "gated":
        d_gate = d * o * sz * (1 + z * (1 - sz))
        d = d * z * sz
    d_w, d_b = (d * n).sum(0), d.sum(0)
    if case["weight"] == "group":
        d_w, d_b = d_w.sum(0), d_b.sum(0)
    d_n = d * w
    d_h = d_n - n * (d_n * n).mean(-1, keepdim=True)
    if case["centered"]:
        d_h = d_h - d_n.mean(-1, keepdim=True)
    d_h = d_h * r
    if case["form"] == "gate_first":
        d_gate = d_h * x * sz * (1 + z * (1 - sz))
        d_h = d_h * z * sz
    shape = st["x"].shape
    return (y, d_h.reshape(shape), d_w.reshape(-1) if st["weight"] is not None else None,
            d_b.reshape(-1) if st["bias"] is not None else None, None if d_gate is None else d_gate.reshape(shape))
