"""Seeded inputs and error bounds of the gated delta rule's tests.

The bounds follow the computation in steps of 64 tokens with running errors
(tests/rounded.py).  From step to step errors are carried by norms: with
beta |k|^2 <= 2 and g <= 0 a token's transition, e^g (1 - beta k k^T), makes no
column of a state longer, so an error of 2-norm d in a column stays within d,
and reaches a token's results with at most |q| d, its correction with |k| d.
The same holds for the state's gradient on its way back.
"""
from __future__ import annotations

import torch

from tests.rounded import E, U, mm, of_type

STEP = 64
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(seed, lead, rows, H, V, G, K, typ, gates, *, state=True, strong=False):
    """CPU tensors: keys and queries of length one, decays up to e^-8 (strong) or about 0.9, beta in (0, 1)."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    unit = lambda v: v / (v.norm(dim=-1, keepdim=True) + 1e-6)
    typ, gates = TYPES[typ], TYPES[gates]
    g = -torch.rand(*lead, H, generator=gen) * (8.0 if strong else 0.2)
    return dict(q=unit(r(*lead, G, K)).to(typ), k=unit(r(*lead, G, K)).to(typ), v=r(*lead, H, V).to(typ),
                g=g.to(gates), beta=torch.sigmoid(r(*lead, H)).to(gates), state=r(rows, H, K, V) if state else None,
                d_y=r(*lead, H, V).to(typ), d_final=r(rows, H, K, V))


def to(p, dev):
    return {k: None if v is None else v.to(dev) for k, v in p.items()}


def _steps(p, H):
    """The tensors of one sequence by step, heads first, padded with tokens that do nothing."""
    L = p["v"].shape[0]
    n = max(1, -(-L // STEP)) if L else 0
    out = []
    for c in range(n):
        cut = {}
        for name in ("q", "k", "v", "g", "beta", "d_y"):
            t = p[name][c * STEP:(c + 1) * STEP].double()
            if name in ("q", "k"):
                t = t.repeat_interleave(H // t.shape[1], 1)
            t = torch.cat([t, torch.zeros(STEP - t.shape[0], *t.shape[1:], dtype=torch.float64)])
            cut[name] = t.transpose(0, 1)
        out.append(cut)
    return out


def _matrices(c, scale):
    q, k, beta = E(c["q"]), E(c["k"]), E(c["beta"])
    cum = torch.clamp(c["g"], min=-760.0).cumsum(-1)
    diff = cum.unsqueeze(-1) - cum.unsqueeze(-2)
    low = torch.ones(STEP, STEP, dtype=torch.float64).tril()
    decay = torch.exp(diff.masked_fill(low == 0, -torch.inf))
    # the exponent is a difference of two floats each: u of the difference, and 4 u of the exponential
    e = E(decay, decay * (diff.abs().clamp(max=100.0) + 6) * U)
    kk, qk = mm(k, k.T), mm(q, k.T)
    strict = low.tril(-1)
    t = (beta.unsqueeze(-1) * (e * kk)).masked(strict)
    m = torch.linalg.inv(torch.eye(STEP, dtype=torch.float64) + t.x)
    a = m.abs()
    inv = E(m, a @ t.e @ a + 2 * (STEP + 4) * U * (a @ (torch.eye(STEP, dtype=torch.float64) + t.x.abs()) @ a))
    p = (scale * (e * qk).masked(low).x, scale * (1 + 4 * U) * ((e * qk).masked(low).e + U * (e * qk).masked(low).x.abs()))
    one = lambda v: E(v, 4 * U * v)
    return dict(q=q, k=k, beta=beta.unsqueeze(-1), e=e, kk=kk, qk=qk, m=inv, p=E(*p), low=low, strict=strict,
                start=one(torch.exp(cum)).unsqueeze(-1), to=one(torch.exp(cum[:, -1:] - cum)).unsqueeze(-1),
                total=one(torch.exp(cum[:, -1])).unsqueeze(-1).unsqueeze(-1), v=E(c["v"]), dy=E(c["d_y"]))


def _norm(e):
    return (e * e).sum(-2).sqrt()  # of every column


def bounds(p, scale, grads=False):
    """{name: (value, bound)} of one sequence's results; p as `inputs` gives them, without a batch axis."""
    typ, gates = p["v"].dtype, p["g"].dtype
    L, H, V = p["v"].shape
    G, K = p["q"].shape[1:]
    two = 0.0 if typ == torch.float32 else 2.0 ** -15  # operands in two bf16 parts, of bf16 results
    s = torch.zeros(H, K, V, dtype=torch.float64) if p["state"] is None else p["state"].double()
    err = torch.zeros(H, V, dtype=torch.float64)  # 2-norms of the state's columns' errors
    ys, kept = [], []
    for c in _steps(p, H):
        x = _matrices(c, scale)
        S = E(s)
        kept.append((x, s, err))
        r = x["beta"] * (x["v"] - x["start"] * mm(x["k"], S))
        u = mm(x["m"], r)
        ye = x["start"] * mm(x["q"], S, two)
        ye = E(scale * ye.x, scale * (ye.e + 2 * U * ye.x.abs())) + mm(x["p"], u, two)
        length = lambda t: t.x.norm(dim=-1, keepdim=True)
        ys.append(ye.wider(scale * length(x["q"]) * err.unsqueeze(1)))
        kept[-1] += (u.wider(x["beta"].x * length(x["k"]) * err.unsqueeze(1)),)
        after = x["total"] * S + mm(x["k"].T, x["to"] * u)
        err = x["total"].x.squeeze(-1) * err + _norm(after.e)
        s = after.x
    flat = lambda parts, n: E(torch.cat([t.x for t in parts], 1)[:, :L].transpose(0, 1),
                              torch.cat([t.e for t in parts], 1)[:, :L].transpose(0, 1)) if parts else E(torch.zeros(0, H, n))
    out = dict(y=of_type(flat(ys, V), typ), final=of_type(E(s, err.unsqueeze(1)), torch.float32))
    if not grads:
        return out
    d = torch.zeros(H, K, V, dtype=torch.float64) if p["d_final"] is None else p["d_final"].double()
    err = torch.zeros(H, V, dtype=torch.float64)
    got = {n: [] for n in ("d_q", "d_k", "d_v", "d_g", "d_beta")}
    for x, s, s_err, u in reversed(kept):
        D, S = E(d), E(s, s_err.unsqueeze(1).expand_as(s))
        du = mm(x["p"].T, x["dy"]) + x["to"] * mm(x["k"], D)
        dr = mm(x["m"].T, du)
        Dw = E(d, err.unsqueeze(1).expand_as(d))
        drw = dr.wider(x["k"].x.norm(dim=-1, keepdim=True) * err.unsqueeze(1))
        got["d_v"].append(x["beta"] * drw)
        ys_, rs, ud = mm(x["dy"], S.T), mm(drw, S.T), mm(u, Dw.T)
        dp, dt = mm(x["dy"], u.T).masked(x["low"]), -mm(drw, u.T).masked(x["strict"])
        sc = E(torch.full((1, 1, 1), scale, dtype=torch.float64))
        pm, et = sc * (x["e"] * dp), x["e"] * dt
        xm = x["beta"] * et
        yq, rk, uk = sc * (x["start"] * ys_), x["start"] * rs, x["to"] * ud
        got["d_q"].append(yq + mm(pm, x["k"], two))
        got["d_k"].append((uk - x["beta"] * rk) + (mm(pm.T, x["q"], two) + (mm(xm, x["k"], two) + mm(xm.T, x["k"], two))))
        kr = (x["k"] * rk).sum(-1)
        got["d_beta"].append(((drw * x["v"]).sum(-1) - kr + (et * x["kk"]).sum(-1)).unsqueeze(-1))
        a = (x["q"] * yq).sum(-1) - x["beta"][..., 0] * kr
        f = (x["k"] * uk).sum(-1)
        z = pm * x["qk"] + xm * x["kk"]
        ends = (x["total"] * (S * Dw))
        ends = E(ends.x.sum((1, 2)), ends.e.sum((1, 2)) + 2 * (K + V) * U * ends.x.abs().sum((1, 2)))
        cols = []
        for t in range(STEP):
            part = E(z.x[:, t:, :t].sum((1, 2)), z.e[:, t:, :t].sum((1, 2)) + 4 * STEP * U * z.x[:, t:, :t].abs().sum((1, 2)))
            cols.append(((a[:, t:].sum(1) + (f[:, :t].sum(1) if t else E(torch.zeros(H)))) + part) + ends)
        got["d_g"].append(E(torch.stack([v.x for v in cols], 1), torch.stack([v.e for v in cols], 1)).unsqueeze(-1))
        before = (x["total"] * D + mm(x["q"].T, sc * (x["start"] * x["dy"]))) - mm(x["k"].T, x["beta"] * (x["start"] * dr))
        err = x["total"].x.squeeze(-1) * err + _norm(before.e)
        d = before.x
    for n, w, t in (("d_q", K, typ), ("d_k", K, typ), ("d_v", V, typ), ("d_g", 1, gates), ("d_beta", 1, gates)):
        v = flat(got[n][::-1], w)
        if n in ("d_q", "d_k"):
            v = E(v.x.unflatten(1, (G, H // G)), v.e.unflatten(1, (G, H // G))).sum(2)
        out[n] = of_type(E(v.x.squeeze(-1), v.e.squeeze(-1)) if n in ("d_g", "d_beta") else v, t)
    out["d_state"] = of_type(E(d, err.unsqueeze(1)), torch.float32)
    return out
