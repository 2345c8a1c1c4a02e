"""Seeded inputs and error bounds of the group norm's tests (tests/rounded.py)."""
from __future__ import annotations

import torch

from tests.rounded import E, U, of_type

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
FORMS = ("plain", "silu", "gated", "gate_first")
# Additions of a term within a group: a lane's own (up to 16), six steps of a wave, a wave's sums (up to 16).
TERMS = 40


def inputs(seed, lead, groups, width, typ, form, weight, bias):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    channels, typ = groups * width, TYPES[typ]
    n = {"channel": channels, "group": width, None: 0}[weight]
    size = torch.exp(torch.rand(groups, generator=gen) * 4 - 2).repeat_interleave(width)
    return dict(x=(r(*lead, channels) * size + 0.2).to(typ), weight=1 + 0.3 * r(n) if n else None,
                bias=0.3 * r(n) if bias else None, gate=r(*lead, channels).to(typ) if form in FORMS[2:] else None,
                d_y=r(*lead, channels).to(typ))


def keywords(groups, form, centered, eps=1e-5):
    return dict(groups=groups, silu=form == "silu", gate_first=form == "gate_first", centered=centered, eps=eps)


def bounds(p, groups, form, centered, eps, grads=False):
    """{name: (value, bound)}; tensors with one leading axis"""
    typ = p["x"].dtype
    rows, channels = p["x"].shape
    width = channels // groups
    cut = lambda t: E(t.double().reshape(rows, groups, width))
    const = lambda v: E(torch.full((1, 1, 1), v, dtype=torch.float64), torch.full((1, 1, 1), 2 * U * abs(v), dtype=torch.float64))
    par = lambda t, v: E(torch.full((groups, width), v, dtype=torch.float64) if t is None
                         else t.double().reshape(-1, width).expand(groups, width))
    mean = lambda v: v.sum(-1, keepdim=True, n=TERMS) * const(1.0 / width)
    x = cut(p["x"])
    w, b = par(p["weight"], 1.0), par(p["bias"], 0.0)
    if p["gate"] is not None:
        z = cut(p["gate"])
        s = z.sigmoid()
        swish, d_swish = z * s, s * (const(1.0) + z * (const(1.0) - s))
    h = x * swish if form == "gate_first" else x
    c = h - mean(h) if centered else h
    r = (mean(c * c) + const(eps)).rsqrt()
    n = c * r
    o = n * w + b
    so = o.sigmoid()
    y = {"plain": lambda: o, "gate_first": lambda: o, "silu": lambda: o * so, "gated": lambda: o * swish}[form]()
    flat = lambda v: E(v.x.reshape(rows, channels), v.e.reshape(rows, channels))
    out = dict(y=of_type(flat(y), typ))
    if not grads:
        return out
    d = cut(p["d_y"])
    d_z = None
    if form == "silu":
        d = d * (so * (const(1.0) + o * (const(1.0) - so)))
    elif form == "gated":
        d_z = d * o * d_swish
        d = d * swish
    dn = d * w
    d_h = dn - n * mean(dn * n)
    if centered:
        d_h = d_h - mean(dn)
    d_h = d_h * r
    if form == "gate_first":
        d_z = d_h * x * d_swish
        d_h = d_h * swish
    out["d_x"] = of_type(flat(d_h), typ)
    if d_z is not None:
        out["d_gate"] = of_type(flat(d_z), typ)
    for name, given, v in (("d_weight", p["weight"], d * n), ("d_bias", p["bias"], d)):
        if given is None:
            continue
        v = v.sum(0, n=rows + 64)
        if given.numel() == width:
            v = v.sum(0, n=groups)
        out[name] = of_type(E(v.x.reshape(-1), v.e.reshape(-1)), torch.float32)
    return out
