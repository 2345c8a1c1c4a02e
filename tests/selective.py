"""Seeded inputs and error bounds of the selective layer's GPU tests.

Bounds.  u = 2^-24 is half a step of fp32, ub = 2^-8 of bf16.  A sum of terms
computed with at most n roundings per term is within n u of the sum of the
terms' absolute values (the oracle's absolute form), whatever the order.  For
the scan n counts: a product over the states (N), over a step of 64 tokens
(64) and over the columns (P), one decay and addition per step (L / 64), the
argument of an exponential (up to 128 before the result is zero, in steps of u)
and 64 for everything of fixed length (softplus, exp, scalings).  bf16 results
add half a step of the result; and where the kernels round an operand of a
product to bf16 (scores, the state as an operand) that is ub per term, twice
for the state's way through a score.  An operand in two bf16 parts is within
2^-16, one in three is whole.  A term below fp32's smallest normal number, 2^-126, may
become zero: up to 2^16 such terms in a sum, each times a factor of the inputs'
size (below 2^10), are within 2^-100, which fp32's arithmetic cannot tell from
zero beside anything larger.
"""
from __future__ import annotations

import torch

U, UB = 2.0 ** -24, 2.0 ** -8
TINY = 2.0 ** -100
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def half_step(t):
    return UB if t == torch.bfloat16 else U


def within(got, want, bound, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if want.numel() == 0:
        return
    assert bool(torch.isfinite(got).all()), what
    over = (got - want).abs() - bound - TINY
    worst = int(over.argmax())
    assert float(over.max()) <= 0, (what, worst, float(got.reshape(-1)[worst]), float(want.reshape(-1)[worst]),
                                    float(bound.expand_as(want).reshape(-1)[worst]))


def gen(seed):
    return torch.Generator().manual_seed(seed)


def scan_inputs(seed, lead, rows, H, P, G, N, typ, dt_typ, *, positive=False, state=True):
    """CPU tensors.  positive: every term of y has the same sign, so the bounds are relative ones."""
    g = gen(seed)

    def r(*s):
        v = torch.randn(*s, generator=g)
        return v.abs() if positive else v

    typ, dt_typ = TYPES[typ], TYPES[dt_typ]
    return dict(x=r(*lead, H, P).to(typ), dt=torch.randn(*lead, H, generator=g).to(dt_typ),
                A=-torch.exp(3 * torch.rand(H, generator=g) - 1), B=r(*lead, G, N).to(typ), C=r(*lead, G, N).to(typ),
                D=r(H), dt_bias=torch.randn(H, generator=g) - 2, state=r(rows, H, N, P) if state else None,
                d_y=r(*lead, H, P).to(typ), d_final=r(rows, H, N, P))


def to(p, dev):
    return {k: None if v is None else v.to(dev) for k, v in p.items()}


def scan_roundings(L, P, N):
    return N + P + 64 + L / 64 + 128 + 64
