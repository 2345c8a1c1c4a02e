"""Running error bounds: values in float64 beside a bound on what fp32 arithmetic makes of them.

An `E` holds the exact value x of an expression and a bound e on how far a
computation of the same expression, rounding after every operation, may be from
it.  u = 2^-24 is half a step of fp32.  Counted per operation: an addition or
product 1 u; a sum or matrix product of n terms 2 n u of its terms' absolute
values, in any order (2: the matrix instructions may cut bits off where an
addition would round); exponentials, sigmoids, reciprocal roots 4 to 8 u and
their argument's error times their derivative.  First-order terms of two
errors are kept, so the bounds hold as they stand.
"""
from __future__ import annotations

import torch

U, UB = 2.0 ** -24, 2.0 ** -8
TINY = 2.0 ** -100  # what denormal terms that became zero may add up to


class E:
    def __init__(self, x, e=None):
        self.x = x.double()
        self.e = torch.zeros_like(self.x) if e is None else e.expand_as(self.x)

    def _of(self, o):
        return o if isinstance(o, E) else E(torch.as_tensor(o, dtype=torch.float64).expand_as(self.x)
                                            if not isinstance(o, torch.Tensor) else o)

    def __add__(self, o):
        o = self._of(o)
        x = self.x + o.x
        return E(x, self.e + o.e + U * x.abs())

    def __neg__(self):
        return E(-self.x, self.e)

    def __sub__(self, o):
        return self + (-self._of(o))

    def __mul__(self, o):
        o = self._of(o)
        x = self.x * o.x
        return E(x, self.x.abs() * o.e + self.e * o.x.abs() + self.e * o.e + U * x.abs())

    def __getitem__(self, i):
        return E(self.x[i], self.e[i])

    @property
    def T(self):
        return E(self.x.transpose(-1, -2), self.e.transpose(-1, -2))

    def masked(self, m):
        return E(self.x * m, self.e * m)

    def sum(self, dim, keepdim=False, n=None):
        """n: additions that a term goes through at most (default: all)."""
        n = self.x.shape[dim] if n is None else n
        return E(self.x.sum(dim, keepdim=keepdim),
                 self.e.sum(dim, keepdim=keepdim) + 2 * n * U * self.x.abs().sum(dim, keepdim=keepdim))

    def unsqueeze(self, d):
        return E(self.x.unsqueeze(d), self.e.unsqueeze(d))

    def wider(self, e):
        """The same value with a further error."""
        return E(self.x, self.e + e)

    def sigmoid(self):
        s = torch.sigmoid(self.x)
        return E(s, 1.01 * self.e * s * (1 - s) + 8 * U * s)

    def rsqrt(self):
        r = self.x ** -0.5
        return E(r, r * (0.51 * self.e / self.x + 4 * U))


def mm(a, b, parts=0.0):
    """a @ b; parts: the relative error of operands that go in in fewer bits than fp32 has."""
    n = a.x.shape[-1]
    size = a.x.abs() @ b.x.abs()
    return E(a.x @ b.x, a.x.abs() @ b.e + a.e @ b.x.abs() + a.e @ b.e + (2 * (n + 4) * U + parts) * size)


def of_type(v, typ):
    """The bound of a result that is rounded to its type once more, and the value itself."""
    step = UB if typ == torch.bfloat16 else U
    return v.x, v.e * (1 + step) + step * v.x.abs() + TINY


def within(got, want, bound, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if want.numel() == 0:
        return
    assert bool(torch.isfinite(got).all()), what
    over = (got - want).abs() - bound
    worst = int(over.argmax())
    assert float(over.max()) <= 0, (what, worst, float(got.reshape(-1)[worst]), float(want.reshape(-1)[worst]),
                                    float(bound.expand_as(want).reshape(-1)[worst]))
