"""The float64 oracle of the gated delta rule and the group norm against closed forms, automatic differentiation,
differences, and the computation in steps that the bounds follow.
"""
from __future__ import annotations

import math

import pytest
import torch

from oracle import delta_oracle as orc
from tests import delta_rule as dr

F = torch.float64


def _one(p):
    return {k: v[0] if k in ("state", "d_final") and v is not None else v for k, v in p.items()}


def _args(p):
    return p["q"], p["k"], p["v"], p["g"], p["beta"]


@pytest.mark.parametrize("strong", [False, True])
@pytest.mark.parametrize("L,H,V,G,K", [(0, 2, 8, 1, 8), (1, 2, 8, 2, 8), (64, 1, 16, 1, 8), (150, 4, 24, 2, 16)])
def test_steps_are_the_rule(L, H, V, G, K, strong):
    p = _one(dr.inputs(1, (L,), 1, H, V, G, K, "f32", "f32", strong=strong))
    b = dr.bounds(p, 0.3, True)
    y, final = orc.delta(*_args(p), 0.3, p["state"])
    want = dict(y=y, final=final, **orc.delta_grads(*_args(p), 0.3, p["state"], p["d_y"], p["d_final"]))
    for name, (value, bound) in b.items():
        assert torch.allclose(value, want[name], rtol=1e-11, atol=1e-12), name
        assert bool((bound >= 0).all()) and bool(torch.isfinite(bound).all())


def test_recall():
    """Orthonormal keys, beta 1 and no decay: a state that returns each key's last value."""
    K, V = 8, 16
    k = torch.eye(K, dtype=F)[torch.tensor([0, 3, 5, 3])].unsqueeze(1)
    v = torch.randn(4, 1, V, dtype=F)
    z, one = torch.zeros(4, 1, dtype=F), torch.ones(4, 1, dtype=F)
    y, s = orc.delta(k, k, v, z, one, 1.0, None)
    assert torch.allclose(y, v)
    for key, t in ((0, 0), (5, 2), (3, 3)):
        assert torch.allclose(s[0, key], v[t, 0])
    assert float(s[0, [1, 2, 4, 6, 7]].abs().max()) == 0


def test_idle_and_forgetting_tokens():
    p = _one(dr.inputs(2, (9,), 1, 2, 8, 1, 8, "f32", "f32"))
    idle = dict(p, g=torch.zeros(9, 2), beta=torch.zeros(9, 2))
    assert torch.equal(orc.delta(*_args(idle), 1.0, p["state"])[1], p["state"].double())
    cut = dict(p, g=p["g"].clone())
    cut["g"][4] = -math.inf
    y, s = orc.delta(*_args(cut), 1.0, p["state"])
    tail = [t[4:] for t in _args(cut)]
    y4, s4 = orc.delta(*tail, 1.0, None)
    assert torch.allclose(y[4:], y4) and torch.allclose(s, s4)
    d = orc.delta_grads(*_args(cut), 1.0, p["state"], p["d_y"], p["d_final"])
    assert float(d["d_g"][4].abs().max()) == 0
    # what was before the token is reached by the results before it alone
    before = orc.delta_grads(*(t[:4] for t in _args(cut)), 1.0, p["state"], p["d_y"][:4], None)
    assert torch.allclose(d["d_state"], before["d_state"]) and torch.allclose(d["d_v"][:4], before["d_v"])


def test_rule_gradients():
    p = {k: v.double() for k, v in _one(dr.inputs(3, (21,), 1, 4, 16, 2, 8, "f32", "f32")).items()}
    names = ("q", "k", "v", "g", "beta", "state")
    d = orc.delta_grads(*_args(p), 0.4, p["state"], p["d_y"], p["d_final"])

    def loss(values):
        y, s = orc.delta(*values[:5], 0.4, values[5])
        return (y * p["d_y"]).sum() + (s * p["d_final"]).sum()

    base = [p[n] for n in names]
    gen = torch.Generator().manual_seed(4)
    for i, n in enumerate(names):  # differences, along one direction each
        w, h = torch.randn(base[i].shape, generator=gen, dtype=F), 1e-5
        at = lambda s: loss([b + s * h * w if j == i else b for j, b in enumerate(base)])
        slope = float((at(1) - at(-1)) / (2 * h))
        want = float((d["d_" + n] * w).sum())
        assert abs(slope - want) <= 1e-7 * max(1.0, abs(want)), n


def test_rule_gradients_by_autograd():
    p = {k: v.double() for k, v in _one(dr.inputs(5, (17,), 1, 2, 8, 1, 8, "f32", "f32")).items()}
    leaves = [p[n].clone().requires_grad_() for n in ("q", "k", "v", "g", "beta", "state")]
    q, k, v, g, beta, s = leaves
    ys = []
    for t in range(17):
        s = torch.exp(g[t])[:, None, None] * s
        kt, qt = k[t].expand(2, 8), q[t].expand(2, 8)
        u = beta[t][:, None] * (v[t] - (s * kt[:, :, None]).sum(1))
        s = s + kt[:, :, None] * u[:, None, :]
        ys.append(0.4 * (s * qt[:, :, None]).sum(1))
    grads = torch.autograd.grad([torch.stack(ys), s], leaves, [p["d_y"], p["d_final"]])
    d = orc.delta_grads(*_args(p), 0.4, p["state"], p["d_y"], p["d_final"])
    for n, e in zip(("q", "k", "v", "g", "beta", "state"), grads):
        assert torch.allclose(d["d_" + n], e, rtol=1e-12, atol=1e-13), n


@pytest.mark.parametrize("form", ["plain", "silu", "gated", "gate_first"])
@pytest.mark.parametrize("centered", [False, True])
@pytest.mark.parametrize("shared", [False, True])
def test_norm_gradients(form, centered, shared):
    gen = torch.Generator().manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=F)
    rows, groups, width = 5, 3, 7
    x, z, d_y = r(rows, 21), r(rows, 21), r(rows, 21)
    n = width if shared else 21
    w, b = 1 + 0.3 * r(n), 0.3 * r(n)
    gate = z if form in ("gated", "gate_first") else None
    d = orc.group_norm_grads(x, w, b, gate, groups, form, centered, 1e-5, d_y)
    names = ["d_x", "d_weight", "d_bias"] + (["d_gate"] if gate is not None else [])
    base = [x, w, b] + ([gate] if gate is not None else [])
    for i, name in enumerate(names):
        v, h = r(*base[i].shape), 1e-5
        f = lambda s: float((orc.group_norm(*[t + s * h * v if j == i else t for j, t in enumerate(base)],
                                            *([None] if gate is None else []), groups, form, centered, 1e-5) * d_y).sum())
        want = float((d[name] * v).sum())
        assert abs((f(1) - f(-1)) / (2 * h) - want) <= 1e-7 * max(1.0, abs(want)), name


def test_norm_closed_forms():
    x = torch.tensor([[3.0, 4.0, 0.0, 0.0, 1.0, 1.0, 1.0, 1.0]])
    y = orc.group_norm(x, None, None, None, 2, "plain", False, 1e-30)
    assert torch.allclose(y[0, :2], torch.tensor([1.2, 1.6], dtype=F)) and torch.allclose(y[0, 4:], torch.ones(4, dtype=F))
    y = orc.group_norm(x, None, None, None, 2, "plain", True, 1e-30)
    assert abs(float(y.sum())) < 1e-12
    # a weight of 1 / sqrt(width) and no mean: length one
    y = orc.group_norm(torch.randn(4, 32), torch.full((16,), 0.25), None, None, 2, "plain", False, 1e-30)
    assert torch.allclose(y.unflatten(1, (2, 16)).norm(dim=-1), torch.ones(4, 2, dtype=F))
    gate = torch.full((1, 8), 40.0)
    assert torch.allclose(orc.group_norm(x, None, None, gate, 2, "gated", False, 1e-5),
                          40 * orc.group_norm(x, None, None, None, 2, "plain", False, 1e-5))
