"""The float64 oracle of the selective layer against closed forms and central differences (CPU)."""
from __future__ import annotations

import math

import pytest
import torch

from oracle import selective_oracle as orc

F64 = torch.float64


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _scan_inputs(seed, L=5, H=4, P=3, G=2, N=2):
    g = _gen(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=F64)
    return dict(x=r(L, H, P), dt=r(L, H), A=-torch.rand(H, generator=g, dtype=F64) - 0.2, B=r(L, G, N), C=r(L, G, N),
                D=r(H), dt_bias=r(H), state=r(H, N, P)), r(L, H, P), r(H, N, P)


def test_scan_of_constant_decay_is_a_geometric_sum():
    # one head, one state, B = C = 1, d = 1: y_t = sum_{s <= t} a^(t - s) x_s
    L, a = 6, 0.7
    x = torch.randn(L, 1, 1, generator=_gen(0), dtype=F64)
    one = torch.ones(L, 1, 1, dtype=F64)
    y, _ = orc.scan(x, torch.ones(L, 1, dtype=F64), torch.tensor([math.log(a)], dtype=F64), one, one, None, None, False,
                    None)
    want = torch.stack([sum(a ** (t - s) * x[s, 0, 0] for s in range(t + 1)) for t in range(L)])
    assert torch.allclose(y[:, 0, 0], want, rtol=1e-13, atol=1e-13)


def test_a_token_without_step_leaves_the_state():
    p, _, _ = _scan_inputs(1)
    p["dt"][2] = -math.inf
    _, states = orc.scan(p["x"], p["dt"], p["A"], p["B"], p["C"], p["D"], p["dt_bias"], True, p["state"])
    assert torch.equal(states[3], states[2])


def test_conv_is_a_sliding_product():
    g = _gen(2)
    x, w = torch.randn(7, 2, generator=g, dtype=F64), torch.randn(2, 3, generator=g, dtype=F64)
    y, _, tail = orc.conv(x, w, None, None, False)
    want = torch.nn.functional.conv1d(x.T[None], w[:, None], padding=2, groups=2)[0, :, :7].T
    assert torch.allclose(y, want) and torch.equal(tail, x[-2:])


@pytest.mark.parametrize("softplus", [True, False])
def test_scan_gradients_against_differences(softplus):
    p, d_y, d_final = _scan_inputs(3)
    if not softplus:
        p["dt"], p["dt_bias"] = p["dt"].abs() * 0.3, None
    names = {"x": "d_x", "dt": "d_dt", "A": "d_A", "B": "d_B", "C": "d_C", "D": "d_D", "dt_bias": "d_dt_bias",
             "state": "d_state"}

    def loss(q):
        y, s = orc.scan(q["x"], q["dt"], q["A"], q["B"], q["C"], q["D"], q["dt_bias"], softplus, q["state"])
        return float((y * d_y).sum() + (s[-1] * d_final).sum())

    grads = orc.scan_grads(*(p[k] for k in ("x", "dt", "A", "B", "C", "D", "dt_bias")), softplus, p["state"], d_y, d_final)
    _differences(p, names, grads, loss)


@pytest.mark.parametrize("silu", [True, False])
def test_conv_gradients_against_differences(silu):
    g = _gen(4)
    r = lambda *s: torch.randn(*s, generator=g, dtype=F64)
    p = dict(x=r(6, 3), weight=r(3, 4), bias=r(3), state=r(3, 3))
    d_y, d_final = r(6, 3), r(3, 3)

    def loss(q):
        y, _, tail = orc.conv(q["x"], q["weight"], q["bias"], q["state"], silu)
        return float((y * d_y).sum() + (tail * d_final).sum())

    grads = orc.conv_grads(p["x"], p["weight"], p["bias"], p["state"], silu, d_y, d_final)
    _differences(p, {"x": "d_x", "weight": "d_weight", "bias": "d_bias", "state": "d_state"}, grads, loss)


def _differences(p, names, grads, loss):
    # central differences of a smooth function: error h^2 f'''/6 + eps |f| / h
    h = 1e-5
    for name, grad in names.items():
        if p[name] is None:
            continue
        flat = p[name].reshape(-1)
        for i in range(0, flat.numel(), 3):
            q = dict(p)
            q[name] = p[name].clone()
            q[name].reshape(-1)[i] += h
            up = loss(q)
            q[name].reshape(-1)[i] -= 2 * h
            got = (up - loss(q)) / (2 * h)
            assert abs(got - float(grads[grad].reshape(-1)[i])) <= 1e-7 * (1 + abs(got)), (name, i)
