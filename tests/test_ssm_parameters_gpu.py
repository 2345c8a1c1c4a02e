"""Decay parameters A that are not finite, in the scan and its single-token form, on an MI355X."""
from __future__ import annotations

import math

import pytest
import torch

import bwd_mamba2_scan_amd as m2
from oracle import selective_oracle as orc
from tests.selective import U, half_step, scan_inputs, scan_roundings, to, within

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
H, P, G, N = 4, 24, 2, 40


def _run(p, **kw):
    d = to(p, DEV)
    args = [d[k] for k in ("x", "dt", "A", "B", "C")]
    kw = dict(D=d["D"], dt_bias=d["dt_bias"], initial_state=d["state"], **kw)
    y, final = m2.ssm_fwd(*args, want_final_state=True, **kw)
    return y, final, m2.ssm_bwd(*args, d["d_y"], d_final_state=d["d_final"], **kw)


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 70, 900])
def test_nan_reaches_its_head_and_no_other(typ, L):
    print("A = NaN", typ, L, flush=True)
    p = scan_inputs(L, (2, L), 2, H, P, G, N, typ, typ)
    y0, f0, g0 = _run(p)
    p["A"][1] = math.nan
    y, f, g = _run(p)
    others = [0, 2, 3]
    for got, want in ((y, y0), (f.transpose(1, 2), f0.transpose(1, 2)), (g["d_x"], g0["d_x"])):
        assert bool(torch.isnan(got[:, :, 1]).all()) and torch.equal(got[:, :, others], want[:, :, others])
    assert bool(torch.isnan(g["d_dt"][:, :, 1]).all()) and torch.equal(g["d_dt"][:, :, others], g0["d_dt"][:, :, others])
    for k in ("d_A", "d_dt_bias"):
        assert bool(torch.isnan(g[k][1])) and torch.equal(g[k][others], g0[k][others]), k
    for k in ("d_B", "d_C"):  # the first group's heads are 0 and 1
        assert bool(torch.isnan(g[k][:, :, 0]).all()) and torch.equal(g[k][:, :, 1], g0[k][:, :, 1]), k


@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_nan_and_infinity_in_a_step(typ):
    p = scan_inputs(3, (3,), 3, H, P, G, N, typ, typ)
    p["A"][1], p["A"][2] = math.nan, -math.inf
    p["dt"][1] = -math.inf                       # a token without a step
    d = to(p, DEV)
    y = m2.ssm_step(*(d[k] for k in ("x", "dt", "A", "B", "C")), d["state"], D=d["D"], dt_bias=d["dt_bias"])
    state, old = d["state"].cpu(), p["state"]
    assert bool(torch.isnan(state[:, 1]).all()) and bool(torch.isnan(y[:, 1]).all())
    assert torch.equal(state[1, [0, 2, 3]], old[1, [0, 2, 3]])
    step = orc.steps(p["dt"], p["dt_bias"], True)
    for s in (0, 2):                             # head 2 keeps nothing but the token
        want = step[s, 2] * p["B"][s, 1].double()[:, None] * p["x"][s, 2].double()[None]
        within(state[s, 2], want, scan_roundings(1, P, N) * U * want.abs(), "state")
    assert bool(torch.isfinite(y[:, [0, 2, 3]]).all())


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 66, 700])
def test_infinite_decay_forgets(typ, L):
    """A = -inf: y_t is the token's own term, and a padded tail (dt = -inf) leaves the last token's state."""
    print("A = -inf", typ, L, flush=True)
    pad = 30
    p = scan_inputs(L + 1, (1, L + pad), 1, H, P, G, N, typ, typ)
    p["A"][0] = -math.inf
    p["dt"][:, L:] = -math.inf
    p["d_y"][:, L:] = 0
    y, final, g = _run(p)
    step = orc.steps(p["dt"], p["dt_bias"], True)[0, :, 0]
    x, B, C = p["x"][0, :, 0].double(), p["B"][0, :, 0].double(), p["C"][0, :, 0].double()
    own = ((B * C).sum(-1) * step)[:, None] * x
    size = (((B * C).abs().sum(-1) * step)[:, None] + p["D"][0].double().abs()) * x.abs()
    want = own + p["D"][0].double() * x
    n = scan_roundings(L, P, N) * U
    rough = 2.02 * half_step(p["x"].dtype) if typ == "bf16" else 0.0     # scores rounded to bf16
    within(y[0, :L, 0], want[:L], (n + rough) * size[:L] + half_step(p["x"].dtype) * want[:L].abs(), "y")
    state = step[L - 1] * B[L - 1][:, None] * x[L - 1][None]
    within(final[0, 0], state, n * state.abs(), "final state")
    short = {k: v[:, :L] if k in ("x", "dt", "B", "C", "d_y") else v for k, v in p.items()}
    y1, f1, g1 = _run(short)
    assert torch.equal(y[:, :L], y1) and torch.equal(final, f1)
    assert torch.equal(g["d_x"][:, :L], g1["d_x"])
