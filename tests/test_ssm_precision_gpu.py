"""bf16 scans give what the formulas give, rounded once: no term loses more than 2^-16 on its way.  On an MI355X.

The bound of a result is half a step of bf16 at that very value (not the most
that a value's binade allows), beside the roundings of fp32 sums and 2^-16 for
each operand that goes into a product in two bf16 parts.  The inputs have both
signs, so the terms cancel and what they lose shows.
"""
from __future__ import annotations

import pytest
import torch

import bwd_mamba2_scan_amd as m2
from oracle import selective_oracle as orc
from tests.selective import TINY, U, scan_inputs, scan_roundings, to

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TWO = 2.0 ** -16    # what an operand in two parts leaves out

# (batch, L, H, P, G, N)
CASES = [(2, 200, 7, 64, 1, 128), (1, 130, 4, 24, 2, 40), (1, 720, 2, 128, 1, 64), (2, 100, 3, 16, 1, 16)]


def _half_step(v):
    """Half the distance of bf16 numbers at |v|."""
    return torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -126))) - 8)


def _within(got, want, size, n, parts, what):
    off = (n + 1.02 * parts * TWO) * size + TINY
    over = (got.cpu().double() - want).abs() - off - _half_step(want.abs() + off)
    assert float(over.max()) <= 0, (what, float(over.max()), int((over > 0).sum()), over.numel())


def _run(case):
    batch, L, H, P, G, N = case
    p = scan_inputs(sum(case), (batch, L), batch, H, P, G, N, "bf16", "f32")
    d = to(p, DEV)
    args = tuple(d[k] for k in ("x", "dt", "A", "B", "C"))
    kw = dict(D=d["D"], dt_bias=d["dt_bias"], initial_state=d["state"])
    n = scan_roundings(L, P, N) * U
    for row in range(batch):
        cpu = tuple(p[k][row] if k in ("x", "dt", "B", "C") else p[k] for k in ("x", "dt", "A", "B", "C", "D", "dt_bias"))
        yield d, args, kw, n, row, cpu + (True, p["state"][row]), (p["d_y"][row], p["d_final"][row])


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward(case):
    print("precision of y", case, flush=True)
    for d, args, kw, n, row, cpu, _ in _run(case):
        y, _ = m2.ssm_fwd(*args, **kw)
        # the scores, or the state, in two parts
        _within(y[row], orc.scan(*cpu)[0], orc.scan(*cpu, absolute=True)[0], n, 1, "y")


def _backward(case, name, parts):
    print(f"precision of {name}", case, flush=True)
    for d, args, kw, n, row, cpu, ups in _run(case):
        g = m2.ssm_bwd(*args, d["d_y"], d_final_state=d["d_final"], **kw)
        _within(g[name][row], orc.scan_grads(*cpu, *ups)[name], orc.scan_grads(*cpu, *ups, absolute=True)[name], n, parts,
                name)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_d_x(case):
    _backward(case, "d_x", 1)       # P


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_d_B_and_d_C(case):
    _backward(case, "d_B", 1)       # Q, or the gradient's state
    _backward(case, "d_C", 1)       # Q


@pytest.mark.parametrize("typ,tiny", [("f32", 2.0 ** -27), ("bf16", 1.875 * 2.0 ** -30)])
def test_small_terms_are_not_lost_in_a_large_state(typ, tiny):
    """A state of 1 that keeps, and terms that are below its half step alone but not 64 of them together: one rounding a
    step (2^-24) is all that the state may be off by, in the scan and in its gradient's reverse recurrence."""
    L, steps, H, P, N = 640, 10, 800, 16, 24        # more heads than work-groups at a time: not cut into segments
    t = torch.float32 if typ == "f32" else torch.bfloat16
    print("small terms", typ, flush=True)
    full = lambda v, *s, dtype=t: torch.full(s, v, dtype=dtype, device=DEV)
    x, one, dt = full(tiny, 1, L, H, P), full(1.0, 1, L, 1, N), full(1.0, 1, L, H)
    A, state = full(0.0, H, dtype=torch.float32), full(1.0, 1, H, N, P, dtype=torch.float32)
    _, final = m2.ssm_fwd(x, dt, A, one, one, softplus=False, initial_state=state, want_final_state=True)
    g = m2.ssm_bwd(x, dt, A, one, one, x, softplus=False, initial_state=state, d_final_state=state)
    want = 1.0 + L * tiny
    for name, got in (("final", final), ("d_initial_state", g["d_initial_state"])):
        assert float((got.double() - want).abs().max()) <= 1.01 * steps * U, name
