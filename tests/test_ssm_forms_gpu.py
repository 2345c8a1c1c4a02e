"""The selective scan's kernels with several heads in a backward work-group, and with the states carried across many
segments, against the float64 oracle (evaluated on the GPU, in plain tensor operations).  On an MI355X.
"""
from __future__ import annotations

import pytest
import torch

import bwd_mamba2_scan_amd as m2
from oracle import selective_oracle as orc
from tests.selective import scan_inputs, to
from tests.ssm_forms import HEADS, SEGMENTS
from tests.test_ssm_gpu import check_forward, check_grads

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CHUNK = 64      # sequences of one length that the oracle takes together


def _together(p, rows, spans, absolute):
    """[(y, [final state], gradients)] of sequences of one length: their heads side by side are one sequence's."""
    n, H = len(rows), p["A"].shape[0]
    side = lambda k: torch.stack([p[k][s] for s in spans], 1).flatten(1, 2)         # [L, n * heads or groups, ...]
    per_head = lambda k: p[k].repeat(n)
    state, d_final = (p[k][rows].flatten(0, 1) for k in ("state", "d_final"))
    args = (side("x"), side("dt"), per_head("A"), side("B"), side("C"), per_head("D"), per_head("dt_bias"), True, state)
    y, states = orc.scan(*args, absolute=absolute)
    g = orc.scan_grads(*args, side("d_y"), d_final, absolute=absolute)
    split = lambda v, dim: v.unflatten(dim, (n, v.shape[dim] // n)).movedim(dim, 0).cpu()
    y, final = split(y, 1), split(states[-1], 0)
    g = {k: split(v, 0 if k in ("d_A", "d_D", "d_dt_bias", "d_state") else 1) for k, v in g.items()}
    return [(y[i], [final[i]], {k: v[i] for k, v in g.items()}) for i in range(n)]


def _oracle(p, spans, absolute):
    res = [None] * len(spans)
    by_length = {}
    for row, s in enumerate(spans):
        by_length.setdefault(len(range(p["x"].shape[0])[s]) if isinstance(s, slice) else p["x"].shape[1], []).append(row)
    for rows in by_length.values():
        for i in range(0, len(rows), CHUNK):
            part = rows[i: i + CHUNK]
            for row, r in zip(part, _together(p, part, [spans[k] for k in part], absolute)):
                res[row] = r
    return res


@pytest.mark.parametrize("case", HEADS + SEGMENTS, ids=lambda c: "-".join(
    str(v) if not isinstance(v, list) else f"{len(v) - 1}of{v[-1]}" for v in c).replace(" ", ""))
def test_against_the_oracle(case):
    lead, H, P, G, N, typ, dt_typ = case
    print("scan", str(case)[:100], flush=True)
    packed = isinstance(lead, list)
    batch = len(lead) - 1 if packed else lead[0]
    rows = (lead[-1],) if packed else lead
    p = scan_inputs(H + N, rows, batch, H, P, G, N, typ, dt_typ)
    d = to(p, DEV)
    off = torch.tensor(lead, dtype=torch.int32, device=DEV) if packed else None
    args = tuple(d[k] for k in ("x", "dt", "A", "B", "C"))
    kw = dict(D=d["D"], dt_bias=d["dt_bias"], initial_state=d["state"], offsets=off)
    y, final = m2.ssm_fwd(*args, want_final_state=True, **kw)
    g = m2.ssm_bwd(*args, d["d_y"], d_final_state=d["d_final"], **kw)
    torch.cuda.synchronize()
    spans = [slice(a, b) for a, b in zip(lead, lead[1:])] if packed else list(range(batch))
    exact, bound = (_oracle(d, spans, a) for a in (False, True))
    check_forward(p, y, final, spans, True, exact, bound)
    check_grads(p, g, spans, exact, bound)
