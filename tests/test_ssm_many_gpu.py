"""More packed sequences than a grid's last dimension has directions for: bitwise as in two calls.  On an MI355X."""
from __future__ import annotations

import pytest
import torch

import bwd_mamba2_scan_amd as m2
from tests.selective import scan_inputs, to

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_backward_of_many_sequences():
    batch, long, at, half = 65535, 1500, 50000, 30000        # one long sequence, carried over 12 segments
    H, P, G, N = 1, 8, 1, 8
    lengths = torch.ones(batch, dtype=torch.int64)
    lengths[at] = long
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), lengths.cumsum(0)])
    p = to(scan_inputs(21, (int(offsets[-1]),), batch, H, P, G, N, "f32", "f32"), DEV)
    print("backward of", batch, "sequences", flush=True)

    def run(first, last):
        lo, hi = int(offsets[first]), int(offsets[last])
        rows = {k: p[k][lo:hi] for k in ("x", "dt", "B", "C", "d_y")}
        off = (offsets[first:last + 1] - lo).int().to(DEV)
        args = (rows["x"], rows["dt"], p["A"], rows["B"], rows["C"])
        kw = dict(D=p["D"], dt_bias=p["dt_bias"], initial_state=p["state"][first:last], offsets=off)
        y, final = m2.ssm_fwd(*args, want_final_state=True, **kw)
        g = m2.ssm_bwd(*args, rows["d_y"], d_final_state=p["d_final"][first:last], **kw)
        return dict(y=y, final=final, **{k: g[k] for k in ("d_x", "d_dt", "d_B", "d_C", "d_initial_state")})

    whole, parts = run(0, batch), [run(0, half), run(half, batch)]
    for k, v in whole.items():
        assert torch.equal(v, torch.cat([q[k] for q in parts])), k
