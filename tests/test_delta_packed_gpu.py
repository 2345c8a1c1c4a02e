"""The gated delta rule over packed sequences whose heads divide among the XCDs, the longest first, against float64.  On
an MI355X.
"""
from __future__ import annotations

import pytest
import torch

import bwd_mamba2_scan_amd as m2
from bwd_mamba2_scan_amd.delta import DeltaDims
from bwd_mamba2_scan_amd.layer import Seqs
from tests import delta_rule as dr
from tests.test_delta_gpu import DEV, _check, _run

pytestmark = pytest.mark.gpu
UNEQUAL = [70, 0, 1, 64, 129, 0, 31, 200, 64, 0]
MANY = [(37 * i) % 23 for i in range(64)]   # as many sequences as the ranking takes


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,H,V,G,K", [
    (UNEQUAL, 8, 40, 2, 24), (UNEQUAL, 4, 128, 4, 128), (UNEQUAL, 16, 24, 1, 72), (UNEQUAL, 8, 72, 8, 40),
    (MANY, 8, 16, 8, 16), (MANY[:63] + [190], 4, 72, 1, 32), ([0, 0, 0], 8, 16, 8, 16),
])
def test_heads_among_the_xcds(lengths, H, V, G, K, typ):
    """64-column slices of all heads are a multiple of eight, sequences at most 64 and too short to be cut."""
    slices = (V + 63) // 64
    rows, n = sum(lengths), len(lengths)
    assert H * slices % 8 == 0 and n <= 64
    d = DeltaDims(1 if typ == "bf16" else 0, 0, H, V, G, K, 1.0)
    off = torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    size = lambda length: m2.lib().mamba2_delta_fwd_workspace_bytes(Seqs(n, length, off.data_ptr()), d) / (length // 64 + n)
    assert size(rows) == size(0), "cut into segments: these have room in the workspace"
    p = dr.inputs(rows + H, (rows,), n, H, V, G, K, typ, "f32")
    got = _run(dr.to(p, DEV), offsets=off)
    ends = off.tolist()
    # all of a few sequences, of many the first and last, the longest, an empty one
    which = range(n) if n <= 10 else sorted({0, 1, n - 1, lengths.index(max(lengths)), lengths.index(0, 1)})
    for i in which:
        _check(p, K ** -0.5, got, i, lengths[i], span=(ends[i], ends[i + 1]))
        if lengths[i] == 0:
            assert torch.equal(got["final"][i].cpu(), p["state"][i]) and torch.equal(got["d_state"][i].cpu(), p["d_final"][i])
