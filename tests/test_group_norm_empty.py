"""Group norms of no rows: what is refused with rows only because nothing is asked for is no refusal without them."""
from __future__ import annotations

import pytest
import torch

import bwd_mamba2_scan_amd as m2
from bwd_mamba2_scan_amd.delta import GATE_FIRST, GATED, PLAIN, SILU, NormDims
from bwd_mamba2_scan_amd.layer import Rows, Seqs

NONE = Rows(None, 0, 0)


@pytest.mark.parametrize("form", [PLAIN, SILU, GATED, GATE_FIRST])
@pytest.mark.parametrize("batch", [1, 3])
def test_backward_of_no_rows(form, batch):
    """An empty tensor has no address.  No kernel is launched: this needs no GPU."""
    L = m2.lib()
    call = lambda length: L.mamba2_norm_bwd(Seqs(batch, length, None), NormDims(1, 2, 8, form, 0, 0, 1e-5), NONE, None, None,
                                            NONE, NONE, NONE, None, None, NONE, None, 0, None)
    assert call(0) == 0
    assert call(1) == m2.ENULL


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["plain", "silu", "gated", "gate_first"])
@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("shape", [(0, 16), (2, 0, 16), "packed"])
def test_no_rows(shape, weight, bias, form):
    dev = "cuda:0"
    kw = dict(groups=2, silu=form == "silu", gate_first=form == "gate_first")
    if shape == "packed":
        shape, kw["offsets"] = (0, 16), torch.zeros(4, dtype=torch.int32, device=dev)
    x = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    w = torch.ones(16, device=dev) if weight else None
    b = torch.ones(16, device=dev) if bias else None
    if form in ("gated", "gate_first"):
        kw["gate"] = torch.empty_like(x)
    assert m2.group_norm_fwd(x, w, b, **kw).shape == x.shape
    g = m2.group_norm_bwd(x, torch.empty_like(x), w, b, **kw)
    assert g["d_x"].shape == x.shape and (g["d_gate"] is not None) == ("gate" in kw)
    for name, t in (("d_weight", w), ("d_bias", b)):
        assert g[name] is None if t is None else float(g[name].abs().max()) == 0, name
