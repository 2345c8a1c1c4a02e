"""Arguments that the selective layer's binding refuses on a GPU (an MI355X)."""
from __future__ import annotations

import pytest
import torch

import bwd_mamba2_scan_amd as m2
from tests.selective import gen, scan_inputs, to

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _conv(batch=2, L=9, C=16, W=4):
    g = gen(1)
    r = lambda *s: torch.randn(*s, generator=g).to(DEV)
    return r(batch, L, C), r(C, W), r(batch, L, C), r(C), r(batch, W - 1, C)


def test_gradients_that_there_are_not():
    x, w, d_y, bias, tail = _conv()
    for name, t, what in (("d_weights", w, "gradients are"), ("y", x, "gradients are"), ("d_bias", bias, "no bias"),
                          ("d_initial_state", tail, "no initial_state")):
        with pytest.raises(ValueError, match=what):
            m2.conv_bwd(x, w, d_y, out={name: torch.empty_like(t)})
    g = m2.conv_bwd(x, w, d_y, bias, out=dict(d_bias=torch.empty_like(bias), d_initial_state=None))
    assert g["d_initial_state"] is None
    p = to(scan_inputs(1, (1, 20), 1, 4, 16, 2, 16, "f32", "f32"), DEV)
    args = [p[k] for k in ("x", "dt", "A", "B", "C", "d_y")]
    for name, t, what in (("dx", "x", "gradients are"), ("d_D", "D", "no D"), ("d_dt_bias", "D", "no dt_bias"),
                          ("d_initial_state", "state", "no initial_state")):
        with pytest.raises(ValueError, match=what):
            m2.ssm_bwd(*args, out={name: torch.empty_like(p[t])})
    g = m2.ssm_bwd(*args, D=p["D"], out=dict(d_D=torch.empty_like(p["D"])))
    assert g["d_dt_bias"] is None and g["d_D"] is not None


def test_outputs_over_the_offsets():
    x, w, d_y, _, _ = _conv(1)
    p = to(scan_inputs(2, (9,), 1, 1, 8, 1, 8, "f32", "f32"), DEV)
    args = [p[k] for k in ("x", "dt", "A", "B", "C")]
    both = torch.zeros(1 << 16, device=DEV)
    offsets = both.view(torch.int32)[:2]
    offsets.copy_(torch.tensor([0, 9]))
    over = lambda *s: both[:torch.Size(s).numel()].view(s)
    for call in (lambda: m2.conv_fwd(x[0], w, offsets=offsets, y=over(9, 16)),
                 lambda: m2.conv_fwd(x[0], w, offsets=offsets, final_state=over(1, 3, 16)),
                 lambda: m2.conv_bwd(x[0], w, d_y[0], offsets=offsets, workspace=both),
                 lambda: m2.conv_bwd(x[0], w, d_y[0], offsets=offsets, out=dict(d_weight=over(16, 4))),
                 lambda: m2.ssm_fwd(*args, offsets=offsets, y=over(9, 1, 8)),
                 lambda: m2.ssm_bwd(*args, p["d_y"], offsets=offsets, out=dict(d_B=over(9, 1, 8))),
                 lambda: m2.ssm_bwd(*args, p["d_y"], offsets=offsets, workspace=both)):
        with pytest.raises(ValueError, match="overlaps offsets"):
            call()
    assert offsets.tolist() == [0, 9] and not bool(both[2:].any())
