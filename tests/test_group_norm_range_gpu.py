"""The group norm's activation over its whole range of arguments, against float64, within running error bounds.  On an
MI355X.
"""
from __future__ import annotations

import pytest
import torch

import bwd_mamba2_scan_amd as m2
from oracle import delta_oracle as orc
from tests import group_norm as gn
from tests import test_group_norm_gpu as base
from tests.rounded import within

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FAR = [-3e38, -1e30, -1e4, 1e4]  # where the sigmoid is 0 or 1


def _every(typ):
    """Every bf16 value within -110 .. 110, or an fp32 one every 1/128 there: past -87.3 e^-v passes fp32's largest."""
    if typ == "bf16":
        v = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
        v = v[v.abs() <= 110].sort().values
    else:
        v = torch.arange(-110 * 128, 110 * 128 + 1).float() / 128 + 2.0 ** -13
    return torch.cat([v, torch.tensor(FAR)])


def _rows_of(v, channels, mixed):
    """The values side by side in rows; mixed: a group has large and small ones."""
    v = torch.cat([v, torch.ones(-len(v) % channels)])
    if mixed:
        v = v[torch.randperm(len(v), generator=torch.Generator().manual_seed(3))]
    return v.reshape(-1, channels)


def _check(p, groups, form, what):
    kw = gn.keywords(groups, form, True)
    d = {k: None if v is None else v.to(DEV) for k, v in p.items()}
    got = dict(m2.group_norm_bwd(d["x"], d["d_y"], d["weight"], d["bias"], gate=d["gate"], **kw),
               y=m2.group_norm_fwd(d["x"], d["weight"], d["bias"], gate=d["gate"], **kw))
    b = gn.bounds(p, groups, form, True, kw["eps"], True)
    args = (p["x"], p["weight"], p["bias"], p["gate"], groups, form, True, kw["eps"])
    want = dict(y=orc.group_norm(*args), **orc.group_norm_grads(*args, p["d_y"]))
    for name, v in want.items():
        if v is not None:
            within(got[name], v, b[name][1], (what, name))


@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("form", ["gated", "gate_first"])
@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("groups,width", [(4, 64), (1, 2048), (2, 97)])
def test_gates(typ, form, groups, width, mixed):
    z = _rows_of(_every(typ), groups * width, mixed)
    p = gn.inputs(11, (z.shape[0],), groups, width, typ, form, "channel", True)
    p["gate"] = z.to(p["x"].dtype)
    _check(p, groups, form, (typ, form, groups, width, mixed))


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("groups,width", [(221, 128), (14, 2048), (29, 971)])
def test_arguments_of_silu(typ, groups, width):
    """SiLU's argument follows the bias, which has every value of the range."""
    v = _every("f32")[:-len(FAR)]
    p = gn.inputs(12, (3,), groups, width, typ, "silu", "channel", True)
    p["weight"] = 0.01 * p["weight"]
    p["bias"] = torch.cat([v, torch.zeros(max(0, groups * width - len(v)))])[:groups * width].contiguous()
    _check(p, groups, "silu", (typ, groups, width))


@pytest.mark.parametrize("form", ["plain", "gated", "gate_first"])
@pytest.mark.parametrize("groups,width,typ", [(8, 97, "bf16"), (5, 3, "bf16"), (64, 1, "bf16"), (7, 120, "f32"), (1, 127, "bf16")])
def test_many_rows_by_elements(groups, width, typ, form):
    """Groups of a wave that fill no vector, a thread's rows one after another."""
    base.test_many_rows(groups, width, typ, form)
