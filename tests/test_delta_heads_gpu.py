"""The gated delta rule's heads that share a query and key, in calls of so many steps that a work-group takes several of
them one after the other, against float64.  On an MI355X.
"""
from __future__ import annotations

import pytest
import torch

from tests import delta_rule as dr
from tests.test_delta_gpu import DEV, _check, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,H,G,V,K", [
    (12, 200, 20, 2, 24, 16),    # 960 steps of heads: three heads to a work-group of the gradients, and one left over
    (40, 200, 20, 2, 16, 40),    # 3200: their matrices by three (of four work-groups a CU), all ten in the gradients
    (40, 200, 20, 2, 16, 72),    # fp32: by six (of two)
    (24, 130, 15, 3, 72, 24), (9, 100, 64, 1, 8, 8),
])
def test_several_heads_to_a_work_group(B, L, H, G, V, K, typ):
    p = dr.inputs(B + K, (B, L), B, H, V, G, K, typ, "f32")
    got = _run(dr.to(p, DEV))
    for i in (0, B // 2, B - 1):
        _check(p, K ** -0.5, got, i, (B, L, H))
    # a call of one sequence has a head to a work-group: sums of heads in another order, else bitwise the same
    one = _run(dr.to({k: v if v is None else v[1:2] for k, v in p.items()}, DEV))
    for n in ("y", "final", "d_v", "d_g", "d_beta", "d_state"):
        assert torch.equal(got[n][1], one[n][0]), n


@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_packed(typ):
    lengths = [130, 1, 64, 0, 77] * 8
    H, G, V, K = 20, 2, 24, 16
    ends = [0]
    for n in lengths:
        ends.append(ends[-1] + n)
    p = dr.inputs(7, (ends[-1],), len(lengths), H, V, G, K, typ, "f32")
    got = _run(dr.to(p, DEV), offsets=torch.tensor(ends, dtype=torch.int32, device=DEV))
    for i in (0, 1, 3, 17, 39):
        _check(p, K ** -0.5, got, i, lengths[i], span=(ends[i], ends[i + 1]))


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("K", [40, 72])
def test_values_that_are_not_finite(K, typ):
    """A head's reach no other head that its work-group takes."""
    B, L, H, G, V = 40, 200, 20, 2, 16
    d = dr.to(dr.inputs(K, (B, L), B, H, V, G, K, typ, "f32"), DEV)
    want = _run(d)
    for name, at in (("v", (1, 70, 3, 5)), ("beta", (1, 70, 3)), ("g", (1, 70, 3)), ("state", (1, 3, 2, 2)), ("d_y", (1, 70, 3, 5))):
        bad = dict(d)
        bad[name] = d[name].clone()
        bad[name][at] = float("nan")
        got = _run(bad)
        for n in ("y", "final", "d_v", "d_g", "d_beta", "d_state"):
            x, y = got[n], want[n]
            axis = 1 if n in ("final", "d_state") else 2
            others = [h for h in range(H) if h != 3]
            keep = torch.tensor(others, device=DEV)
            assert torch.equal(x.index_select(axis, keep), y.index_select(axis, keep)), (name, n)
            assert torch.equal(x[0], y[0]) and torch.equal(x[2:], y[2:]), (name, n)
        for n in ("d_q", "d_k"):
            assert torch.equal(got[n][:, :, 1], want[n][:, :, 1]) and torch.equal(got[n][0], want[n][0]), (name, n)
