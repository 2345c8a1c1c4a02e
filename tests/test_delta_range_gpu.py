"""The gated delta rule at the ends of what it is meant for: beta |k|^2 up to 2, keys that repeat, no decay.  On an
MI355X.
"""
from __future__ import annotations

import pytest
import torch

from tests import delta_rule as dr
from tests.test_delta_gpu import DEV, _check, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("L", [130, 900])
@pytest.mark.parametrize("keys", ["one", "four", "long", "short"])
def test_strong_corrections(keys, L, typ):
    """A token's transition is up to a reflection along its key, which is the same one again and again."""
    B, H, V, G, K = 2, 2, 24, 1, 16
    p = dr.inputs(31 + L, (B, L), B, H, V, G, K, typ, "f32")
    t = p["k"].dtype
    if keys in ("one", "four"):
        n = 1 if keys == "one" else 4
        p["k"] = p["k"][:, :n].repeat(1, -(-L // n), 1, 1)[:, :L].contiguous()
    else:
        p["k"] = (p["k"].float() * (30.0 if keys == "long" else 1 / 30)).to(t)
    p["g"].zero_()
    length = p["k"].float().square().sum(-1)  # [B, L, 1]: beta |k|^2 in 0 .. 2, and 2 in every third token
    share = torch.rand(B, L, H, generator=torch.Generator().manual_seed(5))
    share[:, ::3] = 1.0
    p["beta"] = share * (2 - 2.0 ** -10) / length
    got = _run(dr.to(p, DEV))
    for i in range(B):
        _check(p, K ** -0.5, got, i, (keys, L))
