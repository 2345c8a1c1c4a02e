"""The convolution's weight and bias gradients over long runs of tokens, against the formulas in 64 bits, on an MI355X."""
from __future__ import annotations

import pytest
import torch

import bwd_mamba2_scan_amd as m2
from tests.selective import TYPES, U
from tests.test_conv_gpu import _slack

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
WAVES = 4       # runs of a work-group


def _run(batch, L, channels):
    """Tokens of a wave: about 16 waves on each of 256 CUs, from 8 to 64, in fours."""
    r = -(-(batch * L * -(-channels // 512) // 4096) // 4) * 4
    return min(64, max(8, r))


# (type, batch, L, channels, taps, silu, bias, tokens of a run)
CASES = [("bf16", 4, 4096, 4352, 4, True, True, 36), ("bf16", 8, 4096, 4096, 2, True, True, 64),
         ("f32", 2, 8191, 2056, 4, True, True, 20), ("bf16", 2, 8191, 2055, 3, True, True, 20),
         ("f32", 3, 5000, 1030, 2, False, False, 12)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_sums_over_long_runs(case):
    typ, batch, L, channels, taps, silu, with_bias, run = case
    assert _run(batch, L, channels) == run
    print("convolution's sums", case, flush=True)
    g = torch.Generator(DEV).manual_seed(17)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    x, d_y = r(batch, L, channels).to(TYPES[typ]), r(batch, L, channels).to(TYPES[typ])
    weight, bias = r(channels, taps), r(channels) if with_bias else None
    got = m2.conv_bwd(x, weight, d_y, bias, silu=silu)
    w = weight.double()
    d_weight, d_bias = torch.zeros_like(w), torch.zeros(channels, dtype=torch.float64, device=DEV)
    weight_room, bias_room = torch.zeros_like(d_weight), torch.zeros_like(d_bias)
    # one after another at most: a run's tokens, the work-group's four waves, a quarter of the units and their join
    n = (run + WAVES + -(-L // (run * WAVES)) * batch / 4 + 4) * U
    for row in range(batch):
        xs = torch.nn.functional.pad(x[row].double(), (0, 0, taps - 1, 0))
        terms = [w[:, k] * xs[k:k + L] for k in range(taps)] + ([bias.double()] if with_bias else [])
        dp, off = d_y[row].double(), torch.zeros(L, channels, dtype=torch.float64, device=DEV)
        if silu:
            pre = sum(terms)
            sig = torch.sigmoid(pre)
            # the slope is off by at most the pre-activation's slack (its own slope is below 1) and a dozen roundings
            off = dp.abs() * (_slack(TYPES[typ], sum(t.abs() for t in terms)) + 16 * U)
            dp = dp * sig * (1 + pre * (1 - sig))
        d_bias += dp.sum(0)
        bias_room += (n * dp.abs() + off).sum(0)
        for k in range(taps):
            d_weight[:, k] += (dp * xs[k:k + L]).sum(0)
            weight_room[:, k] += ((n * dp.abs() + off) * xs[k:k + L].abs()).sum(0)
    assert bool(((got["d_weight"].double() - d_weight).abs() <= weight_room).all())
    if with_bias:
        assert bool(((got["d_bias"].double() - d_bias).abs() <= bias_room).all())
