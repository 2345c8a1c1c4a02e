"""The global gradient norm and clipping against float64, on an MI355X."""
from __future__ import annotations

import math

import pytest
import torch

import bwd_mamba2_scan_amd as m2
from oracle import selective_oracle as orc
from tests.selective import U, gen, half_step

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _grads(seed, sizes, scale=1.0):
    g = gen(seed)
    return [(torch.randn(n, generator=g) * scale).to(torch.bfloat16 if i % 3 == 2 else torch.float32)
            for i, n in enumerate(sizes)]


SIZES = [[1], [0, 5, 0], [4096] * 3, [1, 2, 3, 4, 5, 7, 8, 9, 15, 17, 8191, 8192, 8193, 100003], [3] * 250, [0, 0],
         [3_000_000, 11], [5] * 16, [6] * 17, [100] * 97]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("max_norm", [0.5, 1e9, 0.0, math.inf])
def test_against_float64(sizes, max_norm):
    print("clip", len(sizes), max(sizes), max_norm, flush=True)
    grads = _grads(len(sizes), sizes)
    norm, want = orc.clip(grads, max_norm)
    d = [g.to(DEV) for g in grads]
    out = [torch.full_like(g, 7.0) for g in d]
    alone = m2.grad_norm(d)
    n = m2.clip_grads(d, max_norm, out=out)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(d, grads))
    m = m2.clip_grads(d, max_norm)
    assert n.shape == () and torch.equal(n, m) and torch.equal(n, alone)
    # squares of fp32 values are exact in 64 bits: one rounding of the root to fp32
    assert abs(float(n) - norm) <= 1.01 * U * norm
    for g, o, w in zip(d, out, want):
        assert torch.equal(g, o)
        # the factor's rounding, the product's and the result's
        assert bool(((g.cpu().double() - w).abs() <= (2.01 * U + half_step(g.dtype)) * w.abs()).all())


def test_unaligned_tensors():
    base = torch.randn(10_000, generator=gen(1)).to(DEV)
    half = base.bfloat16()
    grads = [base[1:5000], base[5003:5003], base[6001:9998], half[3:4097], half[4099:9999]]
    norm, want = orc.clip([g.cpu() for g in grads], 1.0)
    outs = [torch.empty(g.numel() + 8, dtype=g.dtype, device=DEV)[k: k + g.numel()] for k, g in enumerate(grads)]
    kept = base[0].item(), base[5000:6001].clone(), base[9998:].clone()
    n = m2.clip_grads(grads, 1.0, out=outs)
    m2.clip_grads(grads, 1.0)
    assert abs(float(n) - norm) <= 1.01 * U * norm
    for g, o, w in zip(grads, outs, want):
        assert torch.equal(g, o)
        assert bool(((g.cpu().double() - w).abs() <= (2.01 * U + half_step(g.dtype)) * w.abs()).all())
    assert base[0].item() == kept[0] and torch.equal(base[5000:6001], kept[1]) and torch.equal(base[9998:], kept[2])


def test_squares_beyond_fp32():
    d = [torch.full((1000,), 1e30, device=DEV), torch.full((7,), -3e-30, device=DEV)]
    n = m2.clip_grads(d, 2.0)
    want = 1e30 * math.sqrt(1000)
    assert abs(float(n) - want) <= 1e-6 * want
    assert torch.allclose(d[0].double(), torch.full((1000,), 2 / math.sqrt(1000), dtype=torch.float64, device=DEV), rtol=1e-6)
    big = [torch.full((4,), 3e38, device=DEV)]
    assert math.isinf(float(m2.clip_grads(big, 1.0)))     # the norm itself passes fp32's range, the factor does not
    assert torch.allclose(big[0], torch.full((4,), 0.5, device=DEV), rtol=1e-6)


def test_infinities_and_nan():
    d = [torch.ones(5, device=DEV), torch.tensor([1.0, math.inf], device=DEV)]
    assert math.isinf(float(m2.clip_grads(d, 1.0)))
    assert bool((d[0] == 0).all()) and float(d[1][0]) == 0 and math.isnan(float(d[1][1]))
    d = [torch.ones(5, device=DEV), torch.tensor([1.0, math.nan], device=DEV).bfloat16()]
    assert math.isnan(float(m2.clip_grads(d, 1.0)))
    assert bool(torch.isnan(d[0]).all()) and bool(torch.isnan(d[1]).all())
    d = [torch.tensor([3.0, math.inf], device=DEV)]
    m2.clip_grads(d, math.inf)
    assert float(d[0][0]) == 3.0 and math.isinf(float(d[0][1]))
    d = [torch.tensor([3.0, math.nan], device=DEV)]
    assert math.isnan(float(m2.clip_grads(d, math.inf))) and bool(torch.isnan(d[0]).all())


def test_refusals_of_the_binding():
    a = torch.ones(100, device=DEV)
    for bad in ([a, a], [a[:60], a[50:]]):
        with pytest.raises(m2.Mamba2ScanError) as e:
            m2.clip_grads(bad, 1.0)
        assert e.value.status == -8
    with pytest.raises(m2.Mamba2ScanError):
        m2.clip_grads([a[:50]], 1.0, out=[a[10:60]])
    m2.grad_norm([a, a])    # reading the same tensor twice is no conflict
    with pytest.raises(ValueError, match="contiguous"):
        m2.clip_grads([torch.ones(4, 4, device=DEV).t()[:, :2]], 1.0)
    with pytest.raises(ValueError, match="type and shape"):
        m2.clip_grads([a], 1.0, out=[torch.empty(99, device=DEV)])
    with pytest.raises(ValueError, match="outputs"):
        m2.clip_grads([a], 1.0, out=[])
    with pytest.raises(TypeError):
        m2.clip_grads([a.double()], 1.0)
    with pytest.raises(ValueError, match="one float32"):
        m2.clip_grads([a], 1.0, norm=torch.empty(2, device=DEV))
    with pytest.raises(m2.Mamba2ScanError) as e:
        m2.clip_grads([a], 1.0, workspace=torch.empty(1, device=DEV))
    assert e.value.status == m2.ESIZE
