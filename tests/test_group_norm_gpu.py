"""The group norm's kernels against float64, within running error bounds.  On an MI355X."""
from __future__ import annotations

import math

import pytest
import torch

import bwd_mamba2_scan_amd as m2
from oracle import delta_oracle as orc
from tests import group_norm as gn
from tests.rounded import within

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _to(p):
    return {k: None if v is None else v.to(DEV) for k, v in p.items()}


def _flat(p):
    return {k: v.reshape(-1, v.shape[-1]) if k in ("x", "gate", "d_y") and v is not None else v for k, v in p.items()}


def _check(p, got, groups, form, centered, eps, what):
    f = _flat(p)
    b = gn.bounds(f, groups, form, centered, eps, True)
    args = (f["x"], f["weight"], f["bias"], f["gate"], groups, form, centered, eps)
    want = dict(y=orc.group_norm(*args), **orc.group_norm_grads(*args, f["d_y"]))
    for name, v in want.items():
        if v is None:
            assert got[name] is None, name
            continue
        assert torch.allclose(b[name][0], v, rtol=1e-9, atol=1e-9), name
        within(got[name].reshape(v.shape), v, b[name][1], (what, name))


def _run(d, **kw):
    y = m2.group_norm_fwd(d["x"], d["weight"], d["bias"], gate=d["gate"], **kw)
    return dict(m2.group_norm_bwd(d["x"], d["d_y"], d["weight"], d["bias"], gate=d["gate"], **kw), y=y)


@pytest.mark.parametrize("form", gn.FORMS)
@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("lead,groups,width,centered,weight,bias", [
    ((1, 1), 1, 8, True, "channel", True), ((2, 3), 3, 24, False, "group", True), ((37,), 10, 16, True, "group", False),
    ((2, 33), 5, 97, True, "channel", True), ((5,), 7, 3, False, "channel", False), ((300,), 32, 128, False, "group", False),
    ((9,), 2, 512, True, None, False), ((3, 7), 1, 1000, True, "channel", True), ((4,), 3, 1025, False, "group", True),
    ((11,), 1, 2048, True, "channel", True), ((3,), 2, 5000, False, "channel", True), ((2,), 1, 16384, True, "channel", True),
    ((2,), 1, 16383, True, "group", True), ((2,), 1, 8200, True, "channel", False), ((6,), 300, 1, False, "channel", True),
])
def test_against_float64(form, typ, lead, groups, width, centered, weight, bias):
    p = gn.inputs(width + groups, lead, groups, width, typ, form, weight, bias)
    kw = gn.keywords(groups, form, centered)
    _check(p, _run(_to(p), **kw), groups, form, centered, kw["eps"], (lead, groups, width))


def test_slices_and_given_outputs():
    """Inputs and outputs are slices of wider tensors; between sequences there are rows of others."""
    p = gn.inputs(3, (3, 20), 4, 24, "bf16", "gated", "group", True)
    d = _to(p)
    kw = gn.keywords(4, "gated", False)
    wide = torch.full((3, 25, 3 * 96 + 8), math.nan, dtype=torch.bfloat16, device=DEV)
    put = lambda t, i: wide[:, 2:22, 8 + 96 * i: 104 + 96 * i].copy_(t)
    s = dict(d, x=put(d["x"], 0), gate=put(d["gate"], 1), d_y=put(d["d_y"], 2))
    outs = torch.full((3, 20, 4 * 96), 7.0, dtype=torch.bfloat16, device=DEV)
    y = m2.group_norm_fwd(s["x"], s["weight"], s["bias"], gate=s["gate"], y=outs[..., :96], **kw)
    assert y.data_ptr() == outs.data_ptr()
    g = m2.group_norm_bwd(s["x"], s["d_y"], s["weight"], s["bias"], gate=s["gate"],
                          out=dict(d_x=outs[..., 96:192], d_gate=outs[..., 288:]), **kw)
    _check(p, dict(g, y=y), 4, "gated", False, kw["eps"], "slices")
    assert bool((outs[..., 192:288] == 7).all())
    want = _run(d, **kw)
    for n in ("y", "d_x", "d_gate", "d_weight", "d_bias"):  # unaligned rows add in another order
        assert torch.allclose(dict(g, y=y)[n].float(), want[n].float(), rtol=2 ** -6, atol=1e-5)


def test_rows_outside_the_sequences():
    """Rows before the first sequence and behind the last: not read, not written, in no sum."""
    p = gn.inputs(4, (50,), 2, 40, "f32", "gate_first", "channel", True)
    d = _to(p)
    kw = gn.keywords(2, "gate_first", True)
    off = torch.tensor([5, 20, 20, 41], dtype=torch.int32, device=DEV)
    for t in (d["x"], d["gate"], d["d_y"]):
        t[:5] = math.nan
        t[41:] = math.nan
    y = torch.full_like(d["x"], 3.0)
    out = dict(d_x=torch.full_like(y, 3.0), d_gate=torch.full_like(y, 3.0))
    m2.group_norm_fwd(d["x"], d["weight"], d["bias"], gate=d["gate"], offsets=off, y=y, **kw)
    g = m2.group_norm_bwd(d["x"], d["d_y"], d["weight"], d["bias"], gate=d["gate"], offsets=off, out=out, **kw)
    for t in (y, g["d_x"], g["d_gate"]):
        assert bool((t[:5] == 3).all()) and bool((t[41:] == 3).all())
    mid = {k: v[5:41] if k in ("x", "gate", "d_y") else v for k, v in p.items()}
    got = {k: v[5:41] if k in ("y", "d_x", "d_gate") else v for k, v in dict(g, y=y).items()}
    _check(mid, got, 2, "gate_first", True, kw["eps"], "rows")


def test_no_rows():
    d = _to(gn.inputs(5, (0,), 2, 8, "bf16", "plain", "group", True))
    kw = gn.keywords(2, "plain", False)
    assert m2.group_norm_fwd(d["x"], d["weight"], d["bias"], **kw).shape == (0, 16)
    g = m2.group_norm_bwd(d["x"], d["d_y"], d["weight"], d["bias"], **kw)
    assert float(g["d_weight"].abs().max()) == 0 and float(g["d_bias"].abs().max()) == 0


@pytest.mark.parametrize("form", gn.FORMS)
def test_values_that_are_not_finite(form):
    """They stay in their token and group; the gate's infinities give the formula's values."""
    d = _to(gn.inputs(6, (6,), 3, 16, "f32", form, "group", False))
    kw = gn.keywords(3, form, False)
    clean = m2.group_norm_fwd(d["x"], d["weight"], gate=d["gate"], **kw)
    bad = d["x"].clone()
    bad[2, 17], bad[4, 40] = math.nan, math.inf
    got = m2.group_norm_fwd(bad, d["weight"], gate=d["gate"], **kw)
    same = torch.ones(6, 3, dtype=torch.bool, device=DEV)
    same[2, 1] = same[4, 2] = False
    eq = (got == clean).unflatten(1, (3, 16)).all(-1)
    assert bool((eq == same).all())
    assert not bool(torch.isfinite(got[2, 16:32]).all())
    if form == "gated":
        z = d["gate"].clone()
        z[0, 0], z[0, 1], z[0, 2] = 1e30, -1e30, 120.0
        got = m2.group_norm_fwd(d["x"], d["weight"], gate=z, **kw)
        plain = m2.group_norm_fwd(d["x"], d["weight"], groups=3)
        assert float(got[0, 0]) == float(plain[0, 0] * 1e30) and float(got[0, 1]) == 0
        assert abs(float(got[0, 2]) / float(plain[0, 2]) - 120) < 1e-4


def test_zeros_and_constants():
    """A group of zeros has the norm 0; a constant one, centered, too."""
    x = torch.zeros(2, 64, device=DEV)
    x[1] = 5.0
    assert float(m2.group_norm_fwd(x, groups=2)[0].abs().max()) == 0
    assert float(m2.group_norm_fwd(x, groups=2, centered=True).abs().max()) == 0
    g = m2.group_norm_bwd(x, torch.ones_like(x), groups=2, centered=True)
    assert float(g["d_x"].abs().max()) == 0 and g["d_weight"] is None and g["d_bias"] is None


def test_reproducible_and_refusals():
    d = _to(gn.inputs(7, (4, 700), 6, 40, "bf16", "silu", "channel", True))
    kw = gn.keywords(6, "silu", True)
    a, b = _run(d, **kw), _run(d, **kw)
    for n in a:
        assert (a[n] is None and b[n] is None) or torch.equal(a[n], b[n]), n
    x, w = d["x"], d["weight"]
    bad = ((dict(groups=7), "divide"), (dict(groups=0), "divide"), (dict(gate_first=True), "gate_first"),
           (dict(gate=x, silu=True), "silu"), (dict(y=x), "overlaps"), (dict(weight=w[:30]), "shape"),
           (dict(gate=x[:, :5]), "shape"))
    for k, match in bad:
        with pytest.raises(ValueError, match=match):
            m2.group_norm_fwd(x, **{**dict(weight=w, groups=6), **k})
    with pytest.raises(ValueError, match="needs a weight"):
        m2.group_norm_fwd(x, None, w, groups=6)
    with pytest.raises(ValueError, match="out holds"):
        m2.group_norm_bwd(x, x, w, groups=6, out=dict(d_gate=x.clone()))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        m2.group_norm_fwd(x.half(), groups=6)
    with pytest.raises(m2.Mamba2ScanError):
        m2.group_norm_fwd(x, groups=6, eps=0.0)


def test_rows_far_apart():
    """The last rows are more than 2^31 elements behind the first."""
    rows, stride = 300, (1 << 23) + 8
    p = gn.inputs(9, (rows,), 4, 16, "bf16", "gated", "group", True)
    d = _to(p)
    kw = gn.keywords(4, "gated", True)
    want = _run(d, **kw)
    big = torch.empty((rows - 1) * stride + 5 * 64, dtype=torch.bfloat16, device=DEV)
    at = lambda i: big.as_strided((rows, 64), (stride, 1), 64 * i)
    s = {n: at(i).copy_(d[n]) for i, n in enumerate(("x", "gate", "d_y"))}
    y = m2.group_norm_fwd(s["x"], d["weight"], d["bias"], gate=s["gate"], y=at(3), **kw)
    assert torch.equal(y, want["y"])
    g = m2.group_norm_bwd(s["x"], s["d_y"], d["weight"], d["bias"], gate=s["gate"], out=dict(d_x=at(4)), **kw)
    for n in ("d_x", "d_gate", "d_weight", "d_bias"):
        assert torch.equal(g[n], want[n]), n


@pytest.mark.parametrize("form", ["plain", "gated", "gate_first"])
@pytest.mark.parametrize("groups,width,typ", [(8, 128, "bf16"), (1, 4096, "bf16"), (1, 12288, "bf16"), (3, 97, "f32"),
                                              (1, 8192, "f32"), (1, 5001, "bf16")])
def test_many_rows(groups, width, typ, form):
    """A thread's rows one after another: bitwise the same rows in calls of few, and sums over all of them."""
    rows, few = 9000, 700
    g = torch.Generator(DEV).manual_seed(rows + width)
    dtype = torch.bfloat16 if typ == "bf16" else torch.float32
    x, d_y, z = (torch.randn(rows, groups * width, generator=g, device=DEV).to(dtype) for _ in range(3))
    w = 1 + 0.5 * torch.rand(groups * width, generator=g, device=DEV)
    kw = gn.keywords(groups, form, False)
    gate = {} if form == "plain" else dict(gate=z)
    y = m2.group_norm_fwd(x, w, **gate, **kw)
    got = m2.group_norm_bwd(x, d_y, w, **gate, **kw)
    for at in (0, 4111, rows - few):
        s = slice(at, at + few)
        part = {k: v[s] for k, v in gate.items()}
        assert torch.equal(m2.group_norm_fwd(x[s], w, **part, **kw), y[s])
        want = m2.group_norm_bwd(x[s], d_y[s], w, **part, **kw)
        assert torch.equal(want["d_x"], got["d_x"][s])
        if gate:
            assert torch.equal(want["d_gate"], got["d_gate"][s])
    # d_weight's terms, in 64 bits; up to 16 roundings in a term, and under 112 additions one behind the other
    h, e = x.double(), d_y.double()
    silu = z.double() * torch.sigmoid(z.double())
    if form == "gated":
        e *= silu
    elif form == "gate_first":
        h *= silu
    r = (h.unflatten(-1, (groups, width)).square().mean(-1, keepdim=True) + kw["eps"]).rsqrt()
    terms = e * (h.unflatten(-1, (groups, width)) * r).flatten(-2)
    error = (got["d_weight"].double() - terms.sum(0)).abs()
    assert bool((error <= 128 * 2.0 ** -24 * terms.abs().sum(0)).all())
