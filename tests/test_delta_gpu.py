"""The gated delta rule's kernels against float64, within running error bounds.  On an MI355X."""
from __future__ import annotations

import math

import pytest
import torch

import bwd_mamba2_scan_amd as m2
from oracle import delta_oracle as orc
from tests import delta_rule as dr
from tests.rounded import U, UB, within

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAMES = ("q", "k", "v", "g", "beta")


def _args(p):
    return tuple(p[n] for n in NAMES)


def _seq(p, i, span=None):
    """Sequence i of a batch, or the rows of a packed one, as one sequence."""
    out = {}
    for k, v in p.items():
        if v is None:
            out[k] = None
        elif k in ("state", "d_final"):
            out[k] = v[i]
        else:
            out[k] = v[i] if span is None else v[span[0]:span[1]]
    return out


def _check(p, scale, got, i, what, span=None, grads=True):
    s = _seq(p, i, span)
    b = dr.bounds(s, scale, grads)
    y, final = orc.delta(*_args(s), scale, s["state"])
    want = dict(y=y, final=final)
    if grads:
        want.update(orc.delta_grads(*_args(s), scale, s["state"], s["d_y"], s["d_final"]))
    for name, v in want.items():
        t = got.get(name)
        if t is None:
            continue
        t = t[i] if name in ("final", "d_state") or span is None else t[span[0]:span[1]]
        assert torch.allclose(b[name][0], v, rtol=1e-8, atol=1e-8), name
        within(t, v, b[name][1], (what, i, name))


def _run(d, scale=None, offsets=None, **kw):
    y, final = m2.delta_fwd(*_args(d), scale=scale, initial_state=d["state"], offsets=offsets, want_final_state=True, **kw)
    g = m2.delta_bwd(*_args(d), d["d_y"], scale=scale, initial_state=d["state"], d_final_state=d["d_final"],
                     offsets=offsets, **kw)
    g = dict(g, y=y, final=final)
    g["d_state"] = g.pop("d_initial_state")
    return g


SHAPES = [  # batch, length, heads, width, groups, states
    (1, 1, 1, 8, 1, 8), (2, 5, 2, 16, 1, 16), (1, 63, 3, 40, 3, 24), (1, 64, 2, 64, 2, 32), (2, 65, 4, 72, 2, 40),
    (1, 130, 6, 128, 2, 128), (2, 150, 4, 24, 4, 104), (1, 200, 2, 112, 1, 64), (3, 100, 3, 56, 1, 72),
]


@pytest.mark.parametrize("strong", [False, True])
@pytest.mark.parametrize("typ,gates", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("shape", SHAPES)
def test_against_float64(shape, typ, gates, strong):
    B, L, H, V, G, K = shape
    p = dr.inputs(sum(shape), (B, L), B, H, V, G, K, typ, gates, state=L % 2 == 0, strong=strong)
    got = _run(dr.to(p, DEV), scale=0.7)
    assert (got["d_state"] is None) == (p["state"] is None)
    for i in range(B):
        _check(p, 0.7, got, i, shape)


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1500, 2, 64, 1, 64), (1, 1400, 1, 128, 1, 128), (2, 900, 2, 40, 2, 24)])
def test_segments(shape, typ):
    """Few heads and long sequences: cut into segments that run side by side."""
    B, L, H, V, G, K = shape
    p = dr.inputs(L, (B, L), B, H, V, G, K, typ, "f32")
    got = _run(dr.to(p, DEV))
    for i in range(B):
        _check(p, K ** -0.5, got, i, shape)


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,heads", [([70, 0, 1, 64, 129, 0], 4), ([0], 2), ([900, 3, 0, 700], 1)])
def test_packed(lengths, heads, typ):
    """Packed sequences, empty ones among them; rows outside are neither read nor written."""
    first, behind = 7, 5
    rows, n = sum(lengths), len(lengths)
    ends = [first]
    for v in lengths:
        ends.append(ends[-1] + v)
    p = dr.inputs(rows + 1, (first + rows + behind,), n, heads, 48, 1, 40, typ, "f32")
    d = dr.to(p, DEV)
    for name in (*NAMES, "d_y"):
        d[name][:first] = math.nan
        d[name][first + rows:] = math.nan
    off = torch.tensor(ends, dtype=torch.int32, device=DEV)
    y = torch.full_like(d["v"], 3.0)
    y, final = m2.delta_fwd(*_args(d), initial_state=d["state"], offsets=off, want_final_state=True, y=y)
    out = {"d_" + k: torch.full_like(d[k], 3.0) for k in NAMES}
    g = m2.delta_bwd(*_args(d), d["d_y"], initial_state=d["state"], d_final_state=d["d_final"], offsets=off, out=out)
    got = dict(g, y=y, final=final)
    got["d_state"] = got.pop("d_initial_state")
    for name in ("y", *out):
        assert bool((got[name][:first] == 3).all()) and bool((got[name][first + rows:] == 3).all()), name
    for i in range(n):
        _check(p, 40 ** -0.5, got, i, lengths, span=(ends[i], ends[i + 1]))
        if lengths[i] == 0:
            assert torch.equal(final[i].cpu(), p["state"][i]) and torch.equal(got["d_state"][i].cpu(), p["d_final"][i])


@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_many_sequences(typ):
    """More packed sequences than a wave has lanes, and one tensor as both q and k."""
    lengths = [13 * i % 97 for i in range(70)]
    ends = [0]
    for v in lengths:
        ends.append(ends[-1] + v)
    p = dr.inputs(17, (ends[-1],), 70, 2, 24, 1, 32, typ, "f32")
    d = dr.to(p, DEV)
    p["q"], d["q"] = p["k"], d["k"]
    got = _run(d, offsets=torch.tensor(ends, dtype=torch.int32, device=DEV))
    for i in (0, 1, 33, 65, 69):
        _check(p, 32 ** -0.5, got, i, lengths[i], span=(ends[i], ends[i + 1]))


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("shape,cut", [((2, 70, 2, 24, 1, 40), None), ((1, 1250, 2, 64, 1, 128), None),
                                       ((1, 1000, 4, 40, 4, 24), [0, 1, 66, 66, 900, 1000])])
def test_workspaces_of_any_content(shape, cut, typ):
    """What a workspace held before the call reaches no result."""
    B, L, H, V, G, K = shape
    n = B if cut is None else len(cut) - 1
    d = dr.to(dr.inputs(18, (L,) if cut else (B, L), n, H, V, G, K, typ, "f32"), DEV)
    off = None if cut is None else torch.tensor(cut, dtype=torch.int32, device=DEV)
    want = _run(d, offsets=off)
    spaces = [torch.full((1 << 26,), math.nan, device=DEV), torch.full((1 << 26,), 3e38, device=DEV)]
    for space in spaces:
        got = _run(d, offsets=off, workspace=space)
        for name in want:
            assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_slices(typ):
    """Tensors that are slices of wider ones, gates with any stride, outputs given: bitwise the contiguous result."""
    B, L, H, V, G, K = 2, 90, 4, 24, 2, 16
    d = dr.to(dr.inputs(8, (B, L), B, H, V, G, K, typ, "f32"), DEV)
    want = _run(d)
    wide = torch.full((B, L + 3, 2 * G * K + 2 * H * V + 8), math.nan, dtype=d["v"].dtype, device=DEV)
    at, s = 8, dict(d)
    for name in ("q", "k", "v", "d_y"):
        n = d[name][0, 0].numel()
        s[name] = wide[:, 1:L + 1, at:at + n].copy_(d[name].flatten(2)).unflatten(-1, d[name].shape[2:])
        at += n
    gates = torch.full((B, L, 3 * H + 1), math.nan, device=DEV)
    s["g"], s["beta"] = gates[..., 1:H + 1].copy_(d["g"]), gates[..., 2 * H + 1:].copy_(d["beta"])
    outs = torch.full((B, L, 2 * G * K + H * V), 5.0, dtype=d["v"].dtype, device=DEV)
    cut = lambda a, n, shape: outs[..., a:a + n].unflatten(-1, shape)
    g = m2.delta_bwd(*_args(s), s["d_y"], initial_state=s["state"], d_final_state=s["d_final"],
                     out=dict(d_q=cut(0, G * K, (G, K)), d_k=cut(G * K, G * K, (G, K)), d_v=cut(2 * G * K, H * V, (H, V))))
    y, final = m2.delta_fwd(*_args(s), initial_state=s["state"], want_final_state=True)
    for name, t in (("y", y), ("final", final), *((n, g[n]) for n in ("d_q", "d_k", "d_v", "d_g", "d_beta")),
                    ("d_state", g["d_initial_state"])):
        assert torch.equal(t, want[name]), name


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,V,G,K", [(1, 1, 8, 1, 8), (3, 6, 40, 2, 24), (2, 4, 128, 4, 128), (5, 2, 72, 1, 104)])
def test_tokens(B, H, V, G, K, typ):
    """Single tokens: every one against float64 from the state that the kernel had."""
    p = dr.inputs(B + K, (B, 4), B, H, V, G, K, typ, "f32")
    d = dr.to(p, DEV)
    state = d["state"].clone()
    for t in range(4):
        tok = [d[n][:, t] for n in NAMES]
        kept, new = state.clone(), torch.empty_like(state)
        y0 = m2.delta_step(*tok, kept, new_state=new)
        assert torch.equal(kept, state)
        before = state.cpu()
        y = m2.delta_step(*tok, state)
        assert torch.equal(y, y0) and torch.equal(state, new)
        for i in range(B):
            s = {n: p[n][i, t:t + 1] for n in (*NAMES, "d_y")}
            s.update(state=before[i], d_final=None)
            b = dr.bounds(s, K ** -0.5)
            within(y[i], b["y"][0][0], b["y"][1][0], (t, i, "y"))
            within(state[i], b["final"][0], b["final"][1] + 8 * U * b["final"][0].abs(), (t, i, "state"))


def test_token_slices_and_refusals():
    B, H, V, G, K = 3, 4, 16, 2, 8
    d = dr.to(dr.inputs(9, (B, 1), B, H, V, G, K, "bf16", "f32"), DEV)
    tok = [d[n][:, 0] for n in NAMES]
    state = d["state"].clone()
    want = m2.delta_step(*tok, d["state"].clone())
    wide = torch.zeros(B, H * V + 2 * G * K, dtype=torch.bfloat16, device=DEV)
    v = wide[:, :H * V].copy_(tok[2].flatten(1)).unflatten(-1, (H, V))
    q = wide[:, H * V:H * V + G * K].copy_(tok[0].flatten(1)).unflatten(-1, (G, K))
    k = wide[:, H * V + G * K:].copy_(tok[1].flatten(1)).unflatten(-1, (G, K))
    assert torch.equal(m2.delta_step(q, k, v, *tok[3:], state), want)
    with pytest.raises(ValueError, match="overlaps"):
        m2.delta_step(q, k, v, *tok[3:], state, y=v)
    with pytest.raises(ValueError, match="shape"):
        m2.delta_step(q, k, v, *tok[3:], state[:2])
    with pytest.raises(TypeError):
        m2.delta_step(q.float(), k, v, *tok[3:], state)
    with pytest.raises(TypeError):
        m2.delta_step(q, k, v, tok[3], tok[4].bfloat16(), state)
    with pytest.raises(ValueError, match="overlaps"):
        m2.delta_fwd(*_args(d), y=d["v"])
    with pytest.raises(ValueError, match="out holds"):
        m2.delta_bwd(*_args(d), d["d_y"], out=dict(d_initial_state=torch.empty_like(state)))
    with pytest.raises(ValueError, match="dimensions"):
        m2.delta_fwd(*(t[:, 0] for t in _args(d)))


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("length", [100, 700])
def test_forgetting_tokens(length, typ):
    """g = -inf cuts a sequence in two: what is behind it is as if it began there, and nothing is a NaN."""
    B, H, V, G, K = 1, 2, 24, 1, 16
    p = dr.inputs(10, (B, length), B, H, V, G, K, typ, "f32")
    cut = 70
    p["g"][0, cut] = -math.inf
    p["g"][0, 3, 1] = -1e30
    got = _run(dr.to(p, DEV))
    for name, t in got.items():
        assert bool(torch.isfinite(t).all()), name
    _check(p, K ** -0.5, got, 0, "forget")
    assert float(got["d_g"][0, cut].abs().max()) == 0
    rest = {k: v if k in ("state", "d_final") else v[:, cut:] for k, v in p.items()}
    rest["state"] = None
    again = _run(dr.to(rest, DEV))
    size = float(again["final"].abs().max())
    assert float((got["final"] - again["final"]).abs().max()) <= 2.0 ** -16 * size


@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_padded_batch(typ):
    """Padding, g and beta 0 there, behind sequences of a dense batch: states and gradients as without it."""
    B, L, H, V, G, K = 2, 150, 4, 40, 2, 24
    p = dr.inputs(11, (B, L), B, H, V, G, K, typ, "f32")
    ends = [150, 83]
    p["g"][1, 83:] = 0
    p["beta"][1, 83:] = 0
    p["d_y"][1, 83:] = 0
    got = _run(dr.to(p, DEV))
    for i, n in enumerate(ends):
        s = {k: v[i:i + 1] if v is not None and k in ("state", "d_final") else v[i:i + 1, :n] for k, v in p.items()}
        one = _run(dr.to(s, DEV))
        assert torch.equal(got["final"][i], one["final"][0]) and torch.equal(got["d_state"][i], one["d_state"][0])
        for name in ("y", "d_q", "d_k", "d_v", "d_g", "d_beta"):
            assert torch.equal(got[name][i, :n], one[name][0]), name
    assert float(got["d_v"][1, 83:].abs().max()) == 0


def test_values_that_are_not_finite():
    """They reach their own sequence and head, and of it nothing before their step of 64 tokens."""
    B, L, H, V, G, K = 3, 150, 4, 24, 2, 16
    d = dr.to(dr.inputs(12, (B, L), B, H, V, G, K, "bf16", "f32"), DEV)
    want = _run(d)
    for name, at in (("v", (1, 70, 2, 5)), ("q", (1, 70, 1, 3)), ("k", (1, 70, 1, 3)), ("g", (1, 70, 2)), ("beta", (1, 70, 2))):
        for value in (math.nan, math.inf):
            bad = dict(d)
            bad[name] = d[name].clone()
            bad[name][at] = value
            got = _run(bad)
            for n in ("y", "d_v", "d_g", "d_beta"):
                for i in (0, 2):
                    assert torch.equal(got[n][i], want[n][i]), (name, n)
                assert torch.equal(got[n][1][:, :2], want[n][1][:, :2]), (name, n)
            assert torch.equal(got["y"][1, :64], want["y"][1, :64]), name
            for n in ("d_q", "d_k"):
                assert torch.equal(got[n][0], want[n][0]) and torch.equal(got[n][1][:, 0], want[n][1][:, 0]), (name, n)


def test_idle_gates():
    """beta = 0 everywhere and g = 0: the state stays as it was, bit for bit, over segments too."""
    d = dr.to(dr.inputs(13, (1, 1200), 1, 2, 32, 1, 32, "bf16", "f32"), DEV)
    d["g"].zero_()
    d["beta"].zero_()
    y, final = m2.delta_fwd(*_args(d), initial_state=d["state"], want_final_state=True)
    assert torch.equal(final, d["state"])


@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_precision(typ):
    """fp32 results by their 2-norm.  A result's roundings, about 400 one behind the other, are as often up as down:
    together about sqrt(400) u of it, and with the triangular inverse's share at most 32 u; a bf16 part left out
    of an operand would show as 2^-17 or more."""
    B, L, H, V, G, K = 2, 512, 4, 128, 2, 128
    p = dr.inputs(14, (B, L), B, H, V, G, K, typ, "f32")
    got = _run(dr.to(p, DEV))
    names = ["final", "d_g", "d_beta", "d_state"] + (["y", "d_q", "d_k", "d_v"] if typ == "f32" else [])
    err, size = dict.fromkeys(names, 0.0), dict.fromkeys(names, 0.0)
    half = {}
    for i in range(B):
        s = _seq(p, i)
        y, final = orc.delta(*_args(s), K ** -0.5, s["state"])
        want = dict(y=y, final=final, **orc.delta_grads(*_args(s), K ** -0.5, s["state"], s["d_y"], s["d_final"]))
        for n in names:
            err[n] += float((got[n][i].cpu().double() - want[n]).norm()) ** 2
            size[n] += float(want[n].norm()) ** 2
        if typ == "bf16":  # half a step of every value, and what two parts of 8 bits leave out
            for n in ("y", "d_q", "d_k", "d_v"):
                e = (got[n][i].cpu().double() - want[n]).abs() - UB * want[n].abs()
                half[n] = max(half.get(n, 0.0), float(e.max()) / float(want[n].norm() / want[n].numel() ** 0.5))
    for n in names:
        assert (err[n] / size[n]) ** 0.5 <= 32 * U, (n, (err[n] / size[n]) ** 0.5)
    for n, e in half.items():
        assert e <= 2.0 ** -13, (n, e)


def test_reproducible():
    for shape in ((2, 300, 4, 64, 2, 64), (1, 1500, 2, 32, 1, 64)):
        B, L, H, V, G, K = shape
        d = dr.to(dr.inputs(15, (B, L), B, H, V, G, K, "bf16", "bf16"), DEV)
        a, b = _run(d), _run(d)
        for n in a:
            assert torch.equal(a[n], b[n]), n


def test_far_apart_sequences():
    """Sequences more than 2^31 elements apart."""
    H, V, G, K, L = 2, 16, 1, 16, 70
    p = dr.inputs(16, (2, L), 2, H, V, G, K, "bf16", "f32")
    d = dr.to(p, DEV)
    want = _run(d)
    far = (1 << 31) + 4096
    big = torch.empty(far + L * H * V, dtype=torch.bfloat16, device=DEV)
    s = dict(d, v=big.as_strided((2, L, H, V), (far, H * V, V, 1)).copy_(d["v"]))
    y = m2.delta_fwd(*_args(s), initial_state=s["state"])[0]
    assert torch.equal(y, want["y"])
    g = m2.delta_bwd(*_args(s), s["d_y"], initial_state=s["state"], d_final_state=s["d_final"])
    for n in ("d_q", "d_k", "d_v", "d_g", "d_beta"):
        assert torch.equal(g[n], want[n]), n
    out = big.as_strided((2, L, H, V), (far, H * V, V, 1))
    m2.delta_fwd(*_args(d), initial_state=d["state"], y=out)
    assert torch.equal(out, want["y"])


def test_rows_far_apart():
    """Rows of the largest stride: a sequence's last ones are more than 2^31 elements behind its first."""
    H, V, G, K, L = 2, 16, 1, 16, 300
    d = dr.to(dr.inputs(19, (1, L), 1, H, V, G, K, "bf16", "f32"), DEV)
    want = _run(d)
    stride = (1 << 29) // 65
    big = torch.empty((L - 1) * stride + 4 * H * V, dtype=torch.bfloat16, device=DEV)
    at = lambda i: big.as_strided((1, L, H, V), (L * stride, stride, V, 1), i * H * V)
    s = dict(d, v=at(0).copy_(d["v"]), d_y=at(1).copy_(d["d_y"]))
    y, final = m2.delta_fwd(*_args(s), initial_state=s["state"], want_final_state=True, y=at(2))
    assert torch.equal(y, want["y"]) and torch.equal(final, want["final"])
    g = m2.delta_bwd(*_args(s), s["d_y"], initial_state=s["state"], d_final_state=s["d_final"], out=dict(d_v=at(3)))
    for n in ("d_q", "d_k", "d_v", "d_g", "d_beta"):
        assert torch.equal(g[n], want[n]), n


def test_states_beyond_32_bits():
    """More than 2^31 elements of state: the last sequences' are what they are by themselves."""
    B, H, V, G, K = 1050, 128, 128, 16, 128
    d = dr.to(dr.inputs(20, (2, 1), 2, H, V, G, K, "bf16", "f32"), DEV)
    many = {n: d[n].repeat(B // 2, 1, 1, 1) if d[n].dim() == 4 else d[n].repeat(B // 2, 1, 1) for n in NAMES}
    state = torch.zeros(B, H, K, V, device=DEV)
    assert state.numel() > 1 << 31
    state[-2:] = d["state"]
    y, final = m2.delta_fwd(*_args(d), initial_state=d["state"], want_final_state=True)
    got, ends = m2.delta_fwd(*_args(many), initial_state=state, want_final_state=True)
    assert torch.equal(got[-2:], y) and torch.equal(ends[-2:], final)
    del ends
    new = d["state"].clone()
    y = m2.delta_step(*(d[n][:, 0] for n in NAMES), new)
    got = m2.delta_step(*(many[n][:, 0] for n in NAMES), state)
    assert torch.equal(got[-2:], y) and torch.equal(state[-2:], new)


def test_gates_of_another_type():
    """bf16 gates beside fp32 values."""
    B, L, H, V, G, K = 2, 65, 4, 72, 2, 40
    p = dr.inputs(21, (B, L), B, H, V, G, K, "f32", "bf16")
    got = _run(dr.to(p, DEV))
    assert got["d_g"].dtype == got["d_beta"].dtype == torch.bfloat16
    for i in range(B):
        _check(p, K ** -0.5, got, i, "gates")
    s = {n: p[n][:, 0] for n in NAMES}
    new = p["state"].to(DEV)
    y = m2.delta_step(*(s[n].to(DEV) for n in NAMES), new)
    for i in range(B):
        one = dict({n: p[n][i, :1] for n in NAMES}, d_y=p["d_y"][i, :1], state=p["state"][i], d_final=None)
        b = dr.bounds(one, K ** -0.5)
        within(y[i], b["y"][0][0], b["y"][1][0], (i, "y"))
