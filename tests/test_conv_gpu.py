"""The causal convolution's kernels against the float64 oracle, on an MI355X."""
from __future__ import annotations

import math

import pytest
import torch

import bwd_mamba2_scan_amd as m2
from oracle import selective_oracle as orc
from tests.selective import TYPES, U, gen, half_step, to, within

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# (batch, L, channels, taps, type, bias, silu, state)
CASES = [
    (1, 1, 1, 2, "f32", True, True, True),
    (2, 2, 8, 4, "bf16", True, True, True),
    (3, 3, 9, 4, "bf16", False, True, True),
    (2, 7, 520, 3, "bf16", True, False, False),
    (1, 8, 260, 4, "f32", True, True, False),
    (2, 33, 37, 2, "f32", False, False, True),
    (1, 131, 1032, 4, "bf16", True, True, True),
    (2, 200, 72, 4, "bf16", True, True, False),
    (1, 4000, 24, 4, "bf16", True, True, True),   # runs of several lengths
]


def _inputs(seed, lead, rows, channels, taps, typ, bias, state):
    g = gen(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    t = TYPES[typ]
    tail = (rows, taps - 1, channels)
    return dict(x=r(*lead, channels).to(t), weight=r(channels, taps), bias=r(channels) if bias else None,
                state=r(*tail).to(t) if state else None, d_y=r(*lead, channels).to(t), d_final=r(*tail).to(t))


def _slack(typ, size):
    """Roundings of the pre-activation (a product and a sum per tap, the bias), the exponential's argument (v u, v up
    to a few sizes; bf16 results use the fast one, 2^-21 of v) and a dozen for the SiLU's fixed operations."""
    return ((16 * U if typ == torch.float32 else 2.0 ** -19) * (1 + size)) * size


def check(p, y, final, g, spans, silu):
    typ = p["x"].dtype
    pick = lambda v, row: None if v is None else v[row]
    d_weight = d_bias = wsize = bsize = 0
    tokens = 0
    for row, span in enumerate(spans):
        x, d_y, state, d_final = p["x"][span], p["d_y"][span], pick(p["state"], row), pick(p["d_final"], row)
        want, pre, tail = orc.conv(x, p["weight"], p["bias"], state, silu)
        size = orc.conv(x, p["weight"], p["bias"], state, silu, absolute=True)[1]
        within(y[span], want, _slack(typ, size) + half_step(typ) * want.abs(), f"y of sequence {row}")
        if final is not None:
            assert torch.equal(final[row].cpu().double(), tail), row
        if g is None:
            continue
        e = orc.conv_grads(x, p["weight"], p["bias"], state, silu, d_y, d_final)
        s = orc.conv_grads(x, p["weight"], p["bias"], state, silu, d_y, d_final, absolute=True)
        # a pre-activation gradient is off by the SiLU's slope error times d_y: at most the slack of the largest
        # pre-activation, relative to 1
        rel = float(_slack(typ, size.max() if size.numel() else torch.zeros(()))) + 16 * U
        noise = orc.conv_grads(x, p["weight"], None, state, False, d_y, None, absolute=True)
        for name, got in (("d_x", g["d_x"][span]), ("d_state", None if p["state"] is None else g["d_initial_state"][row])):
            if got is not None:
                within(got, e[name], 16 * U * s[name] + rel * noise[name] + half_step(typ) * e[name].abs(), f"{name} {row}")
        d_weight, d_bias = d_weight + e["d_weight"], d_bias + e["d_bias"]
        wsize = wsize + s["d_weight"] + rel / U * noise["d_weight"]
        bsize = bsize + s["d_bias"] + rel / U * noise["d_bias"]
        tokens += x.shape[0]
    if g is not None:
        # sums over the tokens: at most 32 + units of them one after another, in fp32
        n = 64 + tokens / 8
        sw = sum(orc.conv_grads(p["x"][s], p["weight"], None, pick(p["state"], r), False, p["d_y"][s], None, absolute=True)["d_weight"]
                 for r, s in enumerate(spans))
        sb = sum(p["d_y"][s].double().abs().sum(0) for s in spans)
        within(g["d_weight"], d_weight, U * (wsize + 1.2 * n * sw), "d_weight")
        if p["bias"] is not None:
            within(g["d_bias"], d_bias, U * (bsize + 1.2 * n * sb), "d_bias")
        else:
            assert g["d_bias"] is None


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_against_the_oracle(case):
    batch, L, channels, taps, typ, bias, silu, state = case
    print("conv", case, flush=True)
    p = _inputs(L, (batch, L), batch, channels, taps, typ, bias, state)
    d = to(p, DEV)
    y, final = m2.conv_fwd(d["x"], d["weight"], d["bias"], silu=silu, initial_state=d["state"], want_final_state=True)
    g = m2.conv_bwd(d["x"], d["weight"], d["d_y"], d["bias"], silu=silu, initial_state=d["state"],
                    d_final_state=d["d_final"])
    torch.cuda.synchronize()
    check(p, y, final, g, range(batch), silu)
    assert (g["d_initial_state"] is None) == (not state)


OFFSETS = [([0, 5, 5, 6, 50, 53], 53, 16, 4, "bf16"), ([0, 0, 2], 9, 12, 4, "f32"), ([4, 4, 90, 90], 95, 7, 3, "bf16"),
           ([i * 2 for i in range(200)], 400, 8, 4, "bf16"), ([3, 3], 5, 8, 2, "f32")]


@pytest.mark.parametrize("offsets,rows,channels,taps,typ", OFFSETS, ids=lambda v: str(v)[:20])
def test_packed(offsets, rows, channels, taps, typ):
    print("packed conv", offsets[:6], rows, channels, taps, typ, flush=True)
    batch = len(offsets) - 1
    p = _inputs(rows, (rows,), batch, channels, taps, typ, True, True)
    d = to(p, DEV)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    y, d_x = (torch.full_like(d["x"], 77.0) for _ in range(2))
    _, final = m2.conv_fwd(d["x"], d["weight"], d["bias"], initial_state=d["state"], want_final_state=True, offsets=off, y=y)
    g = m2.conv_bwd(d["x"], d["weight"], d["d_y"], d["bias"], initial_state=d["state"], d_final_state=d["d_final"],
                    offsets=off, out=dict(d_x=d_x))
    torch.cuda.synchronize()
    check(p, y, final, g, [slice(a, b) for a, b in zip(offsets, offsets[1:])], True)
    for t in (y, d_x):
        assert bool((t[: offsets[0]] == 77.0).all()) and bool((t[offsets[-1]:] == 77.0).all())


def test_slices_strides_and_unaligned_rows():
    batch, L, c = 2, 50, 24
    p = to(_inputs(3, (batch, L), batch, c, 4, "bf16", True, True), DEV)
    run = lambda x, dy, **kw: (m2.conv_fwd(x, p["weight"], p["bias"], initial_state=p["state"], want_final_state=True),
                               m2.conv_bwd(x, p["weight"], dy, p["bias"], initial_state=p["state"], d_final_state=p["d_final"], **kw))
    (y0, f0), g0 = run(p["x"], p["d_y"])
    for pad, at in ((8, 8), (3, 1), (5, 0)):   # aligned slices; odd strides and odd starts take element accesses
        wide = torch.full((batch, L, c + pad), 3.0, dtype=torch.bfloat16, device=DEV)
        x = wide[..., at:at + c] if at + c <= c + pad else wide[..., :c]
        x.copy_(p["x"])
        out = torch.full((batch, L, c + pad), 9.0, dtype=torch.bfloat16, device=DEV)
        d_x = out[..., at:at + c] if at + c <= c + pad else out[..., :c]
        (y, f), g = run(x, p["d_y"], out=dict(d_x=d_x))
        assert torch.equal(y, y0) and torch.equal(f, f0)
        assert torch.equal(d_x, g0["d_x"]) and torch.equal(g["d_initial_state"], g0["d_initial_state"])
        # the weights' partial sums cover other channels per block, each in the same order
        assert torch.equal(g["d_weight"], g0["d_weight"]) and torch.equal(g["d_bias"], g0["d_bias"])
        assert bool((out != 9.0).sum() <= batch * L * c)
    xt = p["x"].transpose(0, 1).contiguous().transpose(0, 1)
    (y, f), g = run(xt, p["d_y"])
    assert torch.equal(y, y0) and torch.equal(g["d_x"], g0["d_x"])


@pytest.mark.parametrize("typ,channels,taps", [("f32", 20, 4), ("bf16", 40, 4), ("bf16", 13, 2), ("f32", 5, 3)])
def test_pieces_and_tokens_continue_a_sequence(typ, channels, taps):
    batch, L = 3, 24
    p = _inputs(4, (batch, L), batch, channels, taps, typ, True, True)
    d = to(p, DEV)
    y = torch.empty_like(d["x"])
    state = d["state"]
    for a, b in ((0, 1), (1, 3), (3, 20)):
        y[:, a:b], state = m2.conv_fwd(d["x"][:, a:b], d["weight"], d["bias"], initial_state=state, want_final_state=True)
    for t in range(20, L):
        before, new = state.clone(), torch.empty_like(state)
        other = m2.conv_step(d["x"][:, t], d["weight"], state, d["bias"], new_state=new)
        assert torch.equal(state, before)
        y[:, t] = m2.conv_step(d["x"][:, t], d["weight"], state, d["bias"])
        assert torch.equal(state, new) and torch.equal(other, y[:, t])
    torch.cuda.synchronize()
    check(p, y, state, None, range(batch), True)


@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_values_that_are_not_finite_reach_their_window_alone(typ):
    p = to(_inputs(8, (60,), 2, 24, 4, typ, True, True), DEV)
    off = torch.tensor([2, 31, 58], dtype=torch.int32, device=DEV)
    run = lambda x: (m2.conv_fwd(x, p["weight"], p["bias"], initial_state=p["state"], offsets=off, y=torch.zeros_like(x))[0],
                     m2.conv_bwd(x, p["weight"], p["d_y"], p["bias"], initial_state=p["state"], offsets=off,
                                 out=dict(d_x=torch.zeros_like(x)))["d_x"])
    y0, g0 = run(p["x"])
    x = p["x"].clone()
    x[29] = math.nan                 # two tokens before the first sequence's end
    x[:2] = x[58:] = math.inf        # rows of no sequence
    y, g = run(x)
    rows = torch.arange(60, device=DEV)
    hit = (rows >= 29) & (rows < 31)                        # y of the token and the ones behind
    assert torch.equal(y[~hit], y0[~hit]) and bool(torch.isnan(y[hit]).all())
    hit = (rows >= 26) & (rows < 31)                        # d_x of the inputs of those pre-activations
    assert torch.equal(g[~hit], g0[~hit]) and bool(torch.isnan(g[hit]).all())


def test_parts_of_the_backward():
    p = to(_inputs(5, (1, 30), 1, 16, 4, "f32", True, True), DEV)
    whole = m2.conv_bwd(p["x"], p["weight"], p["d_y"], p["bias"], initial_state=p["state"])
    again = m2.conv_bwd(p["x"], p["weight"], p["d_y"], p["bias"], initial_state=p["state"])
    for k in whole:
        assert torch.equal(whole[k], again[k]), k
    bare = m2.conv_bwd(p["x"], p["weight"], p["d_y"])
    assert bare["d_bias"] is None and bare["d_initial_state"] is None


def test_refusals_of_the_binding():
    p = to(_inputs(6, (2, 9), 2, 16, 4, "bf16", True, True), DEV)
    with pytest.raises(ValueError, match="overlaps"):
        m2.conv_fwd(p["x"], p["weight"], y=p["x"])
    with pytest.raises(ValueError, match="overlaps"):
        m2.conv_step(p["x"][:, 0], p["weight"], p["state"], y=p["state"][:, 0])
    flat = p["weight"].view(-1).view(torch.bfloat16)[:32].view(2, 16)
    with pytest.raises(ValueError, match="overlaps"):
        m2.conv_step(p["x"][:, 0].contiguous(), p["weight"], p["state"], y=flat)
    one, two = p["state"].clone(), p["state"].clone()       # the state's own memory under another name
    m2.conv_step(p["x"][:, 0], p["weight"], one)
    m2.conv_step(p["x"][:, 0], p["weight"], two, new_state=two.view(2, 3, 16))
    assert torch.equal(one, two)
    with pytest.raises(TypeError):
        m2.conv_fwd(p["x"], p["weight"].bfloat16())
    with pytest.raises(TypeError):
        m2.conv_fwd(p["x"], p["weight"], initial_state=p["state"].float())
    with pytest.raises(ValueError, match="shape"):
        m2.conv_fwd(p["x"], p["weight"][:8].contiguous())
    with pytest.raises(m2.Mamba2ScanError) as e:
        m2.conv_fwd(p["x"], torch.zeros(16, 6, device=DEV))
    assert e.value.status == m2.EUNSUPPORTED
    with pytest.raises(m2.Mamba2ScanError) as e:
        m2.conv_fwd(p["x"][:1].expand(2, 9, 16), p["weight"])
    assert e.value.status == m2.EBADDIM


@pytest.mark.parametrize("typ,batch,L,channels", [("bf16", 4, 4096, 4096), ("f32", 2, 8191, 2056)])
def test_long_runs_under_load(typ, batch, L, channels):
    """Enough tokens that a wave walks the longest runs and the memory is busy: every value of several calls,
    against the formulas in 64 bits."""
    taps = 4
    g = torch.Generator(DEV).manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    x, d_y = r(batch, L, channels).to(TYPES[typ]), r(batch, L, channels).to(TYPES[typ])
    weight, bias = r(channels, taps), r(channels)
    print("long conv", typ, batch, L, channels, flush=True)
    calls = [(m2.conv_fwd(x, weight, bias), m2.conv_bwd(x, weight, d_y, bias)) for _ in range(3)]
    for row in range(batch):
        xs = torch.nn.functional.pad(x[row].double(), (0, 0, taps - 1, 0))
        w = weight.double()
        terms = [w[:, k] * xs[k:k + L] for k in range(taps)]
        pre = bias.double() + sum(terms)
        slack = _slack(TYPES[typ], bias.double().abs() + sum(t.abs() for t in terms))
        del terms
        sig = torch.sigmoid(pre)
        want = pre * sig
        for (y, _), _g in calls:
            assert bool(((y[row].double() - want).abs() <= slack + half_step(TYPES[typ]) * want.abs()).all()), row
        # d pre is off by at most d_y times the slack (the slope's slope is below 1) and a dozen roundings
        dp = torch.nn.functional.pad(d_y[row].double() * sig * (1 + pre * (1 - sig)), (0, 0, 0, taps - 1))
        off = torch.nn.functional.pad(d_y[row].double().abs() * (slack + 16 * U), (0, 0, 0, taps - 1))
        want = sum(w[:, k] * dp[taps - 1 - k:taps - 1 - k + L] for k in range(taps))
        size = sum(w[:, k].abs() * dp[taps - 1 - k:taps - 1 - k + L].abs() for k in range(taps))
        room = sum(w[:, k].abs() * off[taps - 1 - k:taps - 1 - k + L] for k in range(taps))
        room = room + 16 * U * size + half_step(TYPES[typ]) * want.abs()
        for _f, grads in calls:
            assert bool(((grads["d_x"][row].double() - want).abs() <= room).all()), row
    for _f, grads in calls:
        for k in ("d_weight", "d_bias"):
            assert torch.equal(grads[k], calls[0][1][k]), k


def test_no_tokens():
    p = to(_inputs(7, (2, 0), 2, 8, 4, "bf16", True, True), DEV)
    y, f = m2.conv_fwd(p["x"], p["weight"], p["bias"], initial_state=p["state"], want_final_state=True)
    g = m2.conv_bwd(p["x"], p["weight"], p["d_y"], p["bias"], initial_state=p["state"], d_final_state=p["d_final"])
    assert y.shape == (2, 0, 8) and torch.equal(f, p["state"]) and torch.equal(g["d_initial_state"], p["d_final"])
    assert bool((g["d_weight"] == 0).all()) and bool((g["d_bias"] == 0).all())
