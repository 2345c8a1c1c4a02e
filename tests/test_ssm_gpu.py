"""The selective scan's kernels against the float64 oracle, on an MI355X."""
from __future__ import annotations

import math

import pytest
import torch

import bwd_mamba2_scan_amd as m2
from oracle import selective_oracle as orc
from tests.selective import U, UB, half_step, scan_inputs, scan_roundings, to, within

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
GRADS = ("d_x", "d_dt", "d_A", "d_B", "d_C", "d_D", "d_dt_bias", "d_state")

# (batch, L, H, P, G, N, type, dt type, what is left out, positive terms)
CASES = [
    (1, 1, 1, 8, 1, 8, "f32", "f32", "", False),
    (2, 1, 4, 16, 2, 16, "bf16", "bf16", "", True),
    (3, 2, 2, 24, 1, 40, "f32", "bf16", "state", False),
    (2, 63, 3, 32, 3, 32, "bf16", "f32", "D", False),
    (1, 64, 6, 64, 2, 64, "bf16", "bf16", "bias", True),
    (2, 65, 4, 40, 1, 24, "f32", "f32", "", False),
    (1, 129, 5, 72, 5, 96, "bf16", "bf16", "state D", False),
    (1, 130, 3, 128, 1, 128, "f32", "f32", "final", False),
    (2, 200, 7, 64, 1, 128, "bf16", "bf16", "", False),
    (1, 200, 2, 128, 2, 128, "bf16", "f32", "", True),
    (1, 777, 2, 8, 1, 8, "bf16", "bf16", "softplus bias", False),      # from here on in segments
    (1, 900, 3, 48, 1, 72, "f32", "bf16", "", False),
    (2, 1029, 2, 64, 2, 16, "bf16", "bf16", "state", True),
]


def _roundings(L, P, N):
    return scan_roundings(L, P, N) * U


def _kw(p, softplus):
    return dict(D=p["D"], dt_bias=p["dt_bias"], softplus=softplus)


def _args(p):
    return tuple(p[k] for k in ("x", "dt", "A", "B", "C"))


def _cut(p, span, row):
    """One sequence of the inputs: tokens `span` and state row `row`."""
    out = {}
    for k, v in p.items():
        if v is None or k in ("A", "D", "dt_bias"):
            out[k] = v
        elif k in ("state", "d_final"):
            out[k] = v[row]
        else:
            out[k] = v[span]
    return out


def _oracle(p, spans, softplus, absolute):
    """[(y, states, gradients)] of every sequence."""
    res = []
    for row, span in enumerate(spans):
        q = _cut(p, span, row)
        args = _args(q) + (q["D"], q["dt_bias"], softplus, q["state"])
        y, states = orc.scan(*args, absolute=absolute)
        res.append((y, states, orc.scan_grads(*args, q["d_y"], q["d_final"], absolute=absolute)))
    return res


def check_forward(p, y, final, spans, softplus, exact, bound):
    typ = p["x"].dtype
    P, N = p["x"].shape[-1], p["B"].shape[-1]
    for row, span in enumerate(spans):
        (want, states, _), (size, states_size, _) = exact[row], bound[row]
        n = _roundings(want.shape[0], P, N)
        tol = n * size + half_step(typ) * want.abs()
        if typ == torch.bfloat16:
            tol = tol + 2.02 * UB * size
        within(y[span], want, tol, f"y of sequence {row}")
        if final is not None:
            within(final[row], states[-1], n * states_size[-1], f"final state of sequence {row}")


def check_grads(p, g, spans, exact, bound, skip=()):
    typ, dt_typ = p["x"].dtype, p["dt"].dtype
    P, N = p["x"].shape[-1], p["B"].shape[-1]
    n = max(_roundings(e[0].shape[0], P, N) for e in exact)
    # operands rounded to bf16: P in d_x, the gradient's state in d_B (one rounding each); Q in two parts in d_B and d_C
    bf16 = typ == torch.bfloat16
    rough = dict(d_x=1.02 * UB, d_B=1.02 * UB, d_C=1.02 * 2.0 ** -16) if bf16 else dict(d_x=0.0, d_B=0.0, d_C=0.0)
    for name in GRADS:
        if name in skip:
            continue
        got = g["d_initial_state" if name == "d_state" else name]
        if name in ("d_A", "d_D", "d_dt_bias"):  # summed over sequences and tokens (n covers the steps)
            if got is None:
                continue
            want, size = (sum(e[2][name] for e in o) for o in (exact, bound))
            tokens = sum(e[0].shape[0] for e in exact)
            within(got, want, (n + tokens / 64 * U) * size, name)
            continue
        for row, span in enumerate(spans):
            want, size = exact[row][2][name], bound[row][2][name]
            at = got[row] if name == "d_state" else got[span]
            if name == "d_state":
                tol = n * size
            elif name == "d_dt":
                tol = n * size + half_step(dt_typ) * want.abs()
            else:
                tol = (n + rough[name]) * size + half_step(typ) * want.abs()
            within(at, want, tol, f"{name} of sequence {row}")


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c[:8]))
def test_against_the_oracle(case):
    batch, L, H, P, G, N, typ, dt_typ, without, positive = case
    print("scan", case, flush=True)
    p = scan_inputs(L + P, (batch, L), batch, H, P, G, N, typ, dt_typ, positive=positive, state="state" not in without)
    softplus = "softplus" not in without
    if not softplus:
        p["dt"] = (p["dt"].float().abs() * 0.2).to(p["dt"].dtype)
    if "D" in without.split():
        p["D"] = None
    if "bias" in without:
        p["dt_bias"] = None
    if "final" in without:
        p["d_final"] = torch.zeros_like(p["d_final"])
    d = to(p, DEV)
    y, final = m2.ssm_fwd(*_args(d), initial_state=d["state"], want_final_state=True, **_kw(d, softplus))
    g = m2.ssm_bwd(*_args(d), d["d_y"], initial_state=d["state"],
                   d_final_state=None if "final" in without else d["d_final"], **_kw(d, softplus))
    torch.cuda.synchronize()
    exact, bound = (_oracle(p, range(batch), softplus, a) for a in (False, True))
    check_forward(p, y, final, range(batch), softplus, exact, bound)
    check_grads(p, g, range(batch), exact, bound, skip=() if p["state"] is not None else ("d_state",))
    assert (g["d_D"] is None) == (p["D"] is None) and (g["d_dt_bias"] is None) == (p["dt_bias"] is None)
    assert (g["d_initial_state"] is None) == (p["state"] is None)


OFFSETS = [
    ([0, 5, 5, 70, 71, 200], 200, "bf16"),          # an empty one, one of a single token
    ([0, 0, 0, 64, 128], 140, "f32"),               # empty at the front, rows behind the last
    ([3, 3, 100, 100], 130, "bf16"),                # rows before the first, empty at the end
    ([7, 7], 16, "f32"),                            # nothing but an empty sequence
    ([0, 650, 1500, 1501], 1510, "bf16"),           # segments
    ([i * 3 for i in range(151)], 450, "f32"),      # more sequences than lanes
]


@pytest.mark.parametrize("offsets,rows,typ", OFFSETS, ids=lambda v: str(v)[:24])
def test_packed(offsets, rows, typ):
    H, P, G, N = 4, 24, 2, 40
    print("packed scan", offsets[:6], rows, typ, flush=True)
    batch = len(offsets) - 1
    p = scan_inputs(rows, (rows,), batch, H, P, G, N, typ, typ)
    d = to(p, DEV)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    mark = 77.0
    y = torch.full((rows, H, P), mark, dtype=p["x"].dtype, device=DEV)
    out = {k: torch.full_like(d[v], mark) for k, v in (("d_x", "x"), ("d_dt", "dt"), ("d_B", "B"), ("d_C", "C"))}
    _, final = m2.ssm_fwd(*_args(d), initial_state=d["state"], want_final_state=True, offsets=off, y=y, **_kw(d, True))
    g = m2.ssm_bwd(*_args(d), d["d_y"], initial_state=d["state"], d_final_state=d["d_final"], offsets=off, out=out,
                   **_kw(d, True))
    torch.cuda.synchronize()
    spans = [slice(a, b) for a, b in zip(offsets, offsets[1:])]
    exact, bound = (_oracle(p, spans, True, a) for a in (False, True))
    check_forward(p, y, final, spans, True, exact, bound)
    check_grads(p, g, spans, exact, bound)
    for row, (a, b) in enumerate(zip(offsets, offsets[1:])):
        if a == b:
            assert torch.equal(final[row], d["state"][row]) and torch.equal(g["d_initial_state"][row], d["d_final"][row])
    for t in (y, g["d_x"], g["d_dt"], g["d_B"], g["d_C"]):
        assert bool((t[: offsets[0]] == mark).all()) and bool((t[offsets[-1]:] == mark).all())


def test_slices_of_one_projection():
    """x, B, C and the gradients as slices of wide tensors, dt with an odd stride: bitwise as with dense ones."""
    L, H, P, G, N, batch = 150, 5, 16, 1, 24, 2
    p = to(scan_inputs(1, (batch, L), batch, H, P, G, N, "bf16", "bf16"), DEV)
    kw = dict(initial_state=p["state"], **_kw(p, True))
    y0, f0 = m2.ssm_fwd(*_args(p), want_final_state=True, **kw)
    g0 = m2.ssm_bwd(*_args(p), p["d_y"], d_final_state=p["d_final"], **kw)

    def wide(*parts, extra):
        buf = torch.full((batch, L, sum(v.shape[2:].numel() for v in parts) + extra), 5.0, dtype=torch.bfloat16, device=DEV)
        views, at = [], 0
        for v in parts:
            n = v.shape[2:].numel()
            view = buf[..., at:at + n]
            views.append(view.unflatten(-1, v.shape[2:]) if v.dim() > 3 else view)
            views[-1].copy_(v)
            at += n
        return buf, views

    _, (x, B, C) = wide(p["x"], p["B"], p["C"], extra=8)
    _, (dt,) = wide(p["dt"], extra=2)
    buf, (d_x, d_B, d_C) = wide(p["x"], p["B"], p["C"], extra=8)
    y, f = m2.ssm_fwd(x, dt, p["A"], B, C, want_final_state=True, **kw)
    g = m2.ssm_bwd(x, dt, p["A"], B, C, p["d_y"], d_final_state=p["d_final"], out=dict(d_x=d_x, d_B=d_B, d_C=d_C), **kw)
    assert torch.equal(y, y0) and torch.equal(f, f0)
    for k, v in g0.items():
        assert torch.equal(g[k], v), k
    assert bool((buf[..., -8:] == 5.0).all())
    # sequences along the second axis: [L, batch, ...] seen as [batch, L, ...]
    xt, Bt, Ct, dtt = (v.transpose(0, 1).contiguous().transpose(0, 1) for v in (p["x"], p["B"], p["C"], p["dt"]))
    yt, ft = m2.ssm_fwd(xt, dtt, p["A"], Bt, Ct, want_final_state=True, **kw)
    assert torch.equal(yt, y0) and torch.equal(ft, f0)


@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_pieces_and_tokens_continue_a_sequence(typ):
    """A prompt in two pieces, then single tokens, against the whole sequence at once; and the step in place."""
    L, H, P, G, N, batch = 75, 6, 40, 3, 24, 2
    p = scan_inputs(2, (batch, L), batch, H, P, G, N, typ, typ)
    d = to(p, DEV)
    exact, bound = (_oracle(p, range(batch), True, a) for a in (False, True))
    at = [0, 30, 70]
    y = torch.empty_like(d["x"])
    state = d["state"]
    for a, b in zip(at, at[1:]):
        part = [d[k][:, a:b] for k in ("x", "dt")] + [d["A"]] + [d[k][:, a:b] for k in ("B", "C")]
        y[:, a:b], state = m2.ssm_fwd(*part, initial_state=state, want_final_state=True, **_kw(d, True))
    for t in range(at[-1], L):
        before = state.clone()
        token = (d["x"][:, t], d["dt"][:, t], d["A"], d["B"][:, t], d["C"][:, t])
        new = torch.empty_like(state)
        other = m2.ssm_step(*token, state, new_state=new, **_kw(d, True))
        assert torch.equal(state, before)
        y[:, t] = m2.ssm_step(*token, state, **_kw(d, True))
        assert torch.equal(state, new) and torch.equal(other, y[:, t])
    torch.cuda.synchronize()
    check_forward(p, y, state, range(batch), True, exact, bound)


STEPS = [(1, 1, 8, 1, 8, "f32"), (3, 6, 128, 2, 128, "bf16"), (2, 5, 24, 5, 88, "bf16"), (7, 4, 64, 1, 16, "f32"),
         (2, 3, 120, 1, 120, "f32")]


@pytest.mark.parametrize("batch,H,P,G,N,typ", STEPS)
def test_step(batch, H, P, G, N, typ):
    p = scan_inputs(P + N, (batch, 1), batch, H, P, G, N, typ, typ)
    d = to(p, DEV)
    y = m2.ssm_step(*(d[k][:, 0] if k != "A" else d[k] for k in ("x", "dt", "A", "B", "C")), d["state"], **_kw(d, True))
    torch.cuda.synchronize()
    for row in range(batch):
        q = _cut(p, row, row)
        args = _args(q) + (q["D"], q["dt_bias"], True, q["state"])
        (want, states), (size, ssize) = orc.scan(*args), orc.scan(*args, absolute=True)
        n = _roundings(1, P, N)
        within(y[row], want[0], n * size[0] + half_step(p["x"].dtype) * want[0].abs(), "y")
        within(d["state"][row], states[1], n * ssize[1], "state")


@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_padding_marked_by_its_step_size(typ):
    """dt = -inf: the token changes neither the state nor any gradient of the others."""
    L, real, H, P, G, N = 100, 70, 3, 32, 1, 32
    p = to(scan_inputs(5, (1, L), 1, H, P, G, N, typ, typ), DEV)
    kw = dict(initial_state=p["state"], **_kw(p, True))
    cut = [p[k][:, :real] if k != "A" else p[k] for k in ("x", "dt", "A", "B", "C")]
    y0, f0 = m2.ssm_fwd(*cut, want_final_state=True, **kw)
    g0 = m2.ssm_bwd(*cut, p["d_y"][:, :real], d_final_state=p["d_final"], **kw)
    p["dt"][:, real:] = -math.inf
    p["d_y"][:, real:] = 0
    y, f = m2.ssm_fwd(*_args(p), want_final_state=True, **kw)
    g = m2.ssm_bwd(*_args(p), p["d_y"], d_final_state=p["d_final"], **kw)
    assert torch.equal(f, f0) and torch.equal(y[:, :real], y0)
    for k in ("d_x", "d_dt", "d_B", "d_C"):
        assert torch.equal(g[k][:, :real], g0[k]), k
        assert bool((g[k][:, real:] == 0).all()), k
    for k in ("d_A", "d_D", "d_dt_bias", "d_initial_state"):
        assert torch.equal(g[k], g0[k]), k


@pytest.mark.parametrize("what", ["forgetful", "one", "huge step", "none", "tiny"])
def test_extreme_decays(what):
    """Decays that underflow at once, in one token only, a decay of one, no step at all, and tiny steps."""
    L, H, P, G, N = 140, 2, 16, 1, 16
    p = scan_inputs(6, (1, L), 1, H, P, G, N, "f32", "f32")
    p["dt_bias"] = None
    p["dt"] = p["dt"].abs() * 0.1
    if what == "forgetful":
        p["A"] = torch.tensor([-1e4, -3e6])
    elif what == "one":
        p["A"] = torch.zeros(H)
        p["dt"] = p["dt"] * 0.1
    elif what == "huge step":
        p["dt"][0, 20] = 3e4
        p["dt"][0, 90] = 1e6
    elif what == "none":
        p["dt"] = torch.zeros(1, L, H)
    else:
        p["dt"] = torch.full((1, L, H), -40.0)
    softplus = what == "tiny"
    d = to(p, DEV)
    y, final = m2.ssm_fwd(*_args(d), initial_state=d["state"], want_final_state=True, **_kw(d, softplus))
    g = m2.ssm_bwd(*_args(d), d["d_y"], initial_state=d["state"], d_final_state=d["d_final"], **_kw(d, softplus))
    torch.cuda.synchronize()
    exact, bound = (_oracle(p, range(1), softplus, a) for a in (False, True))
    check_forward(p, y, final, range(1), softplus, exact, bound)
    check_grads(p, g, range(1), exact, bound)


@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_values_that_are_not_finite_stay_in_their_sequence(typ):
    """NaN and infinities in one sequence: the others, and the steps before, come out bit for bit as without them."""
    H, P, G, N = 4, 24, 2, 40
    offsets = [3, 70, 400, 431]
    p = scan_inputs(9, (440,), 3, H, P, G, N, typ, typ)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)

    def run(q):
        d = to(q, DEV)
        y, final = m2.ssm_fwd(*_args(d), initial_state=d["state"], want_final_state=True, offsets=off, **_kw(d, True))
        g = m2.ssm_bwd(*_args(d), d["d_y"], initial_state=d["state"], d_final_state=d["d_final"], offsets=off, **_kw(d, True))
        return y, final, g

    y0, f0, g0 = run(p)
    for name, bad in (("x", math.inf), ("B", math.nan), ("C", -math.inf), ("d_y", math.nan), ("dt", math.nan)):
        q = {k: v.clone() for k, v in p.items()}
        q[name][70 + 200] = bad
        q[name][:3] = q[name][431:] = math.nan      # rows of no sequence
        y, f, g = run(q)
        whole = [slice(3, 70), slice(400, 431)]
        for s in whole + [slice(70, 70 + 192)]:
            assert torch.equal(y[s], y0[s]), (name, s)
        for s in whole:
            for k in ("d_x", "d_dt", "d_B", "d_C"):
                assert torch.equal(g[k][s], g0[k][s]), (name, k, s)
        for row in (0, 2):
            assert torch.equal(f[row], f0[row]) and torch.equal(g["d_initial_state"][row], g0["d_initial_state"][row])
        if name not in ("d_y", "C"):
            assert not bool(torch.isfinite(f[1]).all()), name


def test_runs_are_bitwise_the_same():
    p = to(scan_inputs(7, (2, 700), 2, 4, 64, 1, 64, "bf16", "bf16"), DEV)
    kw = dict(initial_state=p["state"], **_kw(p, True))
    first = second = None
    for _ in range(2):
        y, f = m2.ssm_fwd(*_args(p), want_final_state=True, **kw)
        g = m2.ssm_bwd(*_args(p), p["d_y"], d_final_state=p["d_final"], **kw)
        first, second = second, [y, f] + [g[k] for k in sorted(g)]
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_refusals_of_the_binding():
    p = to(scan_inputs(8, (1, 20), 1, 4, 16, 2, 16, "f32", "f32"), DEV)
    args = list(_args(p))
    with pytest.raises(TypeError, match="bfloat16"):
        m2.ssm_fwd(args[0].half(), *args[1:])
    with pytest.raises(TypeError):
        m2.ssm_fwd(*args[:3], args[3].bfloat16(), args[4])
    with pytest.raises(ValueError, match="shape"):
        m2.ssm_fwd(*args[:2], args[2][:2], *args[3:])
    with pytest.raises(ValueError, match="dimensions"):
        m2.ssm_fwd(args[0][0], args[1][0], args[2], args[3][0], args[4][0])
    with pytest.raises(ValueError, match="int32"):
        m2.ssm_fwd(args[0][0], args[1][0], args[2], args[3][0], args[4][0],
                   offsets=torch.tensor([0, 20], device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        m2.ssm_fwd(args[0].transpose(2, 3).contiguous().transpose(2, 3), *args[1:])
    with pytest.raises(ValueError, match="overlaps"):
        m2.ssm_fwd(*args, y=args[0])
    with pytest.raises(m2.Mamba2ScanError) as e:
        m2.ssm_fwd(args[0][..., :12].contiguous(), *args[1:])
    assert e.value.status == m2.EUNSUPPORTED
    with pytest.raises(m2.Mamba2ScanError) as e:   # one sequence's rows for all of them
        m2.ssm_fwd(*(v.expand(3, *v.shape[1:]) if v.dim() > 1 else v for v in args))
    assert e.value.status == m2.EBADDIM
    with pytest.raises(m2.Mamba2ScanError) as e:
        m2.ssm_bwd(*args, p["d_y"], workspace=torch.empty(8, device=DEV))
    assert e.value.status == m2.ESIZE
    with pytest.raises(ValueError, match="GPU tensor"):
        m2.ssm_fwd(args[0], args[1].cpu(), *args[2:])
    with pytest.raises(ValueError, match="expected"):
        m2.ssm_step(args[0][:, 0], args[1][:, 0], args[2], args[3][:, 0], args[4][:, 0], p["state"][:, :2])


def test_no_tokens():
    p = to(scan_inputs(9, (2, 0), 2, 2, 16, 1, 16, "bf16", "bf16"), DEV)
    y, f = m2.ssm_fwd(*_args(p), initial_state=p["state"], want_final_state=True, **_kw(p, True))
    g = m2.ssm_bwd(*_args(p), p["d_y"], initial_state=p["state"], d_final_state=p["d_final"], **_kw(p, True))
    assert y.shape == (2, 0, 2, 16) and torch.equal(f, p["state"]) and torch.equal(g["d_initial_state"], p["d_final"])
    for k in ("d_A", "d_D", "d_dt_bias"):
        assert bool((g[k] == 0).all())
