"""Sequences of a single token whose row stride, which no address needs, is anything: bitwise the contiguous call, and
nothing outside the row is written.  Through the C-ABI, on an MI355X.
"""
from __future__ import annotations

import pytest
import torch

import bwd_mamba2_scan_amd as m2
from bwd_mamba2_scan_amd.layer import Rows, Seqs, SsmDims
from tests.selective import TYPES, gen, scan_inputs, to

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
MARK = 77.0
STRIDES = [0, 1, 8, 1 << 20, 1 << 26, (1 << 31) + 8, -8]


def _p(t):
    return None if t is None else t.data_ptr()


def _call(fn, *args):
    status = fn(*args, torch.cuda.current_stream().cuda_stream)
    assert status == m2.OK, status
    torch.cuda.synchronize()


def _seqs(packed, batch):
    off = torch.tensor([0, 1], dtype=torch.int32, device=DEV) if packed else None
    return Seqs(batch, 1, _p(off)), off


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("packed", [False, True])
def test_scan(typ, packed):
    batch, (H, P, G, N) = 1 if packed else 2, (4, 72, 2, 24)
    p = to(scan_inputs(3, (batch,), batch, H, P, G, N, typ, typ), DEV)
    code = {"f32": 0, "bf16": 1}[typ]
    d = SsmDims(code, code, H, P, G, N, 1)
    q, off = _seqs(packed, batch)
    L = m2.lib()
    ws = torch.empty(L.mamba2_ssm_bwd_workspace_bytes(q, d) // 4, device=DEV)
    widths = dict(x=H * P, dt=H, B=G * N, C=G * N)

    def run(stride):
        rows = lambda t, w, batch_stride=None: Rows(_p(t), w if batch_stride is None else batch_stride,
                                                    w if stride is None else stride)
        # outputs with as much behind every row as a kernel could reach by that stride's multiples in one row
        out = {k: torch.full((batch, 3 * w), MARK, dtype=TYPES[typ], device=DEV) for k, w in
               dict(y=H * P, d_x=H * P, d_dt=H, d_B=G * N, d_C=G * N).items()}
        o = {k: rows(t, t.shape[1] // 3, t.shape[1]) for k, t in out.items()}
        vec = {k: torch.empty(H, device=DEV) for k in ("d_A", "d_D", "d_dt_bias")}
        first, final = torch.empty_like(p["state"]), torch.empty_like(p["state"])
        i = {k: rows(p[k], w) for k, w in widths.items()}
        head = (q, d, i["x"], i["dt"], _p(p["A"]), i["B"], i["C"], _p(p["D"]), _p(p["dt_bias"]), _p(p["state"]))
        _call(L.mamba2_ssm_fwd, *head, o["y"], _p(final), None, 0)
        _call(L.mamba2_ssm_bwd, *head, rows(p["d_y"], H * P), _p(p["d_final"]), o["d_x"], o["d_dt"], _p(vec["d_A"]),
              o["d_B"], o["d_C"], _p(vec["d_D"]), _p(vec["d_dt_bias"]), _p(first), _p(ws), ws.numel() * 4)
        return dict(out, final=final, d_initial=first, **vec)

    want = run(None)
    for k in ("y", "d_x", "d_dt", "d_B", "d_C"):
        n = want[k].shape[1] // 3
        assert bool((want[k][:, n:] == MARK).all()) and not bool((want[k][:, :n] == MARK).any()), k
    for stride in STRIDES:
        print("scan of one token", typ, packed, stride, flush=True)
        got = run(stride)
        for k in want:
            assert torch.equal(got[k], want[k]), (stride, k)


def test_through_the_binding():
    """One token of each of two sequences that lie apart: the row stride goes in as the tensor has it."""
    H, P, G, N = 4, 24, 2, 16
    p = to(scan_inputs(5, (2, 1), 2, H, P, G, N, "bf16", "bf16"), DEV)
    kw = dict(D=p["D"], dt_bias=p["dt_bias"], initial_state=p["state"])

    def odd(t, stride):
        wide = torch.zeros(2, 2 * t[0].numel(), dtype=t.dtype, device=DEV)
        strides = list(t.stride())
        strides[0], strides[1] = wide.stride(0), stride
        v = wide.as_strided(t.shape, strides)
        return v.copy_(t)

    names = ("x", "dt", "A", "B", "C")
    args = [p[k] for k in names]
    y0, f0 = m2.ssm_fwd(*args, want_final_state=True, **kw)
    g0 = m2.ssm_bwd(*args, p["d_y"], d_final_state=p["d_final"], **kw)
    for stride in (0, 1, 1 << 40):
        print("binding", stride, flush=True)
        args = [p[k] if k == "A" else odd(p[k], stride) for k in names]
        out = {k: odd(torch.zeros_like(p[v]), stride) for k, v in (("d_x", "x"), ("d_dt", "dt"), ("d_B", "B"), ("d_C", "C"))}
        y, f = m2.ssm_fwd(*args, want_final_state=True, y=odd(p["x"], stride), **kw)
        g = m2.ssm_bwd(*args, odd(p["d_y"], stride), d_final_state=p["d_final"], out=out, **kw)
        assert torch.equal(y, y0) and torch.equal(f, f0)
        for k, v in g0.items():
            assert torch.equal(g[k], v), (stride, k)


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("packed", [False, True])
def test_convolution(typ, packed):
    batch, C, W = 1 if packed else 2, 40, 4
    g = gen(7)
    r = lambda *s: torch.randn(*s, generator=g).to(DEV)
    t = TYPES[typ]
    x, d_y, tail, d_final = r(batch, C).to(t), r(batch, C).to(t), r(batch, W - 1, C).to(t), r(batch, W - 1, C).to(t)
    weight, bias = r(C, W), r(C)
    code = {"f32": 0, "bf16": 1}[typ]
    q, off = _seqs(packed, batch)
    L = m2.lib()
    ws = torch.empty(L.mamba2_conv_bwd_workspace_bytes(q, C, W) // 4, device=DEV)

    def run(stride):
        rows = lambda v: Rows(_p(v), v.shape[1], C if stride is None else stride)
        y, d_x = (torch.full((batch, 3 * C), MARK, dtype=t, device=DEV) for _ in range(2))
        final, first = torch.empty_like(tail), torch.empty_like(tail)
        dw, db = torch.empty_like(weight), torch.empty_like(bias)
        _call(L.mamba2_conv_fwd, code, q, C, W, 1, rows(x), _p(weight), _p(bias), _p(tail), rows(y), _p(final))
        _call(L.mamba2_conv_bwd, code, q, C, W, 1, rows(x), _p(weight), _p(bias), _p(tail), rows(d_y), _p(d_final), rows(d_x),
              _p(dw), _p(db), _p(first), _p(ws), ws.numel() * 4)
        return dict(y=y, d_x=d_x, final=final, first=first, dw=dw, db=db)

    want = run(None)
    for k in ("y", "d_x"):
        assert bool((want[k][:, C:] == MARK).all()) and not bool((want[k][:, :C] == MARK).any()), k
    for stride in STRIDES:
        print("convolution of one token", typ, packed, stride, flush=True)
        got = run(stride)
        for k in want:
            assert torch.equal(got[k], want[k]), (stride, k)


def test_convolution_of_a_slice():
    """One token out of a time-major tensor: its row stride passes the limit of the strides that are used."""
    wide = torch.randn(1, 600, 8000, generator=gen(8)).bfloat16().to(DEV)
    x = wide[..., :16].transpose(0, 1)          # [600, 1, 16], row stride 4.8 million
    weight = torch.randn(16, 4, generator=gen(9)).to(DEV)
    assert torch.equal(m2.conv_fwd(x, weight)[0], m2.conv_fwd(x.contiguous(), weight)[0])
