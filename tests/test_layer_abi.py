"""C-ABI and binding checks of the selective layer that need no GPU: every call below fails an argument check, so
no kernel is launched and no pointer dereferenced.
"""
from __future__ import annotations

import ctypes
import math
import os
import re

import pytest
import torch

import bwd_mamba2_scan_amd as m2
from bwd_mamba2_scan_amd import layer
from bwd_mamba2_scan_amd.layer import Rows, Seqs, SsmDims

EOVERLAP = -8
HEADER = os.path.join(os.path.dirname(m2.HEADER), "mamba2_layer.h")
P = 0x100000


class Grad(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_longlong), ("type", ctypes.c_int)]


@pytest.fixture(scope="module")
def L():
    return m2.lib()


def test_binding_matches_header(L):
    with open(HEADER) as fh:
        text = re.sub(r"/\*.*?\*/", "", fh.read(), flags=re.S)
    names = set(re.findall(r"\b(mamba2_(?:layer|conv|ssm|grad|clip)_\w+)\s*\(", text))
    assert names == set(layer.SIGNATURES)
    for n in names:
        assert hasattr(L, n), n


def test_strerror(L):
    for code in (m2.OK, m2.EBADDIM, m2.EUNSUPPORTED, m2.ENULL, m2.ESIZE, m2.EALIGN, m2.EHIP, EOVERLAP):
        assert L.mamba2_layer_strerror(code) not in (None, b"unknown status")
    assert L.mamba2_layer_strerror(99) == b"unknown status"


# ------------------------------------------------------------- convolution
def _conv(L, typ=1, batch=2, length=9, offsets=None, channels=16, taps=4, x=P, xb=None, xr=16, w=P, bias=P, s0=P, y=P,
          yr=16, s1=P):
    xb = xr * length if xb is None else xb
    return L.mamba2_conv_fwd(typ, Seqs(batch, length, offsets), channels, taps, 1, Rows(x, xb, xr), w, bias, s0,
                             Rows(y, yr * length, yr), s1, None)


@pytest.mark.parametrize("kw,code", [
    (dict(typ=2), m2.EUNSUPPORTED), (dict(batch=0), m2.EBADDIM), (dict(length=-1), m2.EBADDIM),
    (dict(batch=1 << 16, length=1 << 16), m2.EBADDIM), (dict(channels=0), m2.EBADDIM), (dict(taps=1), m2.EUNSUPPORTED),
    (dict(taps=5), m2.EUNSUPPORTED), (dict(x=None), m2.ENULL), (dict(w=None), m2.ENULL), (dict(y=None), m2.ENULL),
    (dict(x=P + 1), m2.EALIGN), (dict(w=P + 2), m2.EALIGN), (dict(s0=P + 1), m2.EALIGN), (dict(s1=P + 1), m2.EALIGN),
    (dict(xr=15), m2.EBADDIM), (dict(xb=8), m2.EBADDIM), (dict(xb=0), m2.EBADDIM), (dict(xr=1 << 23), m2.EUNSUPPORTED),
    (dict(offsets=P + 2), m2.EALIGN),
])
def test_conv_fwd_refuses(L, kw, code):
    assert _conv(L, **kw) == code


def test_conv_bwd_refuses(L):
    q = Seqs(2, 9, None)
    need = L.mamba2_conv_bwd_workspace_bytes(q, 16, 4)
    assert need > 0 and need % 16 == 0
    r = Rows(P, 16 * 9, 16)

    def call(x=r, w=P, dy=r, dx=r, dw=P, db=P, d0=None, ws=P, n=need, taps=4):
        return L.mamba2_conv_bwd(1, q, 16, taps, 1, x, w, P, None, dy, None, dx, dw, db, d0, ws, n, None)

    assert call(n=need - 1) == m2.ESIZE
    assert call(ws=None) == m2.ENULL and call(w=None) == m2.ENULL
    assert call(dy=Rows(None, 144, 16)) == m2.ENULL
    assert call(dx=Rows(None, 0, 0), dw=None, db=None) == m2.ENULL
    assert call(ws=P + 8) == m2.EALIGN and call(dw=P + 2) == m2.EALIGN
    assert call(taps=7) == m2.EUNSUPPORTED
    assert L.mamba2_conv_bwd_workspace_bytes(q, 0, 4) == 0 == L.mamba2_conv_bwd_workspace_bytes(q, 16, 5)
    # more sequences or tokens never need less
    sizes = [L.mamba2_conv_bwd_workspace_bytes(Seqs(1, n, P), 64, 4) for n in (0, 1, 100, 5000, 100000)]
    assert sizes == sorted(sizes) and sizes[0] > 0


def test_conv_step_refuses(L):
    r = Rows(P, 16, 0)

    def call(typ=0, batch=2, x=r, state=P, new=P, taps=3):
        return L.mamba2_conv_step(typ, batch, 16, taps, 1, x, P, None, state, r, new, None)

    assert call(state=None) == m2.ENULL and call(new=None) == m2.ENULL and call(x=Rows(None, 16, 0)) == m2.ENULL
    assert call(batch=0) == m2.EBADDIM and call(batch=70000) == m2.EBADDIM and call(x=Rows(P, 15, 0)) == m2.EBADDIM
    assert call(typ=7) == m2.EUNSUPPORTED and call(state=P + 2) == m2.EALIGN
    far = [P + (i << 20) for i in range(8)]

    def at(x=Rows(far[0], 16, 0), w=far[1], bias=far[2], state=far[3], y=Rows(far[4], 16, 0), new=far[5], batch=2):
        return L.mamba2_conv_step(0, batch, 16, 3, 1, x, w, bias, state, y, new, None)

    # x, y [2][16], weight [16][3], bias [16], states [2][2][16], all fp32
    for bad in (dict(y=Rows(far[0], 16, 0)), dict(y=Rows(far[0] + 124, 16, 0)), dict(y=Rows(far[1] + 188, 16, 0)),
                dict(y=Rows(far[2] + 60, 16, 0)), dict(y=Rows(far[3] + 252, 16, 0)), dict(y=Rows(far[5] + 252, 16, 0)),
                dict(new=far[3] + 4), dict(new=far[3] - 252), dict(new=far[0] + 124), dict(new=far[1]), dict(new=far[2]),
                dict(state=far[0], new=far[0]), dict(x=Rows(far[0], 64, 0), y=Rows(far[0] + 60, 64, 0)),
                dict(x=Rows(far[0], 64, 0), y=Rows(far[0] - 60, 64, 0)), dict(x=Rows(far[0], 64, 0), y=Rows(far[0] + 200, 64, 0))):
        assert at(**bad) == EOVERLAP, bad


# -------------------------------------------------------------------- scan
def _dims(**kw):
    d = dict(type=1, dt_type=1, heads=4, width=16, groups=2, states=24, softplus=1)
    d.update(kw)
    return SsmDims(*(d[k] for k in ("type", "dt_type", "heads", "width", "groups", "states", "softplus")))


def _ssm(L, dims=None, batch=2, length=70, x=None, dt=None, A=P, B=None, C=None, y=None, s0=None, s1=P, ws=P,
         n=1 << 40, bwd=False):
    d = _dims() if dims is None else dims
    xr, br = 64, 48
    q = Seqs(batch, length, None)
    rx, rb, rt = Rows(P, xr * length, xr), Rows(P, br * length, br), Rows(P, 4 * length, 4)
    x, B, C, y, dt = x or rx, B or rb, C or rb, y or rx, dt or rt
    if bwd:
        return L.mamba2_ssm_bwd(q, d, x, dt, A, B, C, P, P, s0, y, None, rx, rt, P, rb, rb, P, P, s1, ws, n, None)
    return L.mamba2_ssm_fwd(q, d, x, dt, A, B, C, P, P, s0, y, s1, ws, n, None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(dims=_dims(type=3)), m2.EUNSUPPORTED), (dict(dims=_dims(dt_type=-1)), m2.EUNSUPPORTED),
    (dict(dims=_dims(heads=0)), m2.EBADDIM), (dict(dims=_dims(groups=3)), m2.EBADDIM),
    (dict(dims=_dims(width=0)), m2.EBADDIM), (dict(dims=_dims(width=12)), m2.EUNSUPPORTED),
    (dict(dims=_dims(width=136)), m2.EUNSUPPORTED), (dict(dims=_dims(states=20)), m2.EUNSUPPORTED),
    (dict(dims=_dims(states=256)), m2.EUNSUPPORTED), (dict(batch=0), m2.EBADDIM), (dict(length=-3), m2.EBADDIM),
    (dict(A=None), m2.ENULL), (dict(A=P + 2), m2.EALIGN), (dict(x=Rows(None, 64 * 70, 64)), m2.ENULL),
    (dict(x=Rows(P + 8, 64 * 70, 64)), m2.EALIGN), (dict(x=Rows(P, 65 * 70, 65)), m2.EALIGN),
    (dict(x=Rows(P, 64 * 70 + 4, 64)), m2.EALIGN), (dict(B=Rows(P, 48 * 70, 40)), m2.EBADDIM),
    (dict(C=Rows(P, 0, 48)), m2.EBADDIM), (dict(y=Rows(P, 64 * 70, 1 << 24)), m2.EUNSUPPORTED),
    (dict(dt=Rows(P, 3, 4)), m2.EBADDIM), (dict(dt=Rows(P + 1, 4 * 70, 4)), m2.EALIGN),
    (dict(dt=Rows(P, 1 << 31, 1 << 24)), m2.EUNSUPPORTED), (dict(s0=P + 8), m2.EALIGN), (dict(s1=P + 4), m2.EALIGN),
])
def test_ssm_refuses(L, kw, code, bwd):
    assert _ssm(L, bwd=bwd, **kw) == code


def test_ssm_workspaces(L):
    d = _dims()
    assert L.mamba2_ssm_fwd_workspace_bytes(Seqs(2, 70, None), d) == 0      # a few steps: no segments
    long = Seqs(1, 100000, None)
    need = L.mamba2_ssm_fwd_workspace_bytes(long, d)
    assert need > 0
    r, b, t = Rows(P, 0, 64), Rows(P, 0, 48), Rows(P, 0, 4)
    call = lambda ws, n: L.mamba2_ssm_fwd(long, d, r, t, P, b, b, None, None, None, r, None, ws, n, None)
    assert call(P, need - 1) == m2.ESIZE and call(None, need) == m2.ENULL and call(P + 8, need) == m2.EALIGN
    need = L.mamba2_ssm_bwd_workspace_bytes(Seqs(2, 70, None), d)
    assert need > 0
    assert _ssm(L, bwd=True, n=need - 1) == m2.ESIZE and _ssm(L, bwd=True, ws=None) == m2.ENULL
    assert _ssm(L, bwd=True, ws=P + 4) == m2.EALIGN
    assert L.mamba2_ssm_bwd_workspace_bytes(Seqs(2, 70, None), _dims(width=7)) == 0
    assert L.mamba2_ssm_fwd_workspace_bytes(Seqs(0, 70, None), d) == 0
    # the workspace covers any split of the packed rows into sequences
    for length in (64, 700, 5000):
        sizes = [L.mamba2_ssm_bwd_workspace_bytes(Seqs(n, length, P), d) for n in (1, 2, 40, 300)]
        assert sizes == sorted(sizes)


def test_ssm_step_refuses(L):
    def call(dims=None, batch=2, x=Rows(P, 64, 0), A=P, state=P, new=P):
        b = Rows(P, 48, 0)
        return L.mamba2_ssm_step(batch, dims or _dims(), x, Rows(P, 4, 0), A, b, b, None, None, state, x, new, None)

    assert call(A=None) == m2.ENULL and call(state=None) == m2.ENULL and call(new=None) == m2.ENULL
    assert call(x=Rows(P, 63, 0)) == m2.EBADDIM and call(batch=0) == m2.EBADDIM
    assert call(state=P + 8) == m2.EALIGN and call(x=Rows(P + 1, 64, 0)) == m2.EALIGN
    assert call(dims=_dims(width=9)) == m2.EUNSUPPORTED
    far = [P + (i << 20) for i in range(10)]

    def at(i=None, p=0):
        """The call with tensor i at p.  bf16: x, y [2][4][16], dt [2][4], B, C [2][2][24]; fp32: A, D, dt_bias [4], states [2][4][24][16]"""
        q = [p if k == i else v for k, v in enumerate(far)]
        return L.mamba2_ssm_step(2, _dims(), Rows(q[0], 64, 0), Rows(q[1], 4, 0), q[2], Rows(q[3], 48, 0),
                                 Rows(q[4], 48, 0), q[5], q[6], q[7], Rows(q[8], 64, 0), q[9], None)

    for i, n in ((0, 256), (1, 16), (2, 16), (3, 192), (4, 192), (5, 16), (6, 16), (7, 12288)):
        assert at(8, far[i]) == EOVERLAP and at(8, far[i] + (n - 1) // 16 * 16) == EOVERLAP, i
        assert at(9, far[i] + (16 if i == 7 else 0)) == EOVERLAP, i
    assert at(8, far[9] + 12272) == EOVERLAP


# --------------------------------------------------------------- gradients
def _table(*entries):
    return (Grad * max(1, len(entries)))(*(Grad(*e) for e in entries))


def test_grad_calls_refuse(L):
    t = _table((P, P, 100, 0), (P + 4096, P + 8192, 8, 1))
    need = L.mamba2_grad_workspace_bytes(t, 2)
    assert need > 0

    def clip(t, n=2, max_norm=1.0, norm=P + (1 << 20), ws=P + (1 << 21), nb=need):
        return L.mamba2_clip_grads(t, n, max_norm, norm, ws, nb, None)

    assert clip(t, n=0) == m2.EBADDIM and clip(None) == m2.ENULL
    assert clip(t, max_norm=-1.0) == m2.EBADDIM and clip(t, max_norm=math.nan) == m2.EBADDIM
    assert clip(t, norm=None) == m2.ENULL and clip(t, ws=None) == m2.ENULL and clip(t, nb=need - 1) == m2.ESIZE
    assert clip(t, norm=P + 2) == m2.EALIGN and clip(t, ws=P + 8) == m2.EALIGN
    assert clip(_table((P, P, 4, 5)), n=1) == m2.EUNSUPPORTED
    assert clip(_table((P, P, -4, 0)), n=1) == m2.EBADDIM
    assert clip(_table((P, P, 1 << 45, 0), (P, P, 1 << 45, 0))) == m2.EBADDIM
    assert clip(_table((None, P, 4, 0)), n=1) == m2.ENULL and clip(_table((P, None, 4, 0)), n=1) == m2.ENULL
    assert clip(_table((P + 2, P, 4, 0)), n=1) == m2.EALIGN
    # the same tensor twice, an output over another gradient, a shifted output
    assert clip(_table((P, P, 4, 0), (P, P, 4, 0))) == EOVERLAP
    assert clip(_table((P, P + 64, 4, 0), (P + 64, P + 128, 4, 0))) == EOVERLAP
    assert clip(_table((P, P + 8, 4, 0)), n=1) == EOVERLAP
    many = _table(*((P + 64 * i, P + 64 * i, 16, 0) for i in range(300)), (P + 5, P + 5, 1, 1))
    assert clip(many, n=301) in (m2.EALIGN, EOVERLAP)
    # the norm or the workspace in a gradient
    assert clip(t, norm=P + 396) == EOVERLAP and clip(t, ws=P + 384) == EOVERLAP and clip(t, norm=P + 4096) == EOVERLAP
    assert L.mamba2_grad_norm(t, 2, None, P, need, None) == m2.ENULL
    assert L.mamba2_grad_workspace_bytes(_table((P, P, 4, 9)), 1) == 0


# ------------------------------------------------------------------ binding
def test_binding_refuses_cpu_tensors_and_bad_arguments():
    f = torch.zeros
    x, w = f(1, 4, 8), f(8, 4)
    for call in (lambda: m2.conv_fwd(x, w), lambda: m2.conv_bwd(x, w, x), lambda: m2.conv_step(x[:, 0], w, f(1, 3, 8)),
                 lambda: m2.ssm_fwd(f(1, 4, 2, 8), f(1, 4, 2), f(2), f(1, 4, 1, 8), f(1, 4, 1, 8)),
                 lambda: m2.ssm_step(f(1, 2, 8), f(1, 2), f(2), f(1, 1, 8), f(1, 1, 8), f(1, 2, 8, 8)),
                 lambda: m2.grad_norm([x]), lambda: m2.clip_grads([x], 1.0)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(TypeError):
        m2.conv_fwd([1.0], w)
    for bad in (-1.0, math.nan):
        with pytest.raises(ValueError, match="max_norm"):
            m2.clip_grads([x], bad)
    with pytest.raises(ValueError, match="no gradients"):
        m2.grad_norm([])


def test_overlap_of_row_slices():
    wide = torch.zeros(3, 5, 40)
    a, b, c = wide[..., :16], wide[..., 16:40], wide[..., 8:24]
    layer._apart((("a", a),), (("b", b),))
    layer._apart((("a", a.unflatten(-1, (2, 8))), ("b", b.unflatten(-1, (3, 8)))), ())
    for one, two in ((a, c), (c, b), (a, a), (wide, a)):
        with pytest.raises(ValueError, match="overlaps"):
            layer._apart((("one", one),), (("two", two),))
    layer._apart((("one", wide[:1]),), (("two", wide[1:]),))
