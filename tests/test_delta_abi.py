"""C-ABI and binding checks of the gated delta rule and the group norm that need no GPU: every call below fails an
argument check, so no kernel is launched and no pointer dereferenced.
"""
from __future__ import annotations

import math
import os
import re

import pytest
import torch

import bwd_mamba2_scan_amd as m2
from bwd_mamba2_scan_amd import delta
from bwd_mamba2_scan_amd.delta import DeltaDims, NormDims
from bwd_mamba2_scan_amd.layer import Rows, Seqs

EOVERLAP = -8
HEADER = os.path.join(os.path.dirname(m2.HEADER), "mamba2_delta.h")
P = 0x100000


@pytest.fixture(scope="module")
def L():
    return m2.lib()


def test_binding_matches_header(L):
    with open(HEADER) as fh:
        text = re.sub(r"/\*.*?\*/", "", fh.read(), flags=re.S)
    names = set(re.findall(r"\b(mamba2_(?:delta|norm)_\w+)\s*\(", text))
    assert names == set(delta.SIGNATURES)
    for n in names:
        assert hasattr(L, n), n


# -------------------------------------------------------------- delta rule
def _dims(**kw):
    d = dict(type=1, gate_type=0, heads=4, width=16, groups=2, states=24, scale=0.5)
    d.update(kw)
    return DeltaDims(*(d[k] for k in ("type", "gate_type", "heads", "width", "groups", "states", "scale")))


def _rule(L, dims=None, batch=2, length=70, q=None, k=None, v=None, g=None, beta=None, y=None, s0=None, s1=P, ws=P,
          n=1 << 40, offsets=None, bwd=False):
    d = _dims() if dims is None else dims
    vr, kr = 64, 48
    sq = Seqs(batch, length, offsets)
    rv, rk, rg = Rows(P, vr * length, vr), Rows(P, kr * length, kr), Rows(P, 4 * length, 4)
    q, k, v, y, g, beta = q or rk, k or rk, v or rv, y or rv, g or rg, beta or rg
    if bwd:
        return L.mamba2_delta_bwd(sq, d, q, k, v, g, beta, s0, y, None, rk, rk, rv, rg, rg, s1, ws, n, None)
    return L.mamba2_delta_fwd(sq, d, q, k, v, g, beta, s0, y, s1, ws, n, None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(dims=_dims(type=3)), m2.EUNSUPPORTED), (dict(dims=_dims(gate_type=-1)), m2.EUNSUPPORTED),
    (dict(dims=_dims(heads=0)), m2.EBADDIM), (dict(dims=_dims(groups=3)), m2.EBADDIM),
    (dict(dims=_dims(groups=0)), m2.EBADDIM), (dict(dims=_dims(width=0)), m2.EBADDIM),
    (dict(dims=_dims(width=12)), m2.EUNSUPPORTED), (dict(dims=_dims(width=136)), m2.EUNSUPPORTED),
    (dict(dims=_dims(states=20)), m2.EUNSUPPORTED), (dict(dims=_dims(states=256)), m2.EUNSUPPORTED),
    (dict(dims=_dims(heads=70000, groups=70000)), m2.EUNSUPPORTED),
    (dict(dims=_dims(scale=math.nan)), m2.EBADDIM), (dict(dims=_dims(scale=math.inf)), m2.EBADDIM),
    (dict(batch=0), m2.EBADDIM), (dict(length=-3), m2.EBADDIM), (dict(batch=1 << 16, length=1 << 16), m2.EBADDIM),
    (dict(dims=_dims(heads=65535, groups=65535), batch=1, length=1 << 20), m2.EBADDIM),
    (dict(q=Rows(None, 48 * 70, 48)), m2.ENULL), (dict(v=Rows(None, 64 * 70, 64)), m2.ENULL),
    (dict(g=Rows(None, 4 * 70, 4)), m2.ENULL), (dict(beta=Rows(None, 4 * 70, 4)), m2.ENULL),
    (dict(k=Rows(P + 8, 48 * 70, 48)), m2.EALIGN), (dict(v=Rows(P, 65 * 70, 65)), m2.EALIGN),
    (dict(v=Rows(P, 64 * 70 + 4, 64)), m2.EALIGN), (dict(q=Rows(P, 48 * 70, 40)), m2.EBADDIM),
    (dict(k=Rows(P, 0, 48)), m2.EBADDIM), (dict(y=Rows(P, 64 * 70, 1 << 24)), m2.EUNSUPPORTED),
    (dict(g=Rows(P, 3, 4)), m2.EBADDIM), (dict(beta=Rows(P + 2, 4 * 70, 4)), m2.EALIGN),
    (dict(g=Rows(P, 1 << 31, 1 << 24)), m2.EUNSUPPORTED), (dict(offsets=P + 2), m2.EALIGN),
    (dict(s0=P + 8), m2.EALIGN), (dict(s1=P + 4), m2.EALIGN), (dict(ws=None), m2.ENULL), (dict(ws=P + 8), m2.EALIGN),
    (dict(n=0), m2.ESIZE),
])
def test_rule_refuses(L, kw, code, bwd):
    assert _rule(L, bwd=bwd, **kw) == code


def test_rule_workspaces(L):
    d = _dims()
    for f, bwd in ((L.mamba2_delta_fwd_workspace_bytes, False), (L.mamba2_delta_bwd_workspace_bytes, True)):
        q = Seqs(2, 70, None)
        need = f(q, d)
        assert need > 0 and need % 16 == 0
        assert _rule(L, n=need - 1, bwd=bwd) == m2.ESIZE
        assert f(q, _dims(width=7)) == 0 and f(Seqs(0, 70, None), d) == 0
        # one long sequence is cut into segments, whose states take room; as many tokens in many sequences are not
        assert f(Seqs(1, 65536, None), d) > f(Seqs(256, 256, None), d)
        # few packed sequences are cut, many are not, and have no states of segments
        one, few, many = (f(Seqs(n, 65536, P), _dims(heads=1, groups=1)) for n in (1, 16, 65535))
        cell = (one - f(Seqs(1, 128, P), _dims(heads=1, groups=1))) / 1022  # of a step, with its share of the segments
        assert one > f(Seqs(256, 256, None), _dims(heads=1, groups=1)) and few > one
        assert many <= cell * (1024 + 65535)
        # more tokens, or the same in more sequences, never need less
        sizes = [f(Seqs(1, n, P), d) for n in (0, 1, 64, 65)]
        assert sizes == sorted(sizes) and sizes[0] > 0


def test_rule_step_refuses(L):
    def call(dims=None, batch=2, q=Rows(P, 48, 0), v=Rows(P, 64, 0), state=P, new=P):
        return L.mamba2_delta_step(batch, dims or _dims(), q, Rows(P, 48, 0), v, Rows(P, 4, 0), Rows(P, 4, 0), state, v, new, None)

    assert call(state=None) == m2.ENULL and call(new=None) == m2.ENULL and call(q=Rows(None, 48, 0)) == m2.ENULL
    assert call(v=Rows(P, 63, 0)) == m2.EBADDIM and call(batch=0) == m2.EBADDIM
    assert call(batch=70000) == m2.EUNSUPPORTED
    assert call(state=P + 8) == m2.EALIGN and call(q=Rows(P + 1, 48, 0)) == m2.EALIGN
    assert call(dims=_dims(width=9)) == m2.EUNSUPPORTED
    far = [P + (i << 20) for i in range(9)]

    def at(i=None, p=0):
        """The call with tensor i at p.  bf16: q, k [2][2][24], v, y [2][4][16]; fp32: g, beta [2][4], states [2][4][24][16]"""
        a = [p if n == i else f for n, f in enumerate(far)]
        return L.mamba2_delta_step(2, _dims(), Rows(a[0], 48, 0), Rows(a[1], 48, 0), Rows(a[2], 64, 0), Rows(a[3], 4, 0),
                                   Rows(a[4], 4, 0), a[5], Rows(a[6], 64, 0), a[7], None)

    for i, n in ((0, 192), (1, 192), (2, 256), (3, 32), (4, 32), (5, 12288)):
        assert at(6, far[i]) == EOVERLAP and at(6, far[i] + n - 16) == EOVERLAP, i
        assert at(7, far[i] + (16 if i == 5 else 0)) == EOVERLAP, i
    assert at(6, far[7] + 12272) == EOVERLAP


# -------------------------------------------------------------- group norm
def _norm_dims(**kw):
    d = dict(type=1, groups=3, width=16, form=2, centered=0, shared=1, eps=1e-5)
    d.update(kw)
    return NormDims(*(d[k] for k in ("type", "groups", "width", "form", "centered", "shared", "eps")))


def _norm(L, dims=None, batch=2, length=9, x=None, gate=None, y=None, w=P, b=None, d_x=None, d_w=P, d_b=None, d_gate=None,
          ws=P, n=1 << 40, bwd=False, offsets=None):
    d = _norm_dims() if dims is None else dims
    sq = Seqs(batch, length, offsets)
    r = Rows(P, 48 * length, 48)
    x, gate, y, d_x, d_gate = x or r, gate or r, y or r, d_x or r, d_gate or r
    if bwd:
        return L.mamba2_norm_bwd(sq, d, x, w, b, gate, y, d_x, d_w, d_b, d_gate, ws, n, None)
    return L.mamba2_norm_fwd(sq, d, x, w, b, gate, y, None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(dims=_norm_dims(type=2)), m2.EUNSUPPORTED), (dict(dims=_norm_dims(form=4)), m2.EUNSUPPORTED),
    (dict(dims=_norm_dims(form=-1)), m2.EUNSUPPORTED), (dict(dims=_norm_dims(groups=0)), m2.EBADDIM),
    (dict(dims=_norm_dims(width=0)), m2.EBADDIM), (dict(dims=_norm_dims(width=16385)), m2.EUNSUPPORTED),
    (dict(dims=_norm_dims(groups=70000)), m2.EUNSUPPORTED), (dict(dims=_norm_dims(groups=1025, width=4096)), m2.EUNSUPPORTED),
    (dict(dims=_norm_dims(eps=0.0)), m2.EBADDIM), (dict(dims=_norm_dims(eps=-1.0)), m2.EBADDIM),
    (dict(dims=_norm_dims(eps=math.nan)), m2.EBADDIM), (dict(dims=_norm_dims(eps=math.inf)), m2.EBADDIM),
    (dict(batch=0), m2.EBADDIM), (dict(length=-1), m2.EBADDIM), (dict(x=Rows(None, 432, 48)), m2.ENULL),
    (dict(gate=Rows(None, 432, 48)), m2.ENULL), (dict(y=Rows(None, 432, 48)), m2.ENULL),
    (dict(x=Rows(P + 1, 432, 48)), m2.EALIGN), (dict(y=Rows(P, 432, 47)), m2.EBADDIM),
    (dict(gate=Rows(P, 47, 48)), m2.EBADDIM), (dict(w=P + 2), m2.EALIGN), (dict(w=None, b=P, d_w=None), m2.ENULL),
    (dict(offsets=P + 2), m2.EALIGN),
])
def test_norm_refuses(L, kw, code, bwd):
    assert _norm(L, bwd=bwd, **kw) == code


def test_norm_bwd_refuses(L):
    need = L.mamba2_norm_bwd_workspace_bytes(Seqs(2, 9, None), _norm_dims())
    assert need > 0 and need % 16 == 0
    none = Rows(None, 0, 0)
    call = lambda **kw: _norm(L, bwd=True, **kw)
    assert call(n=need - 1) == m2.ESIZE and call(ws=None) == m2.ENULL and call(ws=P + 4) == m2.EALIGN
    assert call(d_w=P + 2) == m2.EALIGN and call(d_b=P) == m2.ENULL            # a bias's gradient without one
    assert call(d_x=none, d_w=None, d_gate=none) == m2.ENULL                   # nothing asked for
    assert call(w=None, d_w=P) == m2.ENULL
    assert call(dims=_norm_dims(form=0)) == m2.EUNSUPPORTED                    # a gate's gradient without one
    assert L.mamba2_norm_bwd_workspace_bytes(Seqs(2, 9, None), _norm_dims(width=0)) == 0


# ------------------------------------------------------------------ binding
def test_binding_refuses():
    f = torch.zeros
    q, v, g = f(1, 4, 1, 8), f(1, 4, 2, 8), f(1, 4, 2)
    for call in (lambda: m2.delta_fwd(q, q, v, g, g), lambda: m2.delta_bwd(q, q, v, g, g, v),
                 lambda: m2.delta_step(q[:, 0], q[:, 0], v[:, 0], g[:, 0], g[:, 0], f(1, 2, 8, 8)),
                 lambda: m2.group_norm_fwd(f(4, 8)), lambda: m2.group_norm_bwd(f(4, 8), f(4, 8))):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(TypeError):
        m2.delta_fwd(q, q, [1.0], g, g)
