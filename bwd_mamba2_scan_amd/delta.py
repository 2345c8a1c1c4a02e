"""Python binding of the gated delta rule and of the group norm beside it (include/mamba2_delta.h).

    delta_fwd(q, k, v, g, beta)                -> (y, final_state)
    delta_bwd(q, k, v, g, beta, d_y)           -> dict(d_q, d_k, d_v, d_g, d_beta[, d_initial_state])
    delta_step(q, k, v, g, beta, state)        -> y; the state moves on in place
    group_norm_fwd(x, weight, bias, groups=)   -> y
    group_norm_bwd(x, d_y, weight, bias, ...)  -> dict(d_x[, d_weight, d_bias, d_gate])

Tensors, packed sequences (`offsets`), streams, outputs and workspaces are as in
the selective layer's calls (module `layer`).
"""
from __future__ import annotations

import ctypes

from . import layer as _l
from .layer import (_EOVERLAP, Rows, Seqs, _apart, _c_int, _c_size, _c_vp, _dense, _given, _gpu, _new_dense, _new_rows,
                    _On, _ptr, _raise, _rows, _seqs, _sizes, _start, _token, _type, _workspace)


class DeltaDims(ctypes.Structure):
    """mamba2_delta_dims"""
    _fields_ = [(n, _c_int) for n in ("type", "gate_type", "heads", "width", "groups", "states")] + [
        ("scale", ctypes.c_float)]


class NormDims(ctypes.Structure):
    """mamba2_norm_dims"""
    _fields_ = [(n, _c_int) for n in ("type", "groups", "width", "form", "centered", "shared")] + [
        ("eps", ctypes.c_float)]


PLAIN, SILU, GATED, GATE_FIRST = 0, 1, 2, 3  # MAMBA2_NORM_*

SIGNATURES = {
    "mamba2_norm_fwd": (_c_int, [Seqs, NormDims, Rows, _c_vp, _c_vp, Rows, Rows, _c_vp]),
    "mamba2_norm_bwd_workspace_bytes": (_c_size, [Seqs, NormDims]),
    "mamba2_norm_bwd": (_c_int, [Seqs, NormDims, Rows, _c_vp, _c_vp, Rows, Rows, Rows, _c_vp, _c_vp, Rows, _c_vp,
                                 _c_size, _c_vp]),
    "mamba2_delta_fwd_workspace_bytes": (_c_size, [Seqs, DeltaDims]),
    "mamba2_delta_fwd": (_c_int, [Seqs, DeltaDims, Rows, Rows, Rows, Rows, Rows, _c_vp, Rows, _c_vp, _c_vp, _c_size,
                                  _c_vp]),
    "mamba2_delta_bwd_workspace_bytes": (_c_size, [Seqs, DeltaDims]),
    "mamba2_delta_bwd": (_c_int, [Seqs, DeltaDims, Rows, Rows, Rows, Rows, Rows, _c_vp, Rows, _c_vp, Rows, Rows, Rows,
                                  Rows, Rows, _c_vp, _c_vp, _c_size, _c_vp]),
    "mamba2_delta_step": (_c_int, [_c_int, DeltaDims, Rows, Rows, Rows, Rows, Rows, _c_vp, Rows, _c_vp, _c_vp]),
}


# ---------------------------------------------------------------- delta rule
def _delta_dims(typ, q, v, g, scale):
    _gpu(q, "q")
    _gpu(g, "g")
    if q.dim() != v.dim():
        raise ValueError("q and k must be [..., groups, states] beside v [..., heads, width]")
    heads, width = v.shape[-2:]
    groups, states = q.shape[-2:]
    _sizes(heads, width, groups, states)
    scale = states ** -0.5 if scale is None and states > 0 else float(scale or 0.0)
    return DeltaDims(typ, _type(g, "g"), heads, width, groups, states, scale)


def _delta_inputs(q, k, v, g, beta, lead, d, dev):
    shared, vec = (d.groups, d.states), (d.heads,)
    return (_rows(q, "q", lead, shared, v.dtype, dev), _rows(k, "k", lead, shared, v.dtype, dev),
            _rows(v, "v", lead, (d.heads, d.width), v.dtype, dev), _rows(g, "g", lead, vec, g.dtype, dev),
            _rows(beta, "beta", lead, vec, g.dtype, dev))


def delta_fwd(q, k, v, g, beta, *, scale=None, initial_state=None, offsets=None, want_final_state=False, y=None,
              final_state=None, workspace=None, stream=None):
    """Gated delta rule: S' = e^g_t S_{t-1}, S_t = S' + k_t (beta_t (v_t - S'^T k_t))^T, y_t = scale S_t^T q_t.

    q, k [batch, length, groups, states], v [batch, length, heads, width],
    g, beta [batch, length, heads] (with offsets: no batch axis), float32 or
    bfloat16 (q, k, v alike, g and beta alike); heads / groups neighbouring
    heads share a q and k.  g holds log decays (<= 0), and beta |k|^2 <= 2 is
    meant: keys of length one, say (group_norm_fwd makes them); scale defaults
    to states ** -0.5.  initial_state [batch, heads, states, width] float32
    (default: zeros).  Returns (y, the final state, or None unless
    want_final_state or final_state is given).
    """
    dev, typ = _start(v, "v")
    f32 = _l.torch.float32
    seqs, lead, batch = _seqs(v, offsets, 2, dev, "v")
    d = _delta_dims(typ, q, v, g, scale)
    pq, pk, pv, pg, pb = _delta_inputs(q, k, v, g, beta, lead, d, dev)
    shape = (batch, d.heads, d.states, d.width)
    s0 = _dense(initial_state, "initial_state", shape, f32, dev)
    _apart((("y", y), ("final_state", final_state), ("workspace", workspace)),
           (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("initial_state", initial_state),
            ("offsets", offsets)))
    with _On(dev, stream) as s:
        y, py = _new_rows(y, "y", lead, (d.heads, d.width), v, dev)
        final_state, s1 = _new_state(final_state, "final_state", shape, v, dev, want_final_state)
        workspace, nbytes = _workspace(workspace, _l.lib.mamba2_delta_fwd_workspace_bytes(seqs, d), v, dev)
        st = _l.lib.mamba2_delta_fwd(seqs, d, pq, pk, pv, pg, pb, s0, py, s1, _ptr(workspace), nbytes, s)
    _raise(st, "mamba2_delta_fwd")
    return y, final_state


def _new_state(t, name, shape, like, dev, wanted=True):
    """_new_dense for a float32 tensor beside inputs of any type."""
    if t is not None:
        return t, _dense(t, name, shape, _l.torch.float32, dev)
    if not wanted:
        return None, None
    t = like.new_empty(shape, dtype=_l.torch.float32)
    return t, t.data_ptr()


def delta_bwd(q, k, v, g, beta, d_y, *, scale=None, initial_state=None, d_final_state=None, offsets=None, out=None,
              workspace=None, stream=None):
    """Gradients of delta_fwd for dL/dy = d_y (and dL/dfinal_state): dict with d_q, d_k, d_v, d_g, d_beta and
    d_initial_state (None where the forward had none).  `out` may hold some of them, no others.
    """
    dev, typ = _start(v, "v")
    f32 = _l.torch.float32
    seqs, lead, batch = _seqs(v, offsets, 2, dev, "v")
    d = _delta_dims(typ, q, v, g, scale)
    pq, pk, pv, pg, pb = _delta_inputs(q, k, v, g, beta, lead, d, dev)
    inner, shared, vec = (d.heads, d.width), (d.groups, d.states), (d.heads,)
    shape = (batch, d.heads, d.states, d.width)
    py = _rows(d_y, "d_y", lead, inner, v.dtype, dev)
    s0 = _dense(initial_state, "initial_state", shape, f32, dev)
    sf = _dense(d_final_state, "d_final_state", shape, f32, dev)
    res = _given(out, d_q=True, d_k=True, d_v=True, d_g=True, d_beta=True, d_initial_state=initial_state)
    _apart(tuple(res.items()) + (("workspace", workspace),),
           (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("d_y", d_y), ("initial_state", initial_state),
            ("d_final_state", d_final_state), ("offsets", offsets)))
    with _On(dev, stream) as s:
        ptr = []
        for name, size, like in (("d_q", shared, v), ("d_k", shared, v), ("d_v", inner, v), ("d_g", vec, g),
                                 ("d_beta", vec, g)):
            res[name], p = _new_rows(res.get(name), name, lead, size, like, dev)
            ptr.append(p)
        res["d_initial_state"], s1 = _new_state(res.get("d_initial_state"), "d_initial_state", shape, v, dev,
                                                initial_state is not None)
        workspace, nbytes = _workspace(workspace, _l.lib.mamba2_delta_bwd_workspace_bytes(seqs, d), v, dev)
        st = _l.lib.mamba2_delta_bwd(seqs, d, pq, pk, pv, pg, pb, s0, py, sf, *ptr, s1, _ptr(workspace), nbytes, s)
    _raise(st, "mamba2_delta_bwd")
    return res


def delta_step(q, k, v, g, beta, state, *, scale=None, new_state=None, y=None, stream=None):
    """One token of each sequence: q, k [batch, groups, states], v [batch, heads, width], g, beta [batch, heads] -> y.

    state [batch, heads, states, width] float32 moves on in place, or into
    new_state where that is given.
    """
    dev, typ = _start(v, "v")
    if v.dim() != 3:
        raise ValueError("v must be [batch, heads, width]")
    f32 = _l.torch.float32
    batch = v.shape[0]
    _sizes(batch)
    d = _delta_dims(typ, q, v, g, scale)
    rows = _delta_inputs(q, k, v, g, beta, (batch,), d, dev)
    shape = (batch, d.heads, d.states, d.width)
    s0 = _dense(state, "state", shape, f32, dev)
    if s0 is None:
        raise TypeError("state must be a torch.Tensor")
    s1 = s0 if new_state is None else _dense(new_state, "new_state", shape, f32, dev)
    with _On(dev, stream) as s:
        y, py = _new_rows(y, "y", (batch,), (d.heads, d.width), v, dev)
        for r in (*rows, py):
            _token(r)
        st = _l.lib.mamba2_delta_step(batch, d, *rows, s0, py, s1, s)
    if st == _EOVERLAP:
        raise ValueError("y or new_state overlaps another tensor of the call")
    _raise(st, "mamba2_delta_step")
    return y


# ---------------------------------------------------------------- group norm
_NONE = Rows(None, 0, 0)


def _norm(x, weight, bias, groups, gate, gate_first, silu, centered, eps, offsets):
    """A call's device, dims, sequences, leading shape, channels and parameters."""
    dev, typ = _start(x)
    if offsets is None and x.dim() == 2:  # rows of one sequence
        channels = x.shape[1]
        _sizes(*x.shape)
        seqs, lead = Seqs(1, x.shape[0], None), (x.shape[0],)
    else:
        seqs, lead, _ = _seqs(x, offsets, 1, dev)
        channels = x.shape[-1]
        _sizes(channels)
    groups = int(groups)
    if groups < 1 or channels % groups:
        raise ValueError(f"{channels} channels do not divide into {groups} groups")
    if gate is None:
        if gate_first:
            raise ValueError("gate_first needs a gate")
        form = SILU if silu else PLAIN
    else:
        if silu:
            raise ValueError("silu is the activation of a norm without a gate")
        form = GATE_FIRST if gate_first else GATED
    width = channels // groups
    w = b = None
    shape = (channels,)
    if weight is not None:
        _gpu(weight, "weight", dev)
        if groups > 1 and weight.shape == (width,):
            shape = (width,)
        w = _dense(weight, "weight", shape, _l.torch.float32, dev)
    if bias is not None:
        if weight is None:
            raise ValueError("a bias needs a weight")
        b = _dense(bias, "bias", shape, _l.torch.float32, dev)
    d = NormDims(typ, groups, width, form, bool(centered), shape != (channels,), eps)
    z = _NONE if gate is None else _rows(gate, "gate", lead, (channels,), x.dtype, dev)
    return dev, d, seqs, lead, channels, shape, w, b, z


def group_norm_fwd(x, weight=None, bias=None, *, groups=1, gate=None, gate_first=False, silu=False, centered=False,
                   eps=1e-5, offsets=None, y=None, stream=None):
    """Group norm with an activation, channels last: for every token and group of channels

        n = (h - mean) / sqrt(mean((h - mean)^2) + eps),  o = n weight + bias

    x [batch, length, channels], [rows, channels], or packed rows with offsets,
    float32 or bfloat16.  mean is the group's with centered, 0 without.  h is
    x and the result o, silu(o) with silu, o silu(gate) with a gate; with
    gate_first h is x silu(gate) instead.  gate has x's type and shape; weight
    and bias are float32, [channels], or [channels / groups] for every group.
    A weight of (channels / groups) ** -0.5 makes a group's length one: x /
    sqrt(sum x^2 + eps channels / groups), as queries and keys have.
    Rows outside the sequences that offsets names are neither read nor written.
    """
    dev, d, seqs, lead, channels, _, w, b, z = _norm(x, weight, bias, groups, gate, gate_first, silu, centered, eps,
                                                     offsets)
    rx = _rows(x, "x", lead, (channels,), x.dtype, dev)
    if y is not None:
        _apart((("y", y),), (("x", x), ("weight", weight), ("bias", bias), ("gate", gate), ("offsets", offsets)))
    with _On(dev, stream) as s:
        y, ry = _new_rows(y, "y", lead, (channels,), x, dev)
        st = _l.lib.mamba2_norm_fwd(seqs, d, rx, w, b, z, ry, s)
    _raise(st, "mamba2_norm_fwd")
    return y


def group_norm_bwd(x, d_y, weight=None, bias=None, *, groups=1, gate=None, gate_first=False, silu=False,
                   centered=False, eps=1e-5, offsets=None, out=None, workspace=None, stream=None):
    """Gradients of group_norm_fwd for dL/dy = d_y: dict with d_x, d_weight, d_bias and d_gate (None where the forward
    had no such input).  `out` may hold some of them, no others.
    """
    dev, d, seqs, lead, channels, shape, w, b, z = _norm(x, weight, bias, groups, gate, gate_first, silu, centered,
                                                         eps, offsets)
    rx = _rows(x, "x", lead, (channels,), x.dtype, dev)
    rg = _rows(d_y, "d_y", lead, (channels,), x.dtype, dev)
    res = _given(out, d_x=True, d_weight=weight, d_bias=bias, d_gate=gate)
    _apart(tuple(res.items()) + (("workspace", workspace),),
           (("x", x), ("weight", weight), ("bias", bias), ("gate", gate), ("d_y", d_y), ("offsets", offsets)))
    with _On(dev, stream) as s:
        get = res.get
        res["d_x"], r1 = _new_rows(get("d_x"), "d_x", lead, (channels,), x, dev)
        res["d_weight"], w1 = (_new_dense(get("d_weight"), "d_weight", shape, weight, dev)
                               if weight is not None else (None, None))
        res["d_bias"], b1 = _new_dense(get("d_bias"), "d_bias", shape, bias, dev) if bias is not None else (None, None)
        res["d_gate"], z1 = (_new_rows(get("d_gate"), "d_gate", lead, (channels,), x, dev)
                             if gate is not None else (None, _NONE))
        need = 0 if weight is None else _l.lib.mamba2_norm_bwd_workspace_bytes(seqs, d)
        workspace, nbytes = _workspace(workspace, need, x, dev)
        st = _l.lib.mamba2_norm_bwd(seqs, d, rx, w, b, z, rg, r1, w1, b1, z1, _ptr(workspace), nbytes, s)
    _raise(st, "mamba2_norm_bwd")
    return res
