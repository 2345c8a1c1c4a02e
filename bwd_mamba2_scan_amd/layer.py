"""Python binding of the selective layer's operators (include/mamba2_layer.h).

    conv_fwd(x, weight, bias)                  -> (y, final_state)
    conv_bwd(x, weight, d_y, bias)             -> dict(d_x, d_weight, d_bias[, d_initial_state])
    conv_step(x, weight, state, bias)          -> y; the state moves on in place
    ssm_fwd(x, dt, A, B, C, D=, dt_bias=)      -> (y, final_state)
    ssm_bwd(x, dt, A, B, C, d_y, ...)          -> dict(d_x, d_dt, d_A, d_B, d_C[, d_D, d_dt_bias, d_initial_state])
    ssm_step(x, dt, A, B, C, state, ...)       -> y; the state moves on in place
    grad_norm(grads)                           -> norm
    clip_grads(grads, max_norm)                -> norm; the gradients are scaled in place

Token-major tensors are [batch, length, ...] or, with `offsets`, packed as
[rows, ...] with sequence s in rows offsets[s] .. offsets[s + 1] - 1.  Only
their inner dimensions need be contiguous, so slices of a wider projection go
in as they are.  Work runs on `stream` (default: the current stream of the
tensors' device); outputs and workspaces that a call allocates belong to it.
Tensors that another stream made or will reuse are the caller's to order
(Stream.wait_stream, Tensor.record_stream), as with any kernel.
"""
from __future__ import annotations

import ctypes
import math
import struct

_F32, _BF16 = 0, 1
_EOVERLAP = -8
_MAX_INT = 2 ** 31 - 1

_c_int, _c_size, _c_vp, _c_ll = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_longlong


class Seqs(ctypes.Structure):
    """mamba2_seqs"""
    _fields_ = [("batch", _c_int), ("length", _c_int), ("offsets", _c_vp)]


class Rows(ctypes.Structure):
    """mamba2_rows"""
    _fields_ = [("data", _c_vp), ("batch_stride", _c_ll), ("row_stride", _c_ll)]


class SsmDims(ctypes.Structure):
    """mamba2_ssm_dims"""
    _fields_ = [(n, _c_int) for n in ("type", "dt_type", "heads", "width", "groups", "states", "softplus")]


SIGNATURES = {
    "mamba2_layer_strerror": (ctypes.c_char_p, [_c_int]),
    "mamba2_conv_fwd": (_c_int, [_c_int, Seqs, _c_int, _c_int, _c_int, Rows, _c_vp, _c_vp, _c_vp, Rows, _c_vp, _c_vp]),
    "mamba2_conv_bwd_workspace_bytes": (_c_size, [Seqs, _c_int, _c_int]),
    "mamba2_conv_bwd": (_c_int, [_c_int, Seqs, _c_int, _c_int, _c_int, Rows, _c_vp, _c_vp, _c_vp, Rows, _c_vp, Rows,
                                 _c_vp, _c_vp, _c_vp, _c_vp, _c_size, _c_vp]),
    "mamba2_conv_step": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, Rows, _c_vp, _c_vp, _c_vp, Rows, _c_vp,
                                  _c_vp]),
    "mamba2_ssm_fwd_workspace_bytes": (_c_size, [Seqs, SsmDims]),
    "mamba2_ssm_fwd": (_c_int, [Seqs, SsmDims, Rows, Rows, _c_vp, Rows, Rows, _c_vp, _c_vp, _c_vp, Rows, _c_vp, _c_vp,
                                _c_size, _c_vp]),
    "mamba2_ssm_bwd_workspace_bytes": (_c_size, [Seqs, SsmDims]),
    "mamba2_ssm_bwd": (_c_int, [Seqs, SsmDims, Rows, Rows, _c_vp, Rows, Rows, _c_vp, _c_vp, _c_vp, Rows, _c_vp, Rows,
                                Rows, _c_vp, Rows, Rows, _c_vp, _c_vp, _c_vp, _c_vp, _c_size, _c_vp]),
    "mamba2_ssm_step": (_c_int, [_c_int, SsmDims, Rows, Rows, _c_vp, Rows, Rows, _c_vp, _c_vp, _c_vp, Rows, _c_vp,
                                 _c_vp]),
    "mamba2_grad_workspace_bytes": (_c_size, [_c_vp, _c_int]),
    "mamba2_grad_norm": (_c_int, [_c_vp, _c_int, _c_vp, _c_vp, _c_size, _c_vp]),
    "mamba2_clip_grads": (_c_int, [_c_vp, _c_int, ctypes.c_float, _c_vp, _c_vp, _c_size, _c_vp]),
}


# torch, the loaded library and the element types, looked up once, by the first
# call (importing this package imports no torch).
torch = lib = _TYPES = None


def _load():
    global torch, lib, _TYPES
    import torch as t
    from . import lib as load

    lib = load()
    _TYPES = {t.float32: _F32, t.bfloat16: _BF16}
    torch = t


def _raise(status, where):
    if status != 0:
        from . import Mamba2ScanError
        raise Mamba2ScanError(status, where, lib.mamba2_layer_strerror(status).decode())


class _On:
    """The tensors' device and the stream of a call, made current for its allocations and launches."""

    __slots__ = ("_dev", "_stream", "_guards")

    def __init__(self, dev, stream):
        self._dev, self._stream, self._guards = dev, stream, ()

    def __enter__(self):
        index = self._dev.index
        if self._stream is not None and self._stream.device != self._dev:  # before any guard: none is left behind
            raise ValueError(f"stream is on {self._stream.device}, the tensors on {self._dev}")
        if torch._C._cuda_getDevice() != index:
            self._push(torch.cuda.device(index))
        if self._stream is not None:
            self._push(torch.cuda.stream(self._stream))
        return torch._C._cuda_getCurrentRawStream(index)

    def _push(self, guard):
        guard.__enter__()
        self._guards += (guard,)

    def __exit__(self, *exc):
        for g in reversed(self._guards):
            g.__exit__(*exc)
        return False


def _start(x, name="x"):
    """(device, element type code) of a call's first tensor."""
    if torch is None:
        _load()
    _gpu(x, name)
    return x.device, _type(x, name)


def _type(t, name):
    typ = _TYPES.get(t.dtype)
    if typ is None:
        raise TypeError(f"{name} must be float32 or bfloat16 (got {t.dtype})")
    return typ


def _gpu(t, name, dev=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dev is not None and t.get_device() == dev.index:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (got {t.device})")
    if dev is not None:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _dense(t, name, shape, dtype, dev):
    """The address of a contiguous tensor, or None."""
    if t is None:
        return None
    _gpu(t, name, dev)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name, lead, inner, dtype, dev):
    """A token-major tensor: contiguous inner dimensions, free outer strides."""
    _gpu(t, name, dev)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != lead + inner:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {lead + inner}")
    want = 1
    if t.is_contiguous():
        for size in inner:
            want *= size
        return Rows(t.data_ptr(), want * lead[-1], want)
    strides = t.stride()
    for size, stride in zip(reversed(inner), reversed(strides)):
        if size != 1 and stride != want:
            raise ValueError(f"{name}: the inner dimensions {inner} must be contiguous (strides {strides})")
        want *= size
    if len(lead) == 2:
        return Rows(t.data_ptr(), strides[0], strides[1])
    return Rows(t.data_ptr(), 0, strides[0])


def _token(rows):
    """The rows of a tensor without a token axis: its first axis counts the sequences."""
    rows.batch_stride, rows.row_stride = rows.row_stride, 0
    return rows


def _sizes(*sizes):
    """Refuses sizes that the C ABI's ints do not hold (ctypes would cut them off)."""
    if max(sizes) > _MAX_INT:
        raise ValueError(f"a dimension of {max(sizes)} is too large (at most {_MAX_INT})")


def _seqs(x, offsets, inner_dims, dev, name="x"):
    """(mamba2_seqs, the leading shape, the number of sequences)"""
    if offsets is None:
        if x.dim() != 2 + inner_dims:
            raise ValueError(f"{name} must have {2 + inner_dims} dimensions (got {x.dim()}); packed rows need offsets")
        batch, length = x.shape[:2]
        _sizes(batch, length)
        return Seqs(batch, length, None), (batch, length), batch
    if x.dim() != 1 + inner_dims:
        raise ValueError(f"with offsets {name} must have {1 + inner_dims} dimensions (got {x.dim()})")
    _gpu(offsets, "offsets", dev)
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.numel() < 2 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous int32 vector of at least two elements")
    batch = offsets.numel() - 1
    _sizes(batch, x.shape[0])
    return Seqs(batch, x.shape[0], offsets.data_ptr()), (x.shape[0],), batch


def _span(t):
    """First byte and byte behind the last of a tensor."""
    lo = t.data_ptr()
    if t.is_contiguous():
        return lo, lo + t.nbytes
    if t.numel() == 0:
        return lo, lo
    return lo, lo + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()


def _apart(outs, ins):
    """Refuses outputs that a caller gave and that overlap an input or one another.

    Slices of one wide row-major tensor interleave without overlapping: equal
    row strides and disjoint windows within the row are told apart.
    """
    for i, (n, t) in enumerate(outs):
        if t is None:
            continue
        lo, hi = _span(t)
        if lo == hi:
            continue
        for m, o in (*outs[i + 1:], *ins):
            if o is None:
                continue
            a = o.data_ptr()
            if hi <= a:
                continue
            a, b = _span(o)
            if b > lo and a != b and not _interleaved(t, o):
                raise ValueError(f"{n} overlaps {m}")


def _interleaved(t, o):
    def window(v):  # row strides in bytes, outermost first, and the bytes of a row's window
        sizes, strides = list(v.shape), list(v.stride())
        width = 1
        while sizes and (sizes[-1] == 1 or strides[-1] == width):
            width *= sizes.pop()
            strides.pop()
        return [s * v.element_size() for n, s in zip(sizes, strides) if n > 1], width * v.element_size()

    (st, wt), (so, wo) = window(t), window(o)
    if not st or not so or st[-1] != so[-1] or any(s % st[-1] for s in st + so):
        return False
    row = st[-1]
    gap = (o.data_ptr() - t.data_ptr()) % row
    return wt <= gap and gap + wo <= row


def _given(out, **inputs):
    """The tensors of `out`: gradients of required inputs (True) or of inputs that were given."""
    res = dict(out or {})
    for name, t in res.items():
        if name not in inputs:
            raise ValueError(f"out holds {name!r}; the gradients are {', '.join(inputs)}")
        if t is not None and inputs[name] is None:
            raise ValueError(f"out holds {name}, but no {name[2:]} was given")
    return res


def _ptr(t):
    return None if t is None else t.data_ptr()


def _new_rows(t, name, lead, inner, like, dev):
    """(a token-major output of a tensor's type, its mamba2_rows): the given tensor, or a new one."""
    if t is not None:
        return t, _rows(t, name, lead, inner, like.dtype, dev)
    t = like.new_empty(lead + inner)
    width = 1
    for n in inner:
        width *= n
    return t, Rows(t.data_ptr(), width * lead[-1], width)


def _new_dense(t, name, shape, like, dev, wanted=True):
    """(a contiguous output of a tensor's type or None, its address): the given tensor, or a new one where it is wanted."""
    if t is not None:
        return t, _dense(t, name, shape, like.dtype, dev)
    if not wanted:
        return None, None
    t = like.new_empty(shape)
    return t, t.data_ptr()


# -------------------------------------------------------------- convolution
def _conv_dims(x, weight, dev):
    _gpu(weight, "weight", dev)
    if weight.dim() != 2:
        raise ValueError("weight must be [channels, taps]")
    channels, taps = weight.shape
    _sizes(channels, taps)
    w = _dense(weight, "weight", (channels, taps), torch.float32, dev)
    return channels, taps, w


def conv_fwd(x, weight, bias=None, *, silu=True, initial_state=None, offsets=None, want_final_state=False, y=None,
             final_state=None, stream=None):
    """Short causal depthwise convolution: y_t = f(bias + sum_k weight[:, k] x_{t-W+1+k}), f = SiLU or the identity.

    x [batch, length, channels] (or [rows, channels] with offsets), float32 or
    bfloat16; weight [channels, W], W = 2, 3 or 4, and bias [channels],
    float32.  initial_state [batch, W - 1, channels] holds the inputs before
    the first token (default: zeros).  Returns (y, the last W - 1 inputs, or
    None unless want_final_state or final_state is given).
    """
    dev, typ = _start(x)
    seqs, lead, batch = _seqs(x, offsets, 1, dev)
    channels, taps, w = _conv_dims(x, weight, dev)
    rx = _rows(x, "x", lead, (channels,), x.dtype, dev)
    b = _dense(bias, "bias", (channels,), torch.float32, dev)
    s0 = _dense(initial_state, "initial_state", (batch, taps - 1, channels), x.dtype, dev)
    _apart((("y", y), ("final_state", final_state)),
           (("x", x), ("weight", weight), ("bias", bias), ("initial_state", initial_state), ("offsets", offsets)))
    with _On(dev, stream) as s:
        y, ry = _new_rows(y, "y", lead, (channels,), x, dev)
        final_state, s1 = _new_dense(final_state, "final_state", (batch, taps - 1, channels), x, dev, want_final_state)
        st = lib.mamba2_conv_fwd(typ, seqs, channels, taps, bool(silu), rx, w, b, s0, ry, s1, s)
    _raise(st, "mamba2_conv_fwd")
    return y, final_state


def conv_bwd(x, weight, d_y, bias=None, *, silu=True, initial_state=None, d_final_state=None, offsets=None, out=None,
             workspace=None, stream=None):
    """Gradients of conv_fwd for dL/dy = d_y (and dL/dfinal_state): dict with d_x, d_weight, d_bias (None without
    bias) and d_initial_state (None without initial_state).  `out` may hold some of these tensors, no others.
    """
    dev, typ = _start(x)
    seqs, lead, batch = _seqs(x, offsets, 1, dev)
    channels, taps, w = _conv_dims(x, weight, dev)
    rx = _rows(x, "x", lead, (channels,), x.dtype, dev)
    rg = _rows(d_y, "d_y", lead, (channels,), x.dtype, dev)
    b = _dense(bias, "bias", (channels,), torch.float32, dev)
    tail = (batch, taps - 1, channels)
    s0 = _dense(initial_state, "initial_state", tail, x.dtype, dev)
    sf = _dense(d_final_state, "d_final_state", tail, x.dtype, dev)
    res = _given(out, d_x=True, d_weight=True, d_bias=bias, d_initial_state=initial_state)
    _apart(tuple(res.items()) + (("workspace", workspace),),
           (("x", x), ("weight", weight), ("bias", bias), ("d_y", d_y), ("initial_state", initial_state),
            ("d_final_state", d_final_state), ("offsets", offsets)))
    with _On(dev, stream) as s:
        get = res.get
        res["d_x"], rx1 = _new_rows(get("d_x"), "d_x", lead, (channels,), x, dev)
        res["d_weight"], w1 = _new_dense(get("d_weight"), "d_weight", (channels, taps), weight, dev)
        res["d_bias"], b1 = (_new_dense(get("d_bias"), "d_bias", (channels,), weight, dev)
                             if bias is not None else (None, None))
        res["d_initial_state"], s1 = (_new_dense(get("d_initial_state"), "d_initial_state", tail, x, dev)
                                      if initial_state is not None else (None, None))
        workspace, nbytes = _workspace(workspace, lib.mamba2_conv_bwd_workspace_bytes(seqs, channels, taps), x, dev)
        st = lib.mamba2_conv_bwd(typ, seqs, channels, taps, bool(silu), rx, w, b, s0, rg, sf, rx1, w1, b1, s1,
                                 _ptr(workspace), nbytes, s)
    _raise(st, "mamba2_conv_bwd")
    return res


def _workspace(workspace, need, like, dev):
    """The given workspace or a new one of a tensor's type; (tensor or None, bytes)."""
    if workspace is None:
        if need == 0:
            return None, 0
        return like.new_empty(-(-need // like.element_size())), need
    _gpu(workspace, "workspace", dev)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.numel() * workspace.element_size()


def conv_step(x, weight, state, bias=None, *, silu=True, new_state=None, y=None, stream=None):
    """One token of each sequence: x [batch, channels] -> y; state [batch, W - 1, channels] moves on in place, or
    into new_state where that is given.
    """
    dev, typ = _start(x)
    channels, taps, w = _conv_dims(x, weight, dev)
    batch = x.shape[0]
    _sizes(batch)
    rx = _token(_rows(x, "x", (batch,), (channels,), x.dtype, dev))
    tail = (batch, taps - 1, channels)
    s0 = _dense(state, "state", tail, x.dtype, dev)
    if s0 is None:
        raise TypeError("state must be a torch.Tensor")
    b = _dense(bias, "bias", (channels,), torch.float32, dev)
    s1 = s0 if new_state is None else _dense(new_state, "new_state", tail, x.dtype, dev)
    with _On(dev, stream) as s:
        y, ry = _new_rows(y, "y", (batch,), (channels,), x, dev)
        st = lib.mamba2_conv_step(typ, batch, channels, taps, bool(silu), rx, w, b, s0, _token(ry), s1, s)
    if st == _EOVERLAP:
        raise ValueError("y or new_state overlaps another tensor of the call")
    _raise(st, "mamba2_conv_step")
    return y


# ---------------------------------------------------------------------- scan
def _ssm_dims(typ, x, dt, B, softplus):
    _gpu(dt, "dt")
    _gpu(B, "B")
    if B.dim() != x.dim():
        raise ValueError("B and C must be [..., groups, states] beside x [..., heads, width]")
    heads, width = x.shape[-2:]
    groups, states = B.shape[-2:]
    _sizes(heads, width, groups, states)
    return SsmDims(typ, _type(dt, "dt"), heads, width, groups, states, bool(softplus))


def _ssm_inputs(x, dt, A, B, C, D, dt_bias, lead, d, dev):
    f32 = torch.float32
    inner, shared = (d.heads, d.width), (d.groups, d.states)
    vec = (d.heads,)
    if A is None:
        raise TypeError("A must be a torch.Tensor")
    return (_rows(x, "x", lead, inner, x.dtype, dev), _rows(dt, "dt", lead, vec, dt.dtype, dev),
            _dense(A, "A", vec, f32, dev), _rows(B, "B", lead, shared, x.dtype, dev),
            _rows(C, "C", lead, shared, x.dtype, dev), _dense(D, "D", vec, f32, dev),
            _dense(dt_bias, "dt_bias", vec, f32, dev))


def ssm_fwd(x, dt, A, B, C, *, D=None, dt_bias=None, softplus=True, initial_state=None, offsets=None,
            want_final_state=False, y=None, final_state=None, workspace=None, stream=None):
    """Selective state space scan: S_t = exp(d_t A) S_{t-1} + d_t B_t x_t^T, y_t = S_t^T C_t + D x_t, with
    d_t = softplus(dt_t + dt_bias) (or dt_t + dt_bias).

    x [batch, length, heads, width], dt [batch, length, heads],
    B, C [batch, length, groups, states] (with offsets: no batch axis), float32
    or bfloat16 (x, B, C alike); A, D, dt_bias [heads] float32; heads / groups
    neighbouring heads share a B and C.  initial_state [batch, heads, states,
    width] float32 (default: zeros).  Returns (y, the final state, or None
    unless want_final_state or final_state is given).
    """
    dev, typ = _start(x)
    seqs, lead, batch = _seqs(x, offsets, 2, dev)
    d = _ssm_dims(typ, x, dt, B, softplus)
    px, pdt, pA, pB, pC, pD, pbias = _ssm_inputs(x, dt, A, B, C, D, dt_bias, lead, d, dev)
    shape = (batch, d.heads, d.states, d.width)
    s0 = _dense(initial_state, "initial_state", shape, torch.float32, dev)
    _apart((("y", y), ("final_state", final_state), ("workspace", workspace)),
           (("x", x), ("dt", dt), ("A", A), ("B", B), ("C", C), ("D", D), ("dt_bias", dt_bias),
            ("initial_state", initial_state), ("offsets", offsets)))
    with _On(dev, stream) as s:
        y, py = _new_rows(y, "y", lead, (d.heads, d.width), x, dev)
        final_state, s1 = _new_dense(final_state, "final_state", shape, A, dev, want_final_state)
        workspace, nbytes = _workspace(workspace, lib.mamba2_ssm_fwd_workspace_bytes(seqs, d), A, dev)
        st = lib.mamba2_ssm_fwd(seqs, d, px, pdt, pA, pB, pC, pD, pbias, s0, py, s1, _ptr(workspace), nbytes, s)
    _raise(st, "mamba2_ssm_fwd")
    return y, final_state


def ssm_bwd(x, dt, A, B, C, d_y, *, D=None, dt_bias=None, softplus=True, initial_state=None, d_final_state=None,
            offsets=None, out=None, workspace=None, stream=None):
    """Gradients of ssm_fwd for dL/dy = d_y (and dL/dfinal_state): dict with d_x, d_dt, d_A, d_B, d_C, and d_D,
    d_dt_bias, d_initial_state (each None where the forward had no such input).  `out` may hold some of them, no others.
    """
    dev, typ = _start(x)
    f32 = torch.float32
    seqs, lead, batch = _seqs(x, offsets, 2, dev)
    d = _ssm_dims(typ, x, dt, B, softplus)
    px, pdt, pA, pB, pC, pD, pbias = _ssm_inputs(x, dt, A, B, C, D, dt_bias, lead, d, dev)
    inner, shared, vec = (d.heads, d.width), (d.groups, d.states), (d.heads,)
    shape = (batch, d.heads, d.states, d.width)
    pg = _rows(d_y, "d_y", lead, inner, x.dtype, dev)
    s0 = _dense(initial_state, "initial_state", shape, f32, dev)
    sf = _dense(d_final_state, "d_final_state", shape, f32, dev)
    res = _given(out, d_x=True, d_dt=True, d_A=True, d_B=True, d_C=True, d_D=D, d_dt_bias=dt_bias,
                 d_initial_state=initial_state)
    _apart(tuple(res.items()) + (("workspace", workspace),),
           (("x", x), ("dt", dt), ("A", A), ("B", B), ("C", C), ("D", D), ("dt_bias", dt_bias), ("d_y", d_y),
            ("initial_state", initial_state), ("d_final_state", d_final_state), ("offsets", offsets)))
    with _On(dev, stream) as s:
        ptr = {}
        for name, size, like in (("d_x", inner, x), ("d_dt", vec, dt), ("d_B", shared, x), ("d_C", shared, x)):
            res[name], ptr[name] = _new_rows(res.get(name), name, lead, size, like, dev)
        for name, given, size in (("d_A", A, vec), ("d_D", D, vec), ("d_dt_bias", dt_bias, vec),
                                  ("d_initial_state", initial_state, shape)):
            if given is None:
                res[name] = ptr[name] = None
            else:
                res[name], ptr[name] = _new_dense(res.get(name), name, size, A, dev)
        workspace, nbytes = _workspace(workspace, lib.mamba2_ssm_bwd_workspace_bytes(seqs, d), A, dev)
        st = lib.mamba2_ssm_bwd(seqs, d, px, pdt, pA, pB, pC, pD, pbias, s0, pg, sf, ptr["d_x"], ptr["d_dt"],
                                ptr["d_A"], ptr["d_B"], ptr["d_C"], ptr["d_D"], ptr["d_dt_bias"],
                                ptr["d_initial_state"], _ptr(workspace), nbytes, s)
    _raise(st, "mamba2_ssm_bwd")
    return res


def ssm_step(x, dt, A, B, C, state, *, D=None, dt_bias=None, softplus=True, new_state=None, y=None, stream=None):
    """One token of each sequence: x [batch, heads, width], dt [batch, heads], B, C [batch, groups, states] -> y.

    state [batch, heads, states, width] float32 moves on in place, or into
    new_state where that is given.
    """
    dev, typ = _start(x)
    if x.dim() != 3:
        raise ValueError("x must be [batch, heads, width]")
    batch = x.shape[0]
    _sizes(batch)
    d = _ssm_dims(typ, x, dt, B, softplus)
    px, pdt, pA, pB, pC, pD, pbias = _ssm_inputs(x, dt, A, B, C, D, dt_bias, (batch,), d, dev)
    shape = (batch, d.heads, d.states, d.width)
    s0 = _dense(state, "state", shape, torch.float32, dev)
    if s0 is None:
        raise TypeError("state must be a torch.Tensor")
    s1 = s0 if new_state is None else _dense(new_state, "new_state", shape, torch.float32, dev)
    with _On(dev, stream) as s:
        y, py = _new_rows(y, "y", (batch,), (d.heads, d.width), x, dev)
        for r in (px, pdt, pB, pC, py):
            _token(r)
        st = lib.mamba2_ssm_step(batch, d, px, pdt, pA, pB, pC, pD, pbias, s0, py, s1, s)
    if st == _EOVERLAP:
        raise ValueError("y or new_state overlaps another tensor of the call")
    _raise(st, "mamba2_ssm_step")
    return y


# ----------------------------------------------------------------- gradients
def _grad_table(grads, out):
    """(the mamba2_grad table as bytes, its length, the first gradient)"""
    if torch is None:
        _load()
    grads = list(grads)
    if not grads:
        raise ValueError("no gradients")
    outs = grads if out is None else list(out)
    if len(outs) != len(grads):
        raise ValueError(f"{len(outs)} outputs for {len(grads)} gradients")
    _gpu(grads[0], "grads[0]")
    index = grads[0].get_device()
    fields = []
    Tensor, types = torch.Tensor, _TYPES
    for i, (g, o) in enumerate(zip(grads, outs)):
        if not isinstance(g, Tensor) or g.get_device() != index:
            _gpu(g, f"grads[{i}]", grads[0].device)
        typ = types.get(g.dtype)
        if typ is None:
            _type(g, f"grads[{i}]")
        if not g.is_contiguous():
            raise ValueError(f"grads[{i}] must be contiguous")
        p = g.data_ptr()
        if o is g:
            fields += (p, p, g.numel(), typ)
            continue
        if not isinstance(o, Tensor) or o.get_device() != index:
            _gpu(o, f"out[{i}]", grads[0].device)
        if o.dtype is not g.dtype or o.shape != g.shape or not o.is_contiguous():
            raise ValueError(f"out[{i}] must be contiguous, of the gradient's type and shape")
        fields += (p, o.data_ptr(), g.numel(), typ)
    return struct.pack("=" + "QQqq" * len(grads), *fields), len(grads), grads[0]


def grad_norm(grads, *, norm=None, workspace=None, stream=None):
    """The global 2-norm of a list of float32 / bfloat16 tensors, as a float32 tensor without dimensions."""
    return _grads(grads, None, None, norm, workspace, stream)


def clip_grads(grads, max_norm, *, out=None, norm=None, workspace=None, stream=None):
    """Scales the gradients by min(1, max_norm / (norm + 1e-6)), norm their global 2-norm, and returns the norm.

    In place, or into the tensors of `out`.  Nothing waits for the GPU.
    """
    max_norm = float(max_norm)
    if math.isnan(max_norm) or max_norm < 0:
        raise ValueError(f"max_norm must not be negative (got {max_norm})")
    return _grads(grads, max_norm, out, norm, workspace, stream)


def _grads(grads, max_norm, out, norm, workspace, stream):
    table, count, first = _grad_table(grads, out)
    dev = first.device
    with _On(dev, stream) as s:
        if norm is None:
            norm = first.new_empty((), dtype=torch.float32)
        else:
            _gpu(norm, "norm", dev)
            if norm.dtype != torch.float32 or norm.numel() != 1:
                raise ValueError("norm must be one float32")
        workspace, nbytes = _workspace(workspace, lib.mamba2_grad_workspace_bytes(table, count), first, dev)
        if max_norm is None:
            st = lib.mamba2_grad_norm(table, count, norm.data_ptr(), _ptr(workspace), nbytes, s)
        else:
            st = lib.mamba2_clip_grads(table, count, max_norm, norm.data_ptr(), _ptr(workspace), nbytes, s)
    _raise(st, "mamba2_grad_norm" if max_norm is None else "mamba2_clip_grads")
    return norm
