"""The selective layer's operators in float64 on the CPU: plain loops over the tokens, no chunks.

Independent of the kernels and of the benchmark's plain forms.  Every function
also has an absolute form (absolute=True): the same sums over the absolute
values of their terms, which rounding errors of any order of summation are
bounded by.
"""
from __future__ import annotations

import torch


def _abs(v, absolute):
    return v.abs() if absolute and v is not None else v


# ------------------------------------------------------------ convolution
def conv(x, weight, bias, state, silu, absolute=False):
    """One sequence: x [L, C], state [W - 1, C] -> (y, pre-activation, last W - 1 inputs)."""
    x, weight, bias, state = (_abs(None if v is None else v.double(), absolute) for v in (x, weight, bias, state))
    channels, taps = weight.shape
    if state is None:
        state = torch.zeros(taps - 1, channels, dtype=torch.float64)
    source = torch.cat([state, x])
    pre = torch.zeros_like(x)
    for t in range(x.shape[0]):
        for k in range(taps):
            pre[t] += weight[:, k] * source[t + k]
    if bias is not None:
        pre = pre + bias
    y = pre * torch.sigmoid(pre) if silu and not absolute else pre
    return y, pre, source[x.shape[0]:]


def conv_grads(x, weight, bias, state, silu, d_y, d_final, absolute=False):
    """dict(d_x, d_weight, d_bias, d_state) of one sequence."""
    _, pre, _ = conv(x, weight, bias, state, silu)
    d = d_y.double()
    if silu:
        s = torch.sigmoid(pre)
        d = d * (s + pre * s * (1 - s))
    d, x, weight = (_abs(v.double(), absolute) for v in (d, x, weight))
    channels, taps = weight.shape
    length = x.shape[0]
    state = torch.zeros(taps - 1, channels, dtype=torch.float64) if state is None else _abs(state.double(), absolute)
    source = torch.cat([state, x])
    d_source = torch.zeros_like(source)
    if d_final is not None:
        d_source[length:] += _abs(d_final.double(), absolute)
    d_weight = torch.zeros_like(weight)
    for t in range(length):
        for k in range(taps):
            d_source[t + k] += weight[:, k] * d[t]
            d_weight[:, k] += d[t] * source[t + k]
    return dict(d_x=d_source[taps - 1:], d_weight=d_weight, d_bias=d.sum(0), d_state=d_source[: taps - 1])


# ------------------------------------------------------------------- scan
def steps(dt, dt_bias, softplus):
    raw = dt.double() + (0 if dt_bias is None else dt_bias.double())
    return torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw


def scan(x, dt, A, B, C, D, dt_bias, softplus, state, absolute=False):
    """One sequence: x [L, H, P], dt [L, H], B, C [L, G, N], state [H, N, P] -> (y, states [L + 1, H, N, P])."""
    d = _abs(steps(dt, dt_bias, softplus), absolute)
    decay = torch.exp(steps(dt, dt_bias, softplus) * A.double())
    ratio = x.shape[1] // B.shape[1]
    x, B, C, D, state = (_abs(None if v is None else v.double(), absolute) for v in (x, B, C, D, state))
    length, heads, width = x.shape
    b, c = B.repeat_interleave(ratio, 1), C.repeat_interleave(ratio, 1)
    s = torch.zeros(heads, B.shape[2], width, dtype=torch.float64) if state is None else state
    states, y = [s], torch.zeros_like(x)
    for t in range(length):
        s = decay[t, :, None, None] * s + d[t, :, None, None] * b[t, :, :, None] * x[t, :, None, :]
        y[t] = (s * c[t, :, :, None]).sum(1)
        states.append(s)
    if D is not None:
        y = y + D[:, None] * x
    return y, torch.stack(states)


def scan_grads(x, dt, A, B, C, D, dt_bias, softplus, state, d_y, d_final, absolute=False):
    """dict of the gradients of one sequence."""
    _, states = scan(x, dt, A, B, C, D, dt_bias, softplus, state, absolute)
    raw = dt.double() + (0 if dt_bias is None else dt_bias.double())
    d = steps(dt, dt_bias, softplus)
    decay = torch.exp(d * A.double())
    slope = torch.sigmoid(raw) if softplus else torch.ones_like(raw)
    groups = B.shape[1]
    ratio = x.shape[1] // groups
    d, A, x, B, C, D, d_y, d_final = (_abs(None if v is None else v.double(), absolute)
                                      for v in (d, A, x, B, C, D, d_y, d_final))
    length, heads, width = x.shape
    b, c = B.repeat_interleave(ratio, 1), C.repeat_interleave(ratio, 1)
    g = torch.zeros_like(states[0]) if d_final is None else d_final.clone()
    d_x, d_d, d_b, d_c = (torch.zeros_like(v) for v in (x, d, b, c))
    d_A = torch.zeros_like(A)
    for t in range(length - 1, -1, -1):
        g = g + c[t, :, :, None] * d_y[t, :, None, :]
        d_c[t] = (states[t + 1] * d_y[t, :, None, :]).sum(2)
        gb = (g * b[t, :, :, None]).sum(1)
        d_x[t] = d[t, :, None] * gb
        d_b[t] = (g * x[t, :, None, :]).sum(2) * d[t, :, None]
        m = (g * states[t]).sum((1, 2)) * decay[t]
        d_d[t] = (gb * x[t]).sum(1) + A * m
        d_A += d[t] * m
        g = decay[t, :, None, None] * g
    if D is not None:
        d_x = d_x + D[:, None] * d_y
    d_dt = d_d * slope
    fold = (length, groups, ratio, B.shape[2])
    return dict(d_x=d_x, d_dt=d_dt, d_A=d_A, d_B=d_b.reshape(fold).sum(2), d_C=d_c.reshape(fold).sum(2),
                d_D=(d_y * x).sum((0, 2)), d_dt_bias=d_dt.sum(0), d_state=g)


# -------------------------------------------------------------- gradients
def clip(grads, max_norm):
    norm = sum(float((g.double() ** 2).sum()) for g in grads) ** 0.5
    factor = min(1.0, max_norm / (norm + 1e-6))
    return norm, [g.double() * factor for g in grads]
