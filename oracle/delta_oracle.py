"""The gated delta rule and the group norm in float64 on the CPU: the rule token by token, no chunks.

Independent of the kernels and of the benchmark's plain forms.
"""
from __future__ import annotations

import torch


# -------------------------------------------------------------- delta rule
def _heads(x, heads):
    """[L, G, K] -> [L, H, K]: neighbouring heads share a query and key."""
    return x.double().repeat_interleave(heads // x.shape[1], 1)


def _moved(state, k, v, g, beta):
    """(the faded state, what is missing from the value, the state after the token); all of one token"""
    faded = torch.exp(g)[:, None, None] * state
    missing = v - torch.einsum("hkv,hk->hv", faded, k)
    return faded, missing, faded + k[:, :, None] * (beta[:, None] * missing)[:, None, :]


def delta(q, k, v, g, beta, scale, state):
    """One sequence: q, k [L, G, K], v [L, H, V], g, beta [L, H], state [H, K, V] or None -> (y, final state)."""
    heads = v.shape[1]
    q, k, v, g, beta = _heads(q, heads), _heads(k, heads), v.double(), g.double(), beta.double()
    state = torch.zeros(heads, q.shape[2], v.shape[2], dtype=torch.float64) if state is None else state.double()
    y = torch.zeros_like(v)
    for t in range(v.shape[0]):
        state = _moved(state, k[t], v[t], g[t], beta[t])[2]
        y[t] = scale * torch.einsum("hkv,hk->hv", state, q[t])
    return y, state


def delta_grads(q, k, v, g, beta, scale, state, d_y, d_final):
    """dict(d_q, d_k, d_v, d_g, d_beta, d_state) of one sequence, by the recurrence's reverse."""
    groups, heads = q.shape[1], v.shape[1]
    q, k, v, g, beta = _heads(q, heads), _heads(k, heads), v.double(), g.double(), beta.double()
    d_y = d_y.double()
    state = torch.zeros(heads, q.shape[2], v.shape[2], dtype=torch.float64) if state is None else state.double()
    states = [state]
    for t in range(v.shape[0]):
        states.append(_moved(states[-1], k[t], v[t], g[t], beta[t])[2])
    d_q, d_k, d_v = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    d_g, d_beta = torch.zeros_like(g), torch.zeros_like(beta)
    d_s = torch.zeros_like(state) if d_final is None else d_final.double()
    for t in range(v.shape[0] - 1, -1, -1):
        faded, missing, after = _moved(states[t], k[t], v[t], g[t], beta[t])
        d_q[t] = scale * torch.einsum("hkv,hv->hk", after, d_y[t])
        d_s = d_s + scale * q[t][:, :, None] * d_y[t][:, None, :]
        d_u = torch.einsum("hkv,hk->hv", d_s, k[t])
        d_beta[t] = (d_u * missing).sum(-1)
        d_v[t] = beta[t][:, None] * d_u
        d_k[t] = torch.einsum("hkv,hv->hk", d_s, beta[t][:, None] * missing) - torch.einsum("hkv,hv->hk", faded, d_v[t])
        d_s = d_s - k[t][:, :, None] * d_v[t][:, None, :]
        d_g[t] = (d_s * faded).sum((1, 2))
        d_s = torch.exp(g[t])[:, None, None] * d_s
    shared = lambda d: d.unflatten(1, (groups, heads // groups)).sum(2)
    return dict(d_q=shared(d_q), d_k=shared(d_k), d_v=d_v, d_g=d_g, d_beta=d_beta, d_state=d_s)


# -------------------------------------------------------------- group norm
def _parameter(p, groups, width, without):
    if p is None:
        return torch.full((groups, width), without, dtype=torch.float64)
    return p.double().reshape(-1, width).expand(groups, width)


def _norm_parts(x, weight, bias, gate, groups, form, centered, eps):
    rows, channels = x.shape
    width = channels // groups
    cut = lambda t: t.double().reshape(rows, groups, width)
    x = cut(x)
    z = cut(gate) if gate is not None else None
    h = x * z * torch.sigmoid(z) if form == "gate_first" else x
    c = h - h.mean(-1, keepdim=True) if centered else h
    r = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    n = c * r
    w = _parameter(weight, groups, width, 1.0)
    return x, z, n, r, w, n * w + _parameter(bias, groups, width, 0.0)


def group_norm(x, weight, bias, gate, groups, form, centered, eps):
    """x [rows, channels], form plain, silu, gated or gate_first -> y"""
    _, z, _, _, _, o = _norm_parts(x, weight, bias, gate, groups, form, centered, eps)
    if form == "silu":
        o = o * torch.sigmoid(o)
    elif form == "gated":
        o = o * z * torch.sigmoid(z)
    return o.reshape(x.shape)


def _d_silu(v):
    s = torch.sigmoid(v)
    return s * (1 + v * (1 - s))


def group_norm_grads(x, weight, bias, gate, groups, form, centered, eps, d_y):
    """dict(d_x, d_weight, d_bias, d_gate), None where there is no such input"""
    shape, width = x.shape, x.shape[1] // groups
    x, z, n, r, w, o = _norm_parts(x, weight, bias, gate, groups, form, centered, eps)
    d = d_y.double().reshape(n.shape)
    d_z = None
    if form == "silu":
        d = d * _d_silu(o)
    elif form == "gated":
        d_z = d * o * _d_silu(z)
        d = d * z * torch.sigmoid(z)
    d_w, d_b = (d * n).sum(0), d.sum(0)
    if weight is not None and weight.numel() == width:
        d_w, d_b = d_w.sum(0), d_b.sum(0)
    d_n = d * w
    d_h = d_n - n * (d_n * n).mean(-1, keepdim=True)
    if centered:
        d_h = d_h - d_n.mean(-1, keepdim=True)
    d_h = d_h * r
    if form == "gate_first":
        d_z = d_h * x * _d_silu(z)
        d_h = d_h * z * torch.sigmoid(z)
    return dict(d_x=d_h.reshape(shape), d_weight=None if weight is None else d_w.reshape(-1),
                d_bias=None if bias is None else d_b.reshape(-1), d_gate=None if d_z is None else d_z.reshape(shape))
