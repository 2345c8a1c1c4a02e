"""A layer of the gated delta rule, as a program runs it: convolution, norms of queries and keys, the rule, the gated
norm and the clipping of the gradients; a training step, prompts and then tokens, captured graphs, several streams.
On an MI355X.
"""
from __future__ import annotations

import threading

import pytest
import torch

import bwd_mamba2_scan_amd as m2
from oracle import delta_oracle as orc
from oracle import selective_oracle as sel

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
H, V, G, K, W = 4, 32, 2, 24, 4
QK = G * K
C = 2 * QK + H * V
EPS = 1e-6


def _weights(seed, dev=DEV):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    return {k: v.to(dev) for k, v in dict(conv_w=r(C, W) / 2, conv_b=r(C) / 4, unit=torch.full((K,), K ** -0.5),
                                          norm=1 + 0.2 * r(V)).items()}


def _tokens(seed, batch, L, typ, dev=DEV):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    # one projection gives the convolution's channels and the output's gate
    return dict(proj=r(batch, L, C + H * V).to(typ).to(dev), g=(-torch.rand(batch, L, H, generator=g)).to(dev),
                beta=torch.sigmoid(r(batch, L, H)).to(dev), d_out=r(batch, L, H * V).to(typ).to(dev))


def _parts(mixed):
    return mixed[..., :QK], mixed[..., QK:2 * QK], mixed[..., 2 * QK:]


def _forward(w, t, b, kw, conv=None, rule=None):
    """The layer of a batch: everything that its backward needs."""
    conv, rule = conv or {}, rule or {}
    mixed, tail = m2.conv_fwd(t["proj"][..., :C], w["conv_w"], w["conv_b"], y=b.get("mixed"), **conv, **kw)
    q0, k0, v = _parts(mixed)
    off = {"offsets": rule["offsets"]} if "offsets" in rule else {}
    q = m2.group_norm_fwd(q0, w["unit"], groups=G, eps=EPS, y=b.get("q"), **off, **kw)
    k = m2.group_norm_fwd(k0, w["unit"], groups=G, eps=EPS, y=b.get("k"), **off, **kw)
    cut = lambda x, n: x.unflatten(-1, (n, -1))
    args = (cut(q, G), cut(k, G), cut(v, H), t["g"], t["beta"])
    y, state = m2.delta_fwd(*args, y=b.get("y"), workspace=b.get("ws_fwd"), **rule, **kw)
    out = m2.group_norm_fwd(y.flatten(-2), w["norm"], groups=H, gate=t["proj"][..., C:], y=b.get("out"), **off, **kw)
    return mixed, tail, args, y, state, out


def _step(w, t, bufs=None, stream=None):
    """Forward and backward of the layer and the clipped gradients; every output in a dict."""
    b, kw = bufs or {}, dict(stream=stream)
    mixed, _, args, y, _, out = _forward(w, t, b, kw)
    q0, k0, _ = _parts(mixed)
    d_proj = b["d_proj"] if "d_proj" in b else torch.empty_like(t["proj"])
    d_mixed = b["d_mixed"] if "d_mixed" in b else torch.empty_like(mixed)
    d_q0, d_k0, d_v = _parts(d_mixed)
    n = m2.group_norm_bwd(y.flatten(-2), t["d_out"], w["norm"], groups=H, gate=t["proj"][..., C:],
                          out=dict(d_gate=d_proj[..., C:], **b.get("norm_out", {})), workspace=b.get("ws_norm"), **kw)
    g = m2.delta_bwd(*args, n["d_x"].unflatten(-1, (H, V)), out=dict(d_v=d_v.unflatten(-1, (H, V)), **b.get("rule_out", {})),
                     workspace=b.get("ws_bwd"), **kw)
    for d, x, name in ((d_q0, q0, "d_q"), (d_k0, k0, "d_k")):
        m2.group_norm_bwd(x, g[name].flatten(-2), w["unit"], groups=G, eps=EPS,
                          out=dict(d_x=d, d_weight=b[f"unit_{name}"]) if b else dict(d_x=d), workspace=b.get("ws_unit"), **kw)
    c = m2.conv_bwd(t["proj"][..., :C], w["conv_w"], d_mixed, w["conv_b"], out=dict(d_x=d_proj[..., :C], **b.get("conv", {})),
                    workspace=b.get("ws_conv"), **kw)
    grads = [c["d_weight"], c["d_bias"], n["d_weight"]]
    norm = m2.clip_grads(grads, 0.1, norm=b.get("norm"), workspace=b.get("ws_clip"), **kw)
    return dict(out=out, d_proj=d_proj, d_g=g["d_g"], d_beta=g["d_beta"], norm=norm, **{f"w{i}": v for i, v in enumerate(grads)})


def _bufs(t):
    """Everything that a captured step writes, allocated beforehand."""
    lead, typ = t["proj"].shape[:2], t["proj"].dtype
    e = lambda *s: torch.empty(*lead, *s, dtype=typ, device=DEV)
    f = lambda *s: torch.empty(s, device=DEV)
    big = lambda: torch.empty(1 << 24, device=DEV)
    return dict(mixed=e(C), q=e(QK), k=e(QK), y=e(H, V), out=e(H * V), d_proj=e(C + H * V), d_mixed=e(C),
                norm_out=dict(d_x=e(H * V), d_weight=f(V)), unit_d_q=f(K), unit_d_k=f(K), norm=f(),
                rule_out=dict(d_q=e(G, K), d_k=e(G, K), d_g=torch.empty(*lead, H, device=DEV),
                              d_beta=torch.empty(*lead, H, device=DEV)),
                conv=dict(d_weight=f(C, W), d_bias=f(C)),
                **{"ws_" + n: big() for n in ("fwd", "bwd", "norm", "unit", "conv", "clip")})


@pytest.mark.parametrize("typ", [torch.float32, torch.bfloat16])
def test_training_step(typ):
    """The chain's gradients against the oracle's, stage by stage on the values that the stage was given."""
    batch, L = 2, 130
    w, t = _weights(0), _tokens(1, batch, L, typ)
    out = _step(w, t)
    mixed, _, args, y, _, _ = _forward(w, t, {}, {})
    cpu = lambda v: v.cpu()
    cw = {k: cpu(v) for k, v in w.items()}
    rel = 2.0 ** -7 if typ == torch.bfloat16 else 2.0 ** -16   # of the norm: a few half steps of the type
    grads = [0, 0, 0]

    def near(got, want, times, what):
        assert float((cpu(got).double() - want).norm()) <= times * rel * float(want.norm()), what

    for s in range(batch):
        q, k, v, g, beta = (cpu(a[s]) for a in args)
        want, _ = orc.delta(q, k, v, g, beta, K ** -0.5, None)
        near(y[s], want, 1, "y")
        gate = cpu(t["proj"][s, :, C:])
        near(out["out"][s], orc.group_norm(cpu(y[s]).flatten(1), cw["norm"], None, gate, H, "gated", False, 1e-5), 1, "out")
        n = orc.group_norm_grads(cpu(y[s]).flatten(1), cw["norm"], None, gate, H, "gated", False, 1e-5, cpu(t["d_out"][s]))
        near(out["d_proj"][s, :, C:], n["d_gate"], 1, "d_gate")
        e = orc.delta_grads(q, k, v, g, beta, K ** -0.5, None, n["d_x"].unflatten(1, (H, V)), None)
        near(out["d_g"][s], e["d_g"], 2, "d_g")
        near(out["d_beta"][s], e["d_beta"], 2, "d_beta")
        q0, k0, _ = _parts(cpu(mixed[s]))
        d_q0, d_k0 = (orc.group_norm_grads(x, cw["unit"], None, None, G, "plain", False, EPS, e[n_].flatten(1))["d_x"]
                      for x, n_ in ((q0, "d_q"), (k0, "d_k")))
        d_mixed = torch.cat([d_q0, d_k0, e["d_v"].flatten(1)], 1)
        c = sel.conv_grads(cpu(t["proj"][s, :, :C]), cw["conv_w"], cw["conv_b"], None, True, d_mixed, None)
        near(out["d_proj"][s, :, :C], c["d_x"], 3, "d_proj")
        for i, v_ in enumerate((c["d_weight"], c["d_bias"], n["d_weight"])):
            grads[i] = grads[i] + v_
    norm, clipped = sel.clip(grads, 0.1)
    assert norm > 0.1 and abs(float(out["norm"]) - norm) <= 2 * rel * norm
    for i, v_ in enumerate(clipped):
        near(out[f"w{i}"], v_, 4, i)


@pytest.mark.parametrize("typ", [torch.float32, torch.bfloat16])
def test_prompts_then_tokens(typ):
    """Packed prompts through the layer, their states handed to single tokens: as one longer run gives."""
    lengths, more = [40, 1, 97], 5
    w = _weights(2)
    t = _tokens(3, len(lengths), max(lengths) + more, typ)
    whole = _forward(w, t, {}, {})[-1]
    pack = lambda x: torch.cat([x[i, :n] for i, n in enumerate(lengths)])
    off = torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    packed = {k: pack(v) for k, v in t.items()}
    _, tail, _, _, state, out = _forward(w, packed, {}, {}, dict(offsets=off, want_final_state=True),
                                         dict(offsets=off, want_final_state=True))
    rel = 2.0 ** -6 if typ == torch.bfloat16 else 2.0 ** -17
    size = float(whole.float().abs().max())
    for i, n in enumerate(lengths):
        assert float((out[off[i]:off[i + 1]].float() - whole[i, :n].float()).abs().max()) <= rel * size
    for j in range(more):
        tok = {k: torch.stack([v[i, n + j] for i, n in enumerate(lengths)]) for k, v in t.items()}
        m = m2.conv_step(tok["proj"][:, :C], w["conv_w"], tail, w["conv_b"])
        q0, k0, v = _parts(m)
        q = m2.group_norm_fwd(q0, w["unit"], groups=G, eps=EPS).unflatten(-1, (G, K))
        k = m2.group_norm_fwd(k0, w["unit"], groups=G, eps=EPS).unflatten(-1, (G, K))
        y = m2.delta_step(q, k, v.unflatten(-1, (H, V)), tok["g"], tok["beta"], state)
        out = m2.group_norm_fwd(y.flatten(-2), w["norm"], groups=H, gate=tok["proj"][:, C:])
        for i, n in enumerate(lengths):
            assert float((out[i].float() - whole[i, n + j].float()).abs().max()) <= rel * size


@pytest.mark.parametrize("typ,L", [(torch.float32, 90), (torch.bfloat16, 1300)])
def test_captured_step_replays(typ, L):
    """A captured training step, replayed on changing inputs between eager work: bitwise the eager result."""
    w, t = _weights(4), _tokens(5, 1, L, typ)
    bufs = _bufs(t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(w, t, bufs)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _step(w, t, bufs)
    for seed in (6, 7, 8, 9):
        new = _tokens(seed, 1, L, typ)
        for k in t:
            t[k].copy_(new[k])
        graph.replay()
        got = {k: v.clone() for k, v in out.items()}
        torch.cuda.synchronize()
        want = _step(w, new)
        for k in want:
            assert torch.equal(got[k], want[k]), (seed, k)


def test_two_graphs_side_by_side():
    """Two captured steps with workspaces of their own on two streams."""
    w = _weights(10)
    ins = [_tokens(11 + i, 1, 700, torch.bfloat16) for i in range(2)]
    want = [_step(w, t) for t in ins]
    graphs, outs, kept = [], [], []
    for t in ins:
        bufs = _bufs(t)
        kept.append(bufs)
        _step(w, t, bufs)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_step(w, t, bufs))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in ins]
    for _ in range(4):
        for g, s in zip(graphs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, e in zip(outs, want):
            for k in e:
                assert torch.equal(o[k], e[k]), k


def test_captured_token():
    """A captured token, replayed along a sequence: bitwise the eager tokens."""
    w = _weights(13)
    t = _tokens(14, 3, 6, torch.bfloat16)
    start = torch.randn(3, H, K, V, generator=torch.Generator().manual_seed(15)).to(DEV)
    tok = {k: v[:, 0].clone() for k, v in t.items()}
    state = start.clone()

    def token(tok, state, y=None):
        cut = lambda x, n: x.unflatten(-1, (n, -1))
        q0, k0, v = _parts(tok["proj"][:, :C])
        q, k = (m2.group_norm_fwd(x, w["unit"], groups=G, eps=EPS) for x in (q0, k0))
        return m2.delta_step(cut(q, G), cut(k, G), cut(v, H), tok["g"], tok["beta"], state, y=y)

    y = torch.empty(3, H, V, dtype=torch.bfloat16, device=DEV)
    token(tok, state, y)
    state.copy_(start)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token(tok, state, y)
    state.copy_(start)
    eager = start.clone()
    for i in range(6):
        for k in tok:
            tok[k].copy_(t[k][:, i])
        graph.replay()
        got = y.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, token({k: v[:, i] for k, v in t.items()}, eager))
        assert torch.equal(state, eager)


def test_other_stream_and_threads():
    """A stream that is not the current one; threads with streams of their own."""
    w = _weights(16)
    ins = [_tokens(17 + i, 1, 300, torch.bfloat16) for i in range(3)]
    want = [_step(w, t) for t in ins]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = _step(w, ins[0], stream=side)
    side.synchronize()
    for k in got:
        assert torch.equal(got[k], want[0][k]), k
    res, errors = [None] * 3, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            for _ in range(5):
                res[i] = _step(w, ins[i], stream=s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001 (reported below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for r, e in zip(res, want):
        for k in e:
            assert torch.equal(r[k], e[k]), k
