"""The selective layer's operators together, as a program runs them: a training step, prompts and then tokens,
captured graphs, several streams.  On an MI355X.
"""
from __future__ import annotations

import threading

import pytest
import torch

import bwd_mamba2_scan_amd as m2
from oracle import selective_oracle as orc
from tests.inputs import make_inputs
from tests.selective import U, gen, half_step
from tests.test_parity_gpu import _to_dev

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
H, P, G, N, W = 6, 32, 2, 24, 4
C = H * P + 2 * G * N


def _weights(seed, dev=DEV):
    g = gen(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    return {k: v.to(dev) for k, v in dict(conv_w=r(C, W) / 2, conv_b=r(C) / 4, A=-torch.exp(r(H)), D=r(H),
                                          dt_bias=r(H) - 2).items()}


def _tokens(seed, batch, L, typ):
    g = gen(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(typ).to(DEV)
    # the projection gives the convolution's channels and the step sizes side by side
    return r(batch, L, C + H), r(batch, L, H, P)


def _split(mixed):
    x, b, c = mixed.split((H * P, G * N, G * N), -1)
    return x.unflatten(-1, (H, P)), b.unflatten(-1, (G, N)), c.unflatten(-1, (G, N))


def _step(w, proj, d_y, bufs=None, stream=None):
    """Forward and backward of the layer's operators; every output in a dict."""
    b = bufs or {}
    u, dt = proj[..., :C], proj[..., C:]
    kw = dict(stream=stream)
    mixed, _ = m2.conv_fwd(u, w["conv_w"], w["conv_b"], y=b.get("mixed"), **kw)
    x, Bm, Cm = _split(mixed)
    sc = dict(D=w["D"], dt_bias=w["dt_bias"], **kw)
    y, _ = m2.ssm_fwd(x, dt, w["A"], Bm, Cm, y=b.get("y"), workspace=b.get("ws_fwd"), **sc)
    d_proj = torch.empty_like(proj) if "d_proj" not in b else b["d_proj"]
    d_mixed = torch.empty_like(mixed) if "d_mixed" not in b else b["d_mixed"]
    d_x, d_B, d_C = _split(d_mixed)
    g = m2.ssm_bwd(x, dt, w["A"], Bm, Cm, d_y, out=dict(d_x=d_x, d_B=d_B, d_C=d_C, d_dt=d_proj[..., C:], **b.get("vec", {})),
                   workspace=b.get("ws_bwd"), **sc)
    cg = m2.conv_bwd(u, w["conv_w"], d_mixed, w["conv_b"], out=dict(d_x=d_proj[..., :C], **b.get("conv", {})),
                     workspace=b.get("ws_conv"), **kw)
    grads = [cg["d_weight"], cg["d_bias"], g["d_A"], g["d_D"], g["d_dt_bias"]]
    norm = m2.clip_grads(grads, 0.1, norm=b.get("norm"), workspace=b.get("ws_clip"), **kw)
    return dict(y=y, d_proj=d_proj, norm=norm, **{f"g{i}": v for i, v in enumerate(grads)})


def _bufs(w, proj):
    """Everything a captured step writes, allocated beforehand by one eager step's sizes."""
    f = lambda *s: torch.empty(s, device=DEV)
    lead, typ = proj.shape[:2], proj.dtype
    e = lambda *s: torch.empty(*lead, *s, dtype=typ, device=DEV)
    big = lambda: torch.empty(1 << 24, device=DEV)
    return dict(mixed=e(C), y=e(H, P), d_proj=e(C + H), d_mixed=e(C), norm=f(), ws_fwd=big(), ws_bwd=big(),
                ws_conv=big(), ws_clip=big(), vec=dict(d_A=f(H), d_D=f(H), d_dt_bias=f(H)),
                conv=dict(d_weight=f(C, W), d_bias=f(C)))


@pytest.mark.parametrize("typ", [torch.float32, torch.bfloat16])
def test_training_step(typ):
    """The chain's gradients against the oracle's, stage by stage on the values the stage was given."""
    batch, L = 2, 130
    w = _weights(0)
    proj, d_y = _tokens(1, batch, L, typ)
    out = _step(w, proj, d_y)
    mixed, _ = m2.conv_fwd(proj[..., :C], w["conv_w"], w["conv_b"])
    cpu = lambda v: v.cpu()
    x, Bm, Cm = (cpu(v) for v in _split(mixed))
    dt = cpu(proj[..., C:])
    cw = {k: cpu(v) for k, v in w.items()}
    grads = [0, 0, 0, 0, 0]
    rel = 2.0 ** -7 if typ == torch.bfloat16 else 2.0 ** -16   # of the norm: a few half steps of the type
    for s in range(batch):
        args = (x[s], dt[s], cw["A"], Bm[s], Cm[s], cw["D"], cw["dt_bias"], True, None)
        y, _ = orc.scan(*args)
        assert float((cpu(out["y"][s]).double() - y).norm()) <= rel * float(y.norm())
        e = orc.scan_grads(*args, cpu(d_y[s]), None)
        d_mixed = torch.cat([e[k].flatten(1) for k in ("d_x", "d_B", "d_C")], 1)
        c = orc.conv_grads(cpu(proj[s, :, :C]), cw["conv_w"], cw["conv_b"], None, True, d_mixed, None)
        want = torch.cat([c["d_x"], e["d_dt"]], 1)
        assert float((cpu(out["d_proj"][s]).double() - want).norm()) <= 2 * rel * float(want.norm())
        for i, v in enumerate((c["d_weight"], c["d_bias"], e["d_A"], e["d_D"], e["d_dt_bias"])):
            grads[i] = grads[i] + v
    norm, clipped = orc.clip(grads, 0.1)
    assert abs(float(out["norm"]) - norm) <= rel * norm
    for i, v in enumerate(clipped):
        assert float((cpu(out[f"g{i}"]).double() - v).norm()) <= 2 * rel * float(v.norm()), i
    assert norm > 0.1
    total = sum(float((cpu(out[f"g{i}"]).double() ** 2).sum()) for i in range(5)) ** 0.5
    assert abs(total - 0.1) <= 1e-5


def test_clipping_the_temporal_scans_gradients():
    """mamba2_scan_bwd's weight gradients go straight into clip_grads."""
    inp = _to_dev(make_inputs(70, 5, 128, 32, seed=3))
    _, saved = m2.fwd(inp["h_history"], inp["h_s2"], inp["W_A"], inp["W_B"], inp["W_C"])
    g = m2.bwd(inp["h_history"], inp["h_s2"], saved, inp["d_context"])
    grads = [g[k] for k in ("dW_A", "dW_B", "dW_C")]
    norm, want = orc.clip([v.cpu() for v in grads], 1.0)
    n = m2.clip_grads(grads, 1.0)
    assert abs(float(n) - norm) <= 1.01 * U * norm
    for v, e in zip(grads, want):
        assert bool(((v.cpu().double() - e).abs() <= 3.01 * U * e.abs()).all())


@pytest.mark.parametrize("typ", [torch.float32, torch.bfloat16])
def test_prompts_then_tokens(typ):
    """Packed prompts through both operators, their states handed to single tokens: as one longer run gives."""
    lengths, more = [40, 1, 97], 5
    w = _weights(2)
    proj, _ = _tokens(4, len(lengths), max(lengths) + more, typ)
    whole_mixed, _ = m2.conv_fwd(proj[..., :C], w["conv_w"], w["conv_b"])
    x, Bm, Cm = _split(whole_mixed)
    sc = dict(D=w["D"], dt_bias=w["dt_bias"])
    whole, _ = m2.ssm_fwd(x, proj[..., C:], w["A"], Bm, Cm, **sc)

    packed = torch.cat([proj[i, :n] for i, n in enumerate(lengths)])
    off = torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    mixed, tail = m2.conv_fwd(packed[:, :C], w["conv_w"], w["conv_b"], offsets=off, want_final_state=True)
    x, Bm, Cm = _split(mixed)
    y, state = m2.ssm_fwd(x, packed[:, C:], w["A"], Bm, Cm, offsets=off, want_final_state=True, **sc)
    rel = 2.0 ** -7 if typ == torch.bfloat16 else 2.0 ** -18
    size = float(whole.float().abs().max())
    for i, n in enumerate(lengths):
        assert torch.equal(mixed[off[i]:off[i + 1]], whole_mixed[i, :n])
        assert float((y[off[i]:off[i + 1]].float() - whole[i, :n].float()).abs().max()) <= rel * size
    for k in range(more):
        token = torch.stack([proj[i, n + k] for i, n in enumerate(lengths)])
        m = m2.conv_step(token[:, :C], w["conv_w"], tail, w["conv_b"])
        x, Bm, Cm = _split(m)
        y = m2.ssm_step(x, token[:, C:], w["A"], Bm, Cm, state, **sc)
        for i, n in enumerate(lengths):
            assert torch.equal(m[i], whole_mixed[i, n + k])
            assert float((y[i].float() - whole[i, n + k].float()).abs().max()) <= rel * size


@pytest.mark.parametrize("typ,L", [(torch.float32, 90), (torch.bfloat16, 800)])
def test_captured_step_replays(typ, L):
    """A captured training step, replayed on changing inputs between eager work: bitwise the eager result."""
    w = _weights(5)
    proj, d_y = _tokens(6, 2, L, typ)
    bufs = _bufs(w, proj)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(w, proj, d_y, bufs)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _step(w, proj, d_y, bufs)
    for seed in (7, 8, 9, 10):
        a, b = _tokens(seed, 2, L, typ)
        proj.copy_(a)
        d_y.copy_(b)
        graph.replay()
        got = {k: v.clone() for k, v in out.items()}
        torch.cuda.synchronize()
        want = _step(w, a, b)
        for k in want:
            assert torch.equal(got[k], want[k]), (seed, k)


def test_two_graphs_and_a_token_loop():
    """Two captured steps with workspaces of their own replayed side by side on two streams, and a captured token."""
    w = _weights(11)
    ins = [_tokens(12 + i, 1, 700, torch.bfloat16) for i in range(2)]
    want = [_step(w, *i) for i in ins]
    graphs, outs, kept = [], [], []
    for i in ins:
        bufs = _bufs(w, i[0])
        kept.append(bufs)  # a graph's buffers live as long as it does: capturing releases unused memory
        _step(w, *i, bufs)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_step(w, *i, bufs))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in ins]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, e in zip(outs, want):
            for k in e:
                assert torch.equal(o[k], e[k]), k

    token, _ = _tokens(20, 3, 1, torch.bfloat16)
    token = token[:, 0].contiguous()
    tail, state = torch.zeros(3, W - 1, C, dtype=torch.bfloat16, device=DEV), torch.zeros(3, H, N, P, device=DEV)
    y, m = torch.empty(3, H, P, dtype=torch.bfloat16, device=DEV), torch.empty(3, C, dtype=torch.bfloat16, device=DEV)

    def one(tail, state, y=None, m=None):
        m = m2.conv_step(token[:, :C], w["conv_w"], tail, w["conv_b"], y=m)
        x, Bm, Cm = _split(m)
        return m2.ssm_step(x, token[:, C:], w["A"], Bm, Cm, state, D=w["D"], dt_bias=w["dt_bias"], y=y)

    one(tail, state, y, m)
    tail.zero_()
    state.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        one(tail, state, y, m)
    tail.zero_()
    state.zero_()
    tail2, state2 = tail.clone(), state.clone()
    for seed in range(4):
        token.copy_(_tokens(30 + seed, 3, 1, torch.bfloat16)[0][:, 0])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(one(tail2, state2), y) and torch.equal(state2, state) and torch.equal(tail2, tail)


def test_streams_and_threads():
    """The stream argument, and two host threads enqueuing at once on streams of their own."""
    w = _weights(40)
    proj, d_y = _tokens(41, 2, 300, torch.bfloat16)
    want = _step(w, proj, d_y)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = _step(w, proj, d_y, dict(d_proj=torch.empty_like(proj), d_mixed=torch.empty(2, 300, C, dtype=proj.dtype, device=DEV)),
                stream=side)
    side.synchronize()
    for k in want:
        assert torch.equal(got[k], want[k]), k
    results = {}

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(5):
                results[i] = _step(w, proj, d_y)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        for k in want:
            assert torch.equal(results[i][k], want[k]), (i, k)


def test_offsets_out_of_order_stay_inside():
    """Offsets that are not in order: unspecified results, but nothing outside the given tensors is written."""
    rows, mark = 200, 55.0
    w = _weights(50)
    proj, d_y = _tokens(51, 1, rows, torch.bfloat16)
    proj, d_y = proj[0], d_y[0]
    for offsets in ([0, 150, 40, 500], [-70, 30, 2000000000, 200], [199, 0, -5, 201]):
        print("offsets", offsets, flush=True)
        off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        wide = torch.full((rows + 64, C), mark, dtype=torch.bfloat16, device=DEV)
        mixed, _ = m2.conv_fwd(proj[:, :C], w["conv_w"], w["conv_b"], offsets=off, y=wide[32:-32], want_final_state=True)
        x, Bm, Cm = _split(torch.zeros_like(mixed))
        ywide = torch.full((rows + 64, H, P), mark, dtype=torch.bfloat16, device=DEV)
        m2.ssm_fwd(x, proj[:, C:], w["A"], Bm, Cm, offsets=off, y=ywide[32:-32], want_final_state=True)
        m2.ssm_bwd(x, proj[:, C:], w["A"], Bm, Cm, d_y, offsets=off)
        m2.conv_bwd(proj[:, :C], w["conv_w"], wide[32:-32], w["conv_b"], offsets=off)
        torch.cuda.synchronize()
        for t in (wide, ywide):
            assert bool((t[:32] == mark).all()) and bool((t[-32:] == mark).all())
