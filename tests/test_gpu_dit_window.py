"""WindowLayer and the DiT over it (attention = "window"): the last frames and the first ones, in pages that
come round.  Every step's output against the float64 oracle over the whole rollout's rows, with the bound of
the paged cache's tests (test_gpu_paged.py)."""
import math

import numpy as np
import pytest
import torch

import test_gpu_paged as T
from kv_cache_tempcache_gb300 import _lib as L
from kv_cache_tempcache_gb300.dit import DiT, DiTConfig
from kv_cache_tempcache_gb300.layer import WindowLayer

pytestmark = pytest.mark.gpu

SMALL = DiTConfig(dim=256, heads=2, ffn=512, layers=2, text_dim=256, text_len=64, frames=2, grid_h=4, grid_w=20,
                  steps=2, name="dit_small", qk_norm="head", window_frames=5, sink_frames=1)


def _check(dtype, q, k, v, at, out, lse, scale, block, window, sinks):
    """k, v [Hkv, n, d]: all rows of the rollout, the call's last."""
    pools = [x[None] for x in (k, v)]                       # one page that holds everything
    T.check_attn(dtype, q, *pools, np.zeros((1, 1), np.int32), np.array([at]), None, scale, block, window, sinks, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv,d,nq,window,sinks,block,page", [(4, 2, 64, 40, 100, 30, 0, 16), (2, 2, 128, 24, 24, 0, 8, 32),
                                                              (3, 1, 64, 7, 33, 5, 1, 16), (2, 1, 128, 1, 50, 3, 1, 64)])
def test_a_long_rollout_in_pages_that_come_round(dtype, H, Hkv, d, nq, window, sinks, block, page):
    dt = T.DT[dtype]
    steps = 12 if nq > 1 else 200
    hist = 61
    rows = hist + steps * nq
    layer = WindowLayer(H, d, nq, window, sinks, rows, 8, dtype=dt, Hkv=Hkv, block=block, page=page)
    assert layer.k.shape[0] < layer.table.shape[1]           # fewer pages than the rollout has
    x = T._rand((2, Hkv, hist, d), 1).to(dt)
    layer.load_history(x[0], x[1])
    k, v = x[0], x[1]
    for i in range(steps):
        q, kv = T._rand((H, nq, d), 10 + i, 1.5).to(dt), T._rand((2, Hkv, nq, d), 500 + i).to(dt)
        if i % 5 == 0:
            layer.step_self(q, -kv[0], -kv[1], advance=False)             # a step that is not kept leaves no trace
        out = layer.step_self(q, kv[0], kv[1])
        at = k.shape[1]
        k, v = torch.cat((k, kv[0]), 1), torch.cat((v, kv[1]), 1)
        if nq > 1 or i % 20 == 19:
            _check(dtype, q, k, v, at, out, layer.lse_self, 1 / math.sqrt(d), block, window, sinks)
        assert layer.n == at + nq
    torch.cuda.synchronize()
    assert layer.status() == 0 and layer.len.item() == rows
    layer.step_self(q, kv[0], kv[1])                         # past the rollout's length, once its last page is full
    layer.step_self(T._rand((H, nq, d), 1).to(dt), *T._rand((2, Hkv, nq, d), 2).to(dt))
    for _ in range(page // nq):
        layer.step_self(q, kv[0], kv[1])
    torch.cuda.synchronize()
    assert layer.status() == L.DEV_BAD_LEN and layer.len.item() == layer.cap == layer.n


def test_a_chunk_shorter_than_the_layers_and_refusals():
    layer = WindowLayer(2, 64, 40, 60, 10, 500, 8)
    x = T._rand((3, 2, 25, 64), 1).bfloat16()
    out = layer.step_self(*x)
    torch.cuda.synchronize()
    assert out.shape == (2, 25, 64)
    _check("bf16", x[0], x[1], x[2], 0, out, layer.lse_self[:, :25], 0.125, 0, 60, 10)
    y = T._rand((3, 2, 41, 64), 1).bfloat16()
    with pytest.raises(ValueError, match="chunk"):
        layer.step_self(*y)
    with pytest.raises(ValueError, match="same tokens"):
        layer.step_self(x[0], y[1], y[2])
    for kw in (dict(window=0), dict(sinks=-1), dict(rows=0)):
        a = dict(window=8, sinks=0, rows=100)
        a.update(kw)
        with pytest.raises(ValueError, match="positive"):
            WindowLayer(2, 64, 4, a["window"], a["sinks"], a["rows"], 8)
    with pytest.raises(L.FastarError):
        WindowLayer(2, 64, 40, 60, 10, 500, 8, page=24).step_self(*x)


def _dit(cfg=SMALL, chunks=6):
    dit = DiT(cfg, "window", seed=3, dense_capacity=chunks * cfg.tokens)
    g = torch.Generator(device="cuda").manual_seed(5)
    dit.set_text(torch.randn(cfg.text_len, cfg.text_dim, generator=g, device="cuda").bfloat16())
    return dit, g


def _noise(cfg, g):
    return torch.randn(cfg.tokens, cfg.patch_ch, generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("qk_norm", ["head", "row"])
def test_blocks_attend_over_their_window(qk_norm):
    """Six chunks of two frames, a window of five and the first: pages come round from the fifth on."""
    cfg = SMALL.replace(qk_norm=qk_norm)
    dit, g = _dit(cfg)
    frame = cfg.grid_h * cfg.grid_w
    past = [([], []) for _ in range(cfg.layers)]              # committed rows by layer

    def row_of(a, pool, n0, n1):
        r = torch.arange(n0, n1, device="cuda")
        return pool[a.table[0, r // a.page].long(), :, r % a.page].transpose(0, 1)

    last = {}

    def probe(what, i, a, q, *rest):
        if what != "self":
            return
        k, v, out = rest
        n, m = a.n, a.n + cfg.tokens
        assert a.len.item() == n and a.len_cur.item() == m
        kc, vc = row_of(a, a.k, n, m), row_of(a, a.v, n, m)
        assert torch.equal(vc, v)
        if qk_norm == "row":
            assert torch.equal(kc, k)                         # turned before the append
        else:
            # unit mean square but for the weights and bf16's rounding of each channel (2^-8 of it)
            ms = (kc.double() ** 2).mean(-1)
            w = dit.blocks[i].norm_k.double() ** 2
            assert (ms <= w.max() * 1.02).all() and (ms >= w.min() * 0.98).all()
        kk = torch.cat(past[i][0] + [kc], 1)
        vv = torch.cat(past[i][1] + [vc], 1)
        _check("bf16", q, kk, vv, n, out, a.lse_self, 1 / math.sqrt(cfg.d), 0, 5 * frame, frame)
        last[i] = (kc.clone(), vc.clone())

    for chunk in range(6):
        dit.denoise_chunk(_noise(cfg, g), use_graph=False, probe=probe)
        for i in range(cfg.layers):
            past[i][0].append(last[i][0])
            past[i][1].append(last[i][1])
    torch.cuda.synchronize()
    assert dit.status_word() == 0
    assert dit.attn[0].k.shape[0] < dit.attn[0].table.shape[1]
    with pytest.raises(L.FastarError, match="capacity"):
        dit.denoise_chunk(_noise(cfg, g), use_graph=False)


def test_norm_and_rotation_on_the_way_are_those_before():
    """A chunk through fastar_qk_norm_rope and an append that does not turn, and through one that does.  Each is
    within half a rounding, 2^-8 |y|, and 2^-19 of the pair's magnitudes of the exact value (test_gpu_qk_rope.py:
    they sum a row's squares in another order), so they are within twice that of one another."""
    cfg = SMALL
    qkv = T._rand((cfg.tokens, 3, cfg.heads, cfg.d), 1, 2.0).bfloat16()
    w = 1 + 0.1 * T._rand((2, cfg.d), 2)
    turn = dict(wq=w[0].contiguous(), wk=w[1].contiguous(), eps=cfg.eps, axes=cfg.axes, grid=(cfg.grid_h, cfg.grid_w),
                theta=cfg.theta)
    outs = []
    for way in range(2):
        x = qkv.clone()
        q, k, v = (x[:, i].transpose(0, 1) for i in range(3))
        layer = WindowLayer(cfg.heads, cfg.d, cfg.tokens, 300, 80, 1000, 8)
        layer.load_history(*T._rand((2, cfg.heads, 320, cfg.d), 3).bfloat16())
        if way == 0:
            L.fastar_qk_norm_rope(q, k, q, k, t0=320 // (cfg.grid_h * cfg.grid_w), **turn)
            layer.step_self(q, k, v)
        else:
            layer.step_self(q, k, v, turn=turn)
        torch.cuda.synchronize()
        outs.append((q.double(), layer.k.double(), layer.v.clone()))
    for a, b in zip(outs[0][:2], outs[1][:2]):
        pair = a.abs().unflatten(-1, (-1, 2)).norm(dim=-1, keepdim=True).expand(*a.shape[:-1], a.shape[-1] // 2, 2).flatten(-2)
        # |y0| + |y1| of a pair before its rotation is at most sqrt(2) times its length, which turning keeps
        assert ((a - b).abs() <= 2 * (2.0 ** -8 * torch.maximum(a.abs(), b.abs()) + 2.0 ** -19 * 1.5 * pair)).all()
    assert torch.equal(outs[0][2], outs[1][2])


def test_one_captured_step_serves_every_length():
    outs = []
    for use_graph in (False, True):
        dit, g = _dit()
        outs.append([dit.denoise_chunk(_noise(SMALL, g), use_graph=use_graph).clone() for _ in range(6)])
        torch.cuda.synchronize()
        assert dit.status_word() == 0
        if use_graph:
            assert list(dit._graphs) == [("window",)]
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_a_window_over_everything_equals_the_dense_path():
    """Every row in the window: the same rows as the dense path's, up to what its attention rounds."""
    cfg = SMALL.replace(window_frames=100, sink_frames=0, qk_norm="row")
    outs = []
    for attention in ("window", "dense"):
        dit = DiT(cfg, attention, seed=3, dense_capacity=2 * cfg.tokens)
        g = torch.Generator(device="cuda").manual_seed(5)
        dit.set_text(torch.randn(cfg.text_len, cfg.text_dim, generator=g, device="cuda").bfloat16())
        q = dit._heads(dit.qkv[:, :cfg.dim])
        got = []
        dit.denoise_chunk(_noise(cfg, g), use_graph=False,
                          probe=lambda what, i, a, q, *r: got.append((q.clone(), [x.clone() for x in r])) if i == 0 else None)
        torch.cuda.synchronize()
        outs.append(got)
    (q0, r0), (q1, r1) = outs[0][0], outs[1][0]               # the first block's first step: equal inputs
    assert torch.equal(q0, q1) and torch.equal(r0[0], r1[0]) and torch.equal(r0[1], r1[1])
    # both within 2^-8 |O| + 2^-8 A + ... of the same values: twice that, with A at most the largest |v|
    lim = 2 * 2.0 ** -8 * (r0[2].double().abs() + 1.1 * r0[1].double().abs().amax(1, keepdim=True))
    assert ((r0[2].double() - r1[2].double()).abs() <= lim).all()


def test_a_captured_step_of_the_layer_keeps_its_chunks():
    H, d, nq, chunks = 2, 64, 20, 8
    x = T._rand((3, chunks, H, nq, d), 45).bfloat16()
    layers = [WindowLayer(H, d, nq, 50, 7, 200, 8, page=16) for _ in range(2)]
    bufs = [torch.empty_like(x[0, 0]) for _ in range(3)]
    outs = [[], []]
    for layer in layers:
        layer.load_history(x[1, 0, :, :10], x[2, 0, :, :10])
    eager, layer = layers
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for b in bufs:
            b.zero_()
        layer.step(*bufs, advance=False)                       # warm-up outside the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        layer.step(*bufs)
    torch.cuda.synchronize()
    assert layer.n == 10                                      # nothing has run yet
    for i in range(chunks):
        outs[0].append(eager.step_self(*x[:, i]).clone())
        for b, t in zip(bufs, x[:, i]):
            b.copy_(t)
        g.replay()
        outs[1].append(layer.o_self.clone())
        assert layer.n == eager.n == 10 + (i + 1) * nq
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    layer.load_history(x[1, 1, :, :7], x[2, 1, :, :7])        # and eager calls after replays
    assert layer.n == 7
    layer.step_self(*x[:, 2])
    torch.cuda.synchronize()
    assert layer.n == 27 and layer.len.item() == 27 and layer.status() == 0


def test_reloading_a_layer_whose_step_was_captured():
    """A commit that was captured may be replayed after a new history as well: the length is the device's."""
    H, d, nq = 2, 64, 20
    x = T._rand((3, 6, H, nq, d), 46).bfloat16()
    eager, layer = (WindowLayer(H, d, nq, 50, 7, 300, 8, page=16) for _ in range(2))
    bufs = [t.clone() for t in x[:, 0]]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.step(*bufs, advance=False)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        layer.step(*bufs)
    g.replay()
    torch.cuda.synchronize()
    assert layer.n == nq
    for hist in (7, 33):
        for a in (eager, layer):
            a.load_history(*T._rand((2, H, hist, d), hist).bfloat16())
            assert a.n == hist
        for i in range(1, 4):
            for b, t in zip(bufs, x[:, i]):
                b.copy_(t)
            g.replay()
            want = eager.step_self(*x[:, i])
            assert layer.n == layer.len.item() == eager.n == hist + i * nq
            assert torch.equal(layer.o_self, want)
        layer.step_self(*x[:, 4])                             # and a call outside the graph
        assert layer.n == layer.len.item() == hist + 4 * nq and layer.status() == 0


@pytest.mark.parametrize("n", [25, 1])
def test_a_step_of_a_chunk_shorter_than_the_layers(n):
    """After a full chunk: the short one's outputs, statistics and nothing of the chunk before."""
    H, d, nq, P = 2, 64, 40, 8
    layer, short = WindowLayer(H, d, nq, 60, 10, 500, P), WindowLayer(H, d, n, 60, 10, 500, P)
    kp, vp = T._rand((2, H, P, d), 3).bfloat16()
    x, y = T._rand((3, H, nq, d), 1).bfloat16(), T._rand((3, H, n, d), 2).bfloat16()
    for a in (layer, short):
        a.set_prompt(kp, vp)
    short.load_history(x[1], x[2])
    full = [t.clone() for t in layer.step(*x)]
    assert [t.shape[1] for t in full] == [nq, nq]
    lse = layer.lse_self.clone(), layer.lse_cross.clone()
    got, want = layer.step(*y), short.step(*y)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert a.shape == (H, n, d) and torch.equal(a, b)
    for a, b, before in zip((layer.lse_self, layer.lse_cross), (short.lse_self, short.lse_cross), lse):
        assert torch.equal(a[:, :n], b) and torch.equal(a[:, n:], before[:, n:])
    for a, before in zip((layer.o_self, layer.o_cross), full):
        assert torch.equal(a[:, n:], before[:, n:])
    out = torch.full((H, nq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(layer.step_cross(y[0], out=out), want[1]) and bool((out[:, n:] == 7.0).all())


def test_cross_attention_of_more_tokens_than_the_layers_is_refused():
    layer = WindowLayer(2, 64, 4, 60, 10, 500, 8)
    q = T._rand((2, 5, 64), 1).bfloat16()
    with pytest.raises(ValueError, match="tokens"):
        layer.step_cross(q)
    with pytest.raises(ValueError, match="tokens"):
        layer.step_cross(q[:, :4], out=torch.empty(2, 3, 64, dtype=torch.bfloat16, device="cuda"))


def test_the_blocks_share_a_workspace():
    dit, _ = _dit()
    assert dit.attn[0].ws is not None and len({a.ws.data_ptr() for a in dit.attn}) == 1
    own = [WindowLayer(2, 64, 40, 60, 10, 500, 8) for _ in range(2)]
    assert own[0].ws.data_ptr() != own[1].ws.data_ptr()
    with pytest.raises(ValueError, match="workspace"):
        WindowLayer(2, 64, 40, 60, 10, 500, 8, workspace=own[0].ws[:-16])
    # two layers of a rollout on one workspace, step by step: as with their own
    shared = WindowLayer(2, 64, 40, 60, 10, 500, 8, workspace=own[0].ws)
    for i in range(3):
        x, y = T._rand((2, 3, 2, 40, 64), i).bfloat16()
        own[0].step_self(*x)
        assert torch.equal(shared.step_self(*y), own[1].step_self(*y))
