"""The DiT with its append-only caches in 4 bits (attention = "dense4") and with norms of each
head: every block's self-attention against the float64 oracle on the block's own inputs and the
cache's own values, three chunks, two steps each; one captured step for every length; the layer's
history; a full cache.  The attention bound is the one of the 4-bit cache's tests."""
import math

import numpy as np
import pytest
import torch

import test_gpu_kv4 as T
from kv_cache_tempcache_gb300 import _lib as L
from kv_cache_tempcache_gb300.dit import DiT, DiTConfig
from kv_cache_tempcache_gb300.layer import KV4Layer
from oracle import kv4_oracle as K

pytestmark = pytest.mark.gpu

SMALL = DiTConfig(dim=256, heads=2, ffn=512, layers=2, text_dim=256, text_len=64, frames=2, grid_h=4, grid_w=20,
                  steps=2, name="dit_small", qk_norm="head")


def _dit(cfg=SMALL, chunks=3):
    dit = DiT(cfg, "dense4", seed=3, dense_capacity=chunks * cfg.tokens)
    g = torch.Generator(device="cuda").manual_seed(5)
    dit.set_text(torch.randn(cfg.text_len, cfg.text_dim, generator=g, device="cuda").bfloat16())
    return dit, g


def _noise(cfg, g):
    return torch.randn(cfg.tokens, cfg.patch_ch, generator=g, device="cuda").bfloat16()


def test_blocks_attend_over_the_cache_they_filled():
    cfg = SMALL
    dit, g = _dit()
    for b in dit.blocks:
        b.norm_q.fill_(1.0)
    seen = []

    def probe(what, i, a, q, *rest):
        if what != "self":
            return
        k, v, out = rest
        torch.cuda.synchronize()
        n = a.n + cfg.tokens
        assert a.len.tolist() == [a.n] * cfg.heads and a.len_cur.tolist() == [n] * cfg.heads
        # the norm of each head: unit mean square up to bf16's rounding of each channel (2^-8 of it)
        ms = (q.double() ** 2).mean(-1)
        assert ((ms - 1).abs() <= 2.0 ** -7 + 2.0 ** -12).all()
        codes, scales = K.quantise(T._np(k))
        assert np.array_equal(a.k_codes[:, a.n:n].cpu().numpy(), codes)
        assert np.array_equal(a.k_scales[:, a.n:n].cpu().numpy(), scales)
        vals = [K.values(c[:, :n].cpu().numpy(), s[:, :n].cpu().numpy())
                for c, s in ((a.k_codes, a.k_scales), (a.v_codes, a.v_scales))]
        T._check_attn(out, a.lse_self, q, vals[0], vals[1], [n] * cfg.heads, 1 / math.sqrt(cfg.d), 0)
        seen.append((i, n))

    for chunk in range(3):
        dit.denoise_chunk(_noise(cfg, g), use_graph=False, probe=probe)
    torch.cuda.synchronize()
    assert dit.status_word() == 0
    assert seen == [(i, (c + 1) * cfg.tokens) for c in range(3) for _ in range(cfg.steps) for i in range(cfg.layers)]


def test_one_captured_step_serves_every_length():
    outs = []
    for use_graph in (False, True):
        dit, g = _dit()
        outs.append([dit.denoise_chunk(_noise(SMALL, g), use_graph=use_graph).clone() for _ in range(3)])
        torch.cuda.synchronize()
        assert dit.status_word() == 0
        if use_graph:
            assert list(dit._graphs) == [("dense4",)]
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_row_norms_and_the_dense_path_with_head_norms_run():
    for cfg, attention in ((SMALL.replace(qk_norm="row"), "dense4"), (SMALL, "dense")):
        dit = DiT(cfg, attention, seed=3, dense_capacity=cfg.tokens)
        g = torch.Generator(device="cuda").manual_seed(5)
        dit.set_text(torch.randn(cfg.text_len, cfg.text_dim, generator=g, device="cuda").bfloat16())
        out = dit.denoise_chunk(_noise(cfg, g))
        torch.cuda.synchronize()
        assert torch.isfinite(out.float()).all() and dit.status_word() == 0


def test_an_unknown_norm_is_refused():
    with pytest.raises(ValueError, match="qk_norm"):
        DiT(SMALL.replace(qk_norm="none"), "dense4")


def test_layer_history_shared_heads_and_frames():
    H, Hkv, d, nq = 4, 2, 64, 40
    layer = KV4Layer(H, d, nq, 100, 8, Hkv=Hkv, block=20)
    assert layer.cap == 112
    x = T._rand((2, Hkv, 50, d), 30).bfloat16()
    layer.load_history(x[0], x[1])
    q, kv = T._rand((H, nq, d), 31, 1.5).bfloat16(), T._rand((2, Hkv, nq, d), 32).bfloat16()
    for _ in range(2):                                   # a step that is not kept leaves no trace
        layer.step_self(q, kv[0], kv[1], advance=False)
    out = layer.step_self(q, kv[0], kv[1])
    torch.cuda.synchronize()
    assert layer.n == 90 and layer.len.tolist() == [90, 90] and layer.status() == 0
    k, v = layer.history()
    torch.cuda.synchronize()
    want = [np.concatenate((K.values(*K.quantise(T._np(a))), K.values(*K.quantise(T._np(b)))), axis=1)
            for a, b in ((x[0], kv[0]), (x[1], kv[1]))]
    assert np.array_equal(T._np(k), want[0]) and np.array_equal(T._np(v), want[1])
    T._check_attn(out, layer.lse_self, q, want[0], want[1], [90, 90], 1 / math.sqrt(d), 20)
    layer.step_self(q, kv[0], kv[1])                      # 130 rows do not fit 112
    torch.cuda.synchronize()
    assert layer.status() == L.DEV_BAD_LEN and layer.len.tolist() == [112, 112]


def test_layer_counts_the_rows_that_the_cache_took():
    layer = KV4Layer(2, 64, 24, 64, 8)
    x, q = T._rand((2, 2, 40, 64), 40).bfloat16(), T._rand((2, 24, 64), 41).bfloat16()
    layer.step_self(q, x[0], x[1])                        # more keys than queries
    torch.cuda.synchronize()
    assert layer.n == 40 and layer.len.tolist() == [40, 40] and layer.status() == 0
    layer.step_self(q, x[0], x[1])                        # 24 of 40 rows fit
    k, _ = layer.history()
    torch.cuda.synchronize()
    assert layer.n == 64 and layer.len.tolist() == [64, 64] and layer.status() == L.DEV_BAD_LEN
    want = K.values(*K.quantise(T._np(x[0])))
    assert np.array_equal(T._np(k), np.concatenate((want, want[:, :24]), axis=1))


@pytest.mark.parametrize("use_graph", [False, True])
def test_a_chunk_past_the_capacity_is_refused(use_graph):
    dit, g = _dit(chunks=1)
    dit.denoise_chunk(_noise(SMALL, g), use_graph=use_graph)
    with pytest.raises(L.FastarError, match="capacity"):
        dit.denoise_chunk(_noise(SMALL, g), use_graph=use_graph)
    with pytest.raises(L.FastarError, match="capacity"):
        dit.step(1.0, 0.5, commit=False)
    torch.cuda.synchronize()
    assert dit.status_word() == 0 and dit.attn[0].n == SMALL.tokens


def test_a_captured_step_of_the_layer_keeps_its_chunks():
    H, d, nq, chunks = 2, 64, 20, 4
    x = T._rand((3, chunks, H, nq, d), 45).bfloat16()
    layers = [KV4Layer(H, d, nq, 96, 8) for _ in range(2)]
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
    assert layer.n == 10 and layer.history()[0].shape == (H, 10, d)      # nothing has run yet
    for i in range(chunks):
        outs[0].append(eager.step_self(*x[:, i]).clone())
        for b, t in zip(bufs, x[:, i]):
            b.copy_(t)
        g.replay()
        outs[1].append(layer.o_self.clone())
        assert layer.n == eager.n == 10 + (i + 1) * nq and layer.len.tolist() == [layer.n] * H
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    for a, b in zip(eager.history(), layer.history()):
        assert a.shape == (H, 90, d) and torch.equal(a, b)
    layer.load_history(x[1, 1, :, :7], x[2, 1, :, :7])                   # and an eager call after replays
    assert layer.n == 7
    layer.step_self(*x[:, 2])
    torch.cuda.synchronize()
    assert layer.n == 27 and layer.len.tolist() == [27, 27] and layer.status() == 0
    for a in layers:                                                     # rows can be given up
        a.n = 7
        assert a.n == 7 and a.len.tolist() == [7, 7] and a.history()[0].shape == (H, 7, d)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,nq,block,cap", [(90, 40, 20, 112), (90, 40, 7, 96), (112, 40, 20, 112), (150, 200, 50, 272),
                                            (100, 300, 100, 304)])
def test_frames_that_a_full_cache_cuts(dtype, n, nq, block, cap):
    # rows past the capacity are dropped and flagged; every token sees what is left of the rows it may
    # see, and none of a later frame's
    H, d = 2, 64
    layer = KV4Layer(H, d, nq, cap, 8, dtype=dtype, block=block)
    x = T._rand((2, H, n, d), 46).to(dtype)
    layer.load_history(x[0], x[1])
    q, kv = T._rand((H, nq, d), 47, 1.5).to(dtype), T._rand((2, H, nq, d), 48).to(dtype)
    out = layer.step_self(q, kv[0], kv[1])
    torch.cuda.synchronize()
    assert layer.status() == L.DEV_BAD_LEN and layer.n == cap and layer.len.tolist() == [cap] * H
    vals = [np.concatenate((K.values(*K.quantise(T._np(a))), K.values(*K.quantise(T._np(b)))), axis=1)[:, :cap]
            for a, b in ((x[0], kv[0]), (x[1], kv[1]))]
    for t in range(0, nq, block):
        f = slice(t, min(nq, t + block))
        T._check_attn(out[:, f], layer.lse_self[:, f], q[:, f], vals[0], vals[1], [min(cap, n + f.stop)] * H,
                      1 / math.sqrt(d), 0)


@pytest.mark.parametrize("n,nq,block,cap", [(0, 200, 50, 112), (20, 300, 100, 272)])
def test_a_chunk_larger_than_the_cache_is_refused(n, nq, block, cap):
    layer = KV4Layer(2, 64, nq, cap, 8, block=block)
    x = T._rand((3, 2, nq, 64), 49).bfloat16()
    layer.load_history(x[1, :, :n], x[2, :, :n])
    with pytest.raises(L.FastarError, match="capacity"):
        layer.step_self(*x)
    torch.cuda.synchronize()
    assert layer.n == n and layer.len.tolist() == [n, n] and layer.status() == 0
