"""GPU parity of the paged cache (fastar_paged_append, fastar_paged_attn) against its float64 oracle.

Appended rows: v is moved bit for bit; k and q_out within half a rounding of the type (2^-8, 2^-24 of the
value) plus the fp32 arithmetic before it, 2^-19 of the pair's magnitudes (as the norm and rotation
alone, test_gpu_qk_rope.py).

Attention, from the oracle's own quantities: A = sum_j p_j |v_j| (the mean of |v| under the
softmax), E = the largest sum_c |q_c k_c| * scale of a row, n the rows it sees:
  - a logit is d products summed in fp32, 2 d 2^-24 E at most, then one product; e^x adds 2^-22 and
    the argument's own rounding 2^-23 E; so every p is off by e = (d 2^-23 + 2^-22) E + 2^-22 relative
    (for e < 1/16: doubled covers e^e - 1), and the quotient of two such sums by 2 e;
  - bf16 calls hold p in bf16: 2^-8 relative, at every magnitude (bf16 has fp32's exponents);
  - an exponential under fp32's range is 0: 2^-100 sum_j |v_j| covers it;
  - sums over n keys in fp32: n 2^-23 relative at most, the tensor cores' additions truncate: doubled;
  - the output's rounding: 2^-8 |O| in bf16, 2^-24 |O| in fp32.
  |O - want| <= half |want| + A (4 e + n 2^-22 + [bf16] 2^-8) + 2^-100 n max |v|
  |lse - want| <= 2 e + n 2^-22 + 2^-22 (1 + |want|)."""
import math

import numpy as np
import pytest
import torch

from kv_cache_tempcache_gb300 import _lib as L
from oracle import paged_oracle as P

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


def _np(t):
    return t.detach().double().cpu().numpy()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _rand(shape, seed, std=1.0):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV) * std


def pool_like(pages, H, page, d, dt, layout, fill):
    """[pages, H, page, d], stored so or as [pages, page, H, d]."""
    if layout == "hnd":
        return torch.full((pages, H, page, d), fill, dtype=dt, device=DEV)
    return torch.full((pages, page, H, d), fill, dtype=dt, device=DEV).transpose(1, 2)


def tables(need, page, width, seed, spare=2):
    """A table of pages dealt out at random, -1 where none is needed; and the number of pages."""
    rng = np.random.default_rng(seed)
    table = np.full((len(need), width), -1, np.int32)
    n = sum(len(p) for p in need)
    ids = rng.permutation(n + spare)[:n]
    at = 0
    for b, p in enumerate(need):
        table[b, list(p)] = ids[at:at + len(p)]
        at += len(p)
    return table, n + spare


# ---- append ------------------------------------------------------------------------------------

def run_append(dtype, nq, at, Hq, Hk, d, page, layout, norm, axes, grid, pos, use_cu=True, tail=0, width=None, seed=0,
               in_place=False, theta=1e4):
    dt, B, T = DT[dtype], len(nq), sum(nq) + tail
    width = width or max(-(-(a + n) // page) for a, n in zip(at, nq))
    table, pages = tables([range(min(width, -(-(a + n) // page))) for a, n in zip(at, nq)], page, width, seed)
    qkv = _rand((T, Hq + 2 * Hk, d), seed + 1, 2.0).to(dt)
    before = qkv.clone()
    q, k, v = (x.transpose(0, 1) for x in qkv.split((Hq, Hk, Hk), 1))
    kp, vp = pool_like(pages, Hk, page, d, dt, layout, 3.0), pool_like(pages, Hk, page, d, dt, layout, 5.0)
    wq, wk = (1 + 0.1 * _rand((d,), seed + 2), 1 + 0.1 * _rand((d,), seed + 3)) if norm else (None, None)
    p3 = np.random.default_rng(seed).integers(-50000, 50000, (T, 3)).astype(np.int32) if pos else None
    cu = np.concatenate(([0], np.cumsum(nq))) if use_cu else None
    len_out, status = _i32([-7] * B), _i32([0])
    qo = q if in_place else torch.full((Hq, T, d), 7.0, dtype=dt, device=DEV) if Hq else None
    want = P.append(_np(k), _np(v), _np(kp), _np(vp), table, at, cu, _np(q) if Hq else None,
                    None if wq is None else _np(wq), None if wk is None else _np(wk), 1e-6, axes, p3, grid, theta)
    L.fastar_paged_append(k, v, kp, vp, _i32(table), _i32(at), len_out, q=q if Hq else None, q_out=qo,
                          cu=None if cu is None else _i32(cu), wq=wq, wk=wk, eps=1e-6, axes=axes,
                          pos=None if p3 is None else torch.from_numpy(p3).cuda(), grid=grid, theta=theta,
                          dev_status=status)
    torch.cuda.synchronize()
    wk_, wv, wq_, done, lens, k_pair, q_pair = want
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    assert np.array_equal(_np(vp), wv)
    assert (np.abs(_np(kp) - wk_) <= half * np.abs(wk_) * (k_pair > 0) + 2.0 ** -19 * k_pair).all()
    if Hq:
        got = _np(qo)[:, done]
        assert (np.abs(got - wq_[:, done]) <= half * np.abs(wq_[:, done]) + 2.0 ** -19 * q_pair[:, done]).all()
        rest = qo[:, torch.from_numpy(~done).cuda()]
        assert torch.equal(rest, before.transpose(0, 1)[:Hq, torch.from_numpy(~done).cuda()]) if in_place \
            else bool((rest == 7.0).all())
    if not in_place:
        assert torch.equal(qkv, before)
    assert np.array_equal(len_out.cpu().numpy(), lens)
    return int(status.item())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq,at,Hq,Hk,d,page,layout,norm,axes,grid,pos", [
    ([1], [0], 1, 1, 64, 16, "hnd", True, (64, 0, 0), (1, 1), False),
    ([1], [333], 12, 12, 128, 64, "hnd", True, (44, 42, 42), (6, 13), False),
    ([1] * 8, [0, 15, 16, 17, 100, 3, 64, 1000], 12, 3, 128, 16, "nhd", True, (128, 0, 0), (1, 1), False),
    ([5, 1, 0, 33, 130], [7, 0, 12, 127, 128], 10, 5, 64, 32, "nhd", False, (24, 16, 16), (3, 4), True),
    ([331], [69], 3, 2, 128, 128, "hnd", True, (16, 56, 56), (5, 7), False),
    ([300, 21], [1, 640], 0, 4, 64, 64, "hnd", True, (24, 20, 20), (5, 7), False),
    ([1560, 1560], [14040, 3], 12, 12, 128, 64, "nhd", True, (44, 42, 42), (30, 52), False),
    ([7, 9], [2, 3], 2, 1, 64, 16, "hnd", False, (0, 0, 0), (1, 1), False)])
def test_append(dtype, nq, at, Hq, Hk, d, page, layout, norm, axes, grid, pos):
    assert run_append(dtype, nq, at, Hq, Hk, d, page, layout, norm, axes, grid, pos, tail=3) == 0


def test_append_without_starts_and_in_place():
    assert run_append("bf16", [40, 40, 40], [5, 0, 31], 4, 2, 128, 32, "hnd", True, (44, 42, 42), (3, 5), False,
                      use_cu=False) == 0
    assert run_append("bf16", [37], [5], 4, 2, 128, 32, "nhd", True, (44, 42, 42), (3, 5), False, in_place=True) == 0
    assert run_append("f32", [37, 90], [5, 8], 4, 2, 64, 32, "nhd", True, (24, 20, 20), (3, 5), False, in_place=True,
                      tail=2) == 0


def test_append_many_sequences_and_other_theta():
    rng = np.random.default_rng(0)
    nq = rng.integers(0, 4, 131).tolist()
    at = rng.integers(0, 200, 131).tolist()
    assert run_append("bf16", nq, at, 2, 1, 128, 16, "hnd", True, (128, 0, 0), (1, 1), False, theta=500.0) == 0


def test_append_past_the_pages_drops_rows():
    # 4 pages of 16 a sequence: the first is full before the call, the second fills up in it
    st = run_append("bf16", [3, 20, 5], [64, 50, 0], 2, 2, 64, 16, "hnd", True, (64, 0, 0), (1, 1), False, width=4)
    assert st == L.DEV_BAD_LEN


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_skips_what_makes_no_sense(dtype):
    dt, d, H, page = DT[dtype], 64, 2, 16
    T = 12
    k, v, q = _rand((H, T, d), 1).to(dt), _rand((H, T, d), 2).to(dt), _rand((H, T, d), 3).to(dt)
    table = _i32([[0, 1], [2, 99], [3, 4], [5, -3]])
    at = _i32([-1, 14, 33, 20])
    kp, vp = pool_like(6, H, page, d, dt, "hnd", 3.0), pool_like(6, H, page, d, dt, "hnd", 5.0)
    qo, ln, st = torch.full_like(q, 7.0), _i32([9, 9, 9, 9]), _i32([0])
    L.fastar_paged_append(k, v, kp, vp, table, at, ln, q=q, q_out=qo, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == L.DEV_BAD_LEN | L.DEV_BAD_INDEX
    assert ln.tolist() == [0, 17, 0, 23]
    # sequence 1: rows 14, 15 go to page 2, row 16 to page 99 that is not there; 3: rows 20.. to page -3
    assert torch.equal(kp[2, :, 14:], k[:, 3:5]) and torch.equal(vp[2, :, 14:], v[:, 3:5])
    kp[2, :, 14:], vp[2, :, 14:] = 3.0, 5.0
    assert bool((kp == 3.0).all()) and bool((vp == 5.0).all())
    assert bool((qo[:, 0:3] == 7.0).all()) and bool((qo[:, 6:9] == 7.0).all())
    assert torch.equal(qo[:, 3:6], q[:, 3:6]) and torch.equal(qo[:, 9:], q[:, 9:])
    # starts that fall or leave the call's tokens
    for cu in ([0, 3, 2, 5, 12], [-1, 3, 6, 9, 12], [0, 3, 6, 9, 13]):
        kp.fill_(3.0)
        st.zero_()
        L.fastar_paged_append(k, v, kp, vp, table, _i32([0, 0, 0, 0]), ln, cu=_i32(cu), dev_status=st)
        torch.cuda.synchronize()
        assert st.item() & L.DEV_BAD_LEN


# ---- attention ---------------------------------------------------------------------------------

def attn_case(dtype, nq, at, Hk, G, d, page, layout, block, window, sinks, seed=0, use_cu=True, tail=0, garbage=None,
              width=0, spare_rows=True):
    """The tensors of a call: pages that no token sees have no entry, rows that none sees hold
    `garbage`."""
    dt, B, T = DT[dtype], len(nq), sum(nq) + tail
    width = max(width, max(max(1, -(-(a + n) // page)) for a, n in zip(at, nq)))
    used = []
    for a, n in zip(at, nq):
        m = min(a + n, width * page)
        see = P.sees(n, a, m, block, window, sinks).any(0) if n else np.zeros(m, bool)
        used.append(np.flatnonzero(see))
    # needed: pages with a row between the first and the last of the window, or a sink
    need = [sorted(set((u // page).tolist())) for u in used]
    table, pages = tables(need, page, width, seed)
    g = float("nan") if garbage is None else garbage
    kp, vp = pool_like(pages, Hk, page, d, dt, layout, g), pool_like(pages, Hk, page, d, dt, layout, g)
    for b, u in enumerate(used):
        if len(u):
            x = _rand((2, len(u), Hk, d), seed + 10 + b).to(dt)
            pg, of = torch.from_numpy(table[b, u // page]).long().cuda(), torch.from_numpy(u % page).cuda()
            kp[pg, :, of], vp[pg, :, of] = x[0], x[1]
    q = _rand((T, Hk * G, d), seed + 1, 1.5).to(dt).transpose(0, 1)
    cu = np.concatenate(([0], np.cumsum(nq))) if use_cu else None
    return q, kp, vp, table, np.array(at), cu


def run_attn(q, kp, vp, table, at, cu, scale, block, window, sinks, max_q=None, ws=True, status=0, bits=-1):
    Hq, T, d = q.shape
    out = torch.full((T, Hq, d), 7.0, dtype=q.dtype, device=DEV).transpose(0, 1)
    lse = torch.full((Hq, T), 7.0, device=DEV)
    B, Hk, page = table.shape[0], kp.shape[1], kp.shape[2]
    mq = max_q or (int(np.diff(cu).max()) if cu is not None else T // B)
    nb = L.workspace_bytes(L.OP_PAGED_ATTN, Hq, T, table.shape[1] * page, d, Hk, r=mq, P=B)
    if isinstance(ws, int) and not isinstance(ws, bool):
        nb = min(nb, ws)
    w = torch.full((nb,), 0xA5, dtype=torch.uint8, device=DEV) if nb and ws else None
    st = _i32([0])
    L.fastar_paged_attn(q, kp, vp, _i32(table), _i32(at), scale, out, lse, cu=None if cu is None else _i32(cu),
                        max_q=mq, block=block, window=window, sinks=sinks, dev_status=st, workspace=w)
    torch.cuda.synchronize()
    assert int(st.item()) & bits == status
    return out, lse


def check_attn(dtype, q, kp, vp, table, at, cu, scale, block, window, sinks, out, lse):
    want, wl, A, E, n = P.attention(_np(q), _np(kp), _np(vp), table, at, scale, cu, block, window, sinks)
    d = q.shape[2]
    bf = dtype == "bf16"
    e = (d * 2.0 ** -23 + 2.0 ** -22) * E + 2.0 ** -22
    assert e.max() < 1 / 16
    big = np.nan_to_num(np.abs(_np(vp)), nan=0.0).max()
    tol = (2.0 ** -8 if bf else 2.0 ** -24) * np.abs(want) + n[None, :, None] * 2.0 ** -100 * big
    tol += A * (4 * e + n * 2.0 ** -22 + (2.0 ** -8 if bf else 0))[..., None]
    mine = n >= 0
    got, gl = _np(out), _np(lse)
    assert (np.abs(got - want) <= tol)[:, mine].all(), np.nanmax((np.abs(got - want) / (tol + 1e-300))[:, mine])
    live = mine & (n > 0)
    assert np.isneginf(gl[:, mine & (n == 0)]).all()
    assert (np.abs(gl - wl) <= 2 * e + n * 2.0 ** -22 + 2.0 ** -22 * (1 + np.abs(wl)))[:, live].all()
    assert (got[:, ~mine] == 7.0).all() and (gl[:, ~mine] == 7.0).all()       # tokens of no sequence


MASKS = [(0, 0, 0), (1, 0, 0), (1, 64, 4), (1, 1, 0), (0, 100, 37), (16, 33, 16), (1, 16, 1000), (1000, 5, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block,window,sinks", MASKS)
@pytest.mark.parametrize("nq,at,Hk,G,d,page,layout", [
    ([1], [0], 1, 1, 64, 16, "hnd"), ([1], [332], 12, 1, 128, 64, "hnd"),
    ([1] * 5, [0, 1, 130, 777, 2000], 2, 4, 128, 16, "nhd"), ([4, 0, 7, 1], [900, 3, 0, 128], 2, 4, 64, 32, "nhd"),
    ([33, 1, 130], [7, 500, 128], 2, 2, 128, 32, "hnd"), ([257], [1000], 3, 1, 64, 128, "nhd"),
    ([300, 129], [0, 640], 1, 3, 128, 64, "nhd")])
def test_attention(dtype, block, window, sinks, nq, at, Hk, G, d, page, layout):
    c = attn_case(dtype, nq, at, Hk, G, d, page, layout, block, window, sinks, seed=len(nq) + at[0], tail=2)
    scale = 1 / math.sqrt(d)
    out, lse = run_attn(*c, scale, block, window, sinks)
    check_attn(dtype, *c, scale, block, window, sinks, out, lse)


@pytest.mark.parametrize("dtype,nq,at,Hk,G,d,page,block,window,sinks", [
    ("bf16", [1], [40000], 2, 4, 128, 64, 1, 0, 0), ("bf16", [1, 1, 1], [40000, 13, 9000], 1, 8, 64, 16, 1, 8191, 100),
    ("bf16", [9], [20000], 1, 2, 128, 32, 1, 0, 0), ("bf16", [70], [30000], 1, 1, 128, 128, 1, 15000, 300),
    ("bf16", [600, 40], [12000, 3000], 2, 1, 128, 64, 0, 5000, 1500), ("f32", [3, 1], [20000, 5], 2, 4, 64, 16, 1, 0, 0),
    ("bf16", [700], [5000], 2, 1, 64, 32, 200, 3000, 100), ("f32", [40], [9000], 1, 2, 128, 32, 1, 4000, 7)])
@pytest.mark.parametrize("ws", [True, False, 100000])
def test_attention_over_long_sequences(dtype, nq, at, Hk, G, d, page, block, window, sinks, ws):
    c = attn_case(dtype, nq, at, Hk, G, d, page, "hnd", block, window, sinks, seed=5)
    scale = 1 / math.sqrt(d)
    out, lse = run_attn(*c, scale, block, window, sinks, ws=ws)
    check_attn(dtype, *c, scale, block, window, sinks, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 5, 40, 300])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
def test_what_a_token_does_not_see_cannot_reach_it(dtype, nq, what):
    """K and V of single rows that some tokens see and others do not: causal tokens, a window, sinks."""
    d, page, Hk, G, at, block, window, sinks = 64, 16, 2, 2, 600, 1, 150, 20
    q, kp, vp, table, a, cu = attn_case(dtype, [nq], [at], Hk, G, d, page, "hnd", block, window, sinks, seed=nq)
    scale = 1 / math.sqrt(d)
    clean = run_attn(q, kp, vp, table, a, cu, scale, block, window, sinks)
    see = P.sees(nq, at, at + nq, block, window, sinks)
    for row in sorted({at + nq - 1, at + nq // 2, at - window + 1, at + nq - window, 19}):
        if not see[:, row].any():
            continue
        for pool, ch in ((vp, 3), (vp, slice(0, d)), (kp, 5)):
            pg, of = int(table[0, row // page]), row % page
            keep = pool[pg, 1, of].clone()
            pool[pg, 1, of, ch] = what
            out, lse = run_attn(q, kp, vp, table, a, cu, scale, block, window, sinks)
            pool[pg, 1, of] = keep
            rows = torch.from_numpy(see[:, row]).cuda()
            # tokens that do not see it, and the other KV head's, are as before, bit for bit
            assert torch.equal(out[:G], clean[0][:G]) and torch.equal(lse[:G], clean[1][:G])
            assert torch.equal(out[G:, ~rows], clean[0][G:, ~rows]) and torch.equal(lse[G:, ~rows], clean[1][G:, ~rows])
            if pool is vp:
                assert not bool(torch.isfinite(out[G:, rows][..., ch]).any())
                if ch == 3:
                    other = [c for c in range(d) if c != 3]
                    assert torch.equal(out[G:, rows][..., other], clean[0][G:, rows][..., other])
            elif what != what:
                assert bool(torch.isnan(out[G:, rows]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 3, 30, 200])
def test_a_query_that_is_not_finite_stays_alone(dtype, nq):
    d, Hk, G = 128, 1, 2
    c = attn_case(dtype, [nq], [700], Hk, G, d, 32, "hnd", 1, 300, 10, seed=9)
    clean = run_attn(*c, 0.1, 1, 300, 10)
    c[0][1, nq // 2, 7] = float("nan")
    out, lse = run_attn(*c, 0.1, 1, 300, 10)
    assert bool(torch.isnan(out[1, nq // 2]).all())
    keep = torch.ones(2, nq, dtype=torch.bool, device=DEV)
    keep[1, nq // 2] = False
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 40, 300])
def test_large_and_lopsided_logits(dtype, nq):
    """Logits of hundreds and rows of keys that rise, fall, or lie 30 below one strong key whose V is 0."""
    d, page, n = 64, 16, 1000
    q, kp, vp, table, a, cu = attn_case(dtype, [nq], [n - nq], 1, 1, d, page, "hnd", 0, 0, 0, seed=2)
    row = torch.arange(n, device=DEV)
    pg, of = torch.from_numpy(table[0]).long().cuda()[row // page], row % page
    for shape in (row * 0.5, -row * 0.5, torch.where(row == 17, 30.0, 0.0)):
        kp[pg, :, of] = 0
        kp[pg, 0, of, 0] = shape.to(kp.dtype)
        if float(shape.max()) == 30.0:
            vp[pg[17], :, of[17]] = 0
        q[...] = 0
        q[:, :, 0] = 1.0
        out, lse = run_attn(q, kp, vp, table, a, cu, 1.0, 0, 0, 0)
        check_attn(dtype, q, kp, vp, table, a, cu, 1.0, 0, 0, 0, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 40])
def test_attention_flags_what_makes_no_sense(dtype, nq):
    d, B = 64, 3
    c = attn_case(dtype, [nq] * B, [100, 50, 30], 1, 2, d, 16, "hnd", 1, 0, 0, seed=3)
    q, kp, vp, table, at, cu = c
    clean = run_attn(*c, 0.1, 1, 0, 0)
    # a start outside the pages: the sequence is skipped
    for bad in (-1, table.shape[1] * 16 + 1):
        at2 = at.copy()
        at2[1] = bad
        out, lse = run_attn(q, kp, vp, table, at2, cu, 0.1, 1, 0, 0, status=L.DEV_BAD_LEN)
        assert bool((out[:, nq:2 * nq] == 7.0).all()) and bool((lse[:, nq:2 * nq] == 7.0).all())
        for s in (slice(0, nq), slice(2 * nq, 3 * nq)):
            assert torch.equal(out[:, s], clean[0][:, s]) and torch.equal(lse[:, s], clean[1][:, s])
    # a page that is not there: its rows count as zeros
    for bad in (-1, kp.shape[0], 2 ** 31 - 1, -2 ** 31):
        t2, was = table.copy(), table[0, 2]
        t2[0, 2] = bad
        out, lse = run_attn(q, kp, vp, t2, at, cu, 0.1, 1, 0, 0, status=L.DEV_BAD_INDEX)
        kz, vz = kp.clone(), vp.clone()
        kz[was], vz[was] = 0, 0
        check_attn(dtype, q, kz, vz, table, at, cu, 0.1, 1, 0, 0, out, lse)
    # more tokens than max_q: the first are done
    if nq > 1:
        out, lse = run_attn(*c, 0.1, 1, 0, 0, max_q=nq - 3, status=L.DEV_BAD_LEN)
        for b in range(B):
            s, r = slice(b * nq, b * nq + nq - 3), slice(b * nq + nq - 3, (b + 1) * nq)
            assert torch.allclose(out[:, s].float(), clean[0][:, s].float(), rtol=2e-2, atol=2e-2)
            assert bool((out[:, r] == 7.0).all()) and bool((lse[:, r] == 7.0).all())
    # starts that fall or leave the call's tokens
    for cu2 in ([0, nq, nq - 1, 3 * nq], [-1, nq, 2 * nq, 3 * nq], [0, nq, 2 * nq, 3 * nq + 1]):
        # (a sequence that is left may have become longer than its pages)
        run_attn(q, kp, vp, table, at, np.array(cu2), 0.1, 1, 0, 0, max_q=3 * nq, status=L.DEV_BAD_LEN, bits=L.DEV_BAD_LEN)


def test_more_rows_than_the_pages_hold():
    """Tokens whose rows were dropped see what is there."""
    for nq, at, block, window in ((30, 50, 1, 0), (30, 50, 0, 20), (5, 64, 1, 10), (30, 50, 7, 16)):
        c = attn_case("bf16", [nq], [at], 2, 1, 64, 16, "hnd", block, 0, 0, seed=4)
        q, kp, vp, table, a, cu = c
        table = np.ascontiguousarray(table[:, :4])
        out, lse = run_attn(q, kp, vp, table, a, cu, 0.1, block, window, 0)
        check_attn("bf16", q, kp, vp, table, a, cu, 0.1, block, window, 0, out, lse)


@pytest.mark.parametrize("nq", [1, 20, 200])
def test_offsets_past_32_bits(nq):
    """A pool of 2^32 elements and more: pages at its far end, [pages, page, H, d] with H that counts."""
    d, page, Hk, B = 128, 64, 8, 2
    pages = 2 ** 32 // (page * Hk * d) + 40
    kp = torch.empty(pages, page, Hk, d, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    vp = torch.empty(pages, page, Hk, d, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    at = np.array([500, 0])
    table = (pages - 1 - np.arange(B * 12).reshape(B, 12)).astype(np.int32)
    x = _rand((2, Hk, 500, d), 1).bfloat16()
    L.fastar_paged_append(x[0], x[1], kp, vp, _i32(table[:1]), _i32([0]))
    y = _rand((3, Hk, B * nq, d), 2).bfloat16()
    L.fastar_paged_append(y[0], y[1], kp, vp, _i32(table), _i32(at))
    out, lse = run_attn(y[2], kp, vp, table, at, None, 0.1, 1, 0, 0)
    lo = int(table.min())
    check_attn("bf16", y[2], kp[lo:], vp[lo:], table - lo, at, None, 0.1, 1, 0, 0, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_sequences_than_are_dealt_out(dtype):
    rng = np.random.default_rng(0)
    B = 300
    nq, at = rng.integers(0, 3, B).tolist(), rng.integers(0, 200, B).tolist()
    at[7], nq[7] = 3000, 2
    c = attn_case(dtype, nq, at, 1, 2, 64, 16, "hnd", 1, 0, 0, seed=1, tail=1)
    out, lse = run_attn(*c, 0.125, 1, 0, 0)
    check_attn(dtype, *c, 0.125, 1, 0, 0, out, lse)


@pytest.mark.parametrize("B,most,G,d,block,window,sinks", [(70, 100, 2, 64, 1, 90, 5), (70, 40, 4, 128, 1, 0, 0),
                                                          (3, 1100, 8, 64, 1, 200, 20), (40, 300, 3, 128, 0, 0, 0),
                                                          (2, 1100, 16, 128, 1, 64, 0), (33, 17, 2, 128, 1, 0, 0)])
def test_work_of_many_and_uneven_sequences(B, most, G, d, block, window, sinks):
    """Sequences of very different lengths, some without tokens, more than 32 of them; row tiles of one by the
    dozen."""
    rng = np.random.default_rng(B)
    nq = (most * rng.random(B) ** 3).astype(int)
    nq[rng.integers(0, B, B // 4)] = 0
    nq[-1] = most
    at = (800 * rng.random(B) ** 3).astype(int)
    c = attn_case("bf16", nq.tolist(), at.tolist(), 2 if B > 3 else 1, G, d, 16, "nhd", block, window, sinks, seed=B, tail=2)
    for ws in (True, False):
        out, lse = run_attn(*c, 1 / math.sqrt(d), block, window, sinks, ws=ws)
        check_attn("bf16", *c, 1 / math.sqrt(d), block, window, sinks, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 3, 50])
def test_tokens_before_the_first_sequence_and_other_strides(dtype, nq):
    """cu that does not begin at 0, one KV head, one page, rows of q and out with gaps between, head-major."""
    dt, d, page = DT[dtype], 64, 128
    T = nq + 7
    q = _rand((3, T + 2, d + 8), 1, 1.5).to(dt)[:, :T, :d]
    out = torch.full((3, T + 3, d + 16), 7.0, dtype=dt, device=DEV)[:, :T, 8:8 + d]
    kp, vp = (torch.full((1, 1, page, d + 8), 3.0, dtype=dt, device=DEV)[..., :d] for _ in range(2))
    k, v = (_rand((1, T, d + 24), s).to(dt)[..., 16:16 + d] for s in (2, 3))
    table, at, cu = np.zeros((1, 1), np.int32), np.array([20]), np.array([4, 4 + nq])
    kp[0, 0, :20], vp[0, 0, :20] = _rand((20, d), 4).to(dt), _rand((20, d), 5).to(dt)
    qo = torch.full((3, T, d), 9.0, dtype=dt, device=DEV)
    L.fastar_paged_append(k, v, kp, vp, _i32(table), _i32(at), q=q, q_out=qo, cu=_i32(cu), axes=(24, 20, 20), grid=(3, 4))
    st, lse = _i32([0]), torch.full((3, T), 7.0, device=DEV)
    L.fastar_paged_attn(q, kp, vp, _i32(table), _i32(at), 0.125, out, lse, cu=_i32(cu), max_q=nq, block=1, window=15, sinks=2,
                        dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    want = P.append(_np(k), _np(v), np.full((1, 1, page, d), 3.0), np.full((1, 1, page, d), 3.0), table, at, cu, _np(q), None,
                    None, 1e-6, (24, 20, 20), None, (3, 4))
    assert np.array_equal(_np(vp)[0, 0, 20:], want[1][0, 0, 20:])
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    assert (np.abs(_np(qo) - want[2]) <= half * np.abs(want[2]) + 2.0 ** -19 * want[6])[:, 4:4 + nq].all()
    assert bool((qo[:, :4] == 9.0).all()) and bool((qo[:, 4 + nq:] == 9.0).all())
    check_attn(dtype, q, kp, vp, table, at, cu, 0.125, 1, 15, 2, out, lse)


def test_positions_and_sequences_of_thousands_of_short_ones():
    """A token each of 3000 sequences: every token finds its own."""
    B, d, page = 3000, 64, 16
    rng = np.random.default_rng(3)
    nq, at = (rng.random(B) < 0.7).astype(int).tolist(), rng.integers(0, 40, B).tolist()
    assert run_append("bf16", nq, at, 1, 1, d, page, "hnd", False, (64, 0, 0), (1, 1), False, tail=5) == 0


# ---- both together --------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_rollout_through_both_calls(dtype):
    """Chunks and single tokens of three sequences, appended and attended over, with pages handed back as
    they leave the window; positions turn with the row."""
    dt, B, Hk, G, d, page, window, sinks = DT[dtype], 3, 2, 2, 64, 16, 70, 20
    width, pages = 40, 40
    kp, vp = (pool_like(pages, Hk, page, d, dt, "nhd", float("nan")) for _ in range(2))
    table = np.full((B, width), -1, np.int32)
    free = list(range(pages))
    at, len_out, status = np.zeros(B, np.int64), _i32([0] * B), _i32([0])
    wq, wk = 1 + 0.1 * _rand((d,), 2), 1 + 0.1 * _rand((d,), 3)
    rows = [([], []) for _ in range(B)]
    rng = np.random.default_rng(0)
    for step in range(12):
        nq = [[30, 1, 45], [1, 1, 1], [0, 5, 33], [2, 17, 0]][step % 4]
        T = sum(nq)
        for b in range(B):
            first = max(0, at[b] + 1 - window) if nq[b] else 0
            for p in range(-(-sinks // page), first // page if nq[b] else 0):
                if table[b, p] >= 0:                       # no later token sees it
                    kp[table[b, p]], vp[table[b, p]] = float("nan"), float("nan")
                    free.append(int(table[b, p]))
                    table[b, p] = -1
            for p in range(at[b] // page, -(-(at[b] + nq[b]) // page)):
                if table[b, p] < 0:
                    table[b, p] = free.pop(int(rng.integers(len(free))))
        qkv = _rand((T, (G + 2) * Hk, d), 100 + step).to(dt)
        q, k, v = (x.transpose(0, 1) for x in qkv.split((G * Hk, Hk, Hk), 1))
        cu = np.concatenate(([0], np.cumsum(nq)))
        before = _np(q), _np(k), _np(v)
        L.fastar_paged_append(k, v, kp, vp, _i32(table), _i32(at), len_out, q=q, q_out=q, cu=_i32(cu), wq=wq, wk=wk,
                              axes=(24, 20, 20), grid=(3, 4), dev_status=status)
        out, lse = run_attn(q, kp, vp, table, at, cu, 0.125, 1, window, sinks)
        check_attn(dtype, q, kp, vp, table, at, cu, 0.125, 1, window, sinks, out, lse)
        for b in range(B):
            sl = slice(cu[b], cu[b + 1])
            p = P.positions(int(at[b]), nq[b], (3, 4))
            if nq[b] == 0:
                continue
            rows[b][0].append(P.K.norm_rope(before[1][:, sl], _np(wk), 1e-6, (24, 20, 20), p, 1e4)[0])
            rows[b][1].append(before[2][:, sl])
            # against the whole history in 64 bits, rounded once where the cache is
            kk, vv = np.concatenate(rows[b][0], 1), np.concatenate(rows[b][1], 1)
            qq = P.K.norm_rope(before[0][:, sl], _np(wq), 1e-6, (24, 20, 20), p, 1e4)[0]
            one = np.zeros((1, 1), np.int32)
            w, _, A, _, _ = P.attention(qq, kk[None], vv[None], one, at[b:b + 1], 0.125, None, 1, window, sinks)
            # a normed row has |x| <= 1.5 sqrt(d) (weights up to 1.5): q and k rounded to the type (and to 2^-19 of a
            # pair before) move a logit by 2 half |q| |k| scale <= 2 half * 2.25 d * 0.125 = 36 half, and every p
            # by e^72 half - 1 < 80 half, twice for the quotient; then p, the values and the output rounded
            half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -18
            assert (np.abs(_np(out)[:, sl] - w) <= half * np.abs(w) + A * 162 * half).all()
        at += np.array(nq)
        assert np.array_equal(len_out.cpu().numpy(), at) and status.item() == 0


@pytest.mark.parametrize("nq,G", [(1, 1), (3, 4), (150, 2)])
def test_captured_calls_follow_the_device_and_repeat_bit_for_bit(nq, G):
    d, page, Hk, B, width = 128, 32, 2, 2, 40
    kp, vp = (pool_like(B * width, Hk, page, d, torch.bfloat16, "hnd", 0.0) for _ in range(2))
    kp.copy_(_rand(kp.shape, 1)), vp.copy_(_rand(vp.shape, 2))
    table = _i32(np.random.default_rng(0).permutation(B * width).reshape(B, width))
    qkv = _rand((B * nq, (G + 2) * Hk, d), 3).bfloat16()
    q, k, v = (x.transpose(0, 1) for x in qkv.split((G * Hk, Hk, Hk), 1))
    qo, out = torch.empty_like(q), torch.empty_like(q)
    lse, at, ln, st = torch.empty(G * Hk, B * nq, device=DEV), _i32([0, 0]), _i32([0, 0]), _i32([0])
    nb = L.workspace_bytes(L.OP_PAGED_ATTN, G * Hk, B * nq, width * page, d, Hk, r=nq, P=B)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV) if nb else None

    def go():
        L.fastar_paged_append(k, v, kp, vp, table, at, ln, q=q, q_out=qo, axes=(44, 42, 42), grid=(2, 3), dev_status=st)
        L.fastar_paged_attn(qo, kp, vp, table, at, 0.1, out, lse, block=1, window=300, sinks=7, dev_status=st,
                            workspace=ws)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        go()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        go()
    for a in ([0, 0], [5, 900], [1000, 33], [0, 1]):
        at.copy_(_i32(a))
        g.replay()
        torch.cuda.synchronize()
        first = [x.clone() for x in (qo, out, lse, kp, vp, ln)]
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(first, (qo, out, lse, kp, vp, ln)):
            assert torch.equal(x, y)
        check_attn("bf16", qo, kp, vp, table.cpu().numpy(), np.array(a), None, 0.1, 1, 300, 7, out, lse)
    assert st.item() == 0


def test_two_calls_on_two_streams():
    cs = [attn_case("bf16", [1], [20000], 2, 2, 128, 32, "hnd", 1, 0, 0, seed=s) for s in (1, 2)]
    cs.append(attn_case("bf16", [500], [5000], 2, 2, 128, 32, "hnd", 1, 0, 0, seed=3))
    alone = [run_attn(*c, 0.1, 1, 0, 0) for c in cs]
    outs = []
    torch.cuda.synchronize()
    for c in cs:
        q, kp, vp, table, at, cu = c
        nb = L.workspace_bytes(L.OP_PAGED_ATTN, 4, q.shape[1], table.shape[1] * 32, 128, 2, r=q.shape[1], P=1)
        outs.append((torch.empty_like(q), _i32(table), _i32(at), torch.empty(nb + 16, dtype=torch.uint8, device=DEV),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for c, (o, t, a, w, s) in zip(cs, outs):
            with torch.cuda.stream(s):
                L.fastar_paged_attn(c[0], c[1], c[2], t, a, 0.1, o, block=1, workspace=w)
    torch.cuda.synchronize()
    for o, want in zip(outs, alone):
        assert torch.equal(o[0], want[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq,G", [(1, 1), (3, 4), (70, 2)])
def test_what_follows_finds_the_outputs_of_calls_with_nothing_to_join(dtype, nq, G):
    """Short sequences with long tables: the keys could be split and are not, so that the join has nothing to do; the
    next call reads the outputs."""
    dt, d, page, Hk, B, width, m = DT[dtype], 128, 32, 2, 3, 200, 300
    kp, vp = (_rand((B * width, Hk, page, d), s).to(dt) for s in (1, 2))
    table, at, st = _i32(np.arange(B * width).reshape(B, width)), _i32([m, 0, 11]), _i32([0])
    q = _rand((G * Hk, B * nq, d), 3).to(dt)
    rows = _rand((2, Hk, B * nq, d), 4).to(dt)
    out, moved = torch.empty_like(q), torch.empty_like(q)
    nb = L.workspace_bytes(L.OP_PAGED_ATTN, G * Hk, B * nq, width * page, d, Hk, r=nq, P=B)
    assert nb > 0
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    far = [torch.empty_like(kp) for _ in range(2)]

    def go():
        out.fill_(9.0)
        moved.fill_(8.0)
        L.fastar_paged_attn(q, kp, vp, table, at, 0.1, out, block=1, dev_status=st, workspace=ws)
        L.fastar_paged_append(rows[0], rows[1], far[0], far[1], table, at, q=out, q_out=moved, dev_status=st)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        go()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        go()
    for _ in range(20):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(moved, out) and not bool((out == 9.0).any())
    lse = torch.empty(G * Hk, B * nq, device=DEV)
    L.fastar_paged_attn(q, kp, vp, table, at, 0.1, out, lse, block=1, dev_status=st, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(moved, out) and st.item() == 0
    check_attn(dtype, q, kp, vp, table.cpu().numpy(), at.cpu().numpy(), None, 0.1, 1, 0, 0, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 40])
@pytest.mark.parametrize("scale", [3e38, 1e-44])
def test_the_largest_and_smallest_scales(dtype, nq, scale):
    """Queries of zeros: every key has the same weight, whatever the scale."""
    q, kp, vp, table, at, cu = attn_case(dtype, [nq, nq], [90, 5], 2, 2, 64, 16, "hnd", 1, 0, 0)
    q.zero_()
    out, lse = run_attn(q, kp, vp, table, at, cu, scale * (1 - 2.0 ** -20), 1, 0, 0)
    check_attn(dtype, q, kp, vp, table, at, cu, 1.0, 1, 0, 0, out, lse)


@pytest.mark.parametrize("dtype,nq,Hq,Hk,d,tail", [("bf16", [7001], 1, 1, 64, 0), ("f32", [6000, 0, 1403, 1], 2, 1, 128, 3),
                                                   ("bf16", [1, 9999], 0, 3, 128, 1), ("bf16", [3001, 4002], 8, 8, 64, 0)])
def test_append_of_thousands_of_tokens(dtype, nq, Hq, Hk, d, tail):
    """More tokens than resident warps take in turn: blocks of a few neighbouring tokens, the last one not full."""
    axes = (24, 20, 20) if d == 64 else (44, 42, 42)
    assert run_append(dtype, nq, [5 * i for i in range(len(nq))], Hq, Hk, d, 64, "nhd", True, axes, (30, 52), False,
                      tail=tail) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 5, 7, 9, 11, 15, 16, 31, 32])
def test_few_rows_of_every_kind_of_group(d, G):
    """As many tokens as 32 rows hold, of heads that share one: every row's own token and head."""
    most = 32 // G
    for nq in {1, (most + 1) // 2, most}:
        c = attn_case("bf16", [nq, max(1, nq - 1)], [700, 3], 2, G, d, 16, "nhd", 1, 50, 3, seed=G)
        out, lse = run_attn(*c, 1 / math.sqrt(d), 1, 50, 3)
        check_attn("bf16", *c, 1 / math.sqrt(d), 1, 50, 3, out, lse)
        c = attn_case("bf16", [nq], [1700], 1, G, d, 64, "hnd", 1, 0, 0, seed=G + 1)
        out, lse = run_attn(*c, 1 / math.sqrt(d), 1, 0, 0)
        check_attn("bf16", *c, 1 / math.sqrt(d), 1, 0, 0, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B", [4, 300])
def test_lengths_do_not_grow_by_a_call_whose_starts_make_no_sense(dtype, B):
    """cu that falls or leaves the call's tokens: whose tokens are whose is not known, so no sequence gets longer; rows
    behind the lengths may be written, of sequences whose own bounds make sense, and nothing else."""
    dt, d, H, page, n = DT[dtype], 64, 2, 16, 3
    T = n * B
    k, v = _rand((H, T, d), 1).to(dt), _rand((H, T, d), 2).to(dt)
    width = 40 if B == 4 else 80
    table = np.random.default_rng(1).permutation(B * width).reshape(B, width).astype(np.int32)
    at = [5 + b % 23 for b in range(B)]
    at[2] = -1
    good = [n * b for b in range(B + 1)]
    mid = B - 1
    for at_i, x in ((1, -1), (mid, n * (mid - 1) - 1), (mid, T + 1), (mid, -2 ** 31), (mid, 2 ** 31 - 1), (0, -1), (B, T + 1),
                    (1, n * 3), (B, 0)):
        cu = list(good)
        cu[at_i] = x
        bad = [b for b in range(B) if cu[b] < 0 or cu[b + 1] < cu[b] or cu[b + 1] > T]
        assert bad
        kp, vp = (pool_like(B * width, H, page, d, dt, "nhd", f) for f in (3.0, 5.0))
        ln, st = _i32([-7] * B), _i32([0])
        L.fastar_paged_append(k, v, kp, vp, _i32(table), _i32(at), ln, cu=_i32(cu), dev_status=st)
        torch.cuda.synchronize()
        assert st.item() == L.DEV_BAD_LEN
        assert ln.tolist() == [max(a, 0) for a in at]
        for pool, src, fill in ((kp, k, 3.0), (vp, v, 5.0)):
            flat = pool.transpose(1, 2).reshape(-1, H, d)                  # slots
            touched = (flat != fill).any(-1).any(-1).nonzero()[:, 0].tolist()
            may = {}
            for b in range(B):
                if b not in bad and at[b] >= 0:
                    for i in range(min(cu[b + 1] - cu[b], width * page - at[b])):
                        r = at[b] + i
                        may[int(table[b, r // page]) * page + r % page] = cu[b] + i
            assert set(touched) <= set(may)
            if touched:
                assert torch.equal(flat[touched], src[:, [may[s] for s in touched]].transpose(0, 1))
    ln = _i32([-7] * B)
    L.fastar_paged_append(k, v, kp, vp, _i32(table), _i32(at), ln, cu=_i32(good))
    torch.cuda.synchronize()
    assert ln.tolist() == [a + n if a >= 0 else 0 for a in at]


@pytest.mark.parametrize("nq", [1, 20, 60])
@pytest.mark.parametrize("cu", [[0, 3, 2, 5, 12], [0, 3, 100, 5, 12], [-1, 3, 6, 9, 12]])
def test_attention_of_starts_that_make_no_sense_leaves_other_tokens(nq, cu):
    """Tokens that no sequence has whose own bounds make sense are left as they were."""
    cu, Ts = [c * nq for c in cu], 14 * nq
    c = attn_case("bf16", [3 * nq] * 4, [100, 50, 30, 70], 1, 2, 128, 16, "hnd", 1, 0, 0, seed=3, tail=2 * nq)
    q, kp, vp, table, at, _ = c
    assert q.shape[1] == Ts
    table = np.concatenate((table, np.zeros((4, 64), np.int32)), 1)        # pages for the longest
    out, lse = run_attn(q, kp, vp, table, at, np.array(cu), 0.1, 1, 0, 0, max_q=Ts, status=L.DEV_BAD_LEN, bits=L.DEV_BAD_LEN)
    mine = np.zeros(Ts, bool)
    for b in range(4):
        if 0 <= cu[b] <= cu[b + 1] <= Ts:
            mine[cu[b]:cu[b + 1]] = True
    rest = torch.from_numpy(~mine).cuda()
    assert bool((out[:, rest] == 7.0).all()) and bool((lse[:, rest] == 7.0).all())


def test_starts_that_make_no_sense_are_told_without_lengths():
    """The bounds of a sequence that no token is looked for in."""
    k = _rand((1, 6, 64), 1).bfloat16()
    kp, vp = (pool_like(8, 1, 16, 64, torch.bfloat16, "hnd", 3.0) for _ in range(2))
    table = _i32(np.arange(8).reshape(4, 2))
    for cu, at, want in (([-1, 0, 2, 4, 6], [0] * 4, L.DEV_BAD_LEN), ([0, 2, 2, 4, 6], [0, 33, 0, 0], L.DEV_BAD_LEN),
                         ([0, 2, 2, 4, 6], [0, 32, 0, 0], 0), ([2, 2, 2, 4, 5], [0] * 4, 0)):
        st = _i32([0])
        L.fastar_paged_append(k, k, kp, vp, table, _i32(at), cu=_i32(cu), dev_status=st)
        torch.cuda.synchronize()
        assert st.item() == want


@pytest.mark.parametrize("d,nq", [(64, 130), (128, 130), (128, 300)])
@pytest.mark.parametrize("ws", [True, False])
def test_values_that_are_not_finite_among_many_sequences_that_see_nothing(d, nq, ws):
    """Sequences whose pages end before their window, a run of them between two that see their rows: pieces without
    a key tile go by while the ones before are still written."""
    B, page, cap, window = 700, 32, 448, 40
    full = np.arange(B) % 9 != 4
    at = np.where(full, cap, 430 - nq)
    table = np.full((B, cap // page), -1, np.int32)
    own = np.flatnonzero(~full)                              # they see rows 390 .. 429
    table[own, 12:14] = np.arange(2 * len(own)).reshape(-1, 2)
    kp, vp = (_rand((2 * len(own), 1, page, d), s).bfloat16() for s in (1, 2))
    q = _rand((1, B * nq, d), 3).bfloat16()
    clean = run_attn(q, kp, vp, table, at, None, 0.1, 0, window, 0, ws=ws)
    tok = torch.from_numpy((own[:, None] * nq + np.arange(nq)).reshape(-1)).cuda()
    rest = torch.ones(B * nq, dtype=torch.bool, device=DEV)
    rest[tok] = False
    assert bool((clean[0][:, rest] == 0).all()) and bool(torch.isneginf(clean[1][:, rest]).all())
    check_attn("bf16", q[:, tok], kp, vp, table[own], at[own], None, 0.1, 0, window, 0, clean[0][:, tok], clean[1][:, tok])
    bad, what = vp.clone(), float("inf")
    bad[table[own, 12], 0, 16, 3] = what                     # row 400
    bad[table[own, 12], 0, 17, d - 1] = -what
    for _ in range(3):
        out, lse = run_attn(q, kp, bad, table, at, None, 0.1, 0, window, 0, ws=ws)
        assert torch.equal(lse, clean[1]) and torch.equal(out[:, rest], clean[0][:, rest])
        assert bool((out[:, tok, 3] == what).all()) and bool((out[:, tok, d - 1] == -what).all())
        keep = [c for c in range(d) if c not in (3, d - 1)]
        assert torch.equal(out[:, tok][..., keep], clean[0][:, tok][..., keep])


@pytest.mark.parametrize("d,G,nq", [(64, 2, 70), (128, 2, 70), (128, 1, 90), (128, 3, 200)])
def test_values_that_are_not_finite_are_those_of_their_piece(d, G, nq):
    """Every other sequence that sees something has a NaN, in the channels of one CTA of a pair or of the other; between
    them up to twenty that see nothing: what is taken out of one piece's V comes back to that piece."""
    B, Hk, page, cap, window = 400, 2, 32, 256, 20
    rng = np.random.default_rng(nq)
    full = rng.random(B) < 0.9
    full[:3] = False
    own = np.flatnonzero(~full)
    at = np.where(full, cap, 120 - nq if nq <= 120 else 0)
    end = int(at[own[0]]) + nq
    table = np.full((B, cap // page), -1, np.int32)
    need = list(range(max(0, end - window) // page, (end - 1) // page + 1))
    table[np.ix_(own, need)] = np.arange(len(own) * len(need)).reshape(-1, len(need))
    kp, vp = (_rand((len(own) * len(need), Hk, page, d), s).bfloat16() for s in (1, 2))
    q = _rand((Hk * G, B * nq, d), 3).bfloat16()
    clean = run_attn(q, kp, vp, table, at, None, 0.1, 0, window, 0)
    row, bad = end - 3, vp.clone()
    chs = {}
    for x, b in enumerate(own):
        if x % 2:
            chs[b] = 1 if x % 4 == 1 else d - 2
            bad[int(table[b, row // page]), 1, row % page, chs[b]] = float("nan")
    for _ in range(3):
        out, lse = run_attn(q, kp, bad, table, at, None, 0.1, 0, window, 0)
        assert torch.equal(lse, clean[1]) and torch.equal(out[:G], clean[0][:G])
        want = clean[0].clone()
        for b, ch in chs.items():
            want[G:, b * nq:(b + 1) * nq, ch] = float("nan")
        assert torch.equal(out.isnan(), want.isnan()) and torch.equal(out.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,nq,page,layout", [(64, 20, 128, "nhd"), (128, 1, 16, "hnd"), (128, 10, 128, "nhd"), (128, 16, 64, "hnd"),
                                             (128, 50, 128, "hnd"), (128, 60, 16, "nhd"), (128, 100, 128, "nhd"),
                                             (128, 300, 16, "hnd"), (128, 700, 128, "nhd")])
@pytest.mark.parametrize("ws", [True, False])
def test_values_that_are_not_finite_reach_who_sees_them(dtype, d, nq, page, layout, ws):
    """Infinities and NaN in rows of V that some tokens see and others do not, and in rows that all see: by few rows, a
    CTA alone, a pair with one row tile and with two; in channels of both CTAs of a pair, and in all."""
    Hk, G, at, block, window, sinks = 2, 2, 600, 1, 150, 20
    q, kp, vp, table, a, cu = attn_case(dtype, [nq], [at], Hk, G, d, page, layout, block, window, sinks, seed=nq)
    scale = 1 / math.sqrt(d)
    clean = run_attn(q, kp, vp, table, a, cu, scale, block, window, sinks, ws=ws)
    see = P.sees(nq, at, at + nq, block, window, sinks)
    for i, row in enumerate(sorted({at + nq - 1, at + nq // 2, at - window + 1, at + nq - window, 19, 0})):
        if not see[:, row].any():
            continue
        what = (float("nan"), float("inf"), float("-inf"))[i % 3]
        for ch in ([3], [d - 5], [3, d // 2 + 1], list(range(d))):
            pg, of = int(table[0, row // page]), row % page
            keep = vp[pg, 1, of].clone()
            vp[pg, 1, of, ch] = what
            out, lse = run_attn(q, kp, vp, table, a, cu, scale, block, window, sinks, ws=ws)
            vp[pg, 1, of] = keep
            rows = torch.from_numpy(see[:, row]).cuda()
            assert torch.equal(lse, clean[1]) and torch.equal(out[:G], clean[0][:G])
            assert torch.equal(out[G:, ~rows], clean[0][G:, ~rows])
            got = out[G:, rows]
            assert bool(torch.isnan(got[..., ch]).all() if what != what else (got[..., ch] == what).all())
            other = [c for c in range(d) if c not in ch]
            assert torch.equal(got[..., other], clean[0][G:, rows][..., other])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 30, 40, 100, 200, 600])
def test_large_and_lopsided_logits_of_128_channels(dtype, nq):
    """Logits of hundreds and rows of keys that rise, fall, or lie 30 below one strong key whose V is 0: the reference
    moves in the middle, in every kernel for 128 channels."""
    d, page, n = 128, 128, 1000
    q, kp, vp, table, a, cu = attn_case(dtype, [nq], [n - nq], 1, 1, d, page, "hnd", 0, 0, 0, seed=2)
    row = torch.arange(n, device=DEV)
    pg, of = torch.from_numpy(table[0]).long().cuda()[row // page], row % page
    for shape in (row * 0.5, -row * 0.5, torch.where(row == 517, 30.0, 0.0)):
        kp[pg, :, of] = 0
        kp[pg, 0, of, 70] = shape.to(kp.dtype)
        if float(shape.max()) == 30.0:
            vp[pg[517], :, of[517]] = 0
        q[...] = 0
        q[:, :, 70] = 1.0
        out, lse = run_attn(q, kp, vp, table, a, cu, 1.0, 0, 0, 0)
        check_attn(dtype, q, kp, vp, table, a, cu, 1.0, 0, 0, 0, out, lse)


@pytest.mark.parametrize("ws", [True, False])
@pytest.mark.parametrize("nq,at,Hk,G,d,page,block,window,sinks", [
    ([1], [332], 12, 1, 128, 64, 1, 0, 0), ([1] * 4, [2000, 5, 700, 40], 2, 4, 128, 16, 1, 500, 9),
    ([2, 1], [60, 5000], 1, 8, 64, 32, 1, 0, 0), ([16], [3000], 3, 1, 128, 128, 1, 1000, 70), ([3], [90], 4, 5, 64, 16, 0, 0, 0),
    ([1, 0, 1], [20000, 3, 17], 1, 16, 128, 32, 1, 0, 0)])
def test_weights_of_a_few_rows_keep_their_precision(nq, at, Hk, G, d, page, block, window, sinks, ws):
    """Up to 16 rows a KV head: P as two bf16, the upper half cut off and the rest (below 2^-7 of it) rounded by
    2^-8 of itself, 2^-15 relative; else as this file's bound for bf16, the output's rounding 2^-8."""
    assert max(nq) * G <= 16
    c = attn_case("bf16", nq, at, Hk, G, d, page, "hnd", block, window, sinks, seed=31)
    scale = 1 / math.sqrt(d)
    out, lse = run_attn(*c, scale, block, window, sinks, ws=ws)
    q, kp, vp, table, a, cu = c
    want, _, A, E, n = P.attention(_np(q), _np(kp), _np(vp), table, a, scale, cu, block, window, sinks)
    e = (d * 2.0 ** -23 + 2.0 ** -22) * E + 2.0 ** -22
    big = np.nan_to_num(np.abs(_np(vp)), nan=0.0).max()
    tol = 2.0 ** -8 * np.abs(want) + n[None, :, None] * 2.0 ** -100 * big + A * (4 * e + n * 2.0 ** -22 + 2.0 ** -15)[..., None]
    assert (np.abs(_np(out) - want) <= tol).all(), (np.abs(_np(out) - want) / tol).max()
