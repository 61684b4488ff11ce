"""GPU parity of the 4-bit key/value cache (fastar_kv4_append, fastar_kv4_read,
fastar_kv4_attn) against its float64 oracle.

The stored bits are exact decisions, so codes, scales and read values are compared bit for
bit.  Attention bounds, from the oracle's own quantities: A = sum_j p_j |v_j| (the mean of |v|
under the softmax), E = sum_c |q_c| max_j |k_jc| * scale (no logit's products sum to more):
  - a logit is d products summed in fp32, 2 d 2^-24 E at most (rounded or truncated sums),
    then one product; e^x adds 2^-22 and the argument's own rounding 2^-23 E; so every p is off
    by e = (d 2^-23 + 2^-22) E + 2^-22 relative (for e < 1/16: doubled covers e^e - 1), and the
    quotient of two such sums by 2 e;
  - bf16 calls hold p in fp16: 2^-11 relative, but below 2^-14 absolute, half the spacing 2^-24
    of its subnormals.  That part is not relative to A: a p that rounds to 0 loses its v_j
    however little the other v add up to in that channel (where the strongest key's value is a
    stored 0, O is made of small p alone).  It is at most 2^-25 sum_j |v_j| over a sum of p that
    is at least 1 (the reference maximum was some key's logit, whose p is 1, or is below one);
  - fp32 calls hold p in two fp16 parts of 22 bits (2^-22 relative, in 2 e's doubled terms: n 2^-22
    covers it), and the small ones, whose second part lies below fp16's range, to 2^-25 of a scale
    on which the largest p is at least 2^13: 2^-38 sum_j |v_j|;
  - an exponential under fp32's range is 0: 2^-126 sum_j |v_j| in the same way;
  - sums over n keys in fp32: n 2^-23 relative at most;
  - the output's rounding: 2^-8 |O| in bf16, 2^-24 |O| in fp32.
  |O - want| <= half |want| + A (4 e + n 2^-22 + [bf16] 2^-11) + sum_j |v_j| ([bf16] 2^-25, [fp32] 2^-38)
  |lse - want| <= 2 e + n 2^-22 + 2^-22 (1 + |want|)."""
import math

import numpy as np
import pytest
import torch

from kv_cache_tempcache_gb300 import _lib as L
from oracle import kv4_oracle as K

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


def _np(t):
    return t.detach().double().cpu().numpy()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _empty_cache(H, cap, d, fill=0):
    mk = lambda w: torch.full((H, cap, w), fill, dtype=torch.uint8, device=DEV)
    return mk(d // 2), mk(d // 16), mk(d // 2), mk(d // 16)


def _rand(shape, seed, std=1.0):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV) * std


# ---- append and read ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,n,d,cap,at", [(1, 1, 64, 16, [0]), (3, 5, 128, 32, [0, 27, 11]), (2, 331, 64, 400, [69, 3]),
                                          (12, 1560, 128, 3200, [1640 - i for i in range(12)])])
def test_append_bits_and_read_values(dtype, H, n, d, cap, at):
    dt = DT[dtype]
    x = _rand((2, n, H, d), n, 1.0)
    x[:, :, :, : d // 4] *= torch.exp2(_rand((2, n, H, d // 4), n + 1, 4.0))        # a wide range of scales
    x = x.to(dt)
    k, v = x[0].transpose(0, 1), x[1].transpose(0, 1)                                # token-major
    kc, ks, vc, vs = _empty_cache(H, cap, d, 0xA5)
    len_out, status = _i32([-1] * H), _i32([0])
    L.fastar_kv4_append(k, v, kc, ks, vc, vs, _i32(at), len_out, status)
    torch.cuda.synchronize()
    assert len_out.tolist() == [a + n for a in at] and status.item() == 0
    for t, codes, scales in ((k, kc, ks), (v, vc, vs)):
        wc, ws = K.quantise(_np(t))
        out = torch.empty(H, cap, d, dtype=dt, device=DEV)
        L.fastar_kv4_read(codes, scales, 0, out)
        gc, gs, o = codes.cpu().numpy(), scales.cpu().numpy(), _np(out)
        for h, a in enumerate(at):
            assert np.array_equal(gs[h, a:a + n], ws[h]) and np.array_equal(gc[h, a:a + n], wc[h])
            # rows around the appended ones are left as they were
            assert (gc[h, :a] == 0xA5).all() and (gc[h, a + n:] == 0xA5).all()
            assert (gs[h, :a] == 0xA5).all() and (gs[h, a + n:] == 0xA5).all()
            assert np.array_equal(o[h, a:a + n], K.values(wc[h], ws[h]))


def test_every_bf16_magnitude_at_every_scale_is_rounded_as_defined():
    # one strong channel fixes the block's scale, the other 15 walk through the bf16 values
    # between 0 and the largest: ties included
    rows = []
    for big in torch.arange(1.0, 2.0, 1 / 128).tolist():
        mags = torch.cat([torch.arange(1.0, 2.0, 1 / 128) * 2.0 ** e for e in range(-6, 1)])
        mags = mags[mags <= big]
        pad = (-len(mags)) % 15
        m = torch.cat((mags, torch.zeros(pad))).view(-1, 15)
        rows.append(torch.cat((torch.full((m.shape[0], 1), -big), m), 1))
    x = torch.cat(rows)
    x = torch.cat((x, x * 0.0078125, x * 512.0))
    x = torch.cat((x, torch.zeros((-x.shape[0]) % 4, 16))).view(1, -1, 64)
    n = x.shape[1]
    cap = (n + 15) // 16 * 16
    for dt in (torch.bfloat16, torch.float32):
        y = x.to(dt).cuda()
        c = _empty_cache(1, cap, 64)
        L.fastar_kv4_append(y, -y, *c)
        torch.cuda.synchronize()
        for t, codes, scales in ((y, c[0], c[1]), (-y, c[2], c[3])):
            wc, ws = K.quantise(_np(t))
            assert np.array_equal(scales[:, :n].cpu().numpy(), ws)
            assert np.array_equal(codes[:, :n].cpu().numpy(), wc)


def test_fp32_next_to_the_borders():
    # scales: maxima one step below, at and above 6 x (the middle of two e4m3 numbers);
    # codes: values one step around the middles times the scale
    mids = (K.E4M3[1:] + K.E4M3[:-1]) / 2 * 6
    a = np.concatenate([np.float32(mids), np.nextafter(np.float32(mids), np.float32(0)),
                        np.nextafter(np.float32(mids), np.float32(1e9))])
    x = np.zeros((len(a), 16), np.float32)
    x[:, 0] = a
    s = K.E4M3[K.quantise(x)[1]][:, 0]
    for i in range(7):
        m = np.float32(s * (K.E2M1[i] + K.E2M1[i + 1]) / 2)
        x[:, 1 + 2 * i] = np.nextafter(m, np.float32(0)) if i % 2 else m
        x[:, 2 + 2 * i] = -np.nextafter(m, np.float32(1e9))
    x = np.concatenate((x, np.zeros(((-len(x)) % 4, 16), np.float32))).reshape(1, -1, 64)
    n = x.shape[1]
    c = _empty_cache(1, (n + 15) // 16 * 16, 64)
    y = torch.from_numpy(x).cuda()
    L.fastar_kv4_append(y, y, *c)
    torch.cuda.synchronize()
    wc, ws = K.quantise(x)
    assert np.array_equal(c[1][:, :n].cpu().numpy(), ws) and np.array_equal(c[0][:, :n].cpu().numpy(), wc)
    assert torch.equal(c[0], c[2]) and torch.equal(c[1], c[3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_not_finite_is_stored_as_zero_and_flagged_and_exponents(dtype):
    H, n, d = 2, 6, 64
    k = _rand((H, n, d), 5, 2.0 ** -12).to(DT[dtype])
    v = _rand((H, n, d), 6, 3000.0).to(DT[dtype])
    ke, ve = _i32([-12, -9]), _i32([8, 10])
    c, status = _empty_cache(H, 16, d), _i32([0])
    L.fastar_kv4_append(k, v, *c, None, None, status, ke, ve)
    torch.cuda.synchronize()
    assert status.item() == 0
    for t, codes, scales, e in ((k, c[0], c[1], ke), (v, c[2], c[3], ve)):
        out = torch.empty(H, n, d, dtype=DT[dtype], device=DEV)
        L.fastar_kv4_read(codes, scales, 0, out, exps=e)
        for h in range(H):
            wc, ws = K.quantise(_np(t[h]), int(e[h]))
            assert np.array_equal(codes[h, :n].cpu().numpy(), wc) and np.array_equal(scales[h, :n].cpu().numpy(), ws)
            assert np.array_equal(_np(out[h]), K.values(wc, ws, int(e[h])))
    k[0, 2, 3], k[1, 5, 63] = float("nan"), float("-inf")
    L.fastar_kv4_append(k, v, *c, None, None, status, ke, ve)
    torch.cuda.synchronize()
    assert status.item() == L.DEV_NONFINITE
    for h in range(H):
        wc, ws = K.quantise(_np(k[h]), int(ke[h]))
        assert np.array_equal(c[0][h, :n].cpu().numpy(), wc) and np.array_equal(c[1][h, :n].cpu().numpy(), ws)
    big = torch.full((H, n, d), 3.0e38, dtype=DT[dtype], device=DEV)     # 2^64 times this overflows: held to the largest
    L.fastar_kv4_append(big, -big, *c, None, None, _i32([0]), _i32([-64, 0]), _i32([-64, 0]))
    torch.cuda.synchronize()
    assert (c[1][:, :n] == 126).all() and (c[0][:, :n] == 0x77).all() and (c[2][:, :n] == 0xFF).all()


def test_append_past_the_capacity_and_bad_starts():
    H, n, d, cap = 4, 10, 64, 32
    k = _rand((H, n, d), 8).bfloat16()
    c, len_out, status = _empty_cache(H, cap, d, 0x5A), _i32([0] * H), _i32([0])
    L.fastar_kv4_append(k, k, *c, _i32([3, 25, -1, 33]), len_out, status)
    torch.cuda.synchronize()
    assert status.item() == L.DEV_BAD_LEN and len_out.tolist() == [13, 32, 0, 32]
    wc, _ = K.quantise(_np(k))
    g = c[0].cpu().numpy()
    assert np.array_equal(g[0, 3:13], wc[0]) and np.array_equal(g[1, 25:], wc[1, :7])
    assert (g[2:] == 0x5A).all() and (g[0, 13:] == 0x5A).all()
    empty = torch.empty(H, 0, d, dtype=torch.bfloat16, device=DEV)       # nothing to append: the lengths pass on
    L.fastar_kv4_append(empty, empty, *c, _i32([3, 25, 0, 32]), len_out, _i32([0]))
    torch.cuda.synchronize()
    assert len_out.tolist() == [3, 25, 0, 32] and np.array_equal(c[0].cpu().numpy(), g)


def test_offsets_past_32_bits():
    # the third head's codes start at 2^32 bytes
    H, d, cap, n = 3, 128, 2 ** 25, 7
    mk = lambda w: torch.empty((H, cap, w), dtype=torch.uint8, device=DEV)
    c = (mk(64), mk(8), mk(64), mk(8))
    at = _i32([5, cap - n, cap - n])
    x = _rand((2, H, n, d), 9).bfloat16()
    len_out, status = _i32([0] * H), _i32([0])
    L.fastar_kv4_append(x[0], x[1], *c, at, len_out, status)
    for i in range(2):
        out = torch.empty(H, n, d, dtype=torch.bfloat16, device=DEV)
        L.fastar_kv4_read(c[2 * i], c[2 * i + 1], cap - n, out)
        torch.cuda.synchronize()
        want = K.values(*K.quantise(_np(x[i])))
        assert np.array_equal(_np(out)[1:], want[1:])
    assert status.item() == 0 and len_out.tolist() == [5 + n, cap, cap]
    # attention over short and empty histories of the far heads, with and without splits
    k = _rand((2, H, 40, d), 10).bfloat16()
    L.fastar_kv4_append(k[0], k[1], *c, None, None, status)
    q = _rand((2 * H, 3, d), 11).bfloat16()
    _attend(q, c, [40, 0, 39], 0, vals=[K.values(*K.quantise(_np(k[i]))) for i in range(2)])


# ---- attention -----------------------------------------------------------------------------------

def _check_attn(out, lse, q, kv, vv, lens, scale, block):
    want, wl, A, E = K.attention(_np(q), kv, vv, lens, scale, block)
    d, n = q.shape[2], max(1, max(lens))
    bf16 = q.dtype == torch.bfloat16
    e = (d * 2.0 ** -23 + 2.0 ** -22) * E + 2.0 ** -22
    assert e.max() < 1 / 16
    half = 2.0 ** -8 if bf16 else 2.0 ** -24
    tol = half * np.abs(want) + A * (4 * e + n * 2.0 ** -22 + (2.0 ** -11 if bf16 else 0))[..., None]
    lost = np.stack([np.abs(vv[h * len(lens) // q.shape[0], :lens[h * len(lens) // q.shape[0]]]).sum(0)
                     for h in range(q.shape[0])])
    tol += lost[:, None] * ((2.0 ** -25 if bf16 else 2.0 ** -38) + 2.0 ** -126)
    err = np.abs(_np(out) - want)
    assert not np.isnan(err).any()
    assert (err <= tol).all(), f"{int((err > tol).sum())} of {err.size} outside; worst ratio {(err / np.maximum(tol, 1e-300)).max():.2f}"
    dead = np.isneginf(wl)
    gl = _np(lse)
    assert np.array_equal(np.isneginf(gl), dead)
    live = ~dead
    tl = 2 * e + n * 2.0 ** -22 + 2.0 ** -22 * (1 + np.abs(np.where(live, wl, 0)))
    assert (np.abs(gl[live] - wl[live]) <= tl[live]).all()


def _attend(q, c, lens, block, vals=None, scale=None, split=(True, False), **kw):
    """Runs with and without a workspace, checks both, and returns the first."""
    Hq, nq, d = q.shape
    Hkv, cap = c[0].shape[:2]
    scale = 1 / math.sqrt(d) if scale is None else scale
    if vals is None:
        vals = [K.values(c[2 * i].cpu().numpy(), c[2 * i + 1].cpu().numpy()) for i in range(2)]
    first = None
    for with_ws in split:
        nb = L.workspace_bytes(L.OP_KV4_ATTN, Hq, nq, cap, d, Hkv) if with_ws else 0
        ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device=DEV) if nb else None
        # rows in front of, between and behind the outputs have to stay as they are
        buf = torch.full((nq + 2, Hq + 1, d), 7.0, dtype=q.dtype, device=DEV)
        out = buf[1:-1, :Hq].transpose(0, 1)
        lse = torch.full((Hq, nq), 7.0, device=DEV)
        status = _i32([0])
        L.fastar_kv4_attn(q, *c, _i32(lens), scale, out, lse, block=block, dev_status=status, workspace=ws, **kw)
        torch.cuda.synchronize()
        assert status.item() == 0
        assert (buf[0] == 7).all() and (buf[-1] == 7).all() and (buf[:, Hq] == 7).all()
        _check_attn(out, lse, q, vals[0], vals[1], lens, scale, block)
        if first is None:
            first = out.clone(), lse
    return first


def _filled(Hkv, cap, d, seed, std=1.0):
    x = _rand((2, Hkv, cap, d), seed, std).bfloat16()
    c = _empty_cache(Hkv, cap, d)
    L.fastar_kv4_append(x[0], x[1], *c)
    return c


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hkv,G,nq,d,cap,lens,block", [
    (1, 1, 1, 128, 16, [0], 0), (1, 1, 1, 128, 16, [1], 0), (2, 1, 1, 64, 16, [0, 16], 0),
    (3, 4, 1, 128, 1024, [333, 1, 1024], 0), (1, 8, 2, 64, 528, [517], 1), (2, 2, 5, 128, 2048, [2048, 1999], 0),
    (2, 1, 8, 128, 272, [257, 256], 1), (1, 3, 9, 64, 144, [129], 4), (8, 4, 1, 128, 8192, [8191, 0, 1, 63, 64, 65, 4097, 8192], 0),
    (1, 1, 33, 128, 80, [65], 7), (2, 2, 17, 64, 128, [16, 3], 1)])
def test_few_rows(dtype, Hkv, G, nq, d, cap, lens, block):
    c = _filled(Hkv, cap, d, cap + nq)
    q = _rand((nq, Hkv * G, d), nq, 1.5).to(DT[dtype]).transpose(0, 1)
    _attend(q, c, lens, block)


@pytest.mark.parametrize("Hkv,G,nq,d,cap,lens,block", [
    (1, 1, 127, 128, 144, [129], 0), (1, 1, 128, 128, 128, [128], 1), (2, 1, 129, 128, 272, [127, 257], 0),
    (2, 1, 256, 64, 512, [512, 300], 64), (1, 1, 257, 128, 400, [385], 257), (1, 2, 300, 64, 912, [899], 100),
    (3, 1, 331, 128, 1024, [0, 1000, 100], 1), (2, 3, 90, 128, 256, [255, 91], 1), (1, 1, 700, 128, 2000, [1999], 0),
    (4, 2, 260, 64, 5008, [5000, 4999, 1, 260], 130)])
def test_many_rows(Hkv, G, nq, d, cap, lens, block):
    c = _filled(Hkv, cap, d, cap + nq)
    q = _rand((nq, Hkv * G, d), nq, 1.5).bfloat16().transpose(0, 1)
    _attend(q, c, lens, block)


@pytest.mark.parametrize("Hkv,G,nq,d,cap,lens,block", [
    (1, 1, 17, 128, 16, [0], 0), (1, 1, 17, 128, 16, [1], 1), (4, 4, 8, 128, 400, [127, 128, 129, 385], 0),
    (2, 1, 128, 128, 272, [257, 100], 1), (1, 8, 16, 128, 1040, [1025], 5), (3, 1, 64, 128, 4112, [4100, 0, 2000], 0),
    (2, 1, 100, 128, 60000, [60000, 777], 0), (40, 1, 33, 128, 1008, [25 * h + 8 for h in range(40)], 11),
    (20, 2, 11, 128, 3008, [3000] * 20, 0)])
def test_rows_of_one_tile(Hkv, G, nq, d, cap, lens, block):
    # 17 to 128 rows a KV head: one row tile, on even and odd key tiles; by CTAs alone where the cache
    # is large (the last three), else in pairs
    c = _filled(Hkv, cap, d, cap + nq)
    q = _rand((nq, Hkv * G, d), nq, 1.5).bfloat16().transpose(0, 1)
    _attend(q, c, lens, block)


@pytest.mark.parametrize("Hkv,G,nq,d,cap,lens,block", [
    (1, 1, 300, 128, 912, [899], 100), (2, 2, 90, 64, 2064, [2050, 0], 1), (3, 1, 17, 128, 3008, [3000, 5, 1025], 0)])
def test_many_fp32_rows(Hkv, G, nq, d, cap, lens, block):
    c = _filled(Hkv, cap, d, cap + nq)
    q = _rand((nq, Hkv * G, d), nq, 1.5).transpose(0, 1)
    _attend(q, c, lens, block)


@pytest.mark.parametrize("nq,block", [(1100, 0), (1100, 500), (2100, 0), (2100, 500)])
def test_splits_follow_the_lengths(nq, block):
    # heads that fill the cache, half fill it, need no split, hold less than the call's tokens, or
    # nothing; the last rows of a head fill one row tile; with 2100 tokens the keys are split
    H, d, cap = 24, 128, 16000
    lens = [200 + 37 * h for h in range(H)]
    lens[:6] = [16000, 11000, 0, 1, 1099, 5200]
    c = _empty_cache(H, cap, d)
    x = _rand((2, H, 1100, d), 40).bfloat16()
    for at in range(0, 15400, 1100):                       # the same rows over and over, scaled
        y = (x * (1 + at / 20000)).bfloat16()
        L.fastar_kv4_append(y[0], y[1], *c, _i32([at] * H))
    n = 16000 - 15400
    L.fastar_kv4_append(x[0, :, :n], x[1, :, :n], *c, _i32([15400] * H))
    q = _rand((nq, H, d), 41, 1.5).bfloat16().transpose(0, 1)
    assert nq == 1100 or L.workspace_bytes(L.OP_KV4_ATTN, H, nq, cap, d, H) > 0
    vals = [np.zeros((H, cap, d)) for _ in range(2)]
    for i in range(2):
        codes, scales = c[2 * i].cpu().numpy(), c[2 * i + 1].cpu().numpy()
        for h, m in enumerate(lens):
            vals[i][h, :m] = K.values(codes[h, :m], scales[h, :m])
    a = _attend(q, c, lens, block, vals)
    b = _attend(q, c, lens, block, vals, split=(True,))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_a_zero_query_under_the_largest_scales():
    c = _filled(1, 64, 64, 50)
    for nq in (2, 200):
        for dt in (torch.bfloat16, torch.float32):
            q = torch.zeros(1, nq, 64, dtype=dt, device=DEV)
            out, lse = torch.empty_like(q), torch.empty(1, nq, device=DEV)
            L.fastar_kv4_attn(q, *c, _i32([61]), 2.9e38, out, lse, k_exp=_i32([64]))
            torch.cuda.synchronize()
            want = K.values(c[2][0, :61].cpu().numpy(), c[3][0, :61].cpu().numpy()).mean(0)
            # uniform weights: 61 fp32 products and sums (61 2^-23), and the output's rounding
            half = 2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -24
            assert (np.abs(_np(out)[0] - want) <= half * np.abs(want) + 61 * 2.0 ** -22 * 6).all()
            assert (np.abs(_np(lse) - math.log(61)) <= 2.0 ** -20).all()


@pytest.mark.parametrize("dtype,nq", [("f32", 5), ("bf16", 1), ("bf16", 5), ("bf16", 300)])
def test_rows_behind_the_length_never_count(dtype, nq):
    # behind the lengths: scales that read as NaN and the largest codes
    Hkv, d, cap, lens = 2, 128, 416, [385, 7]
    c = _filled(Hkv, cap, d, 1)
    vals = [K.values(c[2 * i].cpu().numpy(), c[2 * i + 1].cpu().numpy()) for i in range(2)]
    q = _rand((Hkv, nq, d), 2).to(DT[dtype])
    want = _attend(q, c, lens, 0, vals)
    for h, n in enumerate(lens):
        for t, x in zip(c, (0x77, 0x7F, 0x77, 0x7F)):
            t[h, n:] = x
    got = _attend(q, c, lens, 0, vals)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("dtype,nq", [("f32", 5), ("bf16", 5), ("bf16", 200)])
def test_a_query_that_is_not_finite_stays_alone(dtype, nq):
    c = _filled(2, 272, 64, 3)
    q = _rand((2, nq, 64), 4).to(DT[dtype])
    want = _attend(q, c, [259, 130], 0)
    q2 = q.clone()
    q2[0, 1, 5], q2[1, 3, 0] = float("nan"), float("inf")
    out, lse = torch.empty_like(q), torch.empty(2, nq, device=DEV)
    L.fastar_kv4_attn(q2, *c, _i32([259, 130]), 1 / 8, out, lse)
    nb = L.workspace_bytes(L.OP_KV4_ATTN, 2, nq, 272, 64, 2)
    ref, rl = torch.empty_like(q), torch.empty(2, nq, device=DEV)
    L.fastar_kv4_attn(q, *c, _i32([259, 130]), 1 / 8, ref, rl)
    torch.cuda.synchronize()
    bad = torch.zeros(2, nq, dtype=torch.bool, device=DEV)
    bad[0, 1] = bad[1, 3] = True
    assert torch.isnan(out[bad]).all()
    assert torch.equal(out[~bad], ref[~bad]) and torch.equal(lse[~bad], rl[~bad])


@pytest.mark.parametrize("nq", [2, 150])
@pytest.mark.parametrize("mag", [2.0 ** -100, 2.0 ** -20, 2.0 ** 12, 2.0 ** 100])
def test_query_magnitudes(nq, mag):
    # rows far from 1: the scale brings the logits back to order one
    c = _filled(1, 320, 128, 5)
    q = (_rand((1, nq, 128), 6) * mag).bfloat16()
    q[0, 0] = 0                                        # uniform weights
    _attend(q, c, [311], 0, scale=float(np.float32(0.1 / mag)) if mag < 2.0 ** 100 else float(np.float32(2.0 ** -103)))


@pytest.mark.parametrize("dtype,nq", [("f32", 3), ("bf16", 3), ("bf16", 140)])
def test_exponents_of_the_cache(dtype, nq):
    H, d, cap, lens = 2, 64, 528, [517, 300]
    x = _rand((2, H, cap, d), 7)
    x[0] *= 2.0 ** -10
    x[1] *= 2.0 ** 13
    x = x.to(DT[dtype])
    ke, ve = _i32([-10, -11]), _i32([13, 12])
    c = _empty_cache(H, cap, d)
    L.fastar_kv4_append(x[0], x[1], *c, None, None, None, ke, ve)
    q = (_rand((H, nq, d), 8) * 2.0 ** 10).to(DT[dtype])
    vals = [np.stack([K.values(c[2 * i][h].cpu().numpy(), c[2 * i + 1][h].cpu().numpy(), int(e[h])) for h in range(H)])
            for i, e in ((0, ke), (1, ve))]
    _attend(q, c, lens, 0, vals, k_exp=ke, v_exp=ve)


@pytest.mark.parametrize("nq", [1, 200])
def test_sharp_rows(nq):
    # one key dominates, then a later one by far: the running maximum has to move, often
    d, n = 128, 1500
    x = _rand((2, 1, n, d), 9).bfloat16()
    x[0, 0] *= torch.linspace(0.1, 3.0, n, device=DEV)[:, None].bfloat16()
    c = _empty_cache(1, 1504, d)
    L.fastar_kv4_append(x[0], x[1], *c)
    q = (x[0, 0, torch.arange(nq, device=DEV) * 7 + 3][None] * 2).contiguous()
    _attend(q, c, [n], 0)


def test_lengths_out_of_range_are_held_and_flagged():
    c = _filled(2, 64, 64, 11)
    q = _rand((2, 2, 64), 12).bfloat16()
    out, lse, status = torch.empty_like(q), torch.empty(2, 2, device=DEV), _i32([0])
    L.fastar_kv4_attn(q, *c, _i32([-5, 70]), 0.1, out, lse, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == L.DEV_BAD_LEN
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()
    vals = [K.values(c[2 * i].cpu().numpy(), c[2 * i + 1].cpu().numpy()) for i in range(2)]
    _check_attn(out[1:], lse[1:], q[1:], vals[0][1:], vals[1][1:], [64], 0.1, 0)


@pytest.mark.parametrize("nq,G", [(1, 1), (3, 4), (300, 1)])
def test_captured_graph_follows_the_lengths_and_repeats_bit_for_bit(nq, G):
    H, d, cap = 2, 128, 4096
    c = _filled(H, cap, d, 13)
    q = _rand((H * G, nq, d), 14).bfloat16()
    lens = _i32([0, 0])
    out, lse = torch.empty_like(q), torch.empty(H * G, nq, device=DEV)
    nb = L.workspace_bytes(L.OP_KV4_ATTN, H * G, nq, cap, d, H)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV) if nb else None
    call = lambda o, l: L.fastar_kv4_attn(q, *c, lens, 0.09, o, l, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(out, lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(out, lse)
    for n in ([1, 4096], [0, 333], [4000, 129]):
        lens.copy_(_i32(n))
        g.replay()
        torch.cuda.synchronize()
        a, b = out.clone(), lse.clone()
        o2, l2 = torch.empty_like(out), torch.empty_like(lse)
        call(o2, l2)
        torch.cuda.synchronize()
        assert torch.equal(a, o2) and torch.equal(b, l2)
        vals = [K.values(c[2 * i].cpu().numpy(), c[2 * i + 1].cpu().numpy()) for i in range(2)]
        _check_attn(a, b, q, vals[0], vals[1], n, 0.09, 0)


def test_two_calls_on_two_streams():
    c = _filled(2, 2048, 128, 15)
    qs = [_rand((2, n, 128), 16 + n).bfloat16() for n in (1, 400)]
    outs, streams = [torch.empty_like(q) for q in qs], [torch.cuda.Stream() for _ in qs]
    ref = [_attend(q, c, [2000, 1777], 0)[0] for q in qs]
    lens = _i32([2000, 1777])
    wss = []
    for q in qs:
        nb = L.workspace_bytes(L.OP_KV4_ATTN, 2, q.shape[1], 2048, 128, 2)
        wss.append(torch.empty(nb, dtype=torch.uint8, device=DEV) if nb else None)
    torch.cuda.synchronize()
    for _ in range(5):
        for q, o, s, ws in zip(qs, outs, streams, wss):
            L.fastar_kv4_attn(q, *c, lens, 1 / math.sqrt(128), o, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for o, r in zip(outs, ref):
        assert torch.equal(o, r)


def test_norm_append_attend_as_a_block_runs_them():
    """Three chunks through norm and rotation, append and attention, with the lengths on the
    device: each step against the oracle on its own inputs."""
    Hq, Hkv, n, d, cap, axes = 4, 2, 130, 128, 400, (44, 42, 42)
    c = _empty_cache(Hkv, cap, d)
    lens, lens2, status = _i32([0, 0]), _i32([0, 0]), _i32([0])
    wq, wk = 1 + _rand((d,), 20, 0.1), 1 + _rand((d,), 21, 0.1)
    nb = L.workspace_bytes(L.OP_KV4_ATTN, Hq, n, cap, d, Hkv)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV) if nb else None
    for chunk in range(3):
        qkv = _rand((n, Hq + 2 * Hkv, d), 22 + chunk, 2.0).bfloat16()
        q, k, v = (qkv[:, a:b].transpose(0, 1) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
        raw = qkv.clone()
        L.fastar_qk_norm_rope(q, k, q, k, wq=wq, wk=wk, axes=axes, t0=2 * chunk, grid=(5, 13))
        L.fastar_kv4_append(k, v, *c, lens, lens2, status)
        out, lse = torch.empty(Hq, n, d, dtype=torch.bfloat16, device=DEV), torch.empty(Hq, n, device=DEV)
        L.fastar_kv4_attn(q, *c, lens2, 1 / math.sqrt(d), out, lse, block=65, dev_status=status, workspace=ws)
        lens.copy_(lens2)
        torch.cuda.synchronize()
        assert status.item() == 0 and lens.tolist() == [(chunk + 1) * n] * 2
        pos = K.grid_positions(n, 2 * chunk, 5, 13)
        want, pair = K.norm_rope(_np(raw[:, :Hq].transpose(0, 1)), _np(wq), 1e-6, axes, pos, 10000.0)
        assert (np.abs(_np(q) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * pair).all()
        wc, wsc = K.quantise(_np(k))
        at = chunk * n
        assert np.array_equal(c[0][:, at:at + n].cpu().numpy(), wc) and np.array_equal(c[1][:, at:at + n].cpu().numpy(), wsc)
        vals = [K.values(c[2 * i].cpu().numpy(), c[2 * i + 1].cpu().numpy()) for i in range(2)]
        _check_attn(out, lse, q, vals[0], vals[1], lens.tolist(), 1 / math.sqrt(d), 65)


@pytest.mark.parametrize("dtype,G,nq,d", [("bf16", 4, 1, 128), ("bf16", 1, 40, 128), ("bf16", 2, 300, 64), ("f32", 1, 3, 64)])
def test_a_run_of_calls_equals_one_with_a_wait_after_each(dtype, G, nq, d):
    # launches overlap the kernel before them: every call reads what the last one wrote, into buffers
    # and a workspace that the next one uses again
    Hkv, cap, steps = 4, 12000, 40
    dt = DT[dtype]
    nb = L.workspace_bytes(L.OP_KV4_ATTN, Hkv * G, nq, cap, d, Hkv)
    results = []
    for wait in (True, False):
        c = _empty_cache(Hkv, cap, d)
        start = _rand((2, Hkv, 5000, d), 50).to(dt)
        lens, lens2 = _i32([0] * Hkv), _i32([0] * Hkv)
        L.fastar_kv4_append(start[0], start[1], *c, lens, lens2)
        q = _rand((Hkv * G, nq, d), 51).to(dt)
        k, v = _rand((Hkv, nq, d), 52).to(dt), _rand((Hkv, nq, d), 53).to(dt)
        out, lse = torch.empty_like(q), torch.empty(Hkv * G, nq, device=DEV)
        ws = torch.empty(max(nb, 16), dtype=torch.uint8, device=DEV)
        w = torch.ones(d, device=DEV)
        torch.cuda.synchronize()
        for i in range(steps):
            a, b = (lens2, lens) if i % 2 == 0 else (lens, lens2)
            L.fastar_qk_norm_rope(q, k, q, k, wq=w, wk=w, axes=(d // 2, d // 4, d // 4), t0=i, grid=(5, 7))
            if wait:
                torch.cuda.synchronize()
            L.fastar_kv4_append(k, v, *c, a, b)
            if wait:
                torch.cuda.synchronize()
            L.fastar_kv4_attn(q, *c, b, 0.3, out, lse, workspace=ws)
            if wait:
                torch.cuda.synchronize()
            L.fastar_kv4_read(c[2], c[3], 4990 + i, v)            # the next rows of V: what the cache holds
            if wait:
                torch.cuda.synchronize()
            L.fastar_qk_norm_rope(out, None, q, None, wq=w)       # the next queries: this attention's outputs
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        results.append([x.clone() for x in (*c, q, k, v, out, lse, a, b)])
    for x, y in zip(*results):
        assert torch.equal(x, y)
    assert torch.isfinite(results[0][7].float()).all()
    assert results[0][-1].tolist() == [min(cap, 5000 + steps * nq)] * Hkv


def test_lengths_side_by_side_in_one_buffer():
    H, n, d = 3, 5, 64
    k = _rand((H, n, d), 60).bfloat16()
    for a, b in ((slice(0, H), slice(H, 2 * H)), (slice(H, 2 * H), slice(0, H))):
        buf = _i32([4, 5, 6] * 2)
        L.fastar_kv4_append(k, k, *_empty_cache(H, 16, d), buf[a], buf[b])
        with pytest.raises(L.FastarError):
            L.fastar_kv4_append(k, k, *_empty_cache(H, 16, d), buf[:H], buf[1:H + 1])
        torch.cuda.synchronize()
        assert buf[a].tolist() == [4, 5, 6] and buf[b].tolist() == [9, 10, 11]
