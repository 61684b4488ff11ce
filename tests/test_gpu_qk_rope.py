"""GPU parity of the per-head RMS norm with three-axis rotary positions (fastar_qk_norm_rope)
against its float64 oracle.

Bound, per channel: the output's own rounding, half a step, eps/2 = 2^-8 |want| in bf16 and
2^-24 |want| in fp32; and the fp32 arithmetic before it, relative to the pair's magnitude
|y_2j| + |y_2j+1|: the mean of squares (8 products and 4 shuffle sums, 12 roundings of 2^-24,
halved by the root), root, reciprocal, two products and the rotation's three operations (8
roundings), sine and cosine (2 units of 2^-24 and the angle's 2^-31 turns pi), doubled: under
2^-19."""
import numpy as np
import pytest
import torch

from kv_cache_tempcache_gb300 import _lib as L
from oracle import kv4_oracle as K

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _np(t):
    return t.detach().double().cpu().numpy()


def _check(got, x, w, eps, axes, pos, theta=10000.0):
    want, pair = K.norm_rope(_np(x), None if w is None else _np(w), eps, axes, pos, theta)
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    err = np.abs(_np(got) - want)
    bound = half * np.abs(want) + 2.0 ** -19 * pair
    assert not (err > bound).any(), f"worst {err.max():.3e}, {int((err > bound).sum())} of {err.size} outside"


def _make(n, Hq, Hk, d, dt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = (torch.randn(n, Hq + 2 * Hk, d, generator=g, device="cuda") * 2).to(dt)
    wq = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    wk = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    return qkv, qkv[:, :Hq].transpose(0, 1), qkv[:, Hq:Hq + Hk].transpose(0, 1), wq, wk


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,Hq,Hk,d,axes", [(1, 12, 12, 128, (44, 42, 42)), (1, 1, 1, 64, (24, 20, 20)),
                                            (7, 5, 1, 64, (0, 0, 0)), (61, 3, 2, 128, (128, 0, 0)),
                                            (300, 24, 24, 128, (16, 56, 56)), (1001, 10, 5, 64, (24, 16, 16)),
                                            (4680, 12, 12, 128, (44, 42, 42))])
def test_fused_projection_slices(dtype, n, Hq, Hk, d, axes):
    qkv, q, k, wq, wk = _make(n, Hq, Hk, d, DT[dtype], n)
    before = qkv.clone()
    qo = torch.empty(Hq, n, d, dtype=DT[dtype], device="cuda")
    ko = torch.empty(Hk, n, d, dtype=DT[dtype], device="cuda")
    L.fastar_qk_norm_rope(q, k, qo, ko, wq=wq, wk=wk, eps=1e-6, axes=axes, t0=5, grid=(6, 13))
    torch.cuda.synchronize()
    assert torch.equal(qkv, before)                       # out of place: the inputs stay
    pos = K.grid_positions(n, 5, 6, 13)
    _check(qo, q, wq, 1e-6, axes, pos)
    _check(ko, k, wk, 1e-6, axes, pos)


def test_in_place_equals_out_of_place_and_leaves_the_values_alone():
    qkv, q, k, wq, wk = _make(333, 4, 2, 128, torch.bfloat16)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    L.fastar_qk_norm_rope(q, k, qo, ko, wq=wq, wk=wk, axes=(44, 42, 42), t0=9, grid=(10, 11))
    v = qkv[:, 6:].clone()
    L.fastar_qk_norm_rope(q, k, q, k, wq=wq, wk=wk, axes=(44, 42, 42), t0=9, grid=(10, 11))
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(qkv[:, 6:], v)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_far_and_negative_positions_given_one_by_one(dtype):
    n, H, d, axes = 257, 2, 128, (44, 42, 42)
    _, q, k, wq, wk = _make(n, H, H, d, DT[dtype], 3)
    rng = np.random.default_rng(4)
    pos = rng.integers(-2 ** 24, 2 ** 24, (n, 3)).astype(np.int32)
    pos[0] = 0
    pos[1] = (2 ** 31 - 1, -2 ** 31, 1)
    qo, ko = torch.empty(H, n, d, dtype=DT[dtype], device="cuda"), torch.empty(H, n, d, dtype=DT[dtype], device="cuda")
    L.fastar_qk_norm_rope(q, k, qo, ko, wq=wq, wk=None, axes=axes, pos=torch.from_numpy(pos).cuda())
    torch.cuda.synchronize()
    # 2^31 positions away the 64-bit step (53 significant bits, 48 after the products) is good
    # to 2^31 * 2^-48 / 2 pi * 2 pi = 2^-17 rad, and the float64 oracle's own product to 2^-22
    keep = np.arange(n) != 1
    for got, x, w in ((qo, q, wq), (ko, k, None)):
        _check(got[:, keep], x[:, keep], w, 1e-6, axes, pos[keep])
        want, pair = K.norm_rope(_np(x[:, 1:2]), None if w is None else _np(w), 1e-6, axes, pos[1:2], 10000.0)
        half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
        assert (np.abs(_np(got[:, 1:2]) - want) <= half * np.abs(want) + 2.0 ** -16 * pair).all()


def test_one_tensor_alone_device_frame_and_other_theta():
    _, q, _, wq, _ = _make(70, 3, 1, 64, torch.float32)
    qo = torch.empty(3, 70, 64, device="cuda")
    t0 = torch.tensor([1234], dtype=torch.int32, device="cuda")
    L.fastar_qk_norm_rope(q, None, qo, None, wq=wq, eps=1e-5, axes=(24, 20, 20), t0=6, t0_dev=t0, grid=(5, 7), theta=500.0)
    torch.cuda.synchronize()
    _check(qo, q, wq, 1e-5, (24, 20, 20), K.grid_positions(70, 1240, 5, 7), 500.0)


def test_a_row_that_is_not_finite_stays_alone_and_unrotated_channels_pass():
    _, q, k, _, _ = _make(9, 4, 2, 64, torch.float32)
    q, k = q.clone(), k.clone()
    q[2, 4, 10] = float("nan")
    q[1, 3, 63] = float("inf")                 # past the axes: its neighbour 62 must not see it
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    L.fastar_qk_norm_rope(q, k, qo, ko, axes=(24, 16, 16), grid=(3, 3))
    torch.cuda.synchronize()
    assert torch.equal(qo[..., 56:], q[..., 56:])
    bad = torch.isnan(qo)
    assert int(bad.sum()) == 2 and bool(bad[2, 4, 10]) and bool(bad[2, 4, 11])
    zero = torch.zeros(1, 2, 64, device="cuda")
    out = torch.full_like(zero, 7.0)
    L.fastar_qk_norm_rope(zero, None, out, None, wq=torch.ones(64, device="cuda"), axes=(24, 16, 16))
    torch.cuda.synchronize()
    assert torch.equal(out, zero)              # a row of zeros: eps keeps the norm finite


def test_captured_graph_follows_the_device_frame():
    _, q, k, wq, wk = _make(100, 2, 2, 128, torch.bfloat16)
    q, k = q.contiguous(), k.contiguous()
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    t0 = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda: L.fastar_qk_norm_rope(q, k, qo, ko, wq=wq, wk=wk, axes=(44, 42, 42), t0_dev=t0, grid=(4, 5))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    t0.fill_(777)
    g.replay()
    torch.cuda.synchronize()
    _check(qo, q, wq, 1e-6, (44, 42, 42), K.grid_positions(100, 777, 4, 5))


def test_rows_whose_squares_overflow_fp32():
    # the mean of squares is infinite in fp32: every finite channel is x * 0, an infinite one NaN
    x = torch.full((3, 2, 128), 1e25, device="cuda")
    x[1, 1] = 1.0
    x[1, 1, 7] = float("inf")
    x[2] = 1.0
    out = torch.empty_like(x)
    L.fastar_qk_norm_rope(x, None, out, None, wq=torch.ones(128, device="cuda"))
    torch.cuda.synchronize()
    assert (out[0] == 0).all() and (out[1, 0] == 0).all()
    assert torch.isnan(out[1, 1, 7]) and int(torch.isnan(out).sum()) == 1 and (out[1, 1].nan_to_num() == 0).all()
    assert (out[2] - 1).abs().max() <= 2.0 ** -19 + 5e-7      # 1 / sqrt(1 + 1e-6), as the bound above


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,Hq,Hk,d", [(3, 2, 1, 64), (3, 5, 3, 128), (2000, 12, 4, 128), (4000, 10, 5, 64)])
def test_a_nan_makes_its_normed_row_nan_and_no_other(dtype, n, Hq, Hk, d):
    # the mean of the row's squares is NaN, and so is every channel, turned or not
    _, q, k, wq, wk = _make(n, Hq, Hk, d, DT[dtype], 11)
    axes = (d // 4, d // 4, d // 4)
    ref = [torch.empty_like(q), torch.empty_like(k)]
    L.fastar_qk_norm_rope(q, k, *ref, wq=wq, wk=wk, axes=axes, grid=(5, 7))
    q, k = q.clone(), k.clone()
    rows = [(q, (1, n // 2)), (q, (0, 0)), (k, (Hk - 1, n - 1))]
    for i, (t, at) in enumerate(rows):
        t[at][(7 * i + 3, d - 1, 0)[i]] = float("nan")       # channels that turn, and one past the axes
    out = [torch.empty_like(q), torch.empty_like(k)]
    L.fastar_qk_norm_rope(q, k, *out, wq=wq, wk=wk, axes=axes, grid=(5, 7))
    torch.cuda.synchronize()
    for x, y, r in zip((q, k), out, ref):
        bad = torch.isnan(x).any(-1)
        assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], r[~bad])
