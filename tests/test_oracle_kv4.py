"""Pins of the 4-bit cache's oracle: hand-computed scales and codes, the float8 grid against
torch's, rounding by exhaustive search, and the attention's masks by direct sums."""
import numpy as np
import torch

from oracle import kv4_oracle as K


def test_grids():
    assert np.array_equal(K.E4M3, torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy())
    assert list(K.E2M1) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def test_a_block_by_hand():
    x = np.zeros(16)
    x[:8] = [6.0, -3.0, 0.25, 0.75, -1.25, 2.5, 5.0, -0.2]     # amax 6: scale 1 = byte 56
    codes, scales = K.quantise(x[None])
    assert scales[0, 0] == 56
    # 6, -3, 0 (tie to the even code), 1 (tie up), -1 (tie down), 2, 4, -0
    assert [int(c) for c in codes[0, :4]] == [7 | 13 << 4, 0 | 2 << 4, 10 | 4 << 4, 6 | 8 << 4]
    assert list(K.values(codes, scales)[0, :8]) == [6, -3, 0, 1, -1, 2, 4, 0]


def test_rounding_is_nearest_even_by_search():
    rng = np.random.default_rng(0)
    x = np.concatenate((rng.standard_normal((200, 64)) * np.exp(rng.uniform(-9, 9, (200, 1))), np.zeros((1, 64)),
                        np.full((1, 64), 1e9)))
    codes, scales = K.quantise(x)
    amax = np.abs(x.reshape(-1, 4, 16)).max(-1)
    for a, b in zip(amax.ravel(), scales.ravel()):
        dist = np.abs(K.E4M3 - a / 6)
        best = np.flatnonzero(dist == dist.min())
        assert b in best and (len(best) == 1 or b % 2 == 0)
    v = K.values(codes, scales).reshape(-1, 4, 16)
    s = K.E4M3[scales][..., None]
    grid = np.concatenate((-K.E2M1[::-1], K.E2M1))
    dist = np.abs(x.reshape(-1, 4, 16)[..., None] - grid * s[..., None]).min(-1)
    assert np.allclose(np.abs(x.reshape(-1, 4, 16) - v), dist, rtol=0, atol=1e-12 * np.abs(x).max())


def test_not_finite_counts_as_zero_and_exponents_shift():
    x = np.ones((1, 16))
    x[0, 3], x[0, 4] = np.nan, -np.inf
    codes, scales = K.quantise(x)
    v = K.values(codes, scales)
    assert v[0, 3] == 0 and v[0, 4] == 0 and np.all(v[0, 5:] == v[0, 5])
    y = np.random.default_rng(1).standard_normal((3, 32))
    a, b = K.quantise(y), K.quantise(y * 2.0 ** -12, e=-12)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    assert np.array_equal(K.values(*a) * 2.0 ** -12, K.values(*b, e=-12))


def test_visible_rows():
    assert list(K.visible(5, 3, 0)) == [5, 5, 5]
    assert list(K.visible(5, 3, 1)) == [3, 4, 5]
    assert list(K.visible(5, 3, 2)) == [4, 4, 5]
    assert list(K.visible(1, 3, 1)) == [0, 0, 1]          # a cache shorter than the call
    assert list(K.visible(0, 2, 1)) == [0, 0]


def test_attention_by_direct_sums():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((4, 3, 16)), rng.standard_normal((2, 9, 16)), rng.standard_normal((2, 9, 16))
    lens = [9, 2]
    out, lse, _, _ = K.attention(q, k, v, lens, 0.3, block=1)
    for h in range(4):
        for t in range(3):
            n = max(0, lens[h // 2] - 3 + t + 1)
            if n == 0:
                assert np.all(out[h, t] == 0) and lse[h, t] == -np.inf
                continue
            w = np.array([np.exp(0.3 * float(q[h, t] @ k[h // 2, j])) for j in range(n)])
            assert np.allclose(out[h, t], sum(w[j] * v[h // 2, j] for j in range(n)) / w.sum())
            assert np.isclose(lse[h, t], np.log(w.sum()))


def test_norm_rope_keeps_the_length_and_relative_angles():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((2, 5, 64))
    pos = rng.integers(-50, 50, (5, 3))
    y, _ = K.norm_rope(x, None, 1e-6, (24, 16, 16), pos, 10000.0)
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    assert np.array_equal(y[..., 56:], x[..., 56:])
    a, _ = K.norm_rope(x[:, :1].repeat(2, 1), None, 1e-6, (24, 16, 16), pos[:2], 10000.0)
    b, _ = K.norm_rope(x[:, :1].repeat(2, 1), None, 1e-6, (24, 16, 16), pos[:2] + 7, 10000.0)
    assert np.allclose((a[:, 0] * a[:, 1]).sum(-1), (b[:, 0] * b[:, 1]).sum(-1))
    z, _ = K.norm_rope(x, np.ones(64), 1e-12, (0, 0, 0), pos, 10000.0)
    assert np.allclose((z ** 2).mean(-1), 1.0)
