"""Pins of the paged cache's oracle: masks by enumeration, attention against a direct softmax, append
against a dense cache."""
import numpy as np
import pytest

from oracle import kv4_oracle as K
from oracle import paged_oracle as P


@pytest.mark.parametrize("nq,at,cap,block,window,sinks", [(5, 3, 20, 0, 0, 0), (5, 3, 20, 1, 0, 0), (7, 10, 20, 3, 4, 2),
                                                          (6, 0, 20, 1, 2, 3), (4, 18, 20, 2, 5, 0), (1, 9, 10, 1, 1, 9)])
def test_masks(nq, at, cap, block, window, sinks):
    see = P.sees(nq, at, cap, block, window, sinks)
    for i in range(nq):
        end = at + nq if block == 0 else at + min(nq, (i // block + 1) * block)
        for j in range(cap):
            want = j < end and (window == 0 or j >= end - window or j < sinks)
            assert see[i, j] == want, (i, j)


def test_attention_is_a_softmax_over_the_rows_seen():
    rng = np.random.default_rng(0)
    page, d, Hk, G = 4, 8, 2, 3
    kp, vp = rng.normal(size=(2, 9, Hk, page, d))
    table = np.array([[3, 1, 8, -1], [0, 7, 2, 5]])
    at, cu = np.array([4, 9]), np.array([0, 3, 8])
    q = rng.normal(size=(Hk * G, 10, d))                       # two tokens of no sequence
    out, lse, mag, big, n = P.attention(q, kp, vp, table, at, 0.3, cu, 1, 5, 2)
    for b, (t0, m) in enumerate(P.spans(cu, 10, 2)):
        for i in range(m):
            rows = [j for j in range(at[b] + i + 1) if j >= at[b] + i - 4 or j < 2]
            assert n[t0 + i] == len(rows)
            for h in range(Hk * G):
                k = np.stack([kp[table[b, j // page], h // G, j % page] for j in rows])
                v = np.stack([vp[table[b, j // page], h // G, j % page] for j in rows])
                x = k @ q[h, t0 + i] * 0.3
                p = np.exp(x) / np.exp(x).sum()
                np.testing.assert_allclose(out[h, t0 + i], p @ v, rtol=1e-12)
                np.testing.assert_allclose(mag[h, t0 + i], p @ np.abs(v), rtol=1e-12)
                np.testing.assert_allclose(lse[h, t0 + i], np.log(np.exp(x).sum()), rtol=1e-12)
                np.testing.assert_allclose(big[h, t0 + i], (np.abs(k) @ np.abs(q[h, t0 + i])).max() * 0.3, rtol=1e-12)
    assert (n[8:] == -1).all() and (out[:, 8:] == 0).all()


def test_no_rows():
    out, lse, *_ = P.attention(np.ones((1, 2, 4)), np.ones((1, 1, 4, 4)), np.ones((1, 1, 4, 4)), np.array([[0]]),
                               np.array([4]), 1.0, None, 1, 1, 0)
    assert (out == 0).all() and np.isneginf(lse).all()         # both tokens' rows lie past the page


def test_append_equals_a_dense_cache():
    rng = np.random.default_rng(1)
    page, d, Hk, Hq = 4, 8, 2, 3
    kp, vp = rng.normal(size=(2, 8, Hk, page, d))
    table = np.array([[6, 0, 3], [2, 5, 7]])
    at, cu = np.array([2, 7]), np.array([0, 5, 7])
    k, v, q = rng.normal(size=(Hk, 8, d)), rng.normal(size=(Hk, 8, d)), rng.normal(size=(Hq, 8, d))
    w = rng.normal(size=d)
    k2, v2, q2, done, lens, *_ = P.append(k, v, kp, vp, table, at, cu, q, w, None, 1e-6, (4, 2, 0), None, (2, 3))
    assert lens.tolist() == [7, 9] and done.tolist() == [True] * 7 + [False]
    left = np.ones((8, page), bool)
    for b, (t0, n) in enumerate(P.spans(cu, 8, 2)):
        for i in range(n):
            r = at[b] + i
            pos = np.array([[r // 6, r // 3 % 2, r % 3]])
            np.testing.assert_allclose(k2[table[b, r // page], :, r % page],
                                       K.norm_rope(k[:, t0 + i:t0 + i + 1], None, 1e-6, (4, 2, 0), pos, 1e4)[0][:, 0])
            np.testing.assert_allclose(q2[:, t0 + i], K.norm_rope(q[:, t0 + i:t0 + i + 1], w, 1e-6, (4, 2, 0), pos, 1e4)[0][:, 0])
            assert np.array_equal(v2[table[b, r // page], :, r % page], v[:, t0 + i])
            left[table[b, r // page], r % page] = False
    assert np.array_equal(k2.swapaxes(1, 2)[left], kp.swapaxes(1, 2)[left])
    assert np.array_equal(v2.swapaxes(1, 2)[left], vp.swapaxes(1, 2)[left])
