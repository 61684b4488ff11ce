"""Plain float64 restatement of the paged key/value cache (append with norm and rotation, attention
over a window and the first rows): test infrastructure, no code shared with the CUDA path."""
from __future__ import annotations

import numpy as np

from oracle import kv4_oracle as K


def spans(cu, T, B):
    """(first token, tokens) of each sequence."""
    if cu is None:
        return [(b * (T // B), T // B) for b in range(B)]
    return [(int(cu[b]), int(cu[b + 1] - cu[b])) for b in range(B)]


def sees(nq, at, cap, block=0, window=0, sinks=0):
    """Which of a sequence's cap rows each of its nq tokens sees, [nq, cap]."""
    i, j = np.arange(nq)[:, None], np.arange(cap)[None]
    end = at + (np.minimum(nq, (i // block + 1) * block) if block else nq + 0 * i)
    see = j < end
    if window:
        see &= (j >= end - window) | (j < sinks)
    return see


def rows_of(pool, table, n):
    """Rows 0 .. n of one sequence: [n, H, d]; rows of pages that are not there are NaN."""
    pages, H, page, d = pool.shape
    out = np.full((n, H, d), np.nan)
    for p in range((n + page - 1) // page):
        if 0 <= table[p] < pages:
            m = min(page, n - p * page)
            out[p * page:p * page + m] = np.moveaxis(pool[table[p], :, :m], 1, 0)
    return out


def positions(at, n, grid):
    """(frame, row, column) of rows at .. at + n."""
    r = np.arange(at, at + n)
    return np.stack((r // (grid[0] * grid[1]), r // grid[1] % grid[0], r % grid[1]), -1)


def append(k, v, k_pool, v_pool, table, at, cu=None, q=None, wq=None, wk=None, eps=1e-6, axes=(0, 0, 0), pos=None,
           grid=(1, 1), theta=1e4):
    """The pools after the call, q_out, which of its tokens belong to a sequence, len_out; for error bounds
    |y_2j| + |y_2j+1| of each pair before its rotation, as a pool of the rows written and as q_out."""
    k_pool, v_pool = np.array(k_pool, np.float64), np.array(v_pool, np.float64)
    pages, _, page, _ = k_pool.shape
    T, cap = k.shape[1], table.shape[1] * page
    done, lens = np.zeros(T, bool), []
    q_out = None if q is None else np.array(q, np.float64)
    k_pair, q_pair = np.zeros_like(k_pool), None if q is None else np.zeros(q.shape)
    for b, (t0, n) in enumerate(spans(cu, T, len(at))):
        lens.append(min(cap, int(at[b]) + n))
        if n == 0:
            continue
        sl = slice(t0, t0 + n)
        p = positions(int(at[b]), n, grid) if pos is None else np.asarray(pos)[sl]
        kr, kp = K.norm_rope(k[:, sl], wk, eps, axes, p, theta)
        if q is not None:
            q_out[:, sl], q_pair[:, sl] = K.norm_rope(q[:, sl], wq, eps, axes, p, theta)
        done[sl] = True
        for i in range(n):
            r = int(at[b]) + i
            if r < cap and 0 <= table[b, r // page] < pages:
                k_pool[table[b, r // page], :, r % page] = kr[:, i]
                k_pair[table[b, r // page], :, r % page] = kp[:, i]
                v_pool[table[b, r // page], :, r % page] = v[:, t0 + i]
    return k_pool, v_pool, q_out, done, np.array(lens), k_pair, q_pair


def attention(q, k_pool, v_pool, table, at, scale, cu=None, block=0, window=0, sinks=0):
    """out, lse, and for error bounds: the mean of |v| under the softmax [Hq, T, d], the largest
    sum_c |q_c k_c| * scale [Hq, T] and the number of rows seen [T] (-1: no sequence's token)."""
    q = np.asarray(q, np.float64)
    Hq, T, d = q.shape
    page, Hk = k_pool.shape[2], k_pool.shape[1]
    out, mag = np.zeros((Hq, T, d)), np.zeros((Hq, T, d))
    lse, big, count = np.full((Hq, T), -np.inf), np.zeros((Hq, T)), np.full(T, -1)
    for b, (t0, n) in enumerate(spans(cu, T, len(at))):
        if n == 0:
            continue
        m = min(int(at[b]) + n, table.shape[1] * page)
        see = sees(n, int(at[b]), m, block, window, sinks)
        count[t0:t0 + n] = see.sum(1)
        used = see.any(0)
        see = see[:, used]
        if not see.size:
            continue
        k, v = rows_of(k_pool, table[b], m)[used], rows_of(v_pool, table[b], m)[used]
        for h in range(Hq):
            kh, vh = k[:, h // (Hq // Hk)], v[:, h // (Hq // Hk)]
            x = np.where(see, q[h, t0:t0 + n] @ kh.T * scale, -np.inf)
            top = x.max(1, keepdims=True)
            top = np.where(np.isneginf(top), 0.0, top)
            p = np.exp(x - top)
            l = p.sum(1)
            live = l > 0
            p /= np.where(live, l, 1.0)[:, None]
            out[h, t0:t0 + n], mag[h, t0:t0 + n] = p @ vh, p @ np.abs(vh)
            with np.errstate(divide="ignore"):
                lse[h, t0:t0 + n] = top[:, 0] + np.log(l)
            big[h, t0:t0 + n] = np.where(see, np.abs(q[h, t0:t0 + n]) @ np.abs(kh).T * scale, 0.0).max(1)
    return out, lse, mag, big, count
