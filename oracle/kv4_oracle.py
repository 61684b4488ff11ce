"""Plain float64 restatement of the 4-bit key/value cache (quantised append, read, attention)
and of the per-head RMS norm with rotary positions: test infrastructure, no code shared with
the CUDA path."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the finite e4m3 numbers >= 0, by byte
E4M3 = np.array([m / 8 * 2.0 ** -6 for m in range(8)]
                + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1])


def _round_to(a, grid):
    """Index of the grid value nearest to a (>= 0), the even index of two; past the last: the last."""
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    dl, dh = a - grid[hi - 1], grid[hi] - a
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, hi - 1)


def quantise(x, e=0):
    """codes uint8 [..., d / 2] and scales uint8 [..., d / 16] of rows x [..., d]; e: the head's
    exponent.  NaN and infinities count as 0."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isfinite(x), x, 0.0) * 2.0 ** -e
    y = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    scales = _round_to(np.abs(y).max(-1), 6 * E4M3).astype(np.uint8)
    s = E4M3[scales][..., None]
    code = np.zeros(y.shape, np.uint8)
    for i in range(7):
        mid = (E2M1[i] + E2M1[i + 1]) / 2 * s
        code += ((np.abs(y) > mid) | ((np.abs(y) == mid) & (i % 2 == 1) & (s > 0))).astype(np.uint8)
    code = np.where(s > 0, code, 0).astype(np.uint8) | (np.signbit(y).astype(np.uint8) << 3)
    code = code.reshape(*x.shape[:-1], x.shape[-1] // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), scales


def values(codes, scales, e=0):
    """The rows [..., d] that codes and scales stand for."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    v = np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]
    return v * np.repeat(E4M3[scales], 16, axis=-1) * 2.0 ** e


def visible(n, nq, block):
    """How many of n cached rows each of nq tokens sees."""
    t = np.arange(nq)
    if block <= 0:
        return np.full(nq, n)
    return np.maximum(0, n - nq + np.minimum(nq, (t // block + 1) * block))


def attention(q, k, v, lens, scale, block=0):
    """q [Hq, nq, d] over k, v [Hkv, cap, d], lens [Hkv]: out, lse, and for error bounds the
    mean of |v| under the softmax [Hq, nq, d] and the largest sum_c |q_c k_c| * scale [Hq, nq]."""
    q = np.asarray(q, np.float64)
    Hq, nq, d = q.shape
    G = Hq // len(lens)
    out, mag = np.zeros((Hq, nq, d)), np.zeros((Hq, nq, d))
    lse, big = np.full((Hq, nq), -np.inf), np.zeros((Hq, nq))
    for h in range(Hq):
        n = int(lens[h // G])
        if n == 0:
            continue
        kk, vv = k[h // G, :n], v[h // G, :n]
        see = visible(n, nq, block)
        s = q[h] @ kk.T * scale
        s[np.arange(n)[None] >= see[:, None]] = -np.inf
        m = s.max(1, keepdims=True)
        live = np.isfinite(m[:, 0])
        p = np.exp(s[live] - m[live])
        l = p.sum(1, keepdims=True)
        out[h, live] = p @ vv / l
        mag[h, live] = p @ np.abs(vv) / l
        lse[h, live] = (m[live] + np.log(l))[:, 0]
        big[h] = (np.abs(q[h]) @ np.abs(kk).max(0)) * scale
    return out, lse, mag, big


def grid_positions(n, f0, gh, gw):
    i = np.arange(n)
    return np.stack((f0 + i // (gh * gw), (i // gw) % gh, i % gw), -1)


def norm_rope(x, w, eps, axes, pos, theta):
    """x [H, n, d] -> the normed and rotated rows, and for error bounds |y_2j| + |y_2j+1| of each
    pair before the rotation, at both its channels."""
    y = np.asarray(x, np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    out = y.copy()
    at = 0
    for a, width in enumerate(axes):
        for j in range(width // 2):
            ang = pos[:, a].astype(np.float64) * float(theta) ** (-2.0 * j / width)
            c, s = np.cos(ang), np.sin(ang)
            c0, c1 = at + 2 * j, at + 2 * j + 1
            out[..., c0] = y[..., c0] * c - y[..., c1] * s
            out[..., c1] = y[..., c0] * s + y[..., c1] * c
        at += width
    pair = np.abs(y).reshape(*y.shape[:-1], -1, 2).sum(-1)
    return out, np.repeat(pair, 2, axis=-1)
