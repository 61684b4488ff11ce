// What the kernels over a paged cache share: where a sequence's tokens and rows lie, which rows a
// token sees, and how the rows of a piece of work become a list of key tiles.
//
// Row r of sequence b is slot r % page of page table[b, r / page].  Token i of a sequence is its
// row at + i; its end is E(i) = at + nq, or with blocks at + min(nq, (i / block + 1) block); it
// sees the rows j < min(E, cap) with j >= E - window (all with window 0) or j < sinks.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace fastar {
namespace paged {

// The tokens of sequence b: cu[b] .. cu[b] + nq of the call's, behind `at` earlier rows.  nq = 0 where cu
// or at make no sense (FASTAR_DEV_BAD_LEN).
struct Seq {
  int t0, nq, at;
};
__device__ __forceinline__ Seq sequence(const int32_t* cu, const int32_t* at, int B, int64_t T, int64_t cap, int b,
                                        int32_t* status) {
  Seq s;
  if (cu) {
    s.t0 = cu[b];
    const int t1 = cu[b + 1];
    s.nq = t1 - s.t0;
    if (s.t0 < 0 || t1 < s.t0 || t1 > T) s.t0 = 0, s.nq = -1;
  } else {
    s.nq = (int)(T / B);
    s.t0 = b * s.nq;
  }
  s.at = at[b];
  if (s.nq < 0 || s.at < 0 || s.at > cap) {
    flag_status(status, FASTAR_DEV_BAD_LEN);
    s.nq = 0;
    s.at = 0;
  }
  return s;
}

// The rows that token i sees: [lo, hi) and [0, sk).  T is below 2^30, cap 2^30 at most, block T at most.
struct Sees {
  int lo, hi, sk;
};
__device__ __forceinline__ Sees sees(const PagedAttnArgs& a, const Seq& s, int i) {
  int e = s.nq;
  if (a.block > 0) e = min(e, (int)(((uint32_t)i / (uint32_t)a.block + 1) * (uint32_t)a.block));
  e += s.at;
  Sees v;
  v.hi = min(e, (int)a.cap);
  v.lo = a.window > 0 ? min(max(0, e - a.window), v.hi) : 0;
  v.sk = a.window > 0 ? min(a.sinks, v.hi) : 0;
  return v;
}

// Few rows: where the partials of row r (of a KV head of a sequence) of slot v lie.
__device__ __forceinline__ int64_t partial_row(const PagedAttnArgs& a, int64_t v, int h, int r) {
  return (v * a.Hkv + h) * ((int64_t)a.group * a.max_q) + r;
}

// Which of the n <= 32 keys from `key` on are seen, as bits.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }
__device__ __forceinline__ uint32_t seen32(const Sees& v, int key) {
  return (below(v.hi - key) & ~below(v.lo - key)) | below(v.sk - key);
}

// The key tiles of kTile rows that tokens ta .. tb (the first and the last of a piece of work) need:
// tiles [0, s1) and [w0, w1), in this order.  Ends and window starts only grow with the token.
template <int kTile>
struct Tiles {
  Sees first, last;
  int s1, w0, n;
  __device__ __forceinline__ void set(const PagedAttnArgs& a, const Seq& s, int ta, int tb) {
    first = sees(a, s, ta);
    last = sees(a, s, tb);
    s1 = (last.sk + kTile - 1) / kTile;
    w0 = first.lo / kTile;
    int w1 = (last.hi + kTile - 1) / kTile;
    if (last.hi <= first.lo) w1 = w0;
    if (s1 >= w0) {                      // one run of tiles
      w1 = max(w1, s1);
      s1 = w0 = 0;
    }
    n = s1 + w1 - w0;
  }
  // the first row of tile j
  __device__ __forceinline__ int key(int j) const { return (j < s1 ? j : j - s1 + w0) * kTile; }
  // rows that some token sees
  __device__ __forceinline__ bool any(int row) const { return (row >= first.lo && row < last.hi) || row < last.sk; }
  __device__ __forceinline__ bool any(int from, int to) const {     // of rows [from, to)
    return (to > first.lo && from < last.hi) || from < last.sk;
  }
  // every token sees all the rows of the tile at `key`
  __device__ __forceinline__ bool all(int key) const {
    return key + kTile <= first.hi && (key >= last.lo || key + kTile <= first.sk);
  }
};

// The page of a table's entry; -1 and FASTAR_DEV_BAD_INDEX for one that is not there.
__device__ __forceinline__ int page_of(const int32_t* row, int p, int64_t pages, int32_t* status) {
  const int x = row[p];
  if (x >= 0 && x < pages) return x;
  flag_status(status, FASTAR_DEV_BAD_INDEX);
  return -1;
}

// Tiles j0 .. j1 of a list: one of `used` parts.
struct Split {
  int used, j0, j1;
};

// Few rows: what a block of slot v works on.  The blocks are dealt out by the sequences' lengths: with n_b key
// tiles a sequence, a block takes `chunk` of them, the larger of min_tiles and what spreads all the tiles
// over a.extra slots; sequence b has c_b = ceil(n_b / chunk) slots (at least one), side by side.  No more than
// extra + B of them are in use, whatever the lengths.  Every warp finds its block's by itself, the same in
// every lane; sequences in steps of 32.
constexpr int kDealt = 256;              // sequences that are dealt out; with more, each is a slot
struct Work {
  int b, first, count, split;            // sequence, its first slot, its slots, this one's place among them
};
// The work of slot v, or (v < 0) of sequence b; false where there is none.
template <int kTile>
__device__ __forceinline__ bool find_work(const PagedAttnArgs& a, int v, int b, Work& w) {
  w.split = 0;
  w.count = 1;
  if (a.extra == 0) {
    w.b = w.first = v < 0 ? b : v;
    return true;
  }
  const int lane = threadIdx.x & 31;
  int n[kDealt / 32];
  int64_t total = 0;
#pragma unroll
  for (int k = 0; k < kDealt / 32; ++k) {
    n[k] = -1;                           // a sequence without tokens has no slot
    if (32 * k >= a.B) break;
    if (32 * k + lane < a.B) {
      const Seq s = sequence(a.cu, a.at, a.B, a.T, a.cap, 32 * k + lane, blockIdx.x == 0 ? a.status : nullptr);
      if (s.nq > 0) {
        Tiles<kTile> t;
        t.set(a, s, 0, min(s.nq, a.max_q) - 1);
        n[k] = t.n;
        total += t.n;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  // (more than the tiles of 2^30 rows is as good as those)
  const int even = (int)min((total + a.extra - 1) / a.extra, (int64_t)1 << 28);
  const int chunk = max(even, a.min_tiles);
  int base = 0;
  bool here = false;
#pragma unroll
  for (int k = 0; k < kDealt / 32; ++k) {
    if (32 * k >= a.B) break;
    const int c = n[k] < 0 ? 0 : max(1, (n[k] + chunk - 1) / chunk);
    int end = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += x;
    }
    end += base;
    base = __shfl_sync(0xffffffffu, end, 31);
    const uint32_t hit = __ballot_sync(0xffffffffu, v < 0 ? 32 * k + lane == b && c > 0 : v >= end - c && v < end);
    if (hit) {
      const int src = __ffs(hit) - 1;
      w.b = 32 * k + src;
      w.count = __shfl_sync(0xffffffffu, c, src);
      w.first = __shfl_sync(0xffffffffu, end - c, src);
      w.split = v < 0 ? 0 : v - w.first;
      here = true;
    }
  }
  return here;
}
__device__ __forceinline__ Split part_of(int n, const Work& w) {
  Split r;
  r.used = w.count;
  r.j0 = (int)((int64_t)n * w.split / w.count);
  r.j1 = (int)((int64_t)n * (w.split + 1) / w.count);
  return r;
}

// bf16 kernels multiply a tile's P and V as matrices, where a weight of 0 does not keep an infinity or NaN of a row
// that only some tokens see from the others.  So of tiles that not every token sees in full they take such
// values out of V; this is what those add to n channels from c on of a token that sees `see`.
template <int kTile, int n>
__device__ __noinline__ void add_taken_out(const PagedAttnArgs& a, const Tiles<kTile>& tiles, const Split& part, int b, int h,
                                           Sees see, int c, float* o) {
  const int32_t* table = a.table + (int64_t)b * a.max_pages;
  for (int j = part.j0; j < part.j1; ++j) {
    const int key0 = tiles.key(j);
    if (tiles.all(key0)) continue;
    for (int key = key0; key < key0 + kTile; ++key) {
      if (!(seen32(see, key) & 1)) continue;
      const int page = table[key >> a.pool.page_shift];
      if (page < 0 || page >= a.pool.pages) continue;
      const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.pool.v) + page * a.pool.ps + h * a.pool.hs +
                               (key & ((1 << a.pool.page_shift) - 1)) * a.pool.rs + c;
      for (int e = 0; e < n; ++e) {
        const float x = __bfloat162float(v[e]);
        if (!(fabsf(x) < __int_as_float(0x7f800000))) o[e] += x;
      }
    }
  }
}
// Eight channels of such a tile: infinities and NaN become 0; true if there was one.
__device__ __forceinline__ bool take_out(uint4* p) {
  const uint4 u = *p;
  const uint32_t big = __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu),
                                __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
  if (__builtin_expect((big & 0xffffu) < 0x7f80u && (big >> 16) < 0x7f80u, 1)) return false;
  uint32_t y[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if ((y[e] & 0x7fffu) >= 0x7f80u) y[e] &= 0xffff0000u;
    if ((y[e] >> 16 & 0x7fffu) >= 0x7f80u) y[e] &= 0xffffu;
  }
  *p = make_uint4(y[0], y[1], y[2], y[3]);
  return true;
}

}  // namespace paged
}  // namespace fastar
