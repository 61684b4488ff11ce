// How the work of the tensor-core kernel over a paged cache (paged_attn_tc.cu) is dealt out: on the device, where
// the sequences' lengths are.
//
// An item is up to `per` rows of a (sequence, KV head): its row tiles 2 (or 1, where the rows fill half of them or
// less), its key tiles paged.cuh's.  It counts fixed_units and kFull (fewer with one row tile) for each key tile,
// as its time goes: 1.4 us a key tile, 1.15 with one row tile (a pair; it waits for K and V, which it takes twice as
// fast), some 8 us around them (5 at d = 64; a CTA alone at d = 128 goes by the same figure, not measured for it).  Items lie in a row: sequences, their row tiles, the KV heads side by
// side.  Share p of P is the units W p / P .. W (p + 1) / P of that row, so
// that all shares end together, whatever the lengths: borders cut items between two key tiles (12 heads of 4680
// tokens are 120 items on 76 pairs of CTAs: in whole items 2 waves, dealt out 1.53).  A cut may leave a
// part of one key tile (with no part below three, ragged sequences of 7 key tiles a piece took 47.2 us instead of 44.4:
// what one share lost its neighbour had to do); there are no more shares than have an item of four key tiles each.  Without a
// workspace borders move to the nearer end of the item.
#pragma once

#include <climits>

#include "paged.cuh"

namespace fastar {
namespace paged {

constexpr int kFull = 6;
// pairs of CTAs, single ones
__device__ __forceinline__ int half_units(int per) { return per == 512 ? 5 : 4; }
__device__ __forceinline__ int fixed_units(int per) { return per == 512 ? 36 : 18; }
constexpr int kMaxShares = 256;          // the plan asks for no more
constexpr int kItems = 8;                // items of a CTA that are known at once

struct Item {
  Seq s;
  Tiles<128> tiles;
  int64_t at;                            // the item's first unit in the row of all
  uint32_t rows, r0;                     // rows of the sequence's KV head, the item's first
  int units, b, h, nt;                   // nt: row tiles with rows; 0: no item
  int j0, T;                             // the share's key tiles of the item
  int slot;                              // of the partials, -1: the whole item
};

// Where a walk over all items is: those of one head, 32 at a time side by side in the lanes (the row tiles of one
// sequence, or where it has no more than 2^shift < 32, of several).
struct Walk {
  int b0, i, k, rts, shift;              // the lanes' sequences b0 .., the first at work, its 32 row tiles
  Seq mine, s;                           // of sequence b0 + lane; of this lane's item
  int b, rt, units;                      // this lane's item
};

__device__ __forceinline__ int rows_of(const PagedAttnArgs& a, const Seq& s) { return a.group * min(s.nq, a.max_q); }

__device__ __forceinline__ Seq load_seq(const PagedAttnArgs& a, int b, int32_t* status) {
  if (b >= a.B) return Seq{0, 0, 0};
  const Seq s = sequence(a.cu, a.at, a.B, a.T, a.cap, b, status);
  if (s.nq > a.max_q) flag_status(status, FASTAR_DEV_BAD_LEN);
  return s;
}

// Units and row tiles of rows r0 .. of a head.
__device__ __forceinline__ int item_units(const PagedAttnArgs& a, const Seq& s, int r0, int per, Tiles<128>& tiles, int& nt) {
  const int rows = rows_of(a, s);
  nt = 0;
  if (r0 >= rows) return 0;
  nt = rows - r0 > per / 2 ? 2 : 1;
  tiles.set(a, s, r0 / a.group, (r0 + min(per, rows - r0) - 1) / a.group);
  return fixed_units(per) + tiles.n * (nt == 2 ? kFull : half_units(per));
}

__device__ __forceinline__ Seq shfl_seq(const Seq& s, int from) {
  return Seq{__shfl_sync(0xffffffffu, s.t0, from), __shfl_sync(0xffffffffu, s.nq, from),
             __shfl_sync(0xffffffffu, s.at, from)};
}
__device__ __forceinline__ void walk_lane(const PagedAttnArgs& a, Walk& w, int per) {
  const int lane = threadIdx.x & 31, i = min(w.i + (lane >> w.shift), 31);
  w.b = w.b0 + i;
  w.s = shfl_seq(w.mine, i);               // past the last: without tokens
  w.rt = 32 * w.k + (lane & ((1 << w.shift) - 1));
  Tiles<128> t;
  int nt;
  w.units = w.rt < w.rts ? item_units(a, w.s, w.rt * per, per, t, nt) : 0;
}
__device__ __forceinline__ void walk_start(const PagedAttnArgs& a, Walk& w, int per, int32_t* status) {
  w.rts = (int)(((int64_t)a.group * a.max_q + per - 1) / per);
  w.shift = w.rts >= 32 ? 5 : w.rts <= 1 ? 0 : 32 - __clz(w.rts - 1);
  w.b0 = w.i = w.k = 0;
  w.mine = load_seq(a, threadIdx.x & 31, status);
  walk_lane(a, w, per);
}
// The next 32 items; false (and the walk stays) at the end.
__device__ __forceinline__ bool walk_on(const PagedAttnArgs& a, Walk& w, int per, int32_t* status) {
  const int step = 32 >> w.shift;
  if (w.shift == 5 && (int64_t)(w.k + 1) * 32 * per < rows_of(a, w.s)) {      // w.s: the same in every lane
    ++w.k;
  } else if (w.i + step < 32 && w.b0 + w.i + step < a.B) {
    w.i += step;
    w.k = 0;
  } else if (w.b0 + 32 < a.B) {
    w.b0 += 32;
    w.i = w.k = 0;
    w.mine = load_seq(a, w.b0 + (threadIdx.x & 31), status);
  } else {
    return false;
  }
  walk_lane(a, w, per);
  return true;
}

struct Share {
  int p, shares;
  int64_t all, from, to;                 // units of all items, the share's
  bool cuts, end;
  // the item at hand: in the walk's lane L, head h, its first unit
  Walk w;
  int L, h;
  int64_t at;
};

__device__ __forceinline__ int64_t share_border(const Share& sh, int p) {
  // (64-bit divisions are slow)
  if (sh.all < (1 << 24)) return (uint32_t)sh.all * (uint32_t)p / (uint32_t)sh.shares;
  return sh.all * p / sh.shares;
}

// Share p's part of the row (one warp, the same in every lane).
__device__ __forceinline__ void find_share(const PagedAttnArgs& a, Share& sh, int p, int per) {
  int32_t* status = p == 0 ? a.status : nullptr;
  sh.p = p;
  sh.cuts = a.part_o != nullptr;
  walk_start(a, sh.w, per, status);
  int64_t sum = sh.w.units;
  bool one = true;                         // 32 items hold them all
  while (walk_on(a, sh.w, per, status)) sum += sh.w.units, one = false;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  sh.all = sum * a.Hkv;
  const int64_t most = sh.all / (fixed_units(per) + 4 * kFull);
  sh.shares = most < 1 ? 1 : most < a.shares ? (int)most : a.shares;
  sh.end = p >= sh.shares;
  sh.from = share_border(sh, p);
  sh.to = share_border(sh, p + 1);
  if (sh.end || sh.from >= sh.to) {
    sh.end = true;
    return;
  }
  // the item that holds unit `from`
  const int lane = threadIdx.x & 31;
  int64_t base = 0;
  if (!one) walk_start(a, sh.w, per, nullptr);
  do {
    int64_t end = (int64_t)sh.w.units * a.Hkv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += x;
    }
    end += base;
    const uint32_t hit = __ballot_sync(0xffffffffu, end > sh.from);
    if (hit) {
      sh.L = __ffs(hit) - 1;
      const int64_t first = __shfl_sync(0xffffffffu, end - (int64_t)sh.w.units * a.Hkv, sh.L);
      const int u = __shfl_sync(0xffffffffu, sh.w.units, sh.L);
      sh.h = sh.all < INT_MAX ? (int)(sh.from - first) / u : (int)((sh.from - first) / u);
      sh.at = first + (int64_t)sh.h * u;
      return;
    }
    base = __shfl_sync(0xffffffffu, end, 31);
  } while (walk_on(a, sh.w, per, nullptr));
  sh.end = true;
}

// The key tile of the item before which unit `unit` of the row falls.
__device__ __forceinline__ int border_tile(const Share& sh, const Item& it, int64_t unit, int per) {
  const int64_t o = unit - it.at;
  const int n = it.tiles.n;
  if (o <= 0) return 0;
  if (o >= it.units) return n;
  if (!sh.cuts) return 2 * o <= it.units ? 0 : n;
  const int fixed = fixed_units(per);
  return o <= fixed ? 0 : (int)(o - fixed) / (it.nt == 2 ? kFull : half_units(per));
}
__device__ __forceinline__ int border(const Share& sh, int p, const Item& it, int per) {
  return border_tile(sh, it, share_border(sh, p), per);
}

// The share's next item, or (nt = 0) none.
__device__ __forceinline__ void next_item(const PagedAttnArgs& a, Share& sh, Item& it, int per) {
  it.nt = 0;
  it.T = 0;
  while (!sh.end && sh.at < sh.to) {
    it.s = shfl_seq(sh.w.s, sh.L);
    it.b = __shfl_sync(0xffffffffu, sh.w.b, sh.L);
    it.r0 = (uint32_t)__shfl_sync(0xffffffffu, sh.w.rt, sh.L) * (uint32_t)per;
    it.units = item_units(a, it.s, (int)it.r0, per, it.tiles, it.nt);
    it.rows = (uint32_t)rows_of(a, it.s);
    it.h = sh.h;
    it.at = sh.at;
    it.j0 = border_tile(sh, it, sh.from, per);
    it.T = border_tile(sh, it, sh.to, per) - it.j0;
    // (an item without keys: its start decides whose it is)
    const bool mine = it.T > 0 || (it.tiles.n == 0 && sh.from <= sh.at);
    it.slot = it.T < it.tiles.n ? 2 * sh.p + (it.j0 == 0) : -1;
    // on to the next
    sh.at += it.units;
    if (++sh.h == a.Hkv) {
      sh.h = 0;
      uint32_t rest = __ballot_sync(0xffffffffu, sh.w.units > 0) & (sh.L == 31 ? 0u : ~0u << (sh.L + 1));
      while (!rest) {
        if (!walk_on(a, sh.w, per, nullptr)) {
          sh.end = true;
          break;
        }
        rest = __ballot_sync(0xffffffffu, sh.w.units > 0);
      }
      if (rest) sh.L = __ffs(rest) - 1;
    }
    if (mine) return;
    it.nt = 0;
    it.T = 0;
  }
}

// What the join of a cut item needs, in the workspace: written by the share that holds the item's last part.
struct Cut {
  int parts, t0, h;                      // parts 0: no cut ends in this share
  uint32_t r0, rows;
  int slots[kMaxShares + 1];             // of the parts, the last first
};
__device__ __forceinline__ void write_cut(const Share& sh, const Item& it, Cut* cut, int per) {
  const int lane = threadIdx.x & 31;
  if (it.nt == 0 || it.j0 == 0 || it.j0 + it.T < it.tiles.n) {
    if (lane == 0) cut->parts = 0;
    return;
  }
  int n = 0, j = INT_MAX;
  for (int p = sh.p; p >= 0 && j > 0; --p) {
    const int from = border(sh, p, it, per);
    if (from < j) {                      // a share without a key tile of the item has no part
      if (lane == 0) cut->slots[n] = 2 * p + (from == 0);
      ++n;
      j = from;
    }
  }
  if (lane == 0) {
    cut->t0 = it.s.t0;
    cut->h = it.h;
    cut->r0 = it.r0;
    cut->rows = it.rows;
    cut->parts = n;
  }
}

}  // namespace paged
}  // namespace fastar
