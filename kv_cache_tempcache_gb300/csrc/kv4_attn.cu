// Softmax attention over the 4-bit cache: the plan (which kernel, how many splits of the
// keys) and the kernel that joins the splits.
//
// The G = Hq / Hkv query heads that share a KV head see the same keys, so the rows of a KV
// head's work are all (head, token) pairs, r = g * nq + t: the cache is read once for the
// G heads.  With few rows the keys are cut into S splits, one block each, whose partial
// (sum of p v, maximum, sum of p) go to the workspace in fp32 and are joined by a second
// launch.
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"
#include "tmap.h"

namespace fastar {

namespace {

// ---- joining the splits ----------------------------------------------------------------------
// O = sum_s e^(m_s - m) o_s / sum_s e^(m_s - m) l_s over a row's S partials, m = max_s m_s; one
// warp a row, D / 32 channels a lane.  The partials are summed in the order of the splits, so
// results do not change from run to run.  A split in which the row sees no key has l = 0 and
// nothing in o; (inf, 0) for the first split says that the output is in place already.
// Bound: latency, so the loads do not wait for one another (kFew: at most 8 splits, all at once).
template <typename T, int D, bool kFew>
__device__ __forceinline__ void join_row(const Kv4AttnArgs& a, int64_t row, int64_t rows, int lane) {
  constexpr int CPL = D / 32;
  float m = neg_inf(), l = 0.f, o[CPL];
#pragma unroll
  for (int i = 0; i < CPL; ++i) o[i] = 0.f;
  if (kFew) {
    float2 ml[8];
    float p[8][CPL];
#pragma unroll
    for (int s = 0; s < 8; ++s) ml[s] = s < a.splits ? a.part_ml[s * rows + row] : make_float2(neg_inf(), 0.f);
    if (ml[0].x == -neg_inf() && ml[0].y == 0.f) return;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const float* src = a.part_o + (s * rows + row) * D + lane * CPL;
#pragma unroll
      for (int c = 0; c < CPL; ++c) p[s][c] = ml[s].y != 0.f ? src[c] : 0.f;
    }
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (ml[s].y != 0.f) m = fmaxf(m, ml[s].x);
    const float ref = m == neg_inf() ? 0.f : m;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const bool in = ml[s].y != 0.f;
      const float w = in ? expf(ml[s].x - ref) : 0.f;
      l = fmaf(w, ml[s].y, l);
#pragma unroll
      for (int c = 0; c < CPL; ++c) o[c] = fmaf(w, p[s][c], o[c]);
    }
  } else {
    // lane s % 32 reads split s's maximum and sum; then the outputs, eight splits' loads at a time
    constexpr int kPer = kKv4MaxSplits / 32;
    float2 ml[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      ml[i] = make_float2(neg_inf(), 0.f);
      if (32 * i + lane < a.splits) ml[i] = a.part_ml[(32 * i + lane) * rows + row];
      if (ml[i].y != 0.f) m = fmaxf(m, ml[i].x);
    }
    if (__any_sync(0xffffffffu, lane == 0 && ml[0].x == -neg_inf() && ml[0].y == 0.f)) return;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    const float ref = m == neg_inf() ? 0.f : m;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (32 * i >= a.splits) break;
      const float w = ml[i].y != 0.f ? expf(ml[i].x - ref) : 0.f;
      const int here = a.splits - 32 * i < 32 ? a.splits - 32 * i : 32;
#pragma unroll 1
      for (int s0 = 0; s0 < here; s0 += 8) {
        float p[8][CPL], ws[8], ls[8];
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const int src = s0 + s < 32 ? s0 + s : 31;
          ls[s] = __shfl_sync(0xffffffffu, ml[i].y, src);
          ws[s] = __shfl_sync(0xffffffffu, w, src);
          const bool in = s0 + s < here && ls[s] != 0.f;
          const float* src_o = a.part_o + ((32 * i + s0 + s) * rows + row) * D + lane * CPL;
#pragma unroll
          for (int c = 0; c < CPL; ++c) p[s][c] = in ? src_o[c] : 0.f;
          if (!in) ws[s] = ls[s] = 0.f;
        }
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          l = fmaf(ws[s], ls[s], l);
#pragma unroll
          for (int c = 0; c < CPL; ++c) o[c] = fmaf(ws[s], p[s][c], o[c]);
        }
      }
    }
  }
  const bool live = l > 0.f || l != l;
  const int64_t head = row / a.nq, t = row - head * a.nq;
  T* out = static_cast<T*>(a.out) + head * a.o_hs + t * a.o_ts + lane * CPL;
#pragma unroll
  for (int i = 0; i < CPL; ++i) out[i] = from_f<T>(live ? o[i] / l : 0.f);
  if (lane == 0 && a.lse) a.lse[row] = live ? m + logf(l) : neg_inf();
}

// A warp takes `per` rows, at most 32: with more than one it looks at all their first splits at once,
// so that a call of many rows whose outputs are in place costs little.
template <typename T, int D, bool kFew>
__global__ void __launch_bounds__(128) kv4_join_kernel(const Kv4AttnArgs a, int per) {
  const int64_t rows = (int64_t)a.Hq * a.nq, row0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 5)) * per;
  const int lane = threadIdx.x & 31;
  pdl_wait();
  if (row0 >= rows) return;
  uint32_t todo = 1;
  if (per > 1) {
    const bool in = lane < per && row0 + lane < rows;
    const float2 ml = in ? a.part_ml[row0 + lane] : make_float2(0.f, 0.f);
    todo = __ballot_sync(0xffffffffu, in && !(ml.x == -neg_inf() && ml.y == 0.f));
  }
  for (; todo; todo &= todo - 1) join_row<T, D, kFew>(a, row0 + __ffs(todo) - 1, rows, lane);
}

template <typename T, int D>
cudaError_t join_go(const Kv4AttnArgs& a, cudaStream_t s) {
  // a row a warp up to as many rows as are resident at once, then up to 8
  const int64_t rows = (int64_t)a.Hq * a.nq, resident = 48 * (int64_t)sm_count();
  const int per = rows <= resident ? 1 : rows <= 8 * resident ? (int)((rows + resident - 1) / resident) : 8;
  const dim3 grid((unsigned)((rows + 4 * per - 1) / (4 * per)));
  const cudaError_t e = a.splits <= 8 ? launch_dependent(kv4_join_kernel<T, D, true>, grid, dim3(128), 0, s, a, per)
                                      : launch_dependent(kv4_join_kernel<T, D, false>, grid, dim3(128), 0, s, a, per);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Rows of a KV head that take the few-rows kernel (kv4_attn_few.cu) in bf16; in fp32 all do.  At 16
// rows it and the tcgen05 kernel take 21 and 23 us over 9000 rows of 8 heads, 64 and 119 over
// 131,071, 17 and 19 over 9000 rows of 64 channels; above 16 it would read the cache twice.
constexpr int64_t kFewRows = 16;

// Splits for it: one CTA a multiprocessor, but none under a block of 32 keys a warp, and none at
// all for fewer than three of those (there the join costs more than they save; 1000 rows: 13 us
// either way).  Against two blocks a warp: one token of 12 heads over 2000 rows 19 -> 15 us, twelve
// tokens 19 -> 17, five fp32 tokens of 16 heads over 3000 rows 18 -> 17.  items: KV heads, in fp32
// times groups of 8 rows; warps: of a CTA.
int splits_few(int64_t items, int64_t cap, int warps) {
  const int64_t want = sm_count() / items, most = cap / (32 * warps);
  int64_t s = want < most ? want : most;
  if (s > kKv4MaxSplits) s = kKv4MaxSplits;
  return s < 1 || most < 3 ? 1 : (int)s;
}

// The tensor-core kernel at d = 128: CTAs alone where the rows are one tile of 128 and the full cache
// gives each multiprocessor two key tiles or more, else in pairs.  A pair halves the unpacking,
// which bounds it with many rows; with one tile half its rows are empty, and what bounds it is one
// tile's way from product to product, of which single CTAs run twice as many.  32 rows over
// 131,071 keys of 8 heads take 74 us alone and 119 in pairs, 64 over 2000 of 12 heads 20 either
// way, 64 over 500 of 12 heads 17 and 15.
bool tc_alone(int d, int64_t rows, int Hkv, int64_t cap) {
  return d == 128 && rows <= 128 && (cap + 127) / 128 * Hkv >= 2 * sm_count();
}

// Splits for the tensor-core kernel, by a model of its time over a full cache: waves of CTAs
// (pairs of them at d = 128), each a fixed part and so much a key tile; items with one row
// tile, half as long a tile, fill the last wave's gaps; and with splits the partials' way through
// memory and the join.  The fewest splits within 2 % of the best.  (Measured: 1.5 us a tile of
// 128 keys and 512 rows at d = 128, 8 us around them; 1.2 us a tile of a CTA alone.)
// The cache's lengths are the device's, and may be far below its capacity: *min_tiles is what the
// kernel keeps a split's key tiles to, 3 where all the splits run at once, else 40, beside which
// the fixed part is small.
int splits_tc(int d, int64_t rows, int Hkv, int64_t cap, int* min_tiles) {
  const bool alone = tc_alone(d, rows, Hkv, cap);
  const int cta = alone ? 1 : d / 64;     // CTAs that work as one (kv4_attn_tc.cu)
  const int64_t slots = sm_count() / cta, tiles = (cap + 127) / 128;
  const int64_t half = (rows - 1) % (256 * cta) < 128 * cta ? Hkv : 0;
  const int64_t full = (rows + 256 * cta - 1) / (256 * cta) * Hkv - half;
  const double tile = 1.5, fixed = 8.0;
  auto cost = [&](int64_t s) {
    const int64_t waves = (full * s + slots - 1) / slots, gaps = 2 * (waves * slots - full * s);
    const int64_t rest = half * s > gaps ? (half * s - gaps + slots - 1) / slots : 0;
    const double keys = (double)((tiles + s - 1) / s) * (alone ? 1.5 * tile : tile);
    const double join = s > 1 ? 4.0 + 2e-6 * s * rows * Hkv * (d + 2) * 4 / 4.0 : 0.0;
    return waves * (fixed + keys) + rest * (fixed + 0.6 * keys) + join;
  };
  int64_t most = (4 * slots + full + half - 1) / (full + half);
  if (most > tiles) most = tiles;
  if (most > kKv4MaxSplits) most = kKv4MaxSplits;
  double best = cost(1);
  int64_t pick = 1;
  for (int64_t s = 2; s <= most; s += 1 + s / 8) {   // every few: this runs on each call
    const double c = cost(s);
    if (c < 0.98 * best) best = c, pick = s;
  }
  if (min_tiles) *min_tiles = (full + half) * pick <= slots ? 3 : 40;
  return (int)pick;
}

size_t partial_bytes(int splits, int d, int Hq, int64_t nq) {
  return splits == 1 ? 0 : (size_t)splits * Hq * nq * (d + 2) * sizeof(float);
}

cudaError_t run(int dtype, int d, Kv4AttnArgs a, void* ws, cudaStream_t s) {
  if (a.splits > 1) {
    a.part_o = static_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + (int64_t)a.splits * a.Hq * a.nq * d);
  }
  const bool few = dtype == FASTAR_F32 || a.rows <= kFewRows;
  a.alone = tc_alone(d, a.rows, a.Hkv, a.cap);
  if (!few && a.min_tiles == 0) a.min_tiles = 1;         // one split
  const cudaError_t e = few ? launch_kv4_attn_few(dtype, d, a, s) : launch_kv4_attn_tc(d, a, s);
  if (e != cudaSuccess || a.splits == 1) return e;
  if (dtype == FASTAR_F32) return d == 128 ? join_go<float, 128>(a, s) : join_go<float, 64>(a, s);
  return d == 128 ? join_go<__nv_bfloat16, 128>(a, s) : join_go<__nv_bfloat16, 64>(a, s);
}

}  // namespace

int kv4_attn_splits(int dtype, int d, int Hq, int Hkv, int64_t nq, int64_t cap, int* min_tiles) {
  const int64_t rows = (int64_t)(Hq / Hkv) * nq;
  if (dtype == FASTAR_F32) return splits_few((rows + 7) / 8 * Hkv, cap, 8);
  return rows <= kFewRows ? splits_few(Hkv, cap, rows > 8 ? 8 : 16) : splits_tc(d, rows, Hkv, cap, min_tiles);
}

size_t kv4_attn_workspace(int d, int Hq, int Hkv, int64_t nq, int64_t cap) {
  int s = 1;
  for (int dt : {FASTAR_F32, FASTAR_BF16}) {
    const int x = kv4_attn_splits(dt, d, Hq, Hkv, nq, cap, nullptr);
    s = x > s ? x : s;
  }
  return partial_bytes(s, d, Hq, nq);
}

bool launch_kv4_attn(int dtype, int d, Kv4AttnArgs a, void* ws, size_t ws_bytes, cudaStream_t s, cudaError_t* err) {
  a.group = a.Hq / a.Hkv;
  a.rows = (uint32_t)(a.group * a.nq);       // Hq * nq fits 31 bits
  a.min_tiles = 0;
  a.splits = ws ? kv4_attn_splits(dtype, d, a.Hq, a.Hkv, a.nq, a.cap, &a.min_tiles) : 1;
  if (a.splits > 1 && ws_bytes < partial_bytes(a.splits, d, a.Hq, a.nq)) return false;
  *err = run(dtype, d, a, ws, s);
  return true;
}

}  // namespace fastar
