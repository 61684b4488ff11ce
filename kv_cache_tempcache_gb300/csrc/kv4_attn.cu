// Softmax attention over the 4-bit cache: the plan (which kernel, how many splits of the
// keys), the fp32 kernel, and the kernel that joins the splits.
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

// ---- the fp32 kernel -----------------------------------------------------------------------
// For fp32 queries (bf16 ones go to the tensor cores, kv4_attn_tc.cu): one block takes 8 rows of a KV head
// and a range of keys, unpacks 64 keys at a time to fp32 in shared memory and forms the 8 x 64
// logits, their softmax and 8 x d outputs with fp32 arithmetic throughout.  Bound: the fp32
// units (2 flops a row, key and channel twice over), and below them latency.
constexpr int kRows = 8, kKeys = 64, kThreadsF = 128;

template <int D>
struct FSmem {
  float k[kKeys][D + 4];
  float v[kKeys][D];
  float q[kRows][D];
  float p[kRows][kKeys];
  float alpha[kRows], l[kRows], m[kRows];
};

template <int D>
__global__ void __launch_bounds__(kThreadsF) kv4_attn_f32_kernel(const Kv4AttnArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  FSmem<D>& sm = *reinterpret_cast<FSmem<D>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;
  const int64_t rows = (int64_t)G * a.nq;
  const int64_t groups = (rows + kRows - 1) / kRows;
  int64_t u = blockIdx.x;
  const int split = (int)(u % a.splits);
  u /= a.splits;
  const int64_t r0 = u % groups * kRows;
  const int h = (int)(u / groups);
  const int64_t len = kv4::head_len(a.len, h, a.cap, a.status);
  // the keys that any of the rows sees, cut evenly into whole tiles
  int64_t most = 0;
  for (int i = 0; i < kRows; ++i)
    if (r0 + i < rows) {
      const int64_t v = kv4::visible(len, a.nq, (r0 + i) % a.nq, a.block);
      most = v > most ? v : most;
    }
  const int64_t tiles = (most + kKeys - 1) / kKeys;
  const int64_t j0 = tiles * split / a.splits * kKeys;
  const int64_t j1 = tiles * (split + 1) / a.splits * kKeys < most ? tiles * (split + 1) / a.splits * kKeys : most;
  const float sl = a.scale * kv4::pow2i(kv4::head_exp(a.k_exp, h));

  for (int i = tid; i < kRows * D; i += kThreadsF) {
    const int64_t r = r0 + i / D;
    const int64_t g = r / a.nq;
    sm.q[i / D][i % D] =
        r < rows ? static_cast<const float*>(a.q.p)[(h * G + g) * a.q.hs + (r - g * a.nq) * a.q.ts + i % D] : 0.f;
  }
  if (tid < kRows) {
    sm.m[tid] = neg_inf();
    sm.l[tid] = 0.f;
  }
  constexpr int CPT = kRows * D / kThreadsF;     // outputs of a thread: one channel, CPT rows
  const int oc = tid % D, or0 = tid / D * CPT;
  float o[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) o[i] = 0.f;

  for (int64_t j = j0; j < j1; j += kKeys) {
    __syncthreads();
    const int nk = (int)(j1 - j < kKeys ? j1 - j : kKeys);
    for (int i = tid; i < kKeys * (D / 8); i += kThreadsF) {
      const int row = i / (D / 8), c = i % (D / 8);
      uint32_t pk[4] = {0, 0, 0, 0}, pv[4] = {0, 0, 0, 0};   // rows past the range count as 0
      if (row < nk) {
        const int64_t at = (int64_t)h * a.cap + j + row;
        kv4::unpack8(reinterpret_cast<const uint32_t*>(a.kc)[at * (D / 8) + c],
                     kv4::scale_f16x2(a.ks[at * (D / 16) + c / 2]), pk);
        kv4::unpack8(reinterpret_cast<const uint32_t*>(a.vc)[at * (D / 8) + c],
                     kv4::scale_f16x2(a.vs[at * (D / 16) + c / 2]), pv);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = kv4::f16x2_to_f32(pk[e]), y = kv4::f16x2_to_f32(pv[e]);
        *reinterpret_cast<float2*>(&sm.k[row][c * 8 + 2 * e]) = x;
        *reinterpret_cast<float2*>(&sm.v[row][c * 8 + 2 * e]) = y;
      }
    }
    __syncthreads();
    // warp w: rows 2w and 2w + 1; lane: keys lane and lane + 32
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      const int row = warp * 2 + rr;
      const int64_t r = r0 + row;
      const int64_t see = r < rows ? kv4::visible(len, a.nq, r % a.nq, a.block) - j : 0;
      float s0 = 0.f, s1 = 0.f;
#pragma unroll 8
      for (int c = 0; c < D; c += 4) {
        const float4 x = *reinterpret_cast<const float4*>(&sm.q[row][c]);
        const float4 k0 = *reinterpret_cast<const float4*>(&sm.k[lane][c]);
        const float4 k1 = *reinterpret_cast<const float4*>(&sm.k[lane + 32][c]);
        s0 = fmaf(x.x, k0.x, fmaf(x.y, k0.y, fmaf(x.z, k0.z, fmaf(x.w, k0.w, s0))));
        s1 = fmaf(x.x, k1.x, fmaf(x.y, k1.y, fmaf(x.z, k1.z, fmaf(x.w, k1.w, s1))));
      }
      const int64_t lim = see < nk ? see : nk;
      s0 = lane < lim ? s0 * sl : neg_inf();
      s1 = lane + 32 < lim ? s1 * sl : neg_inf();
      float mx = fmaxf(s0, s1);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float mo = sm.m[row], mn = fmaxf(mo, mx);
      const float ref = mn == neg_inf() ? 0.f : mn;
      const float p0 = expf(s0 - ref), p1 = expf(s1 - ref);
      const float al = expf(mo - ref);
      const float sum = warp_sum(p0 + p1);
      sm.p[row][lane] = p0;
      sm.p[row][lane + 32] = p1;
      __syncwarp();
      if (lane == 0) {
        sm.alpha[row] = al;
        sm.l[row] = sm.l[row] * al + sum;
        sm.m[row] = mn;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < CPT; ++i) o[i] *= sm.alpha[or0 + i];
#pragma unroll 4
    for (int key = 0; key < kKeys; ++key) {
      const float v = sm.v[key][oc];
#pragma unroll
      for (int i = 0; i < CPT; ++i) o[i] = fmaf(sm.p[or0 + i][key], v, o[i]);
    }
  }
  __syncthreads();
  const float up = kv4::pow2i(kv4::head_exp(a.v_exp, h));
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int64_t r = r0 + or0 + i;
    if (r >= rows) continue;
    const int64_t g = r / a.nq, t = r - g * a.nq, head = h * G + g;
    const float l = sm.l[or0 + i], m = sm.m[or0 + i];
    if (a.splits > 1) {
      const int64_t at = (split * (int64_t)a.Hq + head) * a.nq + t;
      a.part_o[at * D + oc] = o[i] * up;
      if (oc == 0) a.part_ml[at] = make_float2(m, l);
    } else {
      static_cast<float*>(a.out)[head * a.o_hs + t * a.o_ts + oc] = l > 0.f || l != l ? o[i] * up / l : 0.f;
      if (oc == 0 && a.lse) a.lse[head * a.nq + t] = l > 0.f || l != l ? m + logf(l) : neg_inf();
    }
  }
}

// ---- joining the splits ----------------------------------------------------------------------
// O = sum_s e^(m_s - m) o_s / sum_s e^(m_s - m) l_s over a row's S partials, m = max_s m_s; one
// warp a row, D / 32 channels a lane.  The partials are summed in the order of the splits, so
// results do not change from run to run.  A split in which the row sees no key has l = 0 and
// nothing in o; (inf, 0) for the first split says that the output is in place already.
// Bound: latency, so the loads do not wait for one another (kFew: at most 8 splits, all at once).
template <typename T, int D, bool kFew>
__global__ void __launch_bounds__(128) kv4_join_kernel(const Kv4AttnArgs a) {
  constexpr int CPL = D / 32;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)a.Hq * a.nq;
  pdl_wait();
  if (row >= rows) return;
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

template <typename T, int D>
cudaError_t join_go(const Kv4AttnArgs& a, cudaStream_t s) {
  const int64_t rows = (int64_t)a.Hq * a.nq;
  const dim3 grid((unsigned)((rows + 3) / 4));
  const cudaError_t e = a.splits <= 8 ? launch_dependent(kv4_join_kernel<T, D, true>, grid, dim3(128), 0, s, a)
                                      : launch_dependent(kv4_join_kernel<T, D, false>, grid, dim3(128), 0, s, a);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D>
cudaError_t f32_go(const Kv4AttnArgs& a, cudaStream_t s) {
  const int64_t rows = (int64_t)(a.Hq / a.Hkv) * a.nq;
  const int64_t blocks = (rows + kRows - 1) / kRows * a.Hkv * a.splits;
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  const cudaError_t e = opt_in_smem((const void*)kv4_attn_f32_kernel<D>, (int)sizeof(FSmem<D>));
  if (e != cudaSuccess) return e;
  kv4_attn_f32_kernel<D><<<(unsigned)blocks, kThreadsF, sizeof(FSmem<D>), s>>>(a);
  count_launches(1);
  const cudaError_t r = cudaGetLastError();
  return r != cudaSuccess || a.splits == 1 ? r : join_go<float, D>(a, s);
}

// Splits of the keys for the fp32 kernel: two blocks a multiprocessor, none under 256 keys.
int splits_f32(int64_t blocks, int64_t cap) {
  const int64_t want = (2 * (int64_t)sm_count() + blocks - 1) / blocks;
  const int64_t most = cap / 256;
  int64_t s = want < most ? want : most;
  if (s > kKv4MaxSplits) s = kKv4MaxSplits;
  return s < 1 ? 1 : (int)s;
}

// Rows of a KV head that take the few-rows kernel (kv4_attn_few.cu).
constexpr int64_t kFewRows = 16;

// Splits for it: one CTA a multiprocessor, but none under 512 keys (64 a warp).
int splits_few(int Hkv, int64_t cap) {
  const int64_t want = sm_count() / Hkv, most = cap / 512;
  int64_t s = want < most ? want : most;
  if (s > kKv4MaxSplits) s = kKv4MaxSplits;
  return s < 1 ? 1 : (int)s;
}

// Splits for the tensor-core kernel, by a model of its time over a full cache: waves of CTAs
// (pairs of them at d = 128), each a fixed part and so much a key tile; items with one row
// tile, half as long a tile, fill the last wave's gaps; and with splits the partials' way through
// memory and the join.  The fewest splits within 2 % of the best.  (Measured: 1.5 us a tile of
// 128 keys and 512 rows at d = 128, 8 us around them.)
// The cache's lengths are the device's, and may be far below its capacity: *min_tiles is what the
// kernel keeps a split's key tiles to, 3 where all the splits run at once, else 40, beside which
// the fixed part is small.
int splits_tc(int d, int64_t rows, int Hkv, int64_t cap, int* min_tiles) {
  const int cta = d / 64;                 // CTAs that work as one (kv4_attn_tc.cu)
  const int64_t slots = sm_count() / cta, tiles = (cap + 127) / 128;
  const int64_t half = (rows - 1) % (256 * cta) < 128 * cta ? Hkv : 0;
  const int64_t full = (rows + 256 * cta - 1) / (256 * cta) * Hkv - half;
  const double tile = 1.5, fixed = 8.0;
  auto cost = [&](int64_t s) {
    const int64_t waves = (full * s + slots - 1) / slots, gaps = 2 * (waves * slots - full * s);
    const int64_t rest = half * s > gaps ? (half * s - gaps + slots - 1) / slots : 0;
    const double keys = (double)((tiles + s - 1) / s) * tile;
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
  if (dtype == FASTAR_F32) return d == 128 ? f32_go<128>(a, s) : f32_go<64>(a, s);
  const bool few = (int64_t)(a.Hq / a.Hkv) * a.nq <= kFewRows;
  if (!few && a.min_tiles == 0) a.min_tiles = 1;         // one split
  const cudaError_t e = few ? launch_kv4_attn_few(d, a, s) : launch_kv4_attn_tc(d, a, s);
  if (e != cudaSuccess || a.splits == 1) return e;
  return d == 128 ? join_go<__nv_bfloat16, 128>(a, s) : join_go<__nv_bfloat16, 64>(a, s);
}

}  // namespace

int kv4_attn_splits(int dtype, int d, int Hq, int Hkv, int64_t nq, int64_t cap, int* min_tiles) {
  const int64_t rows = (int64_t)(Hq / Hkv) * nq;
  if (dtype == FASTAR_BF16 && rows > kFewRows) return splits_tc(d, rows, Hkv, cap, min_tiles);
  if (dtype == FASTAR_BF16) return splits_few(Hkv, cap);
  return splits_f32((rows + kRows - 1) / kRows * Hkv, cap);
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
  a.min_tiles = 0;
  a.splits = ws ? kv4_attn_splits(dtype, d, a.Hq, a.Hkv, a.nq, a.cap, &a.min_tiles) : 1;
  if (a.splits > 1 && ws_bytes < partial_bytes(a.splits, d, a.Hq, a.nq)) return false;
  *err = run(dtype, d, a, ws, s);
  return true;
}

}  // namespace fastar
