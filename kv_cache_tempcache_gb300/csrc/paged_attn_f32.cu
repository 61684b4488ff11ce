// Softmax attention over a paged cache in fp32: 32 rows and 64 keys at a time.
//
// Two rows a half warp: a thread forms the logits of two rows and four keys, then two rows and D / 16
// channels of the output.  Keys that no row of the block sees are zeros in shared memory; where only
// some rows see a key the others leave it out (not by a weight of 0: its value may be infinite).
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"
#include "paged_attn.h"
#include "tmap.h"

namespace fastar {

namespace {

constexpr int kRows = kF32Rows, kKeys = kF32Keys;

template <int D>
struct F32Layout {
  static constexpr int ld = D + 4;                       // float4 reads of 8 rows hit 8 bank groups
  static constexpr int q = 0, k = q + kRows * ld, v = k + kKeys * ld, p = v + kKeys * ld;
  static constexpr int ldp = kKeys + 4;
  static constexpr int bytes = (p + kRows * ldp) * 4;
};

template <int D>
__global__ void __launch_bounds__(256) paged_attn_f32_kernel(const PagedAttnArgs a, int row_tiles) {
  using Lay = F32Layout<D>;
  extern __shared__ __align__(16) float sm[];
  float *sq = sm + Lay::q, *sk = sm + Lay::k, *sv = sm + Lay::v, *sp = sm + Lay::p;
  pdl_wait();
  // heads side by side, then row tiles from the last, then slots
  int u = blockIdx.x;
  const int h = u % a.Hkv;
  u /= a.Hkv;
  const int slot = u / row_tiles, r0 = (row_tiles - 1 - u % row_tiles) * kRows;
  paged::Work work;
  if (!paged::find_work<kKeys>(a, slot, 0, work)) return;
  const int b = work.b;
  const paged::Seq s = paged::sequence(a.cu, a.at, a.B, a.T, a.cap, b, a.status);
  if (s.nq > a.max_q && threadIdx.x == 0) flag_status(a.status, FASTAR_DEV_BAD_LEN);
  const int G = a.group, rows = G * min(s.nq, a.max_q);
  if (r0 >= rows) return;
  const int rl = min(r0 + kRows, rows) - 1;
  paged::Tiles<kKeys> tiles;
  tiles.set(a, s, r0 / G, rl / G);
  const paged::Split part = paged::part_of(tiles.n, work);
  const bool partial = part.used > 1;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  paged::Sees see[2];
  int64_t tok[2];
  int head[2];
  bool has[2];
  float m[2], l[2], o[2][D / 16];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = min(r0 + 2 * ty + i, rl);
    has[i] = r0 + 2 * ty + i <= rl;
    see[i] = paged::sees(a, s, r / G);
    tok[i] = s.t0 + r / G;
    head[i] = h * G + r % G;
    m[i] = neg_inf();
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) o[i][c] = 0.f;
  }
  for (int x = threadIdx.x; x < kRows * (D / 8); x += 256) {
    const int row = x / (D / 8), c = x % (D / 8) * 8, r = min(r0 + row, rl);
    float f[8];
    load8(static_cast<const float*>(a.q.p) + (int64_t)(h * G + r % G) * a.q.hs + (int64_t)(s.t0 + r / G) * a.q.ts + c, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) sq[row * Lay::ld + c + e] = f[e];
  }
  const float sl2 = a.scale * 1.4426950408889634f;
  const int32_t* table = a.table + (int64_t)b * a.max_pages;
  for (int j = part.j0; j < part.j1; ++j) {
    const int key0 = tiles.key(j);
    __syncthreads();
    for (int x = threadIdx.x; x < kKeys * (D / 8); x += 256) {
      const int row = x / (D / 8), c = x % (D / 8) * 8, key = key0 + row;
      float fk[8] = {}, fv[8] = {};
      if (tiles.any(key)) {
        const int page = paged::page_of(table, key >> a.pool.page_shift, a.pool.pages, a.status);
        if (page >= 0) {
          const int64_t at = page * a.pool.ps + h * a.pool.hs + (key & ((1 << a.pool.page_shift) - 1)) * a.pool.rs + c;
          load8(static_cast<const float*>(a.pool.k) + at, fk);
          load8(static_cast<const float*>(a.pool.v) + at, fv);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sk[row * Lay::ld + c + e] = fk[e], sv[row * Lay::ld + c + e] = fv[e];
    }
    __syncthreads();
    float x[2][4] = {};
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      const float4 q0 = *reinterpret_cast<const float4*>(&sq[2 * ty * Lay::ld + c]);
      const float4 q1 = *reinterpret_cast<const float4*>(&sq[(2 * ty + 1) * Lay::ld + c]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 kv = *reinterpret_cast<const float4*>(&sk[(tx + 16 * k) * Lay::ld + c]);
        x[0][k] = fmaf(q0.x, kv.x, fmaf(q0.y, kv.y, fmaf(q0.z, kv.z, fmaf(q0.w, kv.w, x[0][k]))));
        x[1][k] = fmaf(q1.x, kv.x, fmaf(q1.y, kv.y, fmaf(q1.z, kv.z, fmaf(q1.w, kv.w, x[1][k]))));
      }
    }
    uint64_t bits[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      bits[i] = paged::seen32(see[i], key0) | (uint64_t)paged::seen32(see[i], key0 + 32) << 32;
      float top = neg_inf();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[i][k] = bits[i] >> (tx + 16 * k) & 1 ? x[i][k] * sl2 : neg_inf();
        top = fmaxf(top, x[i][k]);
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      const float mn = fmaxf(m[i], top), ref = mn == neg_inf() ? 0.f : mn;
      const float f = exp2f(m[i] - ref);
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float p = exp2f(x[i][k] - ref);
        sum += p;
        sp[(2 * ty + i) * Lay::ldp + tx + 16 * k] = p;
      }
      m[i] = mn;
      l[i] = l[i] * f + sum;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[i][c] *= f;
    }
    __syncwarp();
    const bool whole = tiles.all(key0);
#pragma unroll 2
    for (int k = 0; k < kKeys; ++k) {
      const float p0 = sp[2 * ty * Lay::ldp + k], p1 = sp[(2 * ty + 1) * Lay::ldp + k];
      const bool in0 = whole || (bits[0] >> k & 1), in1 = whole || (bits[1] >> k & 1);
#pragma unroll
      for (int c = 0; c < D / 16; c += 4) {
        const float4 v = *reinterpret_cast<const float4*>(&sv[k * Lay::ld + tx * 4 + c * 16]);
        if (in0) {
          o[0][c] = fmaf(p0, v.x, o[0][c]), o[0][c + 1] = fmaf(p0, v.y, o[0][c + 1]);
          o[0][c + 2] = fmaf(p0, v.z, o[0][c + 2]), o[0][c + 3] = fmaf(p0, v.w, o[0][c + 3]);
        }
        if (in1) {
          o[1][c] = fmaf(p1, v.x, o[1][c]), o[1][c + 1] = fmaf(p1, v.y, o[1][c + 1]);
          o[1][c + 2] = fmaf(p1, v.z, o[1][c + 2]), o[1][c + 3] = fmaf(p1, v.w, o[1][c + 3]);
        }
      }
    }
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
    if (!has[i]) continue;
    const bool live = l[i] > 0.f || l[i] != l[i];
    const int64_t row = paged::partial_row(a, slot, h, r0 + 2 * ty + i);
    const float mn = m[i] * 0.6931471805599453f;
    if (tx == 0) {
      if (partial) a.part_ml[row] = make_float2(live ? mn : neg_inf(), l[i]);
      if (!partial && a.lse) a.lse[head[i] * a.T + tok[i]] = live ? mn + logf(l[i]) : neg_inf();
    }
    const float f = partial ? 1.f : 1.f / l[i];
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      const int ch = tx * 4 + (c >> 2) * 64 + (c & 3);
      const float y = live ? o[i][c] * f : 0.f;
      if (partial) a.part_o[row * D + ch] = y;
      else static_cast<float*>(a.out)[head[i] * a.o_hs + tok[i] * a.o_ts + ch] = y;
    }
  }
}

template <int D>
cudaError_t f32_go(const PagedAttnArgs& a, cudaStream_t s) {
  const int64_t rt = ((int64_t)a.group * a.max_q + kRows - 1) / kRows;
  const int64_t blocks = rt * a.Hkv * (a.B + a.extra);
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  cudaError_t e = opt_in_smem((const void*)paged_attn_f32_kernel<D>, F32Layout<D>::bytes);
  if (e != cudaSuccess) return e;
  e = launch_dependent(paged_attn_f32_kernel<D>, dim3((unsigned)blocks), dim3(256), F32Layout<D>::bytes, s, a,
                       (int)rt);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_attn_f32(int d, const PagedAttnArgs& a, cudaStream_t s) {
  return d == 128 ? f32_go<128>(a, s) : f32_go<64>(a, s);
}

}  // namespace fastar
