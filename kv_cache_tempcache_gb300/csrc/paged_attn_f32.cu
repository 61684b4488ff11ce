// Softmax attention over a paged cache in fp32: 32 rows and 64 keys at a time.
//
// Two rows a half warp: a thread forms the logits of two rows and four keys, then two rows and D / 16
// channels of the output, two products an instruction.  A tile's keys and values come by cp.async while the one before
// is worked on; where their rows lie is looked up one tile earlier still.  Rows that no row of the block
// sees come as zeros; where only some rows see a key the others leave it out (not by a weight of 0: its value may
// be infinite).
// Bound: with few rows latency (a block has one or two tiles), with many the shared memory's 128 bytes a clock, of
// which every warp with rows takes all of a tile; weights are read four at a time, and warps without rows only bring tiles
// (one weight at a time in all warps: 18.2 us instead of 16.7 for the first call below, 169 instead of 130 with 100,000
// rows each).  Measured: up to 20 rows over 2006 rows of three sequences, d = 64, 16.3 us with the join in replayed graphs;
// one row over 100,000 rows of 4 heads 90 us (2.3 TB/s).
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"
#include "paged_attn.h"
#include "tc.cuh"
#include "tmap.h"

namespace fastar {

namespace {

constexpr int kRows = kF32Rows, kKeys = kF32Keys;

template <int D>
struct F32Layout {
  static constexpr int ld = D + 4;                       // float4 reads of 8 rows hit 8 bank groups
  static constexpr int q = 0, kv = q + kRows * ld, stage = 2 * kKeys * ld, p = kv + 2 * stage;   // K, V; two stages
  static constexpr int ldp = kKeys + 4;
  static constexpr int off = p + kRows * ldp;            // int64: where a tile's rows lie, two tiles'
  static constexpr int bytes = off * 4 + 2 * kKeys * 8;
};

// Two products or sums an instruction, on pairs of registers.
__device__ __forceinline__ void fma2(float2& c, float ax, float ay, float bx, float by) {
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%0, %1};\n"
      " fma.rn.f32x2 z, x, y, z;\n mov.b64 {%0, %1}, z;\n}\n"
      : "+f"(c.x), "+f"(c.y)
      : "f"(ax), "f"(ay), "f"(bx), "f"(by));
}

template <int D>
__global__ void __launch_bounds__(256) paged_attn_f32_kernel(const PagedAttnArgs a, int row_tiles) {
  using Lay = F32Layout<D>;
  extern __shared__ __align__(16) float sm[];
  float *sq = sm + Lay::q, *sp = sm + Lay::p;
  int64_t* rows_at = reinterpret_cast<int64_t*>(sm + Lay::off);
  pdl_wait();                              // the launch overlaps the end of the kernel before
  if (a.extra > 0) pdl_trigger();          // the join's CTAs may come, find their work and wait
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
  const int rl = r0 + min(kRows, rows - r0) - 1;
  paged::Tiles<kKeys> tiles;
  tiles.set(a, s, r0 / G, rl / G);
  const paged::Split part = paged::part_of(tiles.n, work);
  const bool partial = part.used > 1;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  paged::Sees see[2];
  int64_t tok[2];
  int head[2];
  bool has[2];
  float m[2], l[2];
  float2 o[2][D / 32];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + min(2 * ty + i, rl - r0);
    has[i] = 2 * ty + i <= rl - r0;
    see[i] = paged::sees(a, s, r / G);
    tok[i] = s.t0 + r / G;
    head[i] = h * G + r % G;
    m[i] = neg_inf();
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) o[i][c] = make_float2(0.f, 0.f);
  }
  const int32_t* table = a.table + (int64_t)b * a.max_pages;
  // where row threadIdx.x of tile j lies; -1: it comes as zeros
  auto look = [&](int j) {
    if (threadIdx.x >= kKeys || j >= part.j1) return;
    const int key = tiles.key(j) + (int)threadIdx.x;
    int64_t at = -1;
    if (tiles.any(key)) {
      const int page = paged::page_of(table, key >> a.pool.page_shift, a.pool.pages, a.status);
      if (page >= 0) at = page * a.pool.ps + h * a.pool.hs + (key & ((1 << a.pool.page_shift) - 1)) * a.pool.rs;
    }
    rows_at[(j & 1) * kKeys + threadIdx.x] = at;
  };
  auto bring = [&](int j) {
    if (j < part.j1) {
      float* to = sm + Lay::kv + (j & 1) * Lay::stage;
      for (int x = threadIdx.x; x < kKeys * (D / 4); x += 256) {
        const int row = x / (D / 4), c = x % (D / 4) * 4;
        const int64_t at = rows_at[(j & 1) * kKeys + row];
        const int64_t from = at < 0 ? 0 : at + c;
        tc::cp_async16(tc::smem_u32(to + row * Lay::ld + c), static_cast<const float*>(a.pool.k) + from, at < 0 ? 0 : 16);
        tc::cp_async16(tc::smem_u32(to + (kKeys + row) * Lay::ld + c), static_cast<const float*>(a.pool.v) + from,
                       at < 0 ? 0 : 16);
      }
    }
    tc::cp_async_commit();
  };
  look(part.j0);
  for (int x = threadIdx.x; x < kRows * (D / 4); x += 256) {
    const int row = x / (D / 4), c = x % (D / 4) * 4, r = r0 + min(row, rl - r0);
    tc::cp_async16(tc::smem_u32(sq + row * Lay::ld + c),
                   static_cast<const float*>(a.q.p) + (int64_t)(h * G + r % G) * a.q.hs + (int64_t)(s.t0 + r / G) * a.q.ts + c,
                   16);
  }
  __syncthreads();
  bring(part.j0);                                        // with the query rows
  look(part.j0 + 1);
  const float sl2 = fminf(a.scale * 1.4426950408889634f, 3.0e38f);
  const bool idle = (int)(threadIdx.x >> 5) * 4 > rl - r0;         // a warp without rows only brings tiles
  for (int j = part.j0; j < part.j1; ++j) {
    const int key0 = tiles.key(j);
    __syncthreads();                                     // tile j - 1 has been used, and where j + 1's rows lie is known
    bring(j + 1);
    tc::cp_async_wait<1>();
    __syncthreads();
    look(j + 2);
    if (idle) continue;
    const float *sk = sm + Lay::kv + (j & 1) * Lay::stage, *sv = sk + kKeys * Lay::ld;
    float2 x2[2][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x2[0][k] = x2[1][k] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      const float4 q0 = *reinterpret_cast<const float4*>(&sq[2 * ty * Lay::ld + c]);
      const float4 q1 = *reinterpret_cast<const float4*>(&sq[(2 * ty + 1) * Lay::ld + c]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 kv = *reinterpret_cast<const float4*>(&sk[(tx + 16 * k) * Lay::ld + c]);
        fma2(x2[0][k], q0.x, q0.y, kv.x, kv.y);
        fma2(x2[0][k], q0.z, q0.w, kv.z, kv.w);
        fma2(x2[1][k], q1.x, q1.y, kv.x, kv.y);
        fma2(x2[1][k], q1.z, q1.w, kv.z, kv.w);
      }
    }
    float x[2][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[0][k] = x2[0][k].x + x2[0][k].y, x[1][k] = x2[1][k].x + x2[1][k].y;
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
      for (int c = 0; c < D / 32; ++c) o[i][c].x *= f, o[i][c].y *= f;
    }
    __syncwarp();
    const bool whole = tiles.all(key0);
#pragma unroll 2
    for (int k0 = 0; k0 < kKeys; k0 += 4) {
      const float4 p4[2] = {*reinterpret_cast<const float4*>(&sp[2 * ty * Lay::ldp + k0]),
                            *reinterpret_cast<const float4*>(&sp[(2 * ty + 1) * Lay::ldp + k0])};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = k0 + e;
        const float p0 = e == 0 ? p4[0].x : e == 1 ? p4[0].y : e == 2 ? p4[0].z : p4[0].w;
        const float p1 = e == 0 ? p4[1].x : e == 1 ? p4[1].y : e == 2 ? p4[1].z : p4[1].w;
        const bool in0 = whole || (bits[0] >> k & 1), in1 = whole || (bits[1] >> k & 1);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const float4 v = *reinterpret_cast<const float4*>(&sv[k * Lay::ld + tx * 4 + c * 64]);
          if (in0) fma2(o[0][2 * c], p0, p0, v.x, v.y), fma2(o[0][2 * c + 1], p0, p0, v.z, v.w);
          if (in1) fma2(o[1][2 * c], p1, p1, v.x, v.y), fma2(o[1][2 * c + 1], p1, p1, v.z, v.w);
        }
      }
    }
    __syncwarp();
  }
  tc::cp_async_wait<0>();                                // (a block without a tile)
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
    for (int c = 0; c < D / 64; ++c) {
      const int ch = tx * 4 + c * 64;
      const float2 y0 = o[i][2 * c], y1 = o[i][2 * c + 1];
      const float4 y = live ? make_float4(y0.x * f, y0.y * f, y1.x * f, y1.y * f) : make_float4(0.f, 0.f, 0.f, 0.f);
      float* to = partial ? a.part_o + row * D + ch
                          : static_cast<float*>(a.out) + head[i] * a.o_hs + tok[i] * a.o_ts + ch;
      *reinterpret_cast<float4*>(to) = y;
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
