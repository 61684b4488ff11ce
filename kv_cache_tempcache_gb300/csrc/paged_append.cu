// Tokens into the pages of their sequences, with the norm of every head of q and k and the rotation of
// their positions on the way (qk_rope.cu has the mathematics; rope.cuh what is shared).
//
// Bound: HBM, each element of q, k and v read and written once.  A warp takes a token, or with few
// tokens a part of its heads: D / 16 lanes hold a head's row, 16 channels each; the rows of q, then
// k's, which go to their page, then v's, which are only moved there.  What a token needs besides its
// rows (its sequence, its row, its page) hangs on one another, three loads deep: the first rows of
// the token are on their way while it is found.
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"
#include "rope.cuh"
#include "tmap.h"

namespace fastar {

namespace {

constexpr int kWarpsA = 4;

// The sequence of a token: as many as end at or before it come earlier (cu does not fall).
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int64_t T, uint32_t tok, int lane) {
  if (!cu) return B == 1 ? 0 : (int)(tok / (uint32_t)(T / B));
  int n = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const bool before = b0 + lane < B && cu[b0 + lane + 1] <= (int)tok;
    n += __popc(__ballot_sync(0xffffffffu, before));
  }
  return n;
}

// Inputs and outputs may be the same tensor: every lane reads its channels before it writes
// them and no other lane does.  kAll: every pair turns.
template <typename T, int D, bool kAll, int kAhead>
__global__ void __launch_bounds__(kWarpsA * 32)
    paged_append_kernel(const PagedAppendArgs a, const __grid_constant__ RopeTable tab) {
  pdl_wait();                      // the launch overlaps the end of the kernel before
  __shared__ __align__(16) uint64_t steps[64];
  __shared__ uint8_t axes[64];
  __shared__ __align__(16) float ws[2][D];
  if (threadIdx.x < D / 2) {
    steps[threadIdx.x] = tab.step[threadIdx.x];
    axes[threadIdx.x] = tab.axis[threadIdx.x];
  }
  for (int c = threadIdx.x; c < D; c += kWarpsA * 32) {
    ws[0][c] = a.wq ? a.wq[c] : 1.f;
    ws[1][c] = a.wk ? a.wk[c] : 1.f;
  }
  const int64_t cap = a.max_pages << a.pool.page_shift;
  if (blockIdx.x == 0 && a.len_out) {
    for (int b = threadIdx.x; b < a.B; b += kWarpsA * 32) {
      const paged::Seq s = paged::sequence(a.cu, a.at, a.B, a.T, cap, b, a.status);
      const int64_t n = (int64_t)s.at + s.nq;
      a.len_out[b] = (int)(n < cap ? n : cap);
    }
  }
  constexpr int LPR = D / 16;      // lanes of a row
  constexpr int RW = 32 / LPR;     // rows of a warp side by side
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, li = lane % LPR;
  const uint32_t parts = 1u << a.part_shift;
  const int64_t items = a.T << a.part_shift;
  const int64_t stride = (int64_t)gridDim.x * kWarpsA;
  // groups of rows side by side: of q, then of k, then of v
  const int gq = a.qo ? (a.Hq + RW - 1) / RW : 0, gk = (a.Hk + RW - 1) / RW, groups = gq + 2 * gk;
  __syncthreads();
  for (int64_t u = (int64_t)blockIdx.x * kWarpsA + (threadIdx.x >> 5); u < items; u += stride) {
    const uint32_t tok = (uint32_t)(u >> a.part_shift), part = (uint32_t)u & (parts - 1);   // T fits 31 bits
    Raw<T> v[kAhead];
    auto load = [&](Raw<T>& r, int x) {
      const int side = x < gq ? 0 : x < gq + gk ? 1 : 2;
      const int h = (x - (side == 0 ? 0 : side == 1 ? gq : gq + gk)) * RW + sub;
      const bool in = x < groups && h < (side == 0 ? a.Hq : a.Hk);
      const TokView& t = side == 0 ? a.q : side == 1 ? a.k : a.v;
      const T* p = static_cast<const T*>(t.p) + h * t.hs + (int64_t)tok * t.ts;
#pragma unroll
      for (int i = 0; i < (int)sizeof(T); ++i)
        r.u[i] = in ? reinterpret_cast<const uint4*>(p + li * 16)[i] : make_uint4(0, 0, 0, 0);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(v[i], (int)(part + i * parts));
    // the token's sequence and row; tokens of none are left as they are
    const int b = sequence_of(a.cu, a.B, a.T, tok, lane);
    if (b >= a.B) continue;
    const paged::Seq s = paged::sequence(a.cu, a.at, a.B, a.T, cap, b, a.status);
    const int i = (int)tok - s.t0;
    if (i < 0 || i >= s.nq) continue;
    const int64_t row = (int64_t)s.at + i;
    // where the row goes; -1: nowhere
    int64_t dst = -1;
    if (row < cap) {
      const int page = paged::page_of(a.table + (int64_t)b * a.max_pages, (int)(row >> a.pool.page_shift), a.pool.pages,
                                      a.status);
      if (page >= 0) dst = page * a.pool.ps + (row & ((1 << a.pool.page_shift) - 1)) * a.pool.rs;
    } else {
      flag_status(a.status, FASTAR_DEV_BAD_LEN);
    }
    // the token's rotations: lane l forms those of pairs 2 l and 2 l + 1 (d = 64: l and no other)
    int p3[3];
    if (a.pos) {
#pragma unroll
      for (int e = 0; e < 3; ++e) p3[e] = a.pos[(int64_t)tok * 3 + e];
    } else {
      const uint32_t line = (uint32_t)row / (uint32_t)a.gw, fr = line / (uint32_t)a.gh;
      p3[0] = (int)fr;
      p3[1] = (int)(line - fr * (uint32_t)a.gh);
      p3[2] = (int)((uint32_t)row - line * (uint32_t)a.gw);
    }
    float sn0 = 0.f, cs0 = 1.f, sn1 = 0.f, cs1 = 1.f;
    auto one = [&](int j, float& sn, float& cs) {
      const int ax = axes[j];
      rope_turn(ax == 0 ? p3[0] : ax == 1 ? p3[1] : p3[2], steps[j], sn, cs);
    };
    if (D == 128) {
      one(2 * lane, sn0, cs0);
      one(2 * lane + 1, sn1, cs1);
    } else {
      one(lane, sn0, cs0);
    }
    float A[8], B[8], C[8], E[8];
    bool norm = false;
    int side = -1;
#pragma unroll 1
    for (int x0 = (int)part; x0 < groups; x0 += kAhead * (int)parts) {
#pragma unroll
      for (int n = 0; n < kAhead; ++n) {
        const int x = x0 + n * (int)parts;
        if (x >= groups) break;
        const int of = x < gq ? 0 : x < gq + gk ? 1 : 2;
        if (of == 2) {                       // v: as it is
          const int h = (x - gq - gk) * RW + sub;
          const Raw<T> r = v[n];
          if (kAhead > 1) load(v[n], x + kAhead * (int)parts);
          if (h < a.Hk && dst >= 0) {
            uint4* p = reinterpret_cast<uint4*>(static_cast<T*>(a.pool.v) + dst + h * a.pool.hs + li * 16);
#pragma unroll
            for (int e = 0; e < (int)sizeof(T); ++e) p[e] = r.u[e];
          }
          continue;
        }
        if (side != of) {                    // once for q, once for k: rotations times weights
          side = of;
          norm = of ? a.wk != nullptr : a.wq != nullptr;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int src = D == 128 ? li * 4 + (e >> 1) : li * 8 + e;
            const float sn = __shfl_sync(0xffffffffu, D == 128 && (e & 1) ? sn1 : sn0, src);
            const float cs = __shfl_sync(0xffffffffu, D == 128 && (e & 1) ? cs1 : cs0, src);
            const float2 w2 = reinterpret_cast<const float2*>(&ws[of][li * 16])[e];
            A[e] = cs * w2.x, B[e] = sn * w2.y, C[e] = sn * w2.x, E[e] = cs * w2.y;
          }
        }
        float f[16];
        expand(v[n], f);
        if (kAhead > 1) load(v[n], x + kAhead * (int)parts);
        const float r = norm ? rms_scale<D>(f, a.eps) : 1.f;
        turn16<kAll>(f, A, B, C, E, r, axes + li * 8);
        const int h = (of ? x - gq : x) * RW + sub;
        if (h < (of ? a.Hk : a.Hq) && (of == 0 || dst >= 0)) {
          T* p = (of ? static_cast<T*>(a.pool.k) + dst + h * a.pool.hs
                     : static_cast<T*>(a.qo) + h * a.qo_hs + (int64_t)tok * a.qo_ts) + li * 16;
          store8(p, f);
          store8(p + 8, f + 8);
        }
      }
    }
  }
}

template <typename T, int D>
cudaError_t append_go(PagedAppendArgs a, const RopeTable& tab, bool all, cudaStream_t s) {
  // a warp a token, or while that leaves warp schedulers with few warps, several, down to a warp
  // for each group of rows side by side
  constexpr int RW = 32 / (D / 16);
  const int groups = (a.qo ? (a.Hq + RW - 1) / RW : 0) + 2 * ((a.Hk + RW - 1) / RW);
  const int64_t sms = sm_count();
  a.part_shift = 0;
  while ((1 << a.part_shift) < groups && (a.T << a.part_shift) < 16 * sms) ++a.part_shift;
  int64_t blocks = ((a.T << a.part_shift) + kWarpsA - 1) / kWarpsA;
  if (blocks < 1) blocks = 1;                // lengths alone
  // one group a warp: as many warps as there are groups, with few registers; else four resident
  // blocks a multiprocessor, which go on to their next tokens
  const bool one = (1 << a.part_shift) >= groups;
  const int64_t most = one ? 0x7fffffff : 4 * sms;
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  constexpr int kAhead = sizeof(T) == 2 ? 3 : 2;
  const auto kernel = one ? all ? paged_append_kernel<T, D, true, 1> : paged_append_kernel<T, D, false, 1>
                      : all ? paged_append_kernel<T, D, true, kAhead>
                            : paged_append_kernel<T, D, false, kAhead>;
  const cudaError_t e = launch_dependent(kernel, dim3(grid), dim3(kWarpsA * 32), 0, s, a, tab);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(int dtype, int d, PagedAppendArgs a, const int* axes, float theta, cudaStream_t s) {
  bool all;
  const RopeTable tab = rope_table(d, axes, theta, &all);
  if (dtype == FASTAR_BF16)
    return d == 128 ? append_go<__nv_bfloat16, 128>(a, tab, all, s) : append_go<__nv_bfloat16, 64>(a, tab, all, s);
  return d == 128 ? append_go<float, 128>(a, tab, all, s) : append_go<float, 64>(a, tab, all, s);
}

}  // namespace fastar
