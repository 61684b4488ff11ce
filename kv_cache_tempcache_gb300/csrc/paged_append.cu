// Tokens into the pages of their sequences, with the norm of every head of q and k and the rotation of
// their positions on the way (qk_rope.cu has the mathematics; rope.cuh what is shared).
//
// Bound: HBM, each element of q, k and v read and written once.  A warp takes tokens, or with few
// tokens a part of one's heads: D / 16 lanes hold a head's row, 16 channels each; the rows of q, then
// k's, which go to their page, then v's, which are only moved there.  A lane's channels are chunks of 16 bytes, a
// row's lanes side by side in each (with 32 consecutive bytes a lane every load took two half sectors).  Rows come through shared memory by
// cp.async, kSlots groups of them on their way a warp, across the borders of tokens (held in registers, three
// groups a warp and none on their way between two tokens, 4680 tokens of 36 heads took 0.7 us longer); more slots or
// blocks change nothing.  Each lane reads back what it asked for itself, so no barrier is needed.
// Many tokens go to blocks that end, of a few neighbouring tokens each: the multiprocessors do not read and write equally
// fast, and blocks that stay and take an equal share of the tokens wait for the slowest (14,400 tokens of 72 heads 93.5
// us; now 81.1).  Measured, each call on inputs that are not in L2: 4680 tokens of 36 heads 17.5 us (4.9 TB/s; 15.7 where the
// inputs are there), 14,400 of 72 heads 81.1 (6.5 TB/s, 0.96 of the measured copy rate); 100,000 tokens of 6 heads 121 (2.5
// TB/s: where a side has fewer heads than a warp has rows side by side, 4 at d = 128 and 8 at d = 64, lanes idle, and a token's
// sequence, page and sines are found one after the other between two tokens; what each costs is not measured).
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"
#include "rope.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace fastar {

namespace {

constexpr int kWarpsA = 4, kSlots = 4, kBlocks = 5;   // warps of a block, groups of rows on their way, blocks an SM
constexpr int kGroups = 8;               // of rows that a warp of a block that ends has at least

// 16 bytes of a row.
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float* f) { store8(p, f); }
__device__ __forceinline__ void store16(float* p, const float* f) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}

// The sequence of a token: as many as end at or before it come earlier (cu does not fall).  A warp looks at 32 of them
// at a time, spread over what is left.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int64_t T, uint32_t tok, int lane) {
  if (!cu) return B == 1 ? 0 : (int)(tok / (uint32_t)(T / B));
  int lo = 0, hi = B;                        // it is one of lo .. hi (hi: behind the last)
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const int n = __popc(__ballot_sync(0xffffffffu, i < hi && cu[i + 1] <= (int)tok));
    if (n == 0) return lo;
    hi = min(hi, lo + n * step);             // those probes' sequences end before the token, the next one's does not
    lo += (n - 1) * step + 1;
  }
  return lo + __popc(__ballot_sync(0xffffffffu, lo + lane < hi && cu[lo + lane + 1] <= (int)tok));
}

// Inputs and outputs may be the same tensor: every lane reads its channels before it writes
// them and no other lane does.  kAll: every pair turns.
template <typename T, int D, bool kAll>
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
  bool lost = false;               // cu makes no sense: whose tokens are whose is not known
  if (blockIdx.x == 0 && (a.len_out || a.status)) {
    for (int b = threadIdx.x; b < a.B; b += kWarpsA * 32) {
      const paged::Seq s = paged::sequence(a.cu, a.at, a.B, a.T, cap, b, a.status);
      const int64_t n = (int64_t)s.at + s.nq;
      if (!a.len_out) continue;
      a.len_out[b] = (int)(n < cap ? n : cap);
      if (a.cu) lost |= a.cu[b] < 0 || a.cu[b + 1] < a.cu[b] || a.cu[b + 1] > a.T;
    }
  }
  constexpr int LPR = D / 16;      // lanes of a row
  constexpr int RW = 32 / LPR;     // rows of a warp side by side
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, li = lane % LPR;
  const uint32_t parts = 1u << a.part_shift;
  // a block's items: `per` of each warp side by side, or (0) every grid's width of warps
  const int64_t u0 = (int64_t)blockIdx.x * (kWarpsA * max(a.per, 1)) + (threadIdx.x >> 5), all = a.T << a.part_shift;
  const int64_t stride = a.per ? kWarpsA : (int64_t)gridDim.x * kWarpsA;
  const int64_t items = a.per ? min(all, (int64_t)(blockIdx.x + 1) * (kWarpsA * a.per)) : all;
  // groups of rows side by side: of q, then of k, then of v
  const int gq = a.qo ? (a.Hq + RW - 1) / RW : 0, gk = (a.Hk + RW - 1) / RW, groups = gq + 2 * gk;
  // group lx of item lu is the next to be asked for, into slot `to`; 32 sizeof(T) / 2 bytes a lane
  constexpr int NC = sizeof(T), EPC = 16 / NC;   // 16-byte chunks of a lane, channels of a chunk
  extern __shared__ __align__(16) uint8_t ring[];
  uint8_t* mine = ring + (threadIdx.x >> 5) * (kSlots * NC * 512) + lane * 16;
  int64_t lu = u0;
  int lx = (int)((uint32_t)u0 & (parts - 1)), to = 0, from = 0;
  auto skip = [&]() {                      // (parts beyond the groups have none)
    while (lx >= groups && lu < items) {
      lu += stride;
      lx = (int)((uint32_t)lu & (parts - 1));
    }
  };
  skip();
  auto ask = [&]() {
    if (lu < items) {
      const int side = lx < gq ? 0 : lx < gq + gk ? 1 : 2;
      const int h = (lx - (side == 0 ? 0 : side == 1 ? gq : gq + gk)) * RW + sub;
      if (h < (side == 0 ? a.Hq : a.Hk)) {
        const TokView& t = side == 0 ? a.q : side == 1 ? a.k : a.v;
        const T* p = static_cast<const T*>(t.p) + h * t.hs + (lu >> a.part_shift) * t.ts + li * EPC;
#pragma unroll
        for (int i = 0; i < NC; ++i) tc::cp_async16(tc::smem_u32(mine + (to * NC + i) * 512), p + i * (D / NC), 16);
      }
      lx += (int)parts;
      skip();
    }
    tc::cp_async_commit();
    to = to + 1 == kSlots ? 0 : to + 1;
  };
#pragma unroll 1
  for (int i = 0; i < kSlots - 1; ++i) ask();
  // the tables are there; after the first rows are on their way
  if (__builtin_expect(__syncthreads_or(lost), 0)) {
    // no sequence gets longer (a token is looked for as if cu did not fall, so that any may miss rows)
    for (int b = threadIdx.x; b < a.B; b += kWarpsA * 32) {
      const int n = a.at[b];
      a.len_out[b] = n >= 0 && n <= cap ? n : 0;
    }
  }
  uint32_t turns = 0;                      // of this lane's pairs
#pragma unroll
  for (int e = 0; e < 8; ++e)
    turns |= (uint32_t)(axes[(2 * e / EPC * (D / NC) + li * EPC + 2 * e % EPC) / 2] < 3) << e;
#pragma unroll 1
  for (int64_t u = u0; u < items; u += stride) {
    const uint32_t tok = (uint32_t)(u >> a.part_shift), part = (uint32_t)u & (parts - 1);   // T fits 31 bits
    // the token's sequence and row; tokens of none are left as they are
    const int b = sequence_of(a.cu, a.B, a.T, tok, lane);
    const paged::Seq s = b < a.B ? paged::sequence(a.cu, a.at, a.B, a.T, cap, b, a.status) : paged::Seq{0, 0, 0};
    const int i = (int)tok - s.t0;
    const bool known = i >= 0 && i < s.nq;
    const int64_t row = (int64_t)s.at + i;
    // where the row goes; -1: nowhere
    int64_t dst = -1;
    if (known && row < cap) {
      const int page = paged::page_of(a.table + (int64_t)b * a.max_pages, (int)(row >> a.pool.page_shift), a.pool.pages,
                                      a.status);
      if (page >= 0) dst = page * a.pool.ps + (row & ((1 << a.pool.page_shift) - 1)) * a.pool.rs;
    } else if (known) {
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
    for (int x = (int)part; x < groups; x += (int)parts) {
      ask();
      tc::cp_async_wait<kSlots - 1>();
      Raw<T> v;
#pragma unroll
      for (int e = 0; e < NC; ++e) v.u[e] = *reinterpret_cast<const uint4*>(mine + (from * NC + e) * 512);
      from = from + 1 == kSlots ? 0 : from + 1;
      if (!known) continue;
      const int of = x < gq ? 0 : x < gq + gk ? 1 : 2;
      if (of == 2) {                         // v: as it is
        const int h = (x - gq - gk) * RW + sub;
        if (h < a.Hk && dst >= 0) {
          T* p = static_cast<T*>(a.pool.v) + dst + h * a.pool.hs + li * EPC;
#pragma unroll
          for (int e = 0; e < NC; ++e) *reinterpret_cast<uint4*>(p + e * (D / NC)) = v.u[e];
        }
        continue;
      }
      if (side != of) {                      // once for q, once for k: rotations times weights
        side = of;
        norm = of ? a.wk != nullptr : a.wq != nullptr;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = 2 * e / EPC * (D / NC) + li * EPC + 2 * e % EPC;         // the pair's first channel
          const float sn = __shfl_sync(0xffffffffu, D == 128 && (e & 1) ? sn1 : sn0, c / (D / 32));
          const float cs = __shfl_sync(0xffffffffu, D == 128 && (e & 1) ? cs1 : cs0, c / (D / 32));
          const float2 w2 = *reinterpret_cast<const float2*>(&ws[of][c]);
          A[e] = cs * w2.x, B[e] = sn * w2.y, C[e] = sn * w2.x, E[e] = cs * w2.y;
        }
      }
      float f[16];
      expand(v, f);
      const float r = norm ? rms_scale<D>(f, a.eps) : 1.f;
      turn16<kAll>(f, A, B, C, E, r, turns);
      const int h = (of ? x - gq : x) * RW + sub;
      if (h < (of ? a.Hk : a.Hq) && (of == 0 || dst >= 0)) {
        T* p = (of ? static_cast<T*>(a.pool.k) + dst + h * a.pool.hs
                   : static_cast<T*>(a.qo) + h * a.qo_hs + (int64_t)tok * a.qo_ts) + li * EPC;
#pragma unroll
        for (int e = 0; e < NC; ++e) store16(p + e * (D / NC), f + e * EPC);
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
  constexpr int bytes = kWarpsA * kSlots * 512 * (int)sizeof(T);
  int64_t most = INT_MAX;
  a.per = 0;
  if (blocks >= kBlocks * sms * 9 / 4) {
    // blocks that end, from two and a quarter times as many as are resident (9360 tokens of 36 heads, 3.1 times: 32.4 us
    // instead of 31.8, in fp32 55.3 instead of 59.9; 7200 of 72, 2.4 times: 44.0 instead of 44.4; 3600 of 72, 1.2 times: 27.3
    // instead of 23.6); where tokens have few rows a warp takes several, so that a block's start weighs less (100,000 tokens
    // of 6 rows: 147 us with a token each, 122 with kGroups 8, 116 with 32, but then 30,000 of 12 take 57 instead of 49)
    const int here = (groups + (1 << a.part_shift) - 1) >> a.part_shift;
    a.per = here < kGroups ? (kGroups + here - 1) / here : 1;
    blocks = (blocks + a.per - 1) / a.per;
  } else {
    // resident blocks, which go on to their next tokens: of 3 to kBlocks a multiprocessor the number that leaves
    // their last round fullest (4680 tokens are 1.54 rounds of 5 blocks each and 1.92 of 4: 18.2 and 17.6 us)
    int64_t best = 0;
    for (int n = kBlocks; n >= 3; --n) {
      const int64_t rounds = (blocks + n * sms - 1) / (n * sms), fill = (blocks << 10) / (rounds * n * sms);
      if (fill > best) best = fill, most = n * sms;
    }
  }
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  const auto kernel = all ? paged_append_kernel<T, D, true> : paged_append_kernel<T, D, false>;
  cudaError_t e = opt_in_smem((const void*)kernel, bytes);
  if (e != cudaSuccess) return e;
  e = launch_dependent(kernel, dim3(grid), dim3(kWarpsA * 32), bytes, s, a, tab);
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
