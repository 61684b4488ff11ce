// Softmax attention over a paged cache: the plan (which kernel, how many splits of the keys) and the
// kernel that joins the splits.
//
// The G = Hq / Hkv query heads that share a KV head see the same keys, so the rows of a piece of work
// are (token, head) pairs, r = t * G + g: the cache is read once for the G heads, and neighbouring rows
// see nearly the same keys.  With few rows the keys are cut into splits, a block each, whose
// partials (sum of p v, maximum, sum of p) go to a slot of the workspace in fp32 and are joined by a
// second launch.
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"
#include "paged_attn.h"
#include "paged_tc.cuh"
#include "tmap.h"

namespace fastar {

namespace {

constexpr int kMaxSplits = 256;

// ---- joining the splits ----------------------------------------------------------------------
// O = sum_s e^(m_s - m) o_s / sum_s e^(m_s - m) l_s over a row's partials, m = max_s m_s; one warp a
// row, D / 32 channels a lane.  The partials are summed in the order of the splits, so results do
// not change from run to run.  A split in which the row sees no key has l = 0.  (The tensor-core kernel's
// items are joined in its own file.)
template <typename T, int D, int kTile>
__global__ void __launch_bounds__(128) paged_join_kernel(const PagedAttnArgs a) {
  constexpr int CPL = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);       // (sequence, token, head)
  // Where its partials lie is found while the attention still runs: at and cu come from before that, which has
  // waited for them before it let this launch go.
  const int64_t per = (int64_t)a.max_q * a.Hq;
  const bool in = u < per * a.B;
  const int b = in ? (int)(u / per) : 0;
  const paged::Seq s = paged::sequence(a.cu, a.at, a.B, a.T, a.cap, b, nullptr);
  const int i = in ? (int)((u - b * per) / a.Hq) : 0, head = in ? (int)(u - b * per - (int64_t)i * a.Hq) : 0;
  paged::Work work;
  const bool joins = in && i < s.nq && paged::find_work<kTile>(a, -1, b, work) && work.count > 1;
  // The partials.  Rows without any wait too: a join that ended before the attention would let go what comes next in
  // the stream.
  pdl_wait();
  if (!joins) return;
  const int splits = work.count;
  const int h = head / a.group;
  const int64_t row0 = paged::partial_row(a, work.first, h, i * a.group + head - h * a.group);
  const int64_t step = (int64_t)a.Hkv * a.group * a.max_q;               // from split to split
  constexpr int kPer = kMaxSplits / 32;
  float m = neg_inf(), l = 0.f, o[CPL];
#pragma unroll
  for (int c = 0; c < CPL; ++c) o[c] = 0.f;
  // lane s % 32 reads split s's maximum and sum; then the outputs, eight splits' loads at a time
  float2 ml[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    ml[k] = make_float2(neg_inf(), 0.f);
    if (32 * k + lane < splits) ml[k] = a.part_ml[row0 + (32 * k + lane) * step];
    if (ml[k].y != 0.f) m = fmaxf(m, ml[k].x);
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  const float ref = m == neg_inf() ? 0.f : m;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (32 * k >= splits) break;
    const float w = ml[k].y != 0.f ? expf(ml[k].x - ref) : 0.f;
    const int here = splits - 32 * k < 32 ? splits - 32 * k : 32;
#pragma unroll 1
    for (int s0 = 0; s0 < here; s0 += 8) {
      float p[8][CPL], wt[8], ls[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int src = s0 + x < 32 ? s0 + x : 31;
        ls[x] = __shfl_sync(0xffffffffu, ml[k].y, src);
        wt[x] = __shfl_sync(0xffffffffu, w, src);
        const bool in = s0 + x < here && ls[x] != 0.f;
        const float* src_o = a.part_o + (row0 + (32 * k + s0 + x) * step) * D + lane * CPL;
#pragma unroll
        for (int c = 0; c < CPL; ++c) p[x][c] = in ? src_o[c] : 0.f;
        if (!in) wt[x] = ls[x] = 0.f;
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        l = fmaf(wt[x], ls[x], l);
#pragma unroll
        for (int c = 0; c < CPL; ++c) o[c] = fmaf(wt[x], p[x][c], o[c]);
      }
    }
  }
  const bool live = l > 0.f || l != l;
  T* out = static_cast<T*>(a.out) + head * a.o_hs + (s.t0 + i) * a.o_ts + lane * CPL;
#pragma unroll
  for (int c = 0; c < CPL; ++c) out[c] = from_f<T>(live ? o[c] / l : 0.f);
  if (lane == 0 && a.lse) a.lse[head * a.T + s.t0 + i] = live ? m + logf(l) : neg_inf();
}

template <typename T, int D, int kTile>
cudaError_t join_go(const PagedAttnArgs& a, cudaStream_t s) {
  const int64_t blocks = ((int64_t)a.B * a.max_q * a.Hq + 3) / 4;
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  const cudaError_t e = launch_dependent(paged_join_kernel<T, D, kTile>, dim3((unsigned)blocks), dim3(128), 0, s, a);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

enum Kernel { kF32, kFew, kTensor, kTensorAlone };
struct Plan {
  Kernel kernel;
  int extra, min_tiles, shares;          // see PagedAttnArgs
};

// Slots for few rows: `blocks` blocks in all, each of min_tiles key tiles of `tile` rows or more; none beyond one a
// sequence where they fill the GPU, or where no sequence has three times that many.  With fewer to spare than there are
// sequences, equal ones stay whole and the join is for nothing (3.5 of 30 us: 32 sequences of 1100 rows), so that only twice as
// long ones, whose lengths may differ by more, are worth it.
Plan plan_slots(Kernel kernel, int64_t units, int64_t B, int64_t keys, int64_t blocks, int tile, int min_tiles) {
  int64_t e = blocks / units - B;
  if (B > paged::kDealt || keys < (e < B ? 6 : 3) * (int64_t)tile * min_tiles || e < 0) e = 0;
  if (e > kMaxSplits - 1) e = kMaxSplits - 1;
  return Plan{kernel, (int)e, min_tiles, 0};
}

// Slots of the workspace, and the bytes of one: the rows of a sequence, or of an item (with half of its share's entry
// of what is joined).
int64_t slots_of(const Plan& p, int B) { return p.shares > 0 ? 2 * p.shares : p.extra > 0 ? p.extra + B : 0; }
int64_t slot_rows(const Plan& p, int d, int Hq, int max_q) {
  return p.shares > 0 ? paged_tc_rows(d, p.kernel == kTensorAlone) : (int64_t)max_q * Hq;
}
size_t slot_bytes(const Plan& p, int d, int Hq, int max_q) {
  return (size_t)slot_rows(p, d, Hq, max_q) * (d + 2) * sizeof(float) + (p.shares > 0 ? paged_tc_cut_bytes() / 2 : 0);
}

// keys: that a token sees at most.
Plan make_plan(int dtype, int d, int Hq, int Hkv, int B, int max_q, int64_t keys) {
  const int64_t rows = (int64_t)(Hq / Hkv) * max_q;
  if (dtype == FASTAR_F32) {
    // slots for two blocks a multiprocessor, a tile of 64 keys each or more.  At d = 64 both are resident; at d = 128 a block
    // takes 158 KB of shared memory, one fits, and a call that uses all its slots runs in two waves
    const int64_t units = (rows + kF32Rows - 1) / kF32Rows * Hkv;
    return plan_slots(kF32, units, B, keys, 2 * sm_count(), kF32Keys, 1);
  }
  // two blocks a multiprocessor, all resident: one wave (28 rows over six long sequences take 89 us with two blocks, 110 with
  // three, one and a half waves, 102 with four, two, 123 with eight); eight tiles of 16 keys a warp, or with more than one group of eight rows, where
  // a tile takes a warp 1 us instead of 0.4, four (28 rows over six sequences of 900 rows: 20.5 us with eight, 17.8 with
  // four; one token of 12 heads over 6000 rows: 11.8 and 12.4)
  if (rows <= kFewRows) return plan_slots(kFew, Hkv, B, keys, 2 * sm_count(), 16, (rows <= 8 ? 8 : 4) * kFewWarps);
  // one CTA, or pair of them, a multiprocessor or two
  const bool alone = d == 128 && rows <= 128;
  const int shares = d == 128 && !alone ? sm_count() / 2 : sm_count();
  return Plan{alone ? kTensorAlone : kTensor, 0, 0, shares < paged::kMaxShares ? shares : paged::kMaxShares};
}

}  // namespace

size_t paged_attn_workspace(int d, int Hq, int Hkv, int B, int max_q, int64_t keys) {
  size_t most = 0;
  for (int dt : {FASTAR_F32, FASTAR_BF16}) {
    const Plan p = make_plan(dt, d, Hq, Hkv, B, max_q, keys);
    const size_t n = slots_of(p, B) * slot_bytes(p, d, Hq, max_q);
    most = n > most ? n : most;
  }
  return most;
}

cudaError_t launch_paged_attn(int dtype, int d, PagedAttnArgs a, void* ws, size_t ws_bytes, cudaStream_t s) {
  a.group = a.Hq / a.Hkv;
  int64_t keys = a.cap;
  if (a.window > 0 && (int64_t)a.window + a.sinks < keys) keys = (int64_t)a.window + a.sinks;
  Plan plan = make_plan(dtype, d, a.Hq, a.Hkv, a.B, a.max_q, keys);
  const int64_t fit = ws ? (int64_t)(ws_bytes / slot_bytes(plan, d, a.Hq, a.max_q)) : 0;
  if (plan.extra > fit - a.B) plan.extra = fit > a.B ? (int)(fit - a.B) : 0;
  a.extra = plan.extra;
  a.min_tiles = plan.min_tiles;
  a.shares = plan.shares;
  // (a workspace for fewer shares: no cuts, rather than fewer CTAs)
  const int64_t slots = plan.shares > 0 && fit < 2 * plan.shares ? 0 : slots_of(plan, a.B);
  if (slots > 0) {
    const int64_t rows = slots * slot_rows(plan, d, a.Hq, a.max_q);
    a.part_o = static_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + rows * d);
    a.cuts = a.part_ml + rows;
  }
  if (plan.shares > 0) return launch_paged_attn_tc(d, a, plan.kernel == kTensorAlone, s);
  const cudaError_t e = plan.kernel == kF32 ? launch_paged_attn_f32(d, a, s) : launch_paged_attn_few(d, a, s);
  if (e != cudaSuccess || slots == 0) return e;
  if (plan.kernel == kF32) return d == 128 ? join_go<float, 128, kF32Keys>(a, s) : join_go<float, 64, kF32Keys>(a, s);
  return d == 128 ? join_go<__nv_bfloat16, 128, 16>(a, s) : join_go<__nv_bfloat16, 64, 16>(a, s);
}

}  // namespace fastar
