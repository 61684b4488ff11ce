// Softmax attention over the 4-bit cache for few rows: up to 16 (query head, token) pairs of a KV
// head, as in single-token steps.
//
// Bound: the cache's bytes.  A row tile of the tcgen05 kernel is 128 or 256 rows, so with a few
// rows it spends most of its time unpacking for products that are nearly empty; here the 16
// rows are one m16n8k16 product (mma.sync: its rate is not what bounds this), and the unpacked
// codes go from registers straight into the product's operand, without shared memory between.
//   S[16 rows, 8 keys] += Q[16, 16 channels] K^T,   O[16, 8 channels] += P[16, 16 keys] V
// A product may sum its channels in any order as long as both operands agree, so lane t of a
// quad takes channels t d/4 .. (t + 1) d/4 of a key: 16 consecutive bytes of codes at d = 128.
// The columns of P V may be any channels: lane group g takes d/8 consecutive ones; the pairs
// of keys that the operand wants side by side are made from two rows by byte permutes.
// Each warp runs alone over every eighth block of 64 keys of its CTA's range: three blocks on
// their way by bulk copies, its own reference, sums and outputs; the eight warps' results are
// joined in shared memory, in warp order, at the end, and the CTAs' by the join kernel.
// Queries, P and references as in the tcgen05 kernel (kv4_attn_tc.cu): fp16 rows at a power of
// two, P in fp16 against a reference that moves only when a P would pass 2^15.
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace fastar {

namespace {

constexpr int kWarpsW = 8, kKeysW = 64, kStagesW = 3;

template <int D>
struct FewLayout {
  static constexpr int codes = kKeysW * D / 2, scales = kKeysW * D / 16;
  static constexpr int stage = 2 * (codes + scales);                 // K codes, V codes, K scales, V scales
  static constexpr int ring = kWarpsW * kStagesW * stage;
  static constexpr int red = kWarpsW * 16 * D * 4;                   // the joined outputs, over the ring
  static constexpr int ctl = ring > red ? ring : red;
  static constexpr int bytes = ctl + kWarpsW * kStagesW * 8 + kWarpsW * 16 * 8 + 16 + 128;
};

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2w(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16w(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return max(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_maxf(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// A thread's share of two query rows (channels t D/4 ..) as product operands: a[s] of step s;
// returns each row's logit scale in log2 units.
template <int D>
__device__ __forceinline__ void load_q(const Kv4AttnArgs& a, int h, int rows, int g, int t, uint32_t (*qa)[4], float* sl2) {
  constexpr int CH = D / 4;                 // channels of this thread
  const float ks = kv4::pow2i(kv4::head_exp(a.k_exp, h));
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int r = g + 8 * p;
    uint32_t x[CH / 2];
    uint32_t big = 0;
    if (r < rows) {
      const uint32_t nq = (uint32_t)a.nq, gh = (uint32_t)r / nq;
      const int64_t head = h * (int64_t)(a.Hq / a.Hkv) + gh;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q.p) + head * a.q.hs +
                                                        (int64_t)((uint32_t)r - gh * nq) * a.q.ts + t * CH);
#pragma unroll
      for (int i = 0; i < CH / 8; ++i) {
        const uint4 u = src[i];
        x[4 * i] = u.x, x[4 * i + 1] = u.y, x[4 * i + 2] = u.z, x[4 * i + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < CH / 2; ++i) x[i] = 0;
    }
#pragma unroll
    for (int i = 0; i < CH / 2; ++i) big = max(big, max(x[i] & 0x7fffu, (x[i] >> 16) & 0x7fffu));
    big = quad_max(big);
    const int ex = (int)(big >> 7);
    int qe = ex == 0 ? -126 - 12 : ex - 127 - 12;
    if (qe < -120) qe = -120;
    if (big == 0 || ex == 255) qe = 0;
    const float down = kv4::pow2i(-qe);
    sl2[p] = fmaxf(a.scale * kv4::pow2i(qe) * ks * 1.4426950408889634f, 1.2e-38f);
#pragma unroll
    for (int i = 0; i < CH / 2; ++i)        // pair i of the thread's channels: step i / 2, first or second pair
      qa[i >> 1][p + 2 * (i & 1)] = pack_f16w(__uint_as_float(x[i] << 16) * down, __uint_as_float(x[i] & 0xffff0000u) * down);
  }
}

// kTwo: more than 8 rows (else the product's upper 8 rows are empty and skipped).
template <int D, bool kTwo>
__global__ void __launch_bounds__(kWarpsW * 32, 1) kv4_attn_few_kernel(const Kv4AttnArgs a) {
  using Lay = FewLayout<D>;
  constexpr int NT = D / 8;                 // column tiles of O
  constexpr int RH = kTwo ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~(uintptr_t)127);
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + Lay::ctl);
  float2* wml = reinterpret_cast<float2*>(bars + kWarpsW * kStagesW);      // [warp][16]
  int* abort_flag = reinterpret_cast<int*>(wml + kWarpsW * 16);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int split = (int)(blockIdx.x % (uint32_t)a.splits), h = (int)(blockIdx.x / (uint32_t)a.splits);
  const int rows = (a.Hq / a.Hkv) * (int)a.nq;
  const int64_t len = kv4::head_len(a.len, h, a.cap, a.status);
  // the last key any row sees: with blocks, that of the last token, which some row is; that is len
  const uint32_t blocks = (uint32_t)((len + kKeysW - 1) / kKeysW);
  const uint32_t b0 = (uint32_t)((uint64_t)blocks * split / (uint32_t)a.splits);
  const uint32_t b1 = (uint32_t)((uint64_t)blocks * (split + 1) / (uint32_t)a.splits);
  const int count = b0 + warp < b1 ? (int)((b1 - b0 - warp + kWarpsW - 1) / kWarpsW) : 0;   // this warp's blocks
  pdl_trigger();                            // the join's CTAs may come and wait

  uint64_t* full = bars + warp * kStagesW;
  if (lane == 0) {
    for (int i = 0; i < kStagesW; ++i) tc::mbar_init(&full[i], 1);
    if (warp == 0) *abort_flag = 0;
    tc::mbar_fence_init();
  }
  uint8_t* ring = base + warp * kStagesW * Lay::stage;
  // one lane brings block i of the warp: whole 16-row groups, which lie within the head's rows
  auto fetch = [&](int i) {
    const int64_t key = (int64_t)(b0 + warp + (uint32_t)i * kWarpsW) * kKeysW;
    const int64_t left = (len - key + 15) & ~(int64_t)15;
    const uint32_t nr = left < kKeysW ? (uint32_t)left : kKeysW;
    const int64_t at = (int64_t)h * a.cap + key;
    uint8_t* dst = ring + (i % kStagesW) * Lay::stage;
    uint64_t* bar = &full[i % kStagesW];
    tc::mbar_arrive_tx(bar, 2 * nr * (D / 2 + D / 16));
    tc::bulk_load(dst, a.kc + at * (D / 2), nr * (D / 2), bar);
    tc::bulk_load(dst + 2 * Lay::codes, a.ks + at * (D / 16), nr * (D / 16), bar);
    tc::bulk_load(dst + Lay::codes, a.vc + at * (D / 2), nr * (D / 2), bar);
    tc::bulk_load(dst + 2 * Lay::codes + Lay::scales, a.vs + at * (D / 16), nr * (D / 16), bar);
  };
  if (lane == 0)
    for (int i = 0; i < kStagesW && i < count; ++i) fetch(i);
  __syncthreads();                          // the barriers and the flag are set for every lane

  uint32_t qa[D / 16][4];
  float sl2[2];
  load_q<D>(a, h, rows, g, t, qa, sl2);
  int64_t see[2];                           // how many keys the thread's two rows see
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const uint32_t r = (uint32_t)(g + 8 * p), nq = (uint32_t)a.nq;
    see[p] = (int)r < rows ? kv4::visible(len, a.nq, r % nq, a.block) : len;
  }
  float m[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};
  float o[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  volatile int* abort = abort_flag;

#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    const int64_t key = (int64_t)(b0 + warp + (uint32_t)i * kWarpsW) * kKeysW;
    const uint8_t* st = ring + (i % kStagesW) * Lay::stage;
    if (!__all_sync(0xffffffffu, tc::mbar_wait(&full[i % kStagesW], (i / kStagesW) & 1, abort))) break;
    const int nk = len - key < kKeysW ? (int)(len - key) : kKeysW;
    // ---- S = Q K^T: a lane's share of key g of 8; two times 8 keys side by side and two sums
    // each, so that four products are in flight ----
    float s[8][4];
#pragma unroll
    for (int n = 0; n < 8; n += 2) {
      uint32_t b[2][D / 8];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int k = (n + e) * 8 + g;
        if (D == 128) {
          const uint4 c = reinterpret_cast<const uint4*>(st)[k * 4 + t];
          uint32_t sc = reinterpret_cast<const uint16_t*>(st + 2 * Lay::codes)[k * 4 + t];
          if (k >= nk) sc = 0;             // rows behind the length count as 0, whatever lies there
          const uint32_t s0 = kv4::scale_f16x2(sc), s1 = kv4::scale_f16x2(sc >> 8);
          kv4::unpack8(c.x, s0, b[e]);
          kv4::unpack8(c.y, s0, b[e] + 4);
          kv4::unpack8(c.z, s1, b[e] + 8 % (D / 8));
          kv4::unpack8(c.w, s1, b[e] + 12 % (D / 8));
        } else {
          const uint2 c = reinterpret_cast<const uint2*>(st)[k * 4 + t];
          uint32_t sc = (st + 2 * Lay::codes)[k * 4 + t];
          if (k >= nk) sc = 0;
          const uint32_t s0 = kv4::scale_f16x2(sc);
          kv4::unpack8(c.x, s0, b[e]);
          kv4::unpack8(c.y, s0, b[e] + 4);
        }
      }
      float u[2][2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int x = 0; x < 4; ++x) u[e][0][x] = u[e][1][x] = 0.f;
#pragma unroll
      for (int q = 0; q < D / 16; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e) mma16816(u[e][q & 1], qa[q], b[e][2 * q], b[e][2 * q + 1]);
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[n + e][x] = u[e][0][x] + u[e][1][x];
    }
    // ---- masks, reference, P ----
    if (see[0] - key < kKeysW || see[1] - key < kKeysW) {
#pragma unroll
      for (int p = 0; p < RH; ++p) {
        const int valid = see[p] - key < kKeysW ? (int)(see[p] - key) : kKeysW;
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (n * 8 + 2 * t + e >= valid) s[n][2 * p + e] = neg_inf();
      }
    }
    __syncwarp();
    float mt[2] = {neg_inf(), neg_inf()};
#pragma unroll
    for (int p = 0; p < RH; ++p) {
#pragma unroll
      for (int n = 0; n < 8; ++n) mt[p] = fmaxf(mt[p], fmaxf(s[n][2 * p], s[n][2 * p + 1]));
      mt[p] *= sl2[p];
    }
    if (__any_sync(0xffffffffu, i == 0 || mt[0] > m[0] + 15.f || (kTwo && mt[1] > m[1] + 15.f))) {
#pragma unroll
      for (int p = 0; p < RH; ++p) {
        const float mx = quad_maxf(mt[p]);
        float f = 1.f;
        if (i == 0) {
          m[p] = mx == neg_inf() ? 0.f : mx;
        } else if (mx > m[p]) {
          f = ex2w(m[p] - mx);
          m[p] = mx;
        }
        l[p] *= f;
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][2 * p] *= f, o[n][2 * p + 1] *= f;
      }
    }
    uint32_t pa[4][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        if (p < RH) {
          const float e0 = ex2w(fmaf(s[n][2 * p], sl2[p], -m[p])), e1 = ex2w(fmaf(s[n][2 * p + 1], sl2[p], -m[p]));
          l[p] += e0 + e1;
          pa[n >> 1][p + 2 * (n & 1)] = pack_f16w(e0, e1);
        } else {
          pa[n >> 1][p + 2 * (n & 1)] = 0u;
        }
      }
    // ---- O += P V: 16 keys at a time; a lane's keys 2t, 2t + 1, 2t + 8, 2t + 9, channels g D/8 .. ----
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t v[4][NT / 2];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = q * 16 + 2 * t + (e & 1) + 8 * (e >> 1);
        uint32_t sc = (st + 2 * Lay::codes + Lay::scales)[D == 128 ? k * 8 + g : k * 4 + (g >> 1)];
        if (k >= nk) sc = 0;
        const uint32_t s0 = kv4::scale_f16x2(sc);
        if (D == 128) {
          const uint2 c = reinterpret_cast<const uint2*>(st + Lay::codes)[k * 8 + g];
          kv4::unpack8(c.x, s0, v[e]);
          kv4::unpack8(c.y, s0, v[e] + NT / 4);
        } else {
          kv4::unpack8(reinterpret_cast<const uint32_t*>(st + Lay::codes)[k * 8 + g], s0, v[e]);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        mma16816(o[n], pa[q], __byte_perm(v[0][n >> 1], v[1][n >> 1], 0x5410),
                 __byte_perm(v[2][n >> 1], v[3][n >> 1], 0x5410));
        mma16816(o[n + 1], pa[q], __byte_perm(v[0][n >> 1], v[1][n >> 1], 0x7632),
                 __byte_perm(v[2][n >> 1], v[3][n >> 1], 0x7632));
      }
    }
    __syncwarp();                           // every lane has read the block
    if (lane == 0 && i + kStagesW < count) fetch(i + kStagesW);
  }

  // ---- the eight warps' results, in warp order ----
#pragma unroll
  for (int p = 0; p < RH; ++p) {
    l[p] = quad_sum(l[p]);
    if (t == 0) wml[warp * 16 + g + 8 * p] = make_float2(m[p], l[p]);
  }
  __syncthreads();
  float* red = reinterpret_cast<float*>(base);          // the ring has been used: [warp][16][D]
#pragma unroll
  for (int p = 0; p < RH; ++p) {
    const int r = g + 8 * p;
    float mx = neg_inf();
#pragma unroll
    for (int w = 0; w < kWarpsW; ++w) {
      const float2 x = wml[w * 16 + r];
      if (x.y != 0.f) mx = fmaxf(mx, x.x);
    }
    const float f = l[p] != 0.f ? ex2w(m[p] - mx) : 0.f;
    if (r < rows) {
      // a thread's columns of tile n: channels 2t D/8 + n and (2t + 1) D/8 + n
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float4* dst = reinterpret_cast<float4*>(red + (warp * 16 + r) * D + (2 * t + e) * (D / 8));
#pragma unroll
        for (int n = 0; n < NT; n += 4)
          dst[n >> 2] = make_float4(o[n][2 * p + e] * f, o[n + 1][2 * p + e] * f, o[n + 2][2 * p + e] * f,
                                    o[n + 3][2 * p + e] * f);
      }
    }
  }
  __syncthreads();
  const float up = kv4::pow2i(kv4::head_exp(a.v_exp, h));
  for (int x = threadIdx.x; x < rows * (D / 4); x += kWarpsW * 32) {
    const int r = x / (D / 4), c = x % (D / 4) * 4;
    float mx = neg_inf(), sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarpsW; ++w) {
      const float2 y = wml[w * 16 + r];
      if (y.y != 0.f) mx = fmaxf(mx, y.x);
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarpsW; ++w) {
      const float2 y = wml[w * 16 + r];
      if (y.y == 0.f) continue;             // no key of that warp's that the row sees
      sum += y.y * ex2w(y.x - mx);
      const float4 z = *reinterpret_cast<const float4*>(red + (w * 16 + r) * D + c);
      acc.x += z.x, acc.y += z.y, acc.z += z.z, acc.w += z.w;
    }
    const bool live = sum > 0.f || sum != sum;
    const uint32_t nq = (uint32_t)a.nq, gh = (uint32_t)r / nq;
    const int64_t head = h * (int64_t)(a.Hq / a.Hkv) + gh, tok = (uint32_t)r - gh * nq;
    const float mn = mx * 0.6931471805599453f;
    if (a.splits > 1) {
      const int64_t at = (split * (int64_t)a.Hq + head) * a.nq + tok;
      *reinterpret_cast<float4*>(a.part_o + at * D + c) = make_float4(acc.x * up, acc.y * up, acc.z * up, acc.w * up);
      if (c == 0) a.part_ml[at] = make_float2(live ? mn : neg_inf(), sum);
    } else {
      const float f = live ? up / sum : 0.f;
      __nv_bfloat162 v[2] = {__floats2bfloat162_rn(acc.x * f, acc.y * f), __floats2bfloat162_rn(acc.z * f, acc.w * f)};
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + head * a.o_hs + tok * a.o_ts + c) =
          *reinterpret_cast<uint2*>(v);
      if (c == 0 && a.lse) a.lse[head * a.nq + tok] = live ? mn + logf(sum) : neg_inf();
    }
  }
  if (threadIdx.x == 0 && *abort) flag_status(a.status, FASTAR_DEV_TIMEOUT);
}

template <int D, bool kTwo>
cudaError_t few_go(const Kv4AttnArgs& a, cudaStream_t s) {
  const int64_t blocks = (int64_t)a.Hkv * a.splits;
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  const cudaError_t e = opt_in_smem((const void*)kv4_attn_few_kernel<D, kTwo>, FewLayout<D>::bytes);
  if (e != cudaSuccess) return e;
  kv4_attn_few_kernel<D, kTwo><<<(unsigned)blocks, kWarpsW * 32, FewLayout<D>::bytes, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_attn_few(int d, const Kv4AttnArgs& a, cudaStream_t s) {
  const bool two = (int64_t)(a.Hq / a.Hkv) * a.nq > 8;
  if (d == 128) return two ? few_go<128, true>(a, s) : few_go<128, false>(a, s);
  return two ? few_go<64, true>(a, s) : few_go<64, false>(a, s);
}

}  // namespace fastar
