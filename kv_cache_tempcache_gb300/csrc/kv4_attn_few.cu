// Softmax attention over the 4-bit cache for few rows, as in single-token steps: up to 16 (query
// head, token) pairs of a KV head in bf16; and for fp32 queries, 8 rows a CTA.
//
// Bound: the cache's bytes, for which it still takes twice the time: no unit is full over a long cache (issue
// slots 50 %, integer 49 %, DRAM 52 %), a warp's chain of waits, products and exponentials is what
// it waits for, with four warps a scheduler.  A row tile of the tcgen05 kernel is 128 or 256 rows, so with a few
// rows it spends most of its time unpacking for products that are nearly empty; here the rows
// are the 8 columns (twice, above 8 rows) of m16n8k16 products (mma.sync: its rate is not what
// bounds this), and the unpacked codes go from registers straight into the products' operands,
// without shared memory between:
//   S^T[16 keys, 8 rows] += K[16, 16 channels] Q^T,   O^T[16 channels, 8 rows] += V^T[16, 16 keys] P^T
// P^T is S^T's registers after an 8 x 8 transpose (movmatrix).  A product may sum its channels in
// any order as long as both operands agree, so lane t of a quad takes channels t d/4 .. of a key,
// 16 consecutive bytes of codes at d = 128; and V^T's rows may be any channels: lane group g
// takes d/8 consecutive ones, and the pairs of keys that the operand wants side by side are
// paired as codes, before they are unpacked.
// Each warp runs alone over its share of the CTA's blocks of 32 keys: three (six) blocks on
// their way by bulk copies, its own reference, sums and outputs; the warps' results are joined in
// shared memory, in warp order, at the end, and the CTAs' by the join kernel.
// (With the rows as the products' 16 rows, half of them empty up to 8, 8 warps of 250 registers
// waited for one another's latencies: one token over 131,071 rows of 8 heads 45 us.)
// fp32: a query row (24 bits) is three fp16 rows, P two (22 bits), each a product of its own on
// the codes unpacked once; the unpacking, not the products, is most of the work.  P goes into
// its parts times 2^14, so that they keep 22 bits down to 2^-17 of the largest and 2^-39 of it
// below.
// Queries, P and references otherwise as in the tcgen05 kernel (kv4_attn_tc.cu): fp16 rows at a power of
// two, P in fp16 against a reference that moves only when a P would pass what fp16 holds.
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace fastar {

namespace {

constexpr int kKeysW = 32;

// NR: groups of 8 rows.
template <typename T, int D, int NR>
struct FewLayout {
  static constexpr bool f32 = sizeof(T) == 4;
  static constexpr int warps = NR == 1 && !f32 ? 16 : 8, stages = NR == 1 && !f32 ? 3 : 6;
  static constexpr int codes = kKeysW * D / 2, scales = kKeysW * D / 16;
  static constexpr int stage = 2 * (codes + scales);                 // K codes, V codes, K scales, V scales
  static constexpr int ring = warps * stages * stage;
  static constexpr int red = warps * 8 * NR * D * 4;                 // the joined outputs, over the ring
  static constexpr int ctl = ring > red ? ring : red;
  static constexpr int bytes = ctl + warps * stages * 8 + warps * 8 * NR * 8 + 16 + 128;
  static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
};

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Eight bytes of codes as four fp16 pairs each (scaled): cvt takes a byte of a register at no cost.
__device__ __forceinline__ void unpack_bytes(uint32_t w, uint32_t s2, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  uint32_t o[4];
  kv4::unpack8(w, s2, o);
  a = o[0], b = o[1], c = o[2], d = o[3];
}
// The codes of two keys, channel by channel side by side: even channels of the word, odd ones.
__device__ __forceinline__ void pair_codes(uint32_t ka, uint32_t kb, uint32_t& even, uint32_t& odd) {
  even = (ka & 0x0f0f0f0fu) | ((kb << 4) & 0xf0f0f0f0u);
  odd = ((ka >> 4) & 0x0f0f0f0fu) | (kb & 0xf0f0f0f0u);
}
// The fp16 pair of two scale bytes (lo, hi), and one of them twice.
__device__ __forceinline__ uint32_t scales_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
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
// Over the eight lanes of equal t.
__device__ __forceinline__ float group_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
__device__ __forceinline__ float group_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  return v + __shfl_xor_sync(0xffffffffu, v, 16);
}
// Lane (g, t) holds elements (g, 2t), (g, 2t + 1) of an 8 x 8 matrix of 16-bit values; gets (2t, g), (2t + 1, g).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// A lane's share of query row r (channels t D/4 ..) as product operands: qb[part][s] of step s;
// returns the row's logit scale in log2 units.
template <typename T, int D, int QP>
__device__ __forceinline__ float load_q(const Kv4AttnArgs& a, int h, uint32_t rows, uint32_t r, int t,
                                        uint32_t (*qb)[D / 16][2]) {
  constexpr int CH = D / 4;                 // channels of this lane
  float x[CH];
  uint32_t big = 0;                         // the largest magnitude's bits
  if (r < rows) {
    const uint32_t nq = (uint32_t)a.nq, gh = r / nq;
    const int64_t head = h * (int64_t)a.group + gh;
    const T* src = static_cast<const T*>(a.q.p) + head * a.q.hs + (int64_t)(r - gh * nq) * a.q.ts + t * CH;
#pragma unroll
    for (int i = 0; i < CH; i += 8) load8(src + i, x + i);
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i) x[i] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) big = max(big, __float_as_uint(x[i]) & 0x7fffffffu);
  big = quad_max(big);
  const int ex = (int)(big >> 23);
  int qe = ex == 0 ? -126 - 12 : ex - 127 - 12;
  if (qe < -120) qe = -120;
  if (big == 0 || ex == 255) qe = 0;
  const float down = kv4::pow2i(-qe);
#pragma unroll
  for (int i = 0; i < CH / 2; ++i) {        // pair i of the lane's channels: step i / 2, first or second pair
    float a0 = x[2 * i] * down, a1 = x[2 * i + 1] * down;
#pragma unroll
    for (int part = 0; part < QP; ++part) {
      const uint32_t p = pack_f16w(a0, a1);
      qb[part][i >> 1][i & 1] = p;
      const float2 f = kv4::f16x2_to_f32(p);
      a0 -= f.x;
      a1 -= f.y;
    }
  }
  // a product of scales outside fp32's range: positive and finite
  return fminf(fmaxf(a.scale * kv4::pow2i(qe) * kv4::pow2i(kv4::head_exp(a.k_exp, h)) * 1.4426950408889634f, 1.2e-38f),
               3.0e38f);
}

template <typename T, int D, int NR>
__global__ void __launch_bounds__(FewLayout<T, D, NR>::warps * 32, 1) kv4_attn_few_kernel(const Kv4AttnArgs a) {
  using Lay = FewLayout<T, D, NR>;
  constexpr int QP = Lay::f32 ? 3 : 1, PP = Lay::f32 ? 2 : 1;        // fp16 parts of Q and of P
  constexpr float kUp = Lay::f32 ? 0x1p14f : 1.f, kRoom = Lay::f32 ? 1.f : kv4::kTop;   // P is at most 2^kRoom
  constexpr float kLift = Lay::f32 ? 0.f : kv4::kLift, kUnlift = Lay::f32 ? 1.f : kv4::kUnlift;
  constexpr int W = Lay::warps, ST = Lay::stages, MT = D / 16;       // MT: row tiles of O^T
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~(uintptr_t)127);
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + Lay::ctl);
  float2* wml = reinterpret_cast<float2*>(bars + W * ST);            // [warp][8 NR]
  int* abort_flag = reinterpret_cast<int*>(wml + W * 8 * NR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  pdl_wait();                               // the launch overlaps the end of the kernel before
  const uint32_t rows = a.rows, groups = (rows + 8 * NR - 1) / (8 * NR);
  const int split = (int)blockIdx.y;
  const int h = (int)(groups == 1 ? blockIdx.x : blockIdx.x / groups);
  const uint32_t gr = blockIdx.x - (uint32_t)h * groups;
  const uint32_t r0 = gr * 8 * NR, rlast = (r0 + 8 * NR < rows ? r0 + 8 * NR : rows) - 1;
  // the keys that any of the rows sees
  const int64_t cached = kv4::head_len(a.len, h, a.cap, a.status);
  const int64_t len = kv4::item_keys(cached, (uint32_t)a.nq, a.block, r0, rlast, 1, 1).most;
  const uint32_t blocks = (uint32_t)((len + kKeysW - 1) / kKeysW);
  const uint32_t b0 = (uint32_t)((uint64_t)blocks * split / (uint32_t)a.splits);
  const uint32_t b1 = (uint32_t)((uint64_t)blocks * (split + 1) / (uint32_t)a.splits);
  const int count = b0 + warp < b1 ? (int)((b1 - b0 - warp + W - 1) / W) : 0;   // this warp's blocks
  pdl_trigger();                            // the join's CTAs may come and wait

  uint64_t* full = bars + warp * ST;
  if (lane == 0) {
    for (int i = 0; i < ST; ++i) tc::mbar_init(&full[i], 1);
    if (warp == 0) *abort_flag = 0;
    tc::mbar_fence_init();
  }
  uint8_t* ring = base + warp * ST * Lay::stage;
  // one lane brings block i of the warp: whole 16-row groups, which lie within the head's rows
  auto fetch = [&](int i, int st) {
    const int64_t key = (int64_t)(b0 + warp + (uint32_t)i * W) * kKeysW;
    const int64_t left = (len - key + 15) & ~(int64_t)15;
    const uint32_t nr = left < kKeysW ? (uint32_t)left : kKeysW;
    const int64_t at = (int64_t)h * a.cap + key;
    uint8_t* dst = ring + st * Lay::stage;
    tc::mbar_arrive_tx(&full[st], 2 * nr * (D / 2 + D / 16));
    tc::bulk_load(dst, a.kc + at * (D / 2), nr * (D / 2), &full[st]);
    tc::bulk_load(dst + 2 * Lay::codes, a.ks + at * (D / 16), nr * (D / 16), &full[st]);
    tc::bulk_load(dst + Lay::codes, a.vc + at * (D / 2), nr * (D / 2), &full[st]);
    tc::bulk_load(dst + 2 * Lay::codes + Lay::scales, a.vs + at * (D / 16), nr * (D / 16), &full[st]);
  };
  if (lane == 0)
    for (int i = 0; i < ST && i < count; ++i) fetch(i, i);
  __syncthreads();                          // the barriers and the flag are set for every lane

  uint32_t qb[NR][QP][D / 16][2];
  float sl2[NR][2], m[NR][2], l[NR][2];     // of rows 2t and 2t + 1 of each group
  int see[NR][2];                           // how many keys they see
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const float s = load_q<T, D, QP>(a, h, rows, r0 + 8 * n + g, t, qb[n]);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      sl2[n][p] = __shfl_sync(0xffffffffu, s, (2 * t + p) * 4);
      const uint32_t r = r0 + (uint32_t)(8 * n + 2 * t + p), nq = (uint32_t)a.nq;
      see[n][p] = (int)(r < rows ? a.block > 0 ? kv4::visible(cached, a.nq, r % nq, a.block) : cached : len);
      m[n][p] = l[n][p] = 0.f;
    }
  }
  float o[NR][MT][4];
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int i = 0; i < MT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
  volatile int* abort = abort_flag;

  int stage = 0;
  uint32_t ph = 0;
  int i = 0;
#pragma unroll 1
  for (; i < count; ++i) {
    const int key = (int)(b0 + warp + (uint32_t)i * W) * kKeysW;        // the capacity fits 31 bits
    uint8_t* st = ring + stage * Lay::stage;
    if (!__all_sync(0xffffffffu, tc::mbar_wait(&full[stage], ph, abort))) break;
    if ((int)len - key < kKeysW) {
      // rows behind the length count as 0, whatever lies there: their scales do (a scale each of
      // K's and V's D / 16 a row; a lane a row)
      if (lane >= (int)len - key)
        for (int x = 0; x < D / 16; ++x)
          st[2 * Lay::codes + lane * (D / 16) + x] = st[2 * Lay::codes + Lay::scales + lane * (D / 16) + x] = 0;
      __syncwarp();
    }
    // ---- S^T = K Q^T: 16 keys at a time, a lane's shares of keys g and g + 8 of them ----
    float s[NR][2][4];
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
      uint32_t kf[2][D / 8];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int k = kt * 16 + e * 8 + g;
        if (D == 128) {
          const uint4 c = reinterpret_cast<const uint4*>(st)[k * 4 + t];
          const uint32_t s2 = scales_f16x2(reinterpret_cast<const uint16_t*>(st + 2 * Lay::codes)[k * 4 + t]);
          const uint32_t s0 = __byte_perm(s2, 0, 0x1010), s1 = __byte_perm(s2, 0, 0x3232);
          kv4::unpack8(c.x, s0, kf[e]);
          kv4::unpack8(c.y, s0, kf[e] + 4);
          kv4::unpack8(c.z, s1, kf[e] + 8 % (D / 8));
          kv4::unpack8(c.w, s1, kf[e] + 12 % (D / 8));
        } else {
          const uint2 c = reinterpret_cast<const uint2*>(st)[k * 4 + t];
          const uint32_t s0 = kv4::scale_f16x2((st + 2 * Lay::codes)[k * 4 + t]);
          kv4::unpack8(c.x, s0, kf[e]);
          kv4::unpack8(c.y, s0, kf[e] + 4);
        }
      }
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        float u[2][4];                      // two sums, so that two products are in flight
#pragma unroll
        for (int x = 0; x < 4; ++x) u[0][x] = u[1][x] = 0.f;
#pragma unroll
        for (int q = 0; q < D / 16; ++q) {
          const uint32_t ka[4] = {kf[0][2 * q], kf[1][2 * q], kf[0][2 * q + 1], kf[1][2 * q + 1]};
#pragma unroll
          for (int part = 0; part < QP; ++part) mma16816(u[(q + part) & 1], ka, qb[n][part][q][0], qb[n][part][q][1]);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) s[n][kt][x] = u[0][x] + u[1][x];
      }
    }
    // ---- masks, reference, P ----
    bool cut = false;
#pragma unroll
    for (int n = 0; n < NR; ++n) cut |= min(see[n][0], see[n][1]) - key < kKeysW;
    if (__any_sync(0xffffffffu, cut)) {
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (key + kt * 16 + (x >> 1) * 8 + g >= see[n][x & 1]) s[n][kt][x] = neg_inf();
    }
    float top[NR][2];                       // the largest logits, not scaled yet
    bool grow = i == 0;
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        top[n][p] = fmaxf(fmaxf(s[n][0][p], s[n][0][2 + p]), fmaxf(s[n][1][p], s[n][1][2 + p]));
        grow |= fmaf(top[n][p], sl2[n][p], -m[n][p]) > kRoom;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const float mx = group_max(top[n][p]) * sl2[n][p], to = mx - kLift;
          float f = 1.f;
          if (i == 0) {
            m[n][p] = mx == neg_inf() ? 0.f : to;
          } else if (to > m[n][p]) {
            f = ex2w(m[n][p] - to);
            m[n][p] = to;
          }
          l[n][p] *= f;
#pragma unroll
          for (int x = 0; x < MT; ++x) o[n][x][p] *= f, o[n][x][2 + p] *= f;
        }
    }
    uint32_t pb[NR][PP][2][2];
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float e0 = ex2w(fmaf(s[n][kt][2 * e], sl2[n][0], -m[n][0]));
          float e1 = ex2w(fmaf(s[n][kt][2 * e + 1], sl2[n][1], -m[n][1]));
          l[n][0] += e0;
          l[n][1] += e1;
          e0 *= kUp;
          e1 *= kUp;
#pragma unroll
          for (int part = 0; part < PP; ++part) {
            const uint32_t x = pack_f16w(e0, e1);
            pb[n][part][kt][e] = transpose8(x);
            const float2 y = kv4::f16x2_to_f32(x);
            e0 -= y.x;
            e1 -= y.y;
          }
        }
    // ---- O^T += V^T P^T: a lane's keys 2t, 2t + 1, 2t + 8, 2t + 9 of 16, channels g D/8 .. ----
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
      // va[x]: the operand of row tile x: channels 2 x (rows g) and 2 x + 1 (rows g + 8), each a
      // pair of keys: the codes are paired before they are unpacked
      uint32_t va[MT][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {         // keys 2t, 2t + 1 of the first or second 8
        const int k = kt * 16 + 8 * e + 2 * t;
        const uint8_t* sc = st + 2 * Lay::codes + Lay::scales + (D == 128 ? k * 8 + g : k * 4 + (g >> 1));
        const uint32_t s2 = scales_f16x2(sc[0] | (uint32_t)sc[D / 16] << 8);
        if (D == 128) {
          const uint2 ca = reinterpret_cast<const uint2*>(st + Lay::codes)[k * 8 + g];
          const uint2 cb = reinterpret_cast<const uint2*>(st + Lay::codes)[(k + 1) * 8 + g];
          uint32_t even, odd;
          pair_codes(ca.x, cb.x, even, odd);
          unpack_bytes(even, s2, va[0][2 * e], va[1][2 * e], va[2][2 * e], va[3][2 * e]);
          unpack_bytes(odd, s2, va[0][2 * e + 1], va[1][2 * e + 1], va[2][2 * e + 1], va[3][2 * e + 1]);
          pair_codes(ca.y, cb.y, even, odd);
          unpack_bytes(even, s2, va[4 % MT][2 * e], va[5 % MT][2 * e], va[6 % MT][2 * e], va[7 % MT][2 * e]);
          unpack_bytes(odd, s2, va[4 % MT][2 * e + 1], va[5 % MT][2 * e + 1], va[6 % MT][2 * e + 1],
                       va[7 % MT][2 * e + 1]);
        } else {
          const uint32_t* c = reinterpret_cast<const uint32_t*>(st + Lay::codes) + k * 8 + g;
          uint32_t even, odd;
          pair_codes(c[0], c[8], even, odd);
          unpack_bytes(even, s2, va[0][2 * e], va[1][2 * e], va[2][2 * e], va[3][2 * e]);
          unpack_bytes(odd, s2, va[0][2 * e + 1], va[1][2 * e + 1], va[2][2 * e + 1], va[3][2 * e + 1]);
        }
      }
#pragma unroll
      for (int x = 0; x < MT; ++x)
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int part = 0; part < PP; ++part) mma16816(o[n][x], va[x], pb[n][part][kt][0], pb[n][part][kt][1]);
    }
    __syncwarp();                           // every lane has read the block
    if (lane == 0 && i + ST < count) fetch(i + ST, stage);
    if (++stage == ST) stage = 0, ph ^= 1;
  }
  // after a wait that gave up: the copies in flight land before the ring is used or given back
  volatile int never = 0;
  for (int x = i; x < count && x < i + ST; ++x) {
    tc::mbar_wait(&full[stage], ph, &never, 400000000LL);
    if (++stage == ST) stage = 0, ph ^= 1;
  }

  // ---- the warps' results, in warp order ----
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      l[n][p] = group_sum(l[n][p]);
      if (g == 0) wml[warp * 8 * NR + 8 * n + 2 * t + p] = make_float2(m[n][p], l[n][p]);
    }
  __syncthreads();
  // the largest reference of a row's warps that hold a key it sees
  auto top = [&](int r) {
    float mx = neg_inf();
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 x = wml[w * 8 * NR + r];
      if (x.y != 0.f) mx = fmaxf(mx, x.x);
    }
    return mx;
  };
  float* red = reinterpret_cast<float*>(base);          // the ring has been used: [warp][8 NR][D]
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int r = 8 * n + 2 * t + p;
      const float f = l[n][p] != 0.f ? ex2w(m[n][p] - top(r)) : 0.f;
      // a lane's channels g D/8 + 2 x and + 2 x + 1 of row r
      float4* dst = reinterpret_cast<float4*>(red + (warp * 8 * NR + r) * D + g * (D / 8));
      if (r0 + r <= rlast)
#pragma unroll
        for (int x = 0; x < MT; x += 2)
          dst[x >> 1] = make_float4(o[n][x][p] * f, o[n][x][2 + p] * f, o[n][x + 1][p] * f, o[n][x + 1][2 + p] * f);
    }
  __syncthreads();
  const float up = kv4::pow2i(kv4::head_exp(a.v_exp, h)) / kUp * kUnlift;
  for (int x = threadIdx.x; x < (int)(rlast - r0 + 1) * (D / 4); x += W * 32) {
    const int r = x / (D / 4), c = x % (D / 4) * 4;
    const float mx = top(r);
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 y = wml[w * 8 * NR + r];
      if (y.y == 0.f) continue;             // no key of that warp's that the row sees
      sum += y.y * ex2w(y.x - mx);
      const float4 z = *reinterpret_cast<const float4*>(red + (w * 8 * NR + r) * D + c);
      acc.x += z.x, acc.y += z.y, acc.z += z.z, acc.w += z.w;
    }
    const bool live = sum > 0.f || sum != sum;
    sum *= kUnlift;
    const uint32_t nq = (uint32_t)a.nq, gh = (r0 + (uint32_t)r) / nq;
    const int64_t head = h * (int64_t)a.group + gh, tok = r0 + (uint32_t)r - gh * nq;
    const float mn = (mx + kLift) * 0.6931471805599453f;
    if (a.splits > 1) {
      const int64_t at = (split * (int64_t)a.Hq + head) * a.nq + tok;
      *reinterpret_cast<float4*>(a.part_o + at * D + c) = make_float4(acc.x * up, acc.y * up, acc.z * up, acc.w * up);
      if (c == 0) a.part_ml[at] = make_float2(live ? mn : neg_inf(), sum);
    } else {
      const float f = live ? up / sum : 0.f;
      T* dst = static_cast<T*>(a.out) + head * a.o_hs + tok * a.o_ts + c;
      if (Lay::f32) {
        *reinterpret_cast<float4*>(dst) = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
      } else {
        __nv_bfloat162 v[2] = {__floats2bfloat162_rn(acc.x * f, acc.y * f), __floats2bfloat162_rn(acc.z * f, acc.w * f)};
        *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<uint2*>(v);
      }
      if (c == 0 && a.lse) a.lse[head * a.nq + tok] = live ? mn + logf(sum) : neg_inf();
    }
  }
  if (threadIdx.x == 0 && *abort) flag_status(a.status, FASTAR_DEV_TIMEOUT);
}

template <typename T, int D, int NR>
cudaError_t few_go(const Kv4AttnArgs& a, cudaStream_t s) {
  using Lay = FewLayout<T, D, NR>;
  const int64_t blocks = ((int64_t)a.rows + 8 * NR - 1) / (8 * NR) * a.Hkv;
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  cudaError_t e = opt_in_smem((const void*)kv4_attn_few_kernel<T, D, NR>, Lay::bytes);
  if (e != cudaSuccess) return e;
  e = launch_dependent(kv4_attn_few_kernel<T, D, NR>, dim3((unsigned)blocks, (unsigned)a.splits), dim3(Lay::warps * 32),
                       Lay::bytes, s, a);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_attn_few(int dtype, int d, const Kv4AttnArgs& a, cudaStream_t s) {
  if (dtype == FASTAR_F32) return d == 128 ? few_go<float, 128, 1>(a, s) : few_go<float, 64, 1>(a, s);
  const bool two = a.rows > 8;
  if (d == 128) return two ? few_go<__nv_bfloat16, 128, 2>(a, s) : few_go<__nv_bfloat16, 128, 1>(a, s);
  return two ? few_go<__nv_bfloat16, 64, 2>(a, s) : few_go<__nv_bfloat16, 64, 1>(a, s);
}

}  // namespace fastar
