// Softmax attention over the 4-bit cache on the 5th-generation tensor cores (bf16 queries).
//
// A CTA takes two tiles of 128 rows ((query head, token) pairs of a KV head) and a range of keys,
// 128 at a time; at d = 128 two CTAs of a cluster work as a pair (cta_group::2): every product
// has 256 rows, 128 of each CTA, and each CTA holds half of its K or V operand (64 of the keys
// of Q K^T, 64 of the channels of P V).
//   warps 0-15         softmax: two threads a row, 64 of a tile's 128 keys each (warps 0-3 and 4-7 of
//                      row tile 0, 8-11 and 12-15 of row tile 1): logits from TMEM, exponentials
//                      against a reference that is moved, and the sums rescaled, only when a P
//                      would pass what fp16 holds, P as fp16 over the consumed logits in TMEM, the output;
//   warps 16-19, 20-23 unpack K, V: packed tiles (four on their way, brought by bulk copies that
//                      warp 25 issues) into rings of 128-byte-swizzled fp16 tiles;
//   warp 24            owns TMEM and issues tcgen05.mma from one thread (of the pair's first CTA):
//                      S = Q K^T of both row tiles, O += P V (P from TMEM).
// The order of issue is PV0(j) QK0(j+1) PV1(j) QK1(j+1): while the softmax of one row tile
// runs, the tensor cores work for the other, so a logit buffer a tile is enough and two
// accumulators of 128 columns fit TMEM beside them.  (Two buffers of 64 keys a row tile, so that
// the softmax never waits, were slower: an MMA of 64 columns runs at little over half the rate.)
// A row tile's turn is PV, QK and the softmax between them; with one thread a row the softmax
// was the longest part, which is why it has two.
// Where the rows fill only one row tile, both halves of the CTA take it: one the even key
// tiles, the other the odd ones, and the two results are joined in shared memory at the end.
//
// What bounds it: a 128-key tile is 2048 clocks of MMA a CTA at d = 128.  Shared memory was the
// limit of one CTA alone: operands 192 KB, unpacked tiles 64 KB written, 18 KB in and out, 2300
// clocks at 128 bytes each; a pair halves the K and V part (operands 128 KB, 32 KB written).
// Instruction fetches come next: hot code is one copy, rare paths (masks, rescaling) lie apart.
// Measured, 12 heads of 128, in a replayed graph: 4680 tokens over 93,600 rows 1.81 ms (1490 TFLOP/s, 0.77
// of the bf16 rate measured for a library product; as one call 1.86 ms), 2850 clocks a tile; the
// first 4680 tokens in three frames 98 us, of which a CTA's start and end are 6 us an item.
//
// Numbers: a cache value (code times scale) is exact in fp16 (kv4.cuh).  A query row is scaled
// by a power of two that puts its largest element in [2^12, 2^13) and rounded to fp16: bf16's 8
// bits fit fp16's 11, so only elements 2^-26 of the row's largest and below are not exact (and
// off by at most 2^-37 of it); the power returns in the row's logit scale.  P in fp16 has an
// error of 2^-11, an eighth of bf16's, down to 2^-24 of the row's largest, and 2^-35 of that
// below (kv4.cuh: the reference's lift).  Logits, maxima, sums and outputs are fp32.
//
// Keys past a row's last visible one get P = 0; rows past the CTA's last key are stored as
// zeros in shared memory, so what lies behind the cache's length cannot reach a sum as 0 * NaN.
// Every wait is bounded; a timeout sets FASTAR_DEV_TIMEOUT and unwinds.
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"
#include "tc.cuh"
#include "tc_attn.cuh"
#include "tmap.h"

namespace fastar {

namespace {

constexpr int kRT = 128;               // rows of a row tile in a CTA
constexpr int kKT = 128;               // keys of a tile
constexpr int kStages = 3;             // fp16 tiles of K and of V
constexpr int kIn = 4, kMaxIn = 6;     // packed tiles on their way
constexpr int kSoftWarps = 16, kUnpackWarps = 8;
constexpr int kMmaWarp = kSoftWarps + kUnpackWarps;
constexpr int kThreadsT = 896;         // the last warpgroup: MMA warp, copy warp, two idle ones
// Registers: 896 threads x 72 at launch = 64,512 >= 512 softmax threads x 88 + 384 others x 48.
constexpr int kRegsSoft = 88, kRegsRest = 48;
static_assert(512 * kRegsSoft + 384 * kRegsRest <= kThreadsT * 72, "the launch's registers bound the shares");

// What a CTA works on (the same for both of a pair).
struct Kv4Item {
  int64_t len, most;       // the head's cached rows; keys that any of the CTA's rows sees
  uint32_t rows, r0;       // rows of a KV head, the item's first
  uint32_t j0, split;      // first key tile
  int h, group, nt, T;     // KV head, its query heads, row tiles with rows, key tiles (-1: a split that is not in use)
  bool partial;            // one of several splits
};

// Threads at the barriers that hold the unpacking of all but the first tile of K back until the query
// rows, which the first product waits for, are done (the softmax warps arrive, four warps wait).
constexpr int kHeld = (kSoftWarps + 4) * 32;

struct alignas(16) Kv4Ctl {
  uint64_t in_full[kMaxIn], in_empty[kMaxIn];          // packed tiles: K 0, V 0, K 1, V 1, ...
  uint64_t q_full[2], k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t s_full[2], p_full[2][2], fin;               // by row tile (P: first 32 keys of each half, last 32)
  Kv4Item item;
  uint32_t tmem_base;
  int abort;
  float ex[2][2][kRT];                                 // a row's two threads: half, row tile, row
  float mx[kRT];
};

// C CTAs work as one: at d = 64 one, at d = 128 a pair, or one for calls of a single row tile (kOne).
// What a CTA holds of a tile: KR keys of K, all 128 keys of V with D / C channels; in blocks of 64
// channels.
template <int D, int C>
struct Kv4Layout {
  static constexpr int kCta = C;
  static constexpr bool kOne = D > 64 * C;
  static constexpr int stages = kOne ? 2 : kStages, ins = kOne ? kMaxIn : kIn;
  static constexpr int KR = kKT / kCta;
  static constexpr size_t q_tile = (size_t)kRT * D * 2, q_blk = kRT * 128;
  static constexpr size_t k_tile = (size_t)KR * D * 2, k_blk = KR * 128;
  static constexpr size_t v_tile = (size_t)kKT * (D / C) * 2, v_blk = kKT * 128;
  static constexpr size_t in_codes = (size_t)kKT * D / 2, in_tile = in_codes + (size_t)kKT * D / 16;
  static constexpr size_t q = 0;
  static constexpr size_t k = q + (kOne ? 1 : 2) * q_tile;
  static constexpr size_t v = k + stages * k_tile;
  static constexpr size_t in = v + stages * v_tile;
  // at the end: the odd tiles' output (128 rows of D floats), and 4 KB a softmax warp
  static constexpr size_t odd_o = kOne ? k : q, out = kOne ? v : k;
  static constexpr size_t ctl = in + ins * in_tile;
  static constexpr size_t bytes = ctl + sizeof(Kv4Ctl) + 1024;
  static constexpr uint32_t s_col = 0, o_col = 256;   // two 128-column buffers each
  static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
};

// fp16 operands, fp32 sums; bit 16: B is MN-major.
constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// P = 2^(s sl2 - m) of 32 logits as fp16 pairs into 16 TMEM columns; adds to the row's sum.
__device__ __forceinline__ void row_exp32(const float* x, float sl2, float nm, uint32_t dst, float& s0, float& s1) {
  uint32_t pk[16];
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    float a = x[i], b = x[i + 1];
    fma2(a, b, sl2, nm);
    a = ex2f(a);
    b = ex2f(b);
    add2(s0, s1, a, b);
    pk[i >> 1] = pack_f16(a, b);
  }
  tmem_st16(dst, pk);
}

// Row r of a KV head's work: its query head and token.
struct RowOf {
  int64_t head, t;
};
__device__ __forceinline__ RowOf row_of(const Kv4AttnArgs& a, const Kv4Item& it, int64_t r) {
  const uint32_t nq = (uint32_t)a.nq, g = (uint32_t)r / nq;       // Hq * nq fits 31 bits
  return RowOf{it.h * (int64_t)it.group + g, (int64_t)((uint32_t)r - g * nq)};
}

// A row that sees no key: zeros and lse = -inf.
template <int D>
__device__ __forceinline__ void store_empty(const Kv4AttnArgs& a, RowOf w) {
  uint4* p = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + w.head * a.o_hs + w.t * a.o_ts);
#pragma unroll
  for (int i = 0; i < D / 8; ++i) p[i] = make_uint4(0, 0, 0, 0);
  if (a.lse) a.lse[w.head * a.nq + w.t] = neg_inf();
}

// The work item of this block.  First splits first (a short cache uses no others); in a call in
// blocks the rows that see most keys first, of all heads.  A last item with one row tile takes 0.6
// of a full one's time: it comes at the end, where it fills gaps, or in a call in blocks behind the
// 0.4 of the row tiles that take longer (first chunk in frames: 92 us of the longest chain of
// items become 88).
template <int kCta>
__device__ __forceinline__ Kv4Item item_place(const Kv4AttnArgs& a, int row_tiles) {
  Kv4Item it;
  it.group = a.group;
  const uint32_t rows = it.rows = a.rows;
  const bool odd = row_tiles > 1 && (rows - 1) % (2 * kRT * kCta) < kRT * kCta;
  const int full_tiles = a.block > 0 ? row_tiles : row_tiles - odd;     // in blocks: the odd one among them
  uint32_t u = blockIdx.x / kCta;
  const uint32_t all = (uint32_t)(a.Hkv * full_tiles);
  const bool last = u >= all * (uint32_t)a.splits;
  if (last) u -= all * (uint32_t)a.splits;
  it.split = a.splits == 1 ? 0u : last ? u / (uint32_t)a.Hkv : u / all;
  u -= it.split * (last ? (uint32_t)a.Hkv : all);
  uint32_t rt = (uint32_t)full_tiles;
  if (last) {
    it.h = (int)u;
  } else if (a.block > 0) {
    const uint32_t x = u / (uint32_t)a.Hkv;
    it.h = (int)(u - x * (uint32_t)a.Hkv);
    const uint32_t full = (uint32_t)(row_tiles - odd), at = odd ? (2 * full + 4) / 5 : full;
    rt = x < at ? full - 1 - x : x == at ? full : full - x;
  } else {
    it.h = (int)(u / (uint32_t)full_tiles);
    rt = (uint32_t)full_tiles - 1 - (u - (uint32_t)it.h * (uint32_t)full_tiles);
  }
  it.r0 = rt * (2 * kRT * kCta);
  it.nt = rows - it.r0 > kRT * kCta ? 2 : 1;
  return it;
}
// The keys it works on, from the head's length.
template <int kCta>
__device__ __forceinline__ void item_keys_of(const Kv4AttnArgs& a, Kv4Item& it, int64_t len) {
  it.len = len;
  const uint32_t rlast = (it.r0 + 2 * kRT * kCta < it.rows ? it.r0 + 2 * kRT * kCta : it.rows) - 1;
  const kv4::ItemKeys keys =
      kv4::item_keys(len, (uint32_t)a.nq, a.block, it.r0, rlast, a.splits, a.min_tiles);
  it.most = keys.most;
  it.partial = keys.splits > 1;
  it.j0 = it.partial ? keys.tiles * it.split / keys.splits : 0u;     // tiles times splits fits 32 bits
  it.T = it.split >= keys.splits ? -1
         : it.partial            ? (int)(keys.tiles * (it.split + 1) / keys.splits - it.j0)
                                 : (int)keys.tiles;
}

template <int D, int C>
__global__ void __launch_bounds__(kThreadsT, 1) kv4_attn_tc_kernel(const Kv4AttnArgs a, int row_tiles) {
  using Lay = Kv4Layout<D, C>;
  constexpr int kCta = C;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Kv4Ctl& sm = *reinterpret_cast<Kv4Ctl*>(base + Lay::ctl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kCta == 2 ? (int)cta_rank() : 0;
  pdl_wait();                            // the launch overlaps the end of the kernel before

  // Before the loop a CTA has only latencies to wait for, and instructions to fetch that run once:
  // one thread finds the item (its divisions in all 28 warps took 5000 clocks), another sets the
  // barriers up, and rolled loops move the query rows, which come while the length is on its way.
  const bool finder = threadIdx.x == (kMmaWarp + 1) * 32;
  int cached = 0;                        // the head's length, on its way across the first barrier
  if (finder) {
    for (int i = 0; i < Lay::ins; ++i) {
      tc::mbar_init(&sm.in_full[i], 1);
      tc::mbar_init(&sm.in_empty[i], 4);
    }
    tc::mbar_fence_init();
    const Kv4Item place = item_place<kCta>(a, row_tiles);
    cached = a.len[place.h];
    sm.item = place;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.q_full[i], 8 * kCta);
      tc::mbar_init(&sm.s_full[i], 1);
      tc::mbar_init(&sm.p_full[i][0], 8 * kCta);
      tc::mbar_init(&sm.p_full[i][1], 8 * kCta);
    }
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&sm.k_full[i], 4 * kCta);
      tc::mbar_init(&sm.k_empty[i], 1);
      tc::mbar_init(&sm.v_full[i], 4 * kCta);
      tc::mbar_init(&sm.v_empty[i], 1);
    }
    tc::mbar_init(&sm.fin, 1);
    sm.abort = 0;
    tc::mbar_fence_init();
  }
  __syncthreads();
  // Query rows: warp x of a row tile brings its rows 16 x .. on, four lanes a row, to where the product
  // wants them, then turns them to fp16 in place.  Odd rows take the halves of a block's 16-byte
  // chunks the other way round, so that 8 lanes hit 8 bank groups.
  constexpr int QC = D / 32;                              // a lane's chunks of a row
  const int qw = warp >> 3;                               // row tile
  const bool mine = warp < kSoftWarps && !(sm.item.nt == 1 && qw == 1);
  const int qr = (warp & 7) * 16 + (lane >> 2), qc = (lane & 3) ^ ((lane >> 2 & 1) << 2);
  uint8_t* qd = base + Lay::q + (size_t)qw * Lay::q_tile;
  auto chunk = [&](int i, int j) {                        // chunk j of the lane's row i
    return qd + (j >> 1) * Lay::q_blk + tc::sw128_off(qr + i * 8, qc ^ ((j & 1) << 2));
  };
  if (mine) {
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      const uint32_t x = sm.item.r0 + (uint32_t)(qw * (kRT * kCta) + rank * kRT + qr + i * 8);
      const RowOf from = row_of(a, sm.item, x < a.rows ? x : sm.item.r0);
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q.p) + from.head * a.q.hs + from.t * a.q.ts;
#pragma unroll
      for (int j = 0; j < QC; ++j)
        tc::cp_async16(tc::smem_u32(chunk(i, j)), src + (j >> 1) * 64 + (qc ^ ((j & 1) << 2)) * 8, x < a.rows ? 16 : 0);
    }
    tc::cp_async_commit();
  }
  if (finder) item_keys_of<kCta>(a, sm.item, kv4::held_len(cached, a.cap, a.status));   // fields that no one reads yet
  __syncthreads();
  const Kv4Item& it = sm.item;
  const uint32_t rows = it.rows, r0 = it.r0, split = it.split;
  const int h = it.h, T = it.T;
  const bool partial = it.partial, both = it.nt == 1;    // both: one row tile, even key tiles and odd key tiles
  if (T <= 0 || (a.splits > 1 && !partial)) {
    const uint32_t r = r0 + threadIdx.x / kRT * (kRT * kCta) + rank * kRT + threadIdx.x % kRT;
    if (threadIdx.x < 2 * kRT && r < rows) {
      const RowOf w = row_of(a, it, r);
      // what the join reads of a split that is not in use, and of the first where the output is in place
      if (a.splits > 1)
        a.part_ml[((int64_t)split * a.Hq + w.head) * a.nq + w.t] = make_float2(split == 0 ? -neg_inf() : neg_inf(), 0.f);
      if (T == 0) store_empty<D>(a, w);                  // no keys at all
    }
    if (T <= 0) {                                        // both CTAs of a pair
      tc::cp_async_wait<0>();
      return;
    }
  }
  if (kCta == 2) pair_arrive();                          // this CTA's barriers are ready
  volatile int* abort = &sm.abort;

  if (warp < kSoftWarps) {
    // ---------------- softmax ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    const int w = warp >> 3, half = (warp >> 2) & 1;      // row tile (or parity of the key tiles), half
    const int row = (warp & 3) * 32 + lane;
    const int pair_bar = 1 + w * 4 + (warp & 3);          // the two warps of these rows
    const uint32_t r = r0 + (both ? 0u : (uint32_t)(w * (kRT * kCta))) + (uint32_t)(rank * kRT + row);
    const bool has = r < rows;
    constexpr int HD = D / 2;                             // channels of a row of O a thread takes
    if (mine) {
      tc::cp_async_wait<0>();
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        uint32_t v[4 * QC], big2 = 0;                     // a row's largest magnitude, two channels at a time
#pragma unroll
        for (int j = 0; j < QC; ++j) {
          const uint4 c = *reinterpret_cast<const uint4*>(chunk(i, j));
          v[4 * j] = c.x, v[4 * j + 1] = c.y, v[4 * j + 2] = c.z, v[4 * j + 3] = c.w;
        }
#pragma unroll
        for (int e = 0; e < 4 * QC; ++e) big2 = __vmaxu2(big2, v[e] & 0x7fff7fffu);
        big2 = __vmaxu2(big2, __shfl_xor_sync(0xffffffffu, big2, 1));
        big2 = __vmaxu2(big2, __shfl_xor_sync(0xffffffffu, big2, 2));
        const uint32_t big = max(big2 & 0xffffu, big2 >> 16);
        // exponent of the largest (subnormals count as 2^-126); a row that is zero or not finite
        // stays as it is
        const int ex = (int)(big >> 7);
        int qe = ex == 0 ? -126 - 12 : ex - 127 - 12;
        if (qe < -120) qe = -120;
        if (big == 0 || ex == 255) qe = 0;
        const float down = kv4::pow2i(-qe);
#pragma unroll
        for (int j = 0; j < QC; ++j) {
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[e] = pack_f16(__uint_as_float(v[4 * j + e] << 16) * down, __uint_as_float(v[4 * j + e] & 0xffff0000u) * down);
          *reinterpret_cast<uint4*>(chunk(i, j)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        if ((lane & 3) == 0) sm.ex[0][w][qr + i * 8] = kv4::pow2i(qe);
      }
      tc::fence_proxy_async();
    }
    bar_arrive(11, kHeld);
    bar_arrive(12, kHeld);
    tc::named_bar(10, (kSoftWarps + 1) * 32);             // TMEM is there, and ex
    tc::tc_fence_after();
    if (kCta == 2) pair_wait();                           // the other CTA's barriers are ready
    if (mine && lane == 0) arrive_issuer<kCta>(&sm.q_full[w]);
    const uint32_t tmem = sm.tmem_base;
    const RowOf at = has ? row_of(a, it, r) : RowOf{0, 0};
    // keys the row sees from this thread's first on (a row that is not there: as the last)
    int left = max(0, (int)(has ? kv4::visible(it.len, a.nq, at.t, a.block) : it.most) - (int)it.j0 * kKT - half * 64 -
                          (both ? w * kKT : 0));          // capacities fit 31 bits
    float sl2 = a.scale * sm.ex[0][both ? 0 : w][row] * kv4::pow2i(kv4::head_exp(a.k_exp, h)) * 1.4426950408889634f;
    sl2 = fminf(fmaxf(sl2, 1.2e-38f), 3.0e38f);   // a product of scales outside fp32's range: positive and finite
    tc::named_bar(9, kSoftWarps * 32);     // ex is used again below
    const int step = both ? 2 : 1, count = both ? (T - w + 1) >> 1 : T;      // this row tile's key tiles
    const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_addr = lane_addr + Lay::s_col + (uint32_t)(w * 128 + half * 64);
    const uint32_t o_addr = lane_addr + Lay::o_col + (uint32_t)(w * 128 + half * HD);
    float m = 0.f, l0 = 0.f, l1 = 0.f;      // m: the reference, in log2 units
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < count; ++i, left = max(0, left - step * kKT)) {
      const bool alive = wait_warp(&sm.s_full[w], i & 1, abort);
      tc::tc_fence_after();
      const bool cut = __any_sync(0xffffffffu, left < 64);
      const int valid = min(left, 64);          // keys that the row sees
      float top;                                // the largest of them, not scaled yet
      {
        float x[64];
        tc::tmem_ld32(s_addr, x);
        tc::tmem_ld32(s_addr + 32, x + 32);
        tc::tmem_wait_ld();
        tc::tmem_pin32(x);
        tc::tmem_pin32(x + 32);
        if (__builtin_expect(cut, 0)) {
#pragma unroll
          for (int c = 0; c < 64; ++c) x[c] = c < valid ? x[c] : neg_inf();
        }
        top = row_max<64>(x);
      }
      // Both warps of the rows move the reference together: when a P would pass what fp16 holds (the scale
      // is positive, so the largest logit has the largest P; its exponent is formed as row_exp32
      // forms it), and at the first tile.
      if (__builtin_expect(tc::named_bar_or(pair_bar, 64, fmaf(top, sl2, -m) > kv4::kTop || i == 0 || !alive), 0)) {
        float mt = top * sl2;
        sm.ex[half][w][row] = mt;
        // the warps leave together as well
        if (tc::named_bar_or(pair_bar, 64, !alive)) {
          ok = false;
          break;
        }
        mt = fmaxf(mt, sm.ex[half ^ 1][w][row]);
        float f = 1.f;
        if (i == 0) {
          m = mt == neg_inf() ? 0.f : mt - kv4::kLift;
        } else if (const float to = mt - kv4::kLift; to > m) {
          f = ex2f(m - to);
          m = to;
          l0 *= f;
          l1 *= f;
        }
        __syncwarp();
        if (i > 0) {
          // O holds the products of the tiles before: these logits were issued after them, by the
          // same thread, and their arrival says that all it had issued is complete
#pragma unroll 1
          for (int c = 0; c < HD; c += 16) {
            float o[16];
            tc::tmem_ld16(o_addr + (uint32_t)c, o);
            tc::tmem_wait_ld();
            tc::tmem_pin16(o);
            uint32_t ou[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) ou[e] = __float_as_uint(o[e] * f);
            tmem_st16(o_addr + (uint32_t)c, ou);
          }
          tc::tmem_wait_st();
          tc::tc_fence_before();
          tc::named_bar(pair_bar, 64);                    // all of O is rescaled before either half's P goes
          tc::tc_fence_after();
        }
      }
      // P over the logits' own columns: 32 logits are read again (held since the maximum, 64 took
      // registers that the loads and exponentials need to overlap) and become 16 columns, over
      // logits that have been read
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x[32];
        tc::tmem_ld32(s_addr + (uint32_t)(32 * c), x);
        tc::tmem_wait_ld();
        tc::tmem_pin32(x);
        if (__builtin_expect(cut, 0)) {
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = 32 * c + e < valid ? x[e] : neg_inf();
        }
        row_exp32(x, sl2, -m, s_addr + (uint32_t)(16 * c), l0, l1);
        tc::tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_issuer<kCta>(&sm.p_full[w][c]);
      }
    }
    // the outputs; barriers first, so that every thread passes them whatever has failed
    ok = wait_warp(&sm.fin, 0, abort) && ok;
    tc::tc_fence_after();
    float l = l0 + l1;
    sm.ex[half][w][row] = l;
    float4* shared_o = reinterpret_cast<float4*>(base + Lay::odd_o);   // Q, or K, has been used
    constexpr int CH = D / 4;                                       // 16-byte chunks of a row
    if (both && w == 1) {
      if (half == 0) sm.mx[row] = m;
      if (ok && count > 0)
#pragma unroll 1
        for (int c = 0; c < HD; c += 16) {
          float o[16];
          tc::tmem_ld16(o_addr + (uint32_t)c, o);
          tc::tmem_wait_ld();
          tc::tmem_pin16(o);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            shared_o[row * CH + (((half * HD + c) / 4 + e) ^ (row & (CH - 1)))] =
                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
    }
    tc::named_bar(9, kSoftWarps * 32);
    l += sm.ex[half ^ 1][w][row];
    if (ok && !(both && w == 1)) {
      float f0 = 1.f, f1 = 0.f;             // weights of this sum and of the odd tiles'
      if (both && T > 1) {
        const float lo = sm.ex[0][1][row] + sm.ex[1][1][row], mo = sm.mx[row];
        if (lo != 0.f) {                    // the odd tiles hold a key that the row sees
          const float mn = fmaxf(m, mo);
          f0 = ex2f(m - mn);
          f1 = ex2f(mo - mn);
          l = l * f0 + lo * f1;
          m = mn;
        }
      }
      const bool live = l > 0.f || l != l;
      l *= kv4::kUnlift;
      const float up = kv4::pow2i(kv4::head_exp(a.v_exp, h)) * kv4::kUnlift;
      const float f = partial ? up : live ? up / l : 0.f;
      // Rows of 128 bytes (32 fp32 or 64 bf16 channels; 64 bytes of 32 bf16) go through shared
      // memory (the ring of K, or of V, has been used), so that they leave as whole runs; written
      // 16 bytes a thread, a row each, they took 5 us of a CTA.
      uint8_t* stg = base + Lay::out + warp * 4096;
      uint8_t* out = partial ? reinterpret_cast<uint8_t*>(a.part_o) : static_cast<uint8_t*>(a.out);
      const int64_t off = !has     ? -1
                          : partial ? (((int64_t)split * a.Hq + at.head) * a.nq + at.t) * D * 4 + half * HD * 4
                                    : (at.head * a.o_hs + at.t * a.o_ts + half * HD) * 2;
      const int cp = partial ? 32 : HD, esz = partial ? 4 : 2;   // channels a pass
      const int nc = HD == 64 ? 8 : cp * esz / 16;               // 16-byte chunks of a pass's row
#pragma unroll 1
      for (int c0 = 0; c0 < HD; c0 += cp) {
#pragma unroll 1
        for (int c = c0; c < c0 + cp; c += 16) {
          float o[16];
          __syncwarp();
          tc::tmem_ld16(o_addr + (uint32_t)c, o);
          tc::tmem_wait_ld();
          tc::tmem_pin16(o);
          if (f1 != 0.f) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 v = shared_o[row * CH + (((half * HD + c) / 4 + e) ^ (row & (CH - 1)))];
              o[4 * e] = o[4 * e] * f0 + v.x * f1;
              o[4 * e + 1] = o[4 * e + 1] * f0 + v.y * f1;
              o[4 * e + 2] = o[4 * e + 2] * f0 + v.z * f1;
              o[4 * e + 3] = o[4 * e + 3] * f0 + v.w * f1;
            }
          }
          const int ch = (c - c0) * esz / 16;
          if (partial) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<float4*>(stg + tc::sw128_off(lane, ch + e)) =
                  make_float4(o[4 * e] * f, o[4 * e + 1] * f, o[4 * e + 2] * f, o[4 * e + 3] * f);
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t v[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                __nv_bfloat162 h2 = __floats2bfloat162_rn(o[8 * e + 2 * k] * f, o[8 * e + 2 * k + 1] * f);
                v[k] = live ? *reinterpret_cast<uint32_t*>(&h2) : 0u;
              }
              *reinterpret_cast<uint4*>(stg + tc::sw128_off(lane, ch + e)) = make_uint4(v[0], v[1], v[2], v[3]);
            }
          }
        }
        __syncwarp();
#pragma unroll 4
        for (int i = 0; i < nc; ++i) {
          const int sr = (i * 32 + lane) / nc, ch = (i * 32 + lane) % nc;
          const int64_t to = __shfl_sync(0xffffffffu, off, sr);
          const uint4 v = *reinterpret_cast<const uint4*>(stg + tc::sw128_off(sr, ch));
          if (to >= 0) *reinterpret_cast<uint4*>(out + to + c0 * esz + ch * 16) = v;
        }
        __syncwarp();
      }
      if (has && half == 0) {
        const float mn = (m + kv4::kLift) * 0.6931471805599453f;
        if (partial)
          a.part_ml[((int64_t)split * a.Hq + at.head) * a.nq + at.t] = make_float2(live ? mn : neg_inf(), l);
        else if (a.lse)
          a.lse[at.head * a.nq + at.t] = live ? mn + logf(l) : neg_inf();
      }
    }
  } else if (warp < kMmaWarp) {
    // ---------------- unpack K and V ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (kCta == 2) pair_wait();
    // A thread takes two (four) runs of 32 codes (16 bytes) of a tile: of K's KR rows x D channels, or
    // of V's 128 rows x this CTA's channels.  With four runs to a row (K at d = 128) runs 2 and
    // 3 write their 16-byte chunks in another order: so the 8 lanes of a store phase always
    // hit 8 different bank groups of the swizzled tile.
    const int t = threadIdx.x & 127;
    constexpr int KP = D / 32, VP = D / C / 32;           // runs of a row of K, of V
    constexpr int kRuns = Lay::kOne ? 4 : 2;
    const bool isv = warp >= kSoftWarps + 4;              // warps 16-19: K, 20-23: V
#pragma unroll 1
    for (int n = isv; n < 2 * T; n += 2) {
      const int j = n >> 1, st = j % Lay::stages, in = n % Lay::ins;
      uint64_t* empty = isv ? &sm.v_empty[st] : &sm.k_empty[st];
      uint64_t* full = isv ? &sm.v_full[st] : &sm.k_full[st];
      const bool two = KP == 2 || (VP == 2 && isv);       // runs to a row: two, or four
      const int part = two ? t & 1 : t & 3, row0 = two ? t >> 1 : t >> 2;
      const int rstep = two ? 64 : 32;
      const int flip = part & 2;
      // the run's place in the packed tile: 16 bytes of codes, two scales
      const int run0 = isv && VP < KP ? row0 * KP + 2 * rank + part : t;
      const int runstep = rstep * KP;
      if (n == (isv ? 1 : 2)) tc::named_bar(isv ? 12 : 11, kHeld);
      if (!wait_warp(&sm.in_full[in], (n / Lay::ins) & 1, abort) || !wait_warp(empty, ((j / Lay::stages) & 1) ^ 1, abort)) break;
      const uint8_t* packed = base + Lay::in + in * Lay::in_tile;
      uint8_t* tile = base + (isv ? Lay::v + (size_t)st * Lay::v_tile : Lay::k + (size_t)st * Lay::k_tile);
      // rows past the last key hold what is in memory there, or nothing: they count as 0
      const int left = (int)it.most - (int)(it.j0 + j) * kKT - (isv ? 0 : rank * Lay::KR);
#pragma unroll 1
      for (int g = 0; g < kRuns; g += 2) {
        uint4 c[2];
        uint32_t s[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          c[k] = reinterpret_cast<const uint4*>(packed)[run0 + (g + k) * runstep];
          s[k] = reinterpret_cast<const uint16_t*>(packed + Lay::in_codes)[run0 + (g + k) * runstep];
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int row = row0 + (g + k) * rstep;
          if (row >= left) c[k] = make_uint4(0, 0, 0, 0), s[k] = 0;
          uint32_t wv[4] = {c[k].x, c[k].y, c[k].z, c[k].w};
          uint32_t s0 = kv4::scale_f16x2(s[k]), s1 = kv4::scale_f16x2(s[k] >> 8);
          if (KP == 4 && flip) {
            uint32_t x = wv[0];
            wv[0] = wv[2], wv[2] = x;
            x = wv[1];
            wv[1] = wv[3], wv[3] = x;
            x = s0;
            s0 = s1, s1 = x;
          }
          uint8_t* dst = tile + (KP == 4 && flip ? Lay::k_blk : 0);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t o[4];
            kv4::unpack8(wv[e], e < 2 ? s0 : s1, o);
            *reinterpret_cast<uint4*>(dst + tc::sw128_off(row, (part & 1) * 4 + (e ^ flip))) =
                make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        arrive_issuer<kCta>(full);
        tc::mbar_arrive(&sm.in_empty[in]);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == kMmaWarp) {
      tmem_alloc512<kCta>(&sm.tmem_base);
      tc::tc_fence_before();
      tc::named_bar(10, (kSoftWarps + 1) * 32);
      tc::tc_fence_after();
    }
    if (kCta == 2) pair_wait();
    if (warp == kMmaWarp + 1 && lane == 0) {
      // ---------------- packed tiles into shared memory (one thread) ----------------
      // Whole 16-row groups: the capacity is a multiple of 16, so the group that holds the last
      // key lies within the head's rows, and sizes and addresses are multiples of 16 bytes.  Of
      // K only this CTA's rows; of V whole rows (a bulk copy is contiguous).
      const int64_t first = (int64_t)it.h * a.cap;
      const uint32_t most = (uint32_t)it.most, j0 = it.j0;      // capacities fit 31 bits
      int n = 0;
      for (; n < 2 * T; ++n) {
        const int in = n % Lay::ins;
        const bool isv = n & 1;
        if (!tc::mbar_wait(&sm.in_empty[in], ((n / Lay::ins) & 1) ^ 1, abort)) break;
        const uint32_t key = (j0 + (uint32_t)(n >> 1)) * kKT + (isv ? 0u : (uint32_t)(rank * Lay::KR));
        const uint32_t nr = key < most ? min((most - key + 15) & ~15u, (uint32_t)(isv ? kKT : Lay::KR)) : 0u;
        uint8_t* dst = base + Lay::in + in * Lay::in_tile;
        tc::mbar_arrive_tx(&sm.in_full[in], nr * (D / 2 + D / 16));
        if (nr == 0) continue;
        tc::bulk_load(dst, (isv ? a.vc : a.kc) + (first + key) * (D / 2), nr * (D / 2), &sm.in_full[in]);
        tc::bulk_load(dst + Lay::in_codes, (isv ? a.vs : a.ks) + (first + key) * (D / 16), nr * (D / 16),
                      &sm.in_full[in]);
      }
      // the last copies land before this thread leaves, whether or not anyone waits for them
      volatile int never = 0;
      for (int x = n < Lay::ins ? 0 : n - Lay::ins; x < n; ++x) tc::mbar_wait(&sm.in_full[x % Lay::ins], (x / Lay::ins) & 1, &never, 400000000LL);
    }
    // ---------------- MMA issue (one thread of the pair) ----------------
    if (warp == kMmaWarp && rank == 0 && elect_one()) {
      const uint32_t tmem = sm.tmem_base;
      constexpr uint32_t idesc_qk = idesc_f16(kRT * kCta, kKT, false), idesc_pv = idesc_f16(kRT * kCta, D, true);
      const uint64_t q_desc = tc::sw128_desc(tc::smem_u32(base + Lay::q));
      const uint64_t k_desc = tc::sw128_desc(tc::smem_u32(base + Lay::k));
      const uint64_t v_desc = tc::sw128_mn_desc(tc::smem_u32(base + Lay::v), Lay::v_blk);
      bool ok = true;
      const int step = both ? 2 : 1;
      int kst[2], vst[2], count[2];                       // stages of K and V, key tiles by row tile
      uint32_t kph[2], vph[2];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        kst[w] = vst[w] = both ? w : 0;
        kph[w] = vph[w] = 0;
        count[w] = both ? (T - w + 1) >> 1 : T;
      }
#pragma unroll 1
      for (int i = -1; i < count[0] && ok; ++i) {         // P V of tile i (from 0 on), Q K^T of tile i + 1
#pragma unroll
        for (int w = 0; w < 2; ++w) {                     // unrolled: columns are constants
          if (i >= 0 && i < count[w]) {
            ok = tc::mbar_wait(&sm.v_full[vst[w]], vph[w], abort);
            if (!ok) break;
            const uint64_t vd = v_desc + ((vst[w] * Lay::v_tile) >> 4);
#pragma unroll
            for (int c = 0; c < 2; ++c) {                 // 32 keys of both halves at a time, as their P lands
              ok = tc::mbar_wait(&sm.p_full[w][c], i & 1, abort);
              if (!ok) break;
              tc::tc_fence_after();
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int key = (k >> 1) * 64 + c * 32 + (k & 1) * 16;
                mma_ts<kCta>(tmem + Lay::o_col + w * 128, tmem + Lay::s_col + w * 128 + (k >> 1) * 64 + c * 16 + (k & 1) * 8,
                             vd + ((key * 128) >> 4), idesc_pv, i > 0 || c > 0 || k > 0 ? 1u : 0u);
              }
            }
            if (!ok) break;
            if (w == 1 || both) commit<kCta>(&sm.v_empty[vst[w]]);
            vst[w] += step;
            if (vst[w] >= Lay::stages) vst[w] -= Lay::stages, vph[w] ^= 1;
          }
          if (i + 1 < count[w]) {
            ok = (i >= 0 || tc::mbar_wait(&sm.q_full[both ? 0 : w], 0, abort)) &&
                 tc::mbar_wait(&sm.k_full[kst[w]], kph[w], abort);
            if (!ok) break;
            tc::tc_fence_after();
            const uint64_t qd = q_desc + (((both ? 0 : w) * Lay::q_tile) >> 4);
            const uint64_t kd = k_desc + ((kst[w] * Lay::k_tile) >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_ss<kCta>(tmem + Lay::s_col + w * 128, qd + (((k >> 2) * Lay::q_blk + (k & 3) * 32) >> 4),
                           kd + (((k >> 2) * Lay::k_blk + (k & 3) * 32) >> 4), idesc_qk, k > 0 ? 1u : 0u);
            commit<kCta>(&sm.s_full[w]);
            if (w == 1 || both) commit<kCta>(&sm.k_empty[kst[w]]);
            kst[w] += step;
            if (kst[w] >= Lay::stages) kst[w] -= Lay::stages, kph[w] ^= 1;
          }
        }
      }
      // the outputs are complete; and every issued product ends before TMEM is given back
      commit<kCta>(&sm.fin);
      volatile int never = 0;
      tc::mbar_wait(&sm.fin, 0, &never, 400000000LL);
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (kCta == 2) {                       // neither CTA leaves while the other may signal or use it
    // (after a wait that gave up, signals may be on their way to the other CTA: they land first)
    if (*abort) asm volatile("fence.acq_rel.cluster;" ::: "memory");
    pair_arrive();
    pair_wait();
  }
  if (warp == kMmaWarp) {
    tc::tc_fence_after();
    tmem_free512<kCta>(sm.tmem_base);
  }
  if (threadIdx.x == 0 && sm.abort) flag_status(a.status, FASTAR_DEV_TIMEOUT);
}

template <int D, int C>
cudaError_t tc_go(const Kv4AttnArgs& a, cudaStream_t s) {
  using Lay = Kv4Layout<D, C>;
  const int64_t rt = ((int64_t)a.rows + 2 * kRT * Lay::kCta - 1) / (2 * kRT * Lay::kCta);
  const int64_t blocks = rt * a.Hkv * a.splits * Lay::kCta;
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  cudaError_t e = opt_in_smem((const void*)kv4_attn_tc_kernel<D, C>, (int)Lay::bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreadsT);
  cfg.dynamicSmemBytes = Lay::bytes;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = Lay::kCta;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kv4_attn_tc_kernel<D, C>, a, (int)rt);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_attn_tc(int d, const Kv4AttnArgs& a, cudaStream_t s) {
  if (d == 64) return tc_go<64, 1>(a, s);
  return a.alone ? tc_go<128, 1>(a, s) : tc_go<128, 2>(a, s);
}

}  // namespace fastar
