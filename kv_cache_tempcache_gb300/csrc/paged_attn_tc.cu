// Softmax attention over a paged cache on the 5th-generation tensor cores (bf16).
//
// A CTA takes two tiles of 128 rows ((token, query head) pairs of a KV head) and a list of key tiles of 128
// rows (paged.cuh: those of the first rows, then those of the window); at d = 128 two CTAs of a
// cluster work as a pair (cta_group::2): every product has 256 rows, 128 of each CTA, and each CTA
// holds half of its K or V operand (64 of the keys of Q K^T, 64 of the channels of P V).
//   warps 0-15   softmax: two threads a row, 64 of a tile's 128 keys each (warps 0-3 and 4-7 of row
//                tile 0, 8-11 and 12-15 of row tile 1): logits from TMEM, exponentials against a reference that is
//                moved, and the sums rescaled, only when a P would pass 2^kTop, P as bf16 over the consumed
//                logits in TMEM, the output;
//   warp 16      owns TMEM and issues tcgen05.mma from one thread (of the pair's first CTA): S = Q K^T of
//                both row tiles, O += P V (P from TMEM);
//   warp 17      brings K and V by TMA, a box a lane: a box is a page, or the part of one that a tile
//                has; pages that no row sees, or that are not there, come as zeros (a coordinate past the pool);
//   warp 18      hands K tiles on to the issuing CTA;
//   warp 19      hands V tiles on, and looks into those that not every row sees in full: a key that
//                nobody sees becomes zeros, and an infinity or NaN that only some rows see is taken out (a
//                weight of 0 would not keep it from the others) and returns in the outputs of the rows that see it.
// The order of issue is PV0(j) QK0(j+1) PV1(j) QK1(j+1): while the softmax of one row tile
// runs, the tensor cores work for the other, so a logit buffer a tile is enough and two
// accumulators of 128 columns fit TMEM beside them.  Where the rows fill only one row tile, both halves
// of the CTA take it: one the even key tiles, the other the odd ones, and the two results are joined
// in shared memory at the end.
//
// Numbers: logits, maxima, sums and outputs are fp32.  P is bf16, as V is (a product has one type):
// 2^-8 of itself, at every magnitude, since bf16 has fp32's exponents.
// Every wait is bounded; a timeout sets FASTAR_DEV_TIMEOUT and unwinds.
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"
#include "paged_attn.h"
#include "tc.cuh"
#include "tc_attn.cuh"
#include "tmap.h"

namespace fastar {

namespace {

constexpr int kRT = 128;               // rows of a row tile in a CTA
constexpr int kKT = 128;               // keys of a tile
constexpr int kSoftWarps = 16;
constexpr int kMmaWarp = kSoftWarps, kCopyWarp = kMmaWarp + 1, kKWarp = kMmaWarp + 2, kVWarp = kMmaWarp + 3;
constexpr int kThreadsT = 640;
// Registers: 640 threads x 96 at launch = 61,440 = 512 softmax threads x 104 + 128 others x 64.
constexpr int kRegsSoft = 104, kRegsRest = 64;
static_assert(512 * kRegsSoft + 128 * kRegsRest <= kThreadsT * 96, "the launch's registers bound the shares");
// The reference moves when a P would pass this power of two: sums of 2^30 keys' P times V stay far inside fp32
// for |V| up to 2^88.
constexpr float kTop = 8.f;

// What a CTA works on (the same for both of a pair).
struct Item {
  paged::Seq s;
  paged::Tiles<kKT> tiles;
  paged::Split part;
  uint32_t rows, r0;       // rows of the sequence's KV head, the item's first
  int b, h, split, nt;     // sequence, KV head, split, row tiles with rows
};

struct alignas(16) Ctl {
  uint64_t k_land[4], k_full[4], k_empty[4], v_land[4], v_full[4], v_empty[4];
  uint64_t q_full[2], s_full[2], p_full[2][2], fin;    // by row tile (P: first 32 keys of each half, last 32)
  Item item;
  uint32_t tmem_base;
  int abort, poison;
  float ex[2][2][kRT];                                 // a row's two threads: half, row tile, row
  float mx[kRT];
};

// C CTAs work as one: at d = 64 one, at d = 128 a pair, or one for work of a single row tile (kOne).
// What a CTA holds of a tile: KR keys of K, all 128 keys of V with D / C channels; in blocks of 64
// channels.
template <int D, int C>
struct Layout {
  static constexpr int kCta = C;
  static constexpr bool kOne = D > 64 * C;
  static constexpr int ks = kOne ? 3 : 4, vs = kOne ? 2 : 4;    // tiles of K and of V on their way
  static constexpr int KR = kKT / kCta, VC = D / C;
  static constexpr size_t q_tile = (size_t)kRT * D * 2, q_blk = kRT * 128;
  static constexpr size_t k_tile = (size_t)KR * D * 2, k_blk = KR * 128;
  static constexpr size_t v_tile = (size_t)kKT * VC * 2, v_blk = kKT * 128;
  static constexpr size_t q = 0;
  static constexpr size_t k = q + (kOne ? 1 : 2) * q_tile;
  static constexpr size_t v = k + ks * k_tile;
  // at the end: the odd tiles' output (128 rows of D floats), and 4 KB a softmax warp
  static constexpr size_t odd_o = kOne ? k : q, out = kOne ? v : k;
  static constexpr size_t ctl = v + vs * v_tile;
  static constexpr size_t bytes = ctl + sizeof(Ctl) + 1024;
  static constexpr uint32_t s_col = 0, o_col = 256;   // two 128-column buffers each
  static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
  static_assert((kOne ? ks * k_tile : 2 * q_tile) >= (size_t)kRT * D * 4, "the odd tiles' output");
  static_assert((kOne ? vs * v_tile : ks * k_tile) >= kSoftWarps * 4096, "the outputs on their way");
};

// P = 2^(s sl2 - m) of 32 logits as bf16 pairs into 16 TMEM columns; adds to the row's sum.
__device__ __forceinline__ void row_exp32(const float* x, float sl2, float nm, uint32_t dst, float& s0, float& s1) {
  uint32_t pk[16];
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    float a = x[i], b = x[i + 1];
    fma2(a, b, sl2, nm);
    a = ex2f(a);
    b = ex2f(b);
    add2(s0, s1, a, b);
    pk[i >> 1] = pack_bf16(a, b);
  }
  tmem_st16(dst, pk);
}

// Row r of the item: its token in the sequence and its query head.
struct RowOf {
  int t, head;
};
__device__ __forceinline__ RowOf row_of(const PagedAttnArgs& a, const Item& it, uint32_t r) {
  const uint32_t t = r / (uint32_t)a.group;
  return RowOf{(int)t, it.h * a.group + (int)(r - t * (uint32_t)a.group)};
}

// A row that sees no key: zeros and lse = -inf.
template <int D>
__device__ __forceinline__ void store_empty(const PagedAttnArgs& a, const Item& it, RowOf w) {
  const int64_t tok = it.s.t0 + w.t;
  uint4* p = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + w.head * a.o_hs + tok * a.o_ts);
#pragma unroll
  for (int i = 0; i < D / 8; ++i) p[i] = make_uint4(0, 0, 0, 0);
  if (a.lse) a.lse[w.head * a.T + tok] = neg_inf();
}

// The work of this block: heads side by side, then sequences, then row tiles from the last (whose rows see
// most), then splits.
template <int kCta>
__device__ __forceinline__ void find_item(const PagedAttnArgs& a, Item& it, int row_tiles) {
  uint32_t u = blockIdx.x / kCta;
  uint32_t x = u / (uint32_t)a.Hkv;
  it.h = (int)(u - x * (uint32_t)a.Hkv);
  u = x / (uint32_t)a.B;
  it.b = (int)(x - u * (uint32_t)a.B);
  x = u / (uint32_t)row_tiles;
  it.split = (int)x;
  it.r0 = ((uint32_t)row_tiles - 1 - (u - x * (uint32_t)row_tiles)) * (2 * kRT * kCta);
  it.s = paged::sequence(a.cu, a.at, a.B, a.T, a.cap, it.b, a.status);
  if (it.s.nq > a.max_q) flag_status(a.status, FASTAR_DEV_BAD_LEN);
  it.rows = (uint32_t)(a.group * min(it.s.nq, a.max_q));             // fits 31 bits
  it.nt = 0;
  if (it.r0 >= it.rows) return;
  it.nt = it.rows - it.r0 > kRT * kCta ? 2 : 1;
  const uint32_t last = min(it.r0 + 2 * kRT * kCta, it.rows) - 1;
  it.tiles.set(a, it.s, (int)(it.r0 / (uint32_t)a.group), (int)(last / (uint32_t)a.group));
  it.part = paged::split_of(it.tiles.n, it.split, a.splits, a.min_tiles);
}

template <int D, int C>
__global__ void __launch_bounds__(kThreadsT, 1)
    paged_attn_tc_kernel(const PagedAttnArgs a, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap, int row_tiles) {
  using Lay = Layout<D, C>;
  constexpr int kCta = C;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Ctl& sm = *reinterpret_cast<Ctl*>(base + Lay::ctl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kCta == 2 ? (int)cta_rank() : 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.q_full[i], 8 * kCta);
      tc::mbar_init(&sm.s_full[i], 1);
      tc::mbar_init(&sm.p_full[i][0], 8 * kCta);
      tc::mbar_init(&sm.p_full[i][1], 8 * kCta);
    }
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(&sm.k_land[i], 1);
      tc::mbar_init(&sm.k_full[i], kCta);
      tc::mbar_init(&sm.k_empty[i], 1);
      tc::mbar_init(&sm.v_land[i], 1);
      tc::mbar_init(&sm.v_full[i], kCta);
      tc::mbar_init(&sm.v_empty[i], 1);
    }
    tc::mbar_init(&sm.fin, 1);
    sm.abort = 0;
    sm.poison = 0;
    tc::mbar_fence_init();
  }
  pdl_wait();                            // the launch overlaps the end of the kernel before
  if (threadIdx.x == kCopyWarp * 32) {   // one thread finds the work
    find_item<kCta>(a, sm.item, row_tiles);
    tc::tma_prefetch_desc(&kmap);
    tc::tma_prefetch_desc(&vmap);
  }
  __syncthreads();
  const Item& it = sm.item;
  if (it.nt == 0) return;                                // both CTAs of a pair
  const uint32_t rows = it.rows, r0 = it.r0;
  const int T = it.part.j1 - it.part.j0;
  const bool partial = it.part.used > 1, both = it.nt == 1;   // both: one row tile, even key tiles and odd key tiles
  if (T == 0 || (a.splits > 1 && !partial)) {
    const uint32_t r = r0 + threadIdx.x / kRT * (kRT * kCta) + rank * kRT + threadIdx.x % kRT;
    if (threadIdx.x < 2 * kRT && r < rows) {
      const RowOf w = row_of(a, it, r);
      // what the join reads of a split that is not in use, and of the first where the output is in place
      if (a.splits > 1)
        a.part_ml[paged::partial_row(a, (int64_t)it.split * a.B + it.b, it.h, (int)r)] =
            make_float2(it.split == 0 ? -neg_inf() : neg_inf(), 0.f);
      if (it.tiles.n == 0 && it.split == 0) store_empty<D>(a, it, w);   // no keys at all
    }
    if (T == 0) return;
  }
  if (kCta == 2) pair_arrive();                          // this CTA's barriers are ready
  volatile int* abort = &sm.abort;

  if (warp < kSoftWarps) {
    // ---------------- softmax ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    const int w = warp >> 3, half = (warp >> 2) & 1;      // row tile (or parity of the key tiles), half
    const int row = (warp & 3) * 32 + lane;
    const int pair_bar = 1 + w * 4 + (warp & 3);          // the two warps of these rows
    const bool mine = !(both && w == 1);
    if (mine) {
      // Query rows: warp x of a row tile brings its rows 16 x .. on, four lanes a row, to where the product
      // wants them; odd rows take the halves of a block's 16-byte chunks the other way round, so that
      // 8 lanes hit 8 bank groups.
      constexpr int QC = D / 32;                          // a lane's chunks of a row
      const int qr = (warp & 7) * 16 + (lane >> 2), qc = (lane & 3) ^ ((lane >> 2 & 1) << 2);
      uint8_t* qd = base + Lay::q + (size_t)w * Lay::q_tile;
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        const uint32_t x = r0 + (uint32_t)(w * (kRT * kCta) + rank * kRT + qr + i * 8);
        const RowOf from = row_of(a, it, x < rows ? x : r0);
        const __nv_bfloat16* src =
            static_cast<const __nv_bfloat16*>(a.q.p) + from.head * a.q.hs + (int64_t)(it.s.t0 + from.t) * a.q.ts;
#pragma unroll
        for (int j = 0; j < QC; ++j)
          tc::cp_async16(tc::smem_u32(qd + (j >> 1) * Lay::q_blk + tc::sw128_off(qr + i * 8, qc ^ ((j & 1) << 2))),
                         src + (j >> 1) * 64 + (qc ^ ((j & 1) << 2)) * 8, x < rows ? 16 : 0);
      }
      tc::cp_async_commit();
    }
    const uint32_t r = r0 + (both ? 0u : (uint32_t)(w * (kRT * kCta))) + (uint32_t)(rank * kRT + row);
    const bool has = r < rows;
    const RowOf at = row_of(a, it, has ? r : rows - 1);   // a row that is not there: as the last
    const paged::Sees see = paged::sees(a, it.s, at.t);
    constexpr int HD = D / 2;                             // channels of a row of O a thread takes
    float sl2 = a.scale * 1.4426950408889634f;
    sl2 = fminf(fmaxf(sl2, 1.2e-38f), 3.0e38f);
    const int step = both ? 2 : 1, count = both ? (T - w + 1) >> 1 : T;      // this row tile's key tiles
    if (mine) {
      tc::cp_async_wait<0>();
      tc::fence_proxy_async();
      __syncwarp();
    }
    tc::named_bar(10, (kSoftWarps + 1) * 32);             // TMEM is there
    tc::tc_fence_after();
    if (kCta == 2) pair_wait();                           // the other CTA's barriers are ready
    if (mine && lane == 0) arrive_issuer<kCta>(&sm.q_full[w]);
    const uint32_t tmem = sm.tmem_base;
    const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_addr = lane_addr + Lay::s_col + (uint32_t)(w * 128 + half * 64);
    const uint32_t o_addr = lane_addr + Lay::o_col + (uint32_t)(w * 128 + half * HD);
    float m = neg_inf(), l0 = 0.f, l1 = 0.f;      // m: the reference, in log2 units; -inf: no key seen yet
    bool ok = true;
    int j = it.part.j0 + (both ? w : 0);
#pragma unroll 1
    for (int i = 0; i < count; ++i, j += step) {
      const int key0 = it.tiles.key(j);
      const bool cut = !it.tiles.all(key0);
      uint32_t bits[2];
      if (cut) {
        bits[0] = paged::seen32(see, key0 + half * 64);
        bits[1] = paged::seen32(see, key0 + half * 64 + 32);
      }
      const bool alive = wait_warp(&sm.s_full[w], i & 1, abort);
      tc::tc_fence_after();
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
          for (int c = 0; c < 64; ++c) x[c] = bits[c >> 5] >> (c & 31) & 1 ? x[c] : neg_inf();
        }
        top = row_max<64>(x);
      }
      // Both warps of the rows stop together when a P would pass 2^kTop (the scale is positive, so the
      // largest logit has the largest P), or at a row's first key; of their rows only those that need
      // it move the reference, so that no row's roundings hang on its neighbours' keys.
      if (__builtin_expect(tc::named_bar_or(pair_bar, 64, fmaf(top, sl2, -m) > kTop || i == 0 || !alive), 0)) {
        float mt = top * sl2;
        sm.ex[half][w][row] = mt;
        // the warps leave together as well
        if (tc::named_bar_or(pair_bar, 64, !alive)) {
          ok = false;
          break;
        }
        mt = fmaxf(mt, sm.ex[half ^ 1][w][row]);
        float f = 1.f;
        if (mt - m > kTop) {
          f = ex2f(m - mt);                     // 0 at the first key
          m = mt;
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
      const float nm = m == neg_inf() ? 0.f : -m;
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
          for (int e = 0; e < 32; ++e) x[e] = bits[c] >> e & 1 ? x[e] : neg_inf();
        }
        row_exp32(x, sl2, nm, s_addr + (uint32_t)(16 * c), l0, l1);
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
      const bool poison = *(volatile int*)&sm.poison != 0;
      const float f = partial ? 1.f : live ? 1.f / l : 0.f;
      // Rows of 128 bytes (32 fp32 or 64 bf16 channels; 64 bytes of 32 bf16) go through shared
      // memory (the ring of K, or of V, has been used), so that they leave as whole runs
      uint8_t* stg = base + Lay::out + warp * 4096;
      uint8_t* out = partial ? reinterpret_cast<uint8_t*>(a.part_o) : static_cast<uint8_t*>(a.out);
      const int64_t tok = it.s.t0 + at.t;
      const int64_t prow = paged::partial_row(a, (int64_t)it.split * a.B + it.b, it.h, (int)r);
      const int64_t off = !has      ? -1
                          : partial ? (prow * D + half * HD) * 4
                                    : (at.head * a.o_hs + tok * a.o_ts + half * HD) * 2;
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
          if (__builtin_expect(poison, 0)) {
            float q[16];                    // a copy: o's registers keep no address
#pragma unroll
            for (int e = 0; e < 16; ++e) q[e] = o[e];
            paged::add_taken_out<kKT, 16>(a, it.tiles, it.part, it.b, it.h, see, half * HD + c, q);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = q[e];
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
              for (int k = 0; k < 4; ++k)
                v[k] = live ? pack_bf16(o[8 * e + 2 * k] * f, o[8 * e + 2 * k + 1] * f) : 0u;
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
        const float mn = m * 0.6931471805599453f;
        if (partial)
          a.part_ml[prow] = make_float2(live ? mn : neg_inf(), l);
        else if (a.lse)
          a.lse[at.head * a.T + tok] = live ? mn + logf(l) : neg_inf();
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
    if (warp == kCopyWarp) {
      // ---------------- K and V into shared memory ----------------
      const int shift = a.pool.page_shift, page = 1 << shift;
      const int kr = min(page, Lay::KR), vr = min(page, kKT);      // rows of a box
      const int nk = Lay::KR / kr * (D / 64), nv = kKT / vr * (Lay::VC / 64);
      const int32_t* table = a.table + (int64_t)it.b * a.max_pages;
      const int none = (int)a.pool.pages;                          // past the pool: the box comes as zeros
      const int kb = lane / (D / 64), kc = lane % (D / 64);        // this lane's box: rows, channels
      const int vb = lane / (Lay::VC / 64), vc = lane % (Lay::VC / 64);
      auto page_at = [&](int key, int n) {
        if (!it.tiles.any(key, key + n)) return none;
        const int x = paged::page_of(table, key >> shift, a.pool.pages, a.status);
        return x < 0 ? none : x;
      };
      int kn = 0, vn = 0;                                          // tiles asked for
      // the pages of a tile are looked up while the one before is asked for
      int kp = none, vp = none;
      auto look = [&](int i) {
        const int key = it.tiles.key(it.part.j0 + i);
        if (lane < nk) kp = page_at(key + rank * Lay::KR + kb * kr, kr);
        if (lane < nv) vp = page_at(key + vb * vr, vr);
      };
      look(0);
      for (int i = 0; i < T; ++i) {
        const int key = it.tiles.key(it.part.j0 + i);
        const int kp0 = kp, vp0 = vp;
        if (i + 1 < T) look(i + 1);
        int st = i % Lay::ks;
        if (!wait_warp(&sm.k_empty[st], ((i / Lay::ks) & 1) ^ 1, abort)) break;
        if (lane == 0) tc::mbar_arrive_tx(&sm.k_land[st], (uint32_t)Lay::k_tile);
        __syncwarp();
        if (lane < nk)
          tc::tma_load_4d(base + Lay::k + st * Lay::k_tile + kc * Lay::k_blk + kb * kr * 128, &kmap, kc * 64,
                          (key + rank * Lay::KR + kb * kr) & (page - 1), it.h, kp0, &sm.k_land[st]);
        ++kn;
        st = i % Lay::vs;
        if (!wait_warp(&sm.v_empty[st], ((i / Lay::vs) & 1) ^ 1, abort)) break;
        if (lane == 0) tc::mbar_arrive_tx(&sm.v_land[st], (uint32_t)Lay::v_tile);
        __syncwarp();
        if (lane < nv)
          tc::tma_load_4d(base + Lay::v + st * Lay::v_tile + vc * Lay::v_blk + vb * vr * 128, &vmap,
                          rank * Lay::VC + vc * 64, (key + vb * vr) & (page - 1), it.h, vp0, &sm.v_land[st]);
        ++vn;
      }
      // the last copies land before this warp leaves, whether or not anyone waits for them
      volatile int never = 0;
      for (int x = max(0, kn - Lay::ks); x < kn; ++x)
        tc::mbar_wait(&sm.k_land[x % Lay::ks], (x / Lay::ks) & 1, &never, 400000000LL);
      for (int x = max(0, vn - Lay::vs); x < vn; ++x)
        tc::mbar_wait(&sm.v_land[x % Lay::vs], (x / Lay::vs) & 1, &never, 400000000LL);
    } else if (warp == kKWarp && lane == 0) {
      // ---------------- K tiles handed on ----------------
      for (int i = 0; i < T; ++i) {
        if (!tc::mbar_wait(&sm.k_land[i % Lay::ks], (i / Lay::ks) & 1, abort)) break;
        arrive_issuer<kCta>(&sm.k_full[i % Lay::ks]);
      }
    } else if (warp == kVWarp) {
      // ---------------- V tiles looked into and handed on ----------------
      for (int i = 0; i < T; ++i) {
        const int st = i % Lay::vs, key0 = it.tiles.key(it.part.j0 + i);
        if (!wait_warp(&sm.v_land[st], (i / Lay::vs) & 1, abort)) break;
        if (!it.tiles.all(key0)) {
          uint8_t* tile = base + Lay::v + st * Lay::v_tile;
          bool found = false;
#pragma unroll 1
          for (int x = lane; x < kKT; x += 32) {
            const bool any = it.tiles.any(key0 + x);
#pragma unroll 1
            for (int c = 0; c < Lay::VC / 8; ++c) {
              uint4* p = reinterpret_cast<uint4*>(tile + (c >> 3) * Lay::v_blk + tc::sw128_off(x, c & 7));
              if (!any) {
                *p = make_uint4(0, 0, 0, 0);
                continue;
              }
              found |= paged::take_out(p);
            }
          }
          tc::fence_proxy_async();
          if (__any_sync(0xffffffffu, found) && lane == 0) {
            *(volatile int*)&sm.poison = 1;
            if (kCta == 2) {               // the other CTA's rows see these channels too
              asm volatile(
                  "{\n .reg .b32 p;\n mapa.shared::cluster.u32 p, %0, %1;\n st.shared::cluster.u32 [p], %2;\n}\n" ::"r"(
                      tc::smem_u32(&sm.poison)),
                  "r"(rank ^ 1), "r"(1)
                  : "memory");
              asm volatile("fence.acq_rel.cluster;" ::: "memory");
            }
          }
        }
        __syncwarp();
        if (lane == 0) arrive_issuer<kCta>(&sm.v_full[st]);
      }
    }
    // ---------------- MMA issue (one thread of the pair) ----------------
    if (warp == kMmaWarp && rank == 0 && elect_one()) {
      const uint32_t tmem = sm.tmem_base;
      constexpr uint32_t idesc_qk = tc::idesc_bf16_f32(kRT * kCta, kKT), idesc_pv = tc::idesc_bf16_f32_bmn(kRT * kCta, D);
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
            if (vst[w] >= Lay::vs) vst[w] -= Lay::vs, vph[w] ^= 1;
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
            if (kst[w] >= Lay::ks) kst[w] -= Lay::ks, kph[w] ^= 1;
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
cudaError_t tc_go(const PagedAttnArgs& a, cudaStream_t s) {
  using Lay = Layout<D, C>;
  const int per = 2 * kRT * Lay::kCta;
  const int64_t rt = ((int64_t)a.group * a.max_q + per - 1) / per;
  const int64_t blocks = rt * a.Hkv * a.B * a.splits * Lay::kCta;
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  const int page = 1 << a.pool.page_shift;
  CUtensorMap km, vm;
  if (!make_pool_tmap(&km, a, a.pool.k, D, page < Lay::KR ? page : Lay::KR) || !make_pool_tmap(&vm, a, a.pool.v, D, page))
    return cudaErrorInvalidValue;
  cudaError_t e = opt_in_smem((const void*)paged_attn_tc_kernel<D, C>, (int)Lay::bytes);
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
  e = cudaLaunchKernelEx(&cfg, paged_attn_tc_kernel<D, C>, a, km, vm, (int)rt);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_attn_tc(int d, const PagedAttnArgs& a, bool alone, cudaStream_t s) {
  if (d == 64) return tc_go<64, 1>(a, s);
  return alone ? tc_go<128, 1>(a, s) : tc_go<128, 2>(a, s);
}

}  // namespace fastar
