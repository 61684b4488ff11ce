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
//   warp 17      finds the CTA's work and brings K and V by TMA, a box a lane: a box is a page, or the part of
//                one that a tile has; pages that no row sees, or that are not there, come as zeros (a
//                coordinate past the pool);
//   warp 18      hands K tiles on to the issuing CTA;
//   warp 19      hands V tiles on, and looks into those that not every row sees in full: an infinity or NaN is
//                taken out, since a weight of 0 would not keep it from the rows that do not see its key (of a key
//                that nobody sees, with its row), and returns in the outputs of the rows that do.
// The order of issue is PV0(j) QK0(j+1) PV1(j) QK1(j+1): while the softmax of one row tile
// runs, the tensor cores work for the other, so a logit buffer a tile is enough and two
// accumulators of 128 columns fit TMEM beside them.  Where the rows fill only one row tile, both halves
// of the CTA take it: one the even key tiles, the other the odd ones, and the two results are joined
// in shared memory at the end.
//
// The work is dealt out on the device (paged_tc.cuh): CTAs (pairs) that stay, one a multiprocessor, each with an equal
// share of all the key tiles of all items, in one run; an item that a border between two shares cuts leaves
// partials for a second launch.  While the softmax warps write an item's output, the next one's
// keys, values and queries are on their way.
//
// What bounds it: a key tile is 2048 clocks of MMA a CTA at d = 128 (1.0 us at 2.07 GHz); softmax and its hand-overs make it
// 1.41 us.  Around an item some 8 us: queries to first logits 1.3, last P to complete outputs 1.8, outputs 3.5, which are 16
// warps' instructions as much as bytes.  A tile of one row tile alone waits for K and V: 1.15 us.
// Of the 2850 clocks of a key tile a row tile's softmax takes 1450: its largest logit, and that of the other half's warps,
// 490, exponentials and P 920; then its products are issued, run and reported.  Without the halves' agreement on
// the reference it would be 4 to 8 % less.
// Measured, d = 128: 9728 tokens of 4 heads over 37,440 rows 413 to 430 us (1740 to 1800 TFLOP/s, 0.91 to 0.95 of the bf16 rate
// measured for a library product); 4680 tokens of 12 heads over the same 690 to 704 us in a short run, 760 to 791 in long ones, under
// the power limit; the first 4680 tokens in three frames 90 us; 16,384 causal tokens of 16 heads of 4 with a window of 4096 339 us
// in a short run, 349 to 362 in long ones.  Seven ragged causal sequences of up to 777 tokens, d = 64: 43 us.
//
// Numbers: logits, maxima, sums and outputs are fp32.  P is bf16, as V is (a product has one type):
// 2^-8 of itself, at every magnitude, since bf16 has fp32's exponents.
// Every wait is bounded; a timeout sets FASTAR_DEV_TIMEOUT and unwinds.
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"
#include "paged_attn.h"
#include "paged_tc.cuh"
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

using paged::Item;
using paged::Share;

struct alignas(16) Ctl {
  uint64_t k_land[4], k_full[4], k_empty[4], v_land[4], v_full[4], v_empty[4];
  uint64_t q_full[2], s_full[2], p_full[2][2], fin;    // by row tile (P: first 32 keys of each half, last 32)
  uint64_t item_full[paged::kItems], item_free[paged::kItems];
  Item item[paged::kItems];                            // item x of this CTA in place x % kItems
  // n: infinities or NaN were taken out of the V of the n-th item with key tiles, in place (n - 1) % kItems.  (Not by all
  // items: those without key tiles go by without the other CTA, which may be that far behind and find its mark gone; the
  // tiles of V keep the CTAs of a pair within kItems of one another.)
  int poison[paged::kItems];
  uint32_t tmem_base;
  int abort;
  float ex[2][2][kRT];                                 // a row's two threads: half, row tile, row
  float mx[kRT];
  int see[3][2][2][kRT];                               // what the row sees (kept here: the loop needs the registers)
};

// C CTAs work as one: at d = 64 one, at d = 128 a pair, or one for work of a single row tile (kOne).
// What a CTA holds of a tile: KR keys of K, all 128 keys of V with D / C channels; in blocks of 64
// channels.
template <int D, int C>
struct Layout {
  static constexpr int kCta = C;
  static constexpr bool kOne = D > 64 * C;
  static constexpr int ks = kOne ? 2 : 3, vs = kOne ? 2 : 4;    // tiles of K and of V on their way
  static constexpr int KR = kKT / kCta, VC = D / C;
  static constexpr size_t q_tile = (size_t)kRT * D * 2, q_blk = kRT * 128;
  static constexpr size_t k_tile = (size_t)KR * D * 2, k_blk = KR * 128;
  static constexpr size_t v_tile = (size_t)kKT * VC * 2, v_blk = kKT * 128;
  static constexpr size_t q = 0;
  static constexpr size_t k = q + (kOne ? 1 : 2) * q_tile;
  static constexpr size_t v = k + ks * k_tile;
  static constexpr size_t out = v + vs * v_tile;       // 2 KB a softmax warp
  static constexpr size_t ctl = out + kSoftWarps * 2048;
  static constexpr size_t bytes = ctl + sizeof(Ctl) + 1024;
  static constexpr uint32_t s_col = 0, o_col = 256;   // two 128-column buffers each
  static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
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

// Row r of the sequence's KV head: its token in the sequence and its query head.
struct RowOf {
  int t, head;
};
__device__ __forceinline__ RowOf row_of(const PagedAttnArgs& a, const Item& it, uint32_t r) {
  const uint32_t t = r / (uint32_t)a.group;
  return RowOf{(int)t, it.h * a.group + (int)(r - t * (uint32_t)a.group)};
}
// Byte offset of 16-byte chunk c (0..3) of row `row` among rows of 64 bytes, so that 8 rows hit 8 bank groups.
__device__ __forceinline__ uint32_t out_off(int row, int c) { return (uint32_t)(row * 64 + ((c ^ (row >> 1 & 3)) << 4)); }

// A warp's 32 staged rows to where each goes: rows i * 8 + lane / 4 to to[i] bytes from out (-1: nowhere).
__device__ __forceinline__ void store_rows(uint8_t* out, const int64_t* to, const uint8_t* stg, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 v = *reinterpret_cast<const uint4*>(stg + out_off(i * 8 + (lane >> 2), lane & 3));
    if (to[i] >= 0) *reinterpret_cast<uint4*>(out + to[i] + (lane & 3) * 16) = v;
  }
}

template <int D, int C>
__global__ void __launch_bounds__(kThreadsT, 1)
    paged_attn_tc_kernel(const PagedAttnArgs a, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap) {
  using Lay = Layout<D, C>;
  constexpr int kCta = C, kPer = 2 * kRT * kCta;
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
    for (int i = 0; i < paged::kItems; ++i) {
      tc::mbar_init(&sm.item_full[i], 1);
      tc::mbar_init(&sm.item_free[i], kSoftWarps + 2 + (rank == 0));     // who reads items, but the copy warp
      sm.poison[i] = 0;
    }
    sm.abort = 0;
    tc::mbar_fence_init();
    tc::tma_prefetch_desc(&kmap);
    tc::tma_prefetch_desc(&vmap);
  }
  __syncthreads();
  if (kCta == 2) pair_arrive();                          // this CTA's barriers are ready
  pdl_wait();                            // the launch overlaps the end of the kernel before
  if (a.part_o) pdl_trigger();           // the join's CTAs may come and wait
  volatile int* abort = &sm.abort;
  // Item x of this CTA: null at the end, or after a wait that gave up (`ok` says which).
  auto item_at = [&](int x, bool& ok) -> const Item* {
    ok = wait_warp(&sm.item_full[x % paged::kItems], (x / paged::kItems) & 1, abort);
    const Item* it = &sm.item[x % paged::kItems];
    return ok && it->nt > 0 ? it : nullptr;
  };

  if (warp < kSoftWarps) {
    // ---------------- softmax ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    const int w = warp >> 3, half = (warp >> 2) & 1;      // row tile (or parity of the key tiles), half
    const int row = (warp & 3) * 32 + lane;
    const int pair_bar = 1 + w * 4 + (warp & 3);          // the two warps of these rows
    const int both_bar = 11 + (warp & 3);                 // with those of the other parity
    constexpr int HD = D / 2;                             // channels of a row of O a thread takes
    float sl2 = a.scale * 1.4426950408889634f;
    sl2 = fminf(fmaxf(sl2, 1.2e-38f), 3.0e38f);
    // Query rows: warp x of a row tile brings its rows 16 x .. on, four lanes a row, to where the product
    // wants them; odd rows take the halves of a block's 16-byte chunks the other way round, so that
    // 8 lanes hit 8 bank groups.
    auto bring_q = [&](const Item& it) {
      if (it.nt == 1 && w == 1) return;
      constexpr int QC = D / 32;                          // a lane's chunks of a row
      const int qr = (warp & 7) * 16 + (lane >> 2), qc = (lane & 3) ^ ((lane >> 2 & 1) << 2);
      uint8_t* qd = base + Lay::q + (size_t)w * Lay::q_tile;
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        const uint32_t x = it.r0 + (uint32_t)(w * (kRT * kCta) + rank * kRT + qr + i * 8);
        const RowOf from = row_of(a, it, x < it.rows ? x : it.r0);
        const __nv_bfloat16* src =
            static_cast<const __nv_bfloat16*>(a.q.p) + from.head * a.q.hs + (int64_t)(it.s.t0 + from.t) * a.q.ts;
#pragma unroll
        for (int j = 0; j < QC; ++j)
          tc::cp_async16(tc::smem_u32(qd + (j >> 1) * Lay::q_blk + tc::sw128_off(qr + i * 8, qc ^ ((j & 1) << 2))),
                         src + (j >> 1) * 64 + (qc ^ ((j & 1) << 2)) * 8, x < it.rows ? 16 : 0);
      }
      tc::cp_async_commit();
    };
    auto send_q = [&]() {
      tc::cp_async_wait<0>();
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) arrive_issuer<kCta>(&sm.q_full[w]);
    };
    bool ok = true, q_sent = false;       // the item's queries have been handed over already
    const Item* next = item_at(0, ok);
    if (next && next->T > 0) bring_q(*next);
    tc::named_bar(10, (kSoftWarps + 1) * 32);             // TMEM is there
    tc::tc_fence_after();
    if (kCta == 2) pair_wait();                           // the other CTA's barriers are ready
    const uint32_t tmem = sm.tmem_base;
    const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_addr = lane_addr + Lay::s_col + (uint32_t)(w * 128 + half * 64);
    const uint32_t o_addr = lane_addr + Lay::o_col + (uint32_t)(w * 128 + half * HD);
    uint32_t seen = 0, done = 0;                          // logit tiles of this row tile, items with tiles, so far
#pragma unroll 1
    for (int x = 0; next; ++x) {
      const Item& it = *next;
      const int T = it.T;
      const bool partial = it.slot >= 0, both = it.nt == 1;   // both: one row tile, even key tiles and odd key tiles
      const bool mine = !(both && w == 1);
      {
        const uint32_t r = it.r0 + (both ? 0u : (uint32_t)(w * (kRT * kCta))) + (uint32_t)(rank * kRT + row);
        const paged::Sees see = paged::sees(a, it.s, row_of(a, it, min(r, it.rows - 1)).t);
        sm.see[0][half][w][row] = see.lo;
        sm.see[1][half][w][row] = see.hi;
        sm.see[2][half][w][row] = see.sk;
      }
      const int step = both ? 2 : 1, count = both ? (T - w + 1) >> 1 : T;      // this row tile's key tiles
      if (mine && T > 0 && !q_sent) send_q();
      q_sent = false;
      float m = neg_inf(), l0 = 0.f, l1 = 0.f;      // m: the reference, in log2 units; -inf: no key seen yet
      int j = it.j0 + (both ? w : 0);
#pragma unroll 1
      for (int i = 0; i < count; ++i, j += step) {
        const int key0 = it.tiles.key(j);
        const bool cut = !it.tiles.all(key0);
        uint32_t bits[2];
        if (cut) {
          const paged::Sees see{sm.see[0][half][w][row], sm.see[1][half][w][row], sm.see[2][half][w][row]};
          bits[0] = paged::seen32(see, key0 + half * 64);
          bits[1] = paged::seen32(see, key0 + half * 64 + 32);
        }
        const bool alive = wait_warp(&sm.s_full[w], (seen + i) & 1, abort);
        tc::tc_fence_after();
        float x[64];
        tc::tmem_ld32(s_addr, x);
        tc::tmem_ld32(s_addr + 32, x + 32);
        tc::tmem_wait_ld();
        tc::tmem_pin32(x);
        tc::tmem_pin32(x + 32);
        if (__builtin_expect(cut, 0)) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (!__all_sync(0xffffffffu, bits[k] == 0xffffffffu)) {
#pragma unroll
              for (int c = 0; c < 32; ++c) x[32 * k + c] = bits[k] >> c & 1 ? x[32 * k + c] : neg_inf();
            }
        }
        const float top = row_max<64>(x);         // the largest of them, not scaled yet
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
        // P over the logits' own columns: 32 logits become 16 columns
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          row_exp32(x + 32 * c, sl2, nm, s_addr + (uint32_t)(16 * c), l0, l1);
          tc::tmem_wait_st();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_issuer<kCta>(&sm.p_full[w][c]);
        }
      }
      seen += (uint32_t)count;
      // The next item's queries: this row tile's place is free once its last logits are there (both: once those
      // of both halves are), so that the next item's first product follows this one's last.
      bool more;
      next = item_at(x + 1, more);
      const bool early = !both && count > 0 && next && next->T > 0 && ok;
      if (early) bring_q(*next);
      if (T > 0) {
        ok = ok && wait_warp(&sm.fin, done & 1, abort);
        ++done;
        tc::tc_fence_after();
      }
      ok = ok && more;
      if (early) {
        if (!(next->nt == 1 && w == 1)) send_q();
        q_sent = true;
      }
      // a group of warps that exchange results leaves together
      float l = l0 + l1;
      // (nothing where this row tile has no key tile: the other half may still be reading the sums of the item before,
      // and no barrier of the loop has come since)
      if (count > 0) sm.ex[half][w][row] = l;
      if (both && w == 1 && half == 0) sm.mx[row] = m;
      if (!(both ? tc::named_bar_and(both_bar, 128, ok) : tc::named_bar_and(pair_bar, 64, ok))) {
        ok = false;
        break;
      }
      if (!early && next && next->T > 0) bring_q(*next);
      if (count > 0) l += sm.ex[half ^ 1][w][row];
      float f0 = 1.f, f1 = 0.f;             // weights of this sum and of the odd tiles'
      if (mine && both && T > 1) {
        const float lo = sm.ex[0][1][row] + sm.ex[1][1][row], mo = sm.mx[row];
        if (lo != 0.f) {                    // the odd tiles hold a key that the row sees
          const float mn = fmaxf(m, mo);
          f0 = ex2f(m - mn);
          f1 = ex2f(mo - mn);
          l = l * f0 + lo * f1;
          m = mn;
        }
      }
      const uint32_t i0 = (both ? 0u : (uint32_t)(w * (kRT * kCta))) + (uint32_t)(rank * kRT + row);
      const bool has = it.r0 + i0 < it.rows;
      const RowOf at = row_of(a, it, has ? it.r0 + i0 : it.rows - 1);    // a row that is not there: as the last
      const bool live = l > 0.f || l != l;
      const bool poison = T > 0 && *(volatile int*)&sm.poison[(done - 1) % paged::kItems] == (int)done;
      const float f = live ? 1.f / l : 0.f;
      // Rows of 64 bytes (32 channels) go through shared memory, so that they leave as whole runs
      uint8_t* stg = base + Lay::out + warp * 2048;
      const uint8_t* odd = base + Lay::out + (warp + 8) * 2048;        // (both) the odd tiles' 16 channels
      const int64_t tok = it.s.t0 + at.t;
      const int64_t off = has ? (at.head * a.o_hs + tok * a.o_ts + half * HD) * 2 : -1;
      int64_t to[4];                        // of the rows that this lane stores a part of
#pragma unroll
      for (int i = 0; i < 4; ++i) to[i] = __shfl_sync(0xffffffffu, off, i * 8 + (lane >> 2));
#pragma unroll                              // (as a loop the whole kernel was 1 % slower: its registers were dealt out differently)
      for (int c = 0; c < HD; c += 32) {
        float o[32];
        if (count > 0) {
          tc::tmem_ld32(o_addr + (uint32_t)c, o);
          tc::tmem_wait_ld();
          tc::tmem_pin32(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
        if (both) {                         // the odd tiles' part: 16 channels at a time through its warp's place
#pragma unroll
          for (int d = 0; d < 32; d += 16) {
            if (w == 1) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                *reinterpret_cast<float4*>(stg + out_off(lane, e)) =
                    make_float4(o[d + 4 * e], o[d + 4 * e + 1], o[d + 4 * e + 2], o[d + 4 * e + 3]);
            }
            tc::named_bar(both_bar, 128);
            if (w == 0 && f1 != 0.f) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float4 v = *reinterpret_cast<const float4*>(odd + out_off(lane, e));
                o[d + 4 * e] = o[d + 4 * e] * f0 + v.x * f1;
                o[d + 4 * e + 1] = o[d + 4 * e + 1] * f0 + v.y * f1;
                o[d + 4 * e + 2] = o[d + 4 * e + 2] * f0 + v.z * f1;
                o[d + 4 * e + 3] = o[d + 4 * e + 3] * f0 + v.w * f1;
              }
            }
            tc::named_bar(both_bar, 128);
          }
          if (w == 1) continue;
        }
        if (__builtin_expect(poison, 0)) {
          const paged::Split part{1, it.j0, it.j0 + it.T};
          const paged::Sees see{sm.see[0][half][w][row], sm.see[1][half][w][row], sm.see[2][half][w][row]};
#pragma unroll
          for (int d = 0; d < 32; d += 16) {
            float q[16];                    // a copy: o's registers keep no address
#pragma unroll
            for (int e = 0; e < 16; ++e) q[e] = o[d + e];
            paged::add_taken_out<kKT, 16>(a, it.tiles, part, it.b, it.h, see, half * HD + c + d, q);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[d + e] = q[e];
          }
        }
        if (partial) {                      // four channels of 32 rows side by side: whole runs as they are
          float4* p = reinterpret_cast<float4*>(a.part_o) + ((int64_t)it.slot * (D / 4) + (half * HD + c) / 4) * kPer + i0;
          if (has) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              p[(int64_t)e * kPer] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        } else {
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              v[k] = live ? pack_bf16(o[8 * e + 2 * k] * f, o[8 * e + 2 * k + 1] * f) : 0u;
            *reinterpret_cast<uint4*>(stg + out_off(lane, e)) = make_uint4(v[0], v[1], v[2], v[3]);
          }
          __syncwarp();
          store_rows(static_cast<uint8_t*>(a.out) + c * 2, to, stg, lane);
        }
      }
      tc::tc_fence_before();                // O has been read: the next item's products, which this warp's P let go
      if (has && half == 0 && mine) {
        const float mn = m * 0.6931471805599453f;
        if (partial)
          a.part_ml[(int64_t)it.slot * kPer + i0] = make_float2(live ? mn : neg_inf(), l);
        else if (a.lse)
          a.lse[at.head * a.T + tok] = live ? mn + logf(l) : neg_inf();
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.item_free[x % paged::kItems]);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == kMmaWarp) {
      tmem_alloc512<kCta>(&sm.tmem_base);
      tc::tc_fence_before();
      tc::named_bar(10, (kSoftWarps + 1) * 32);
      tc::tc_fence_after();
    }
    if (warp != kCopyWarp && kCta == 2) pair_wait();
    if (warp == kCopyWarp) {
      // ---------------- the work, and K and V into shared memory ----------------
      Share share;
      paged::find_share(a, share, (int)blockIdx.x / kCta, kPer);
      const int shift = a.pool.page_shift, page = 1 << shift;
      const int kr = min(page, Lay::KR), vr = min(page, kKT);      // rows of a box
      const int nk = Lay::KR / kr * (D / 64), nv = kKT / vr * (Lay::VC / 64);
      const int none = (int)a.pool.pages;                          // past the pool: the box comes as zeros
      const int kb = lane / (D / 64), kc = lane % (D / 64);        // this lane's box: rows, channels
      const int vb = lane / (Lay::VC / 64), vc = lane % (Lay::VC / 64);
      int kn = 0, vn = 0;                                          // tiles asked for
      bool ok = true;
      // what the join needs of the first item; not before its first tiles are asked for
      auto cut_known = [&](const Item& it) {
        if (rank == 0 && a.part_o) paged::write_cut(share, it, static_cast<paged::Cut*>(a.cuts) + share.p, kPer);
      };
#pragma unroll 1
      for (int x = 0; ok; ++x) {
        Item it;
        paged::next_item(a, share, it, kPer);
        if (!(ok = wait_warp(&sm.item_free[x % paged::kItems], ((x / paged::kItems) & 1) ^ 1, abort))) {
          if (x == 0) cut_known(it);
          break;
        }
        if (lane == 0) {
          sm.item[x % paged::kItems] = it;
          tc::mbar_arrive(&sm.item_full[x % paged::kItems]);
        }
        __syncwarp();
        if (it.nt == 0) {
          if (x == 0) cut_known(it);
          break;
        }
        const int32_t* table = a.table + (int64_t)it.b * a.max_pages;
        auto page_at = [&](int key, int n) {
          if (!it.tiles.any(key, key + n)) return none;
          const int y = paged::page_of(table, key >> shift, a.pool.pages, a.status);
          return y < 0 ? none : y;
        };
        // the pages of a tile are looked up while the one before is asked for
        int kp = none, vp = none;
        auto look = [&](int i) {
          const int key = it.tiles.key(it.j0 + i);
          if (lane < nk) kp = page_at(key + rank * Lay::KR + kb * kr, kr);
          if (lane < nv) vp = page_at(key + vb * vr, vr);
        };
        if (it.T > 0) look(0);
#pragma unroll 1
        for (int i = 0; i < it.T; ++i) {
          const int key = it.tiles.key(it.j0 + i);
          const int kp0 = kp, vp0 = vp;
          if (i + 1 < it.T) look(i + 1);
          int st = kn % Lay::ks;
          if (!(ok = wait_warp(&sm.k_empty[st], ((kn / Lay::ks) & 1) ^ 1, abort))) break;
          if (lane == 0) tc::mbar_arrive_tx(&sm.k_land[st], (uint32_t)Lay::k_tile);
          __syncwarp();
          if (lane < nk)
            tc::tma_load_4d(base + Lay::k + st * Lay::k_tile + kc * Lay::k_blk + kb * kr * 128, &kmap, kc * 64,
                            (key + rank * Lay::KR + kb * kr) & (page - 1), it.h, kp0, &sm.k_land[st]);
          ++kn;
          st = vn % Lay::vs;
          if (!(ok = wait_warp(&sm.v_empty[st], ((vn / Lay::vs) & 1) ^ 1, abort))) break;
          if (lane == 0) tc::mbar_arrive_tx(&sm.v_land[st], (uint32_t)Lay::v_tile);
          __syncwarp();
          if (lane < nv)
            tc::tma_load_4d(base + Lay::v + st * Lay::v_tile + vc * Lay::v_blk + vb * vr * 128, &vmap,
                            rank * Lay::VC + vc * 64, (key + vb * vr) & (page - 1), it.h, vp0, &sm.v_land[st]);
          ++vn;
          if (x == 0 && i == 0) cut_known(it);
        }
        if (x == 0 && vn == 0) cut_known(it);                      // no tile, or a wait that gave up
      }
      if (kCta == 2) pair_wait();
      // the last copies land before this warp leaves, whether or not anyone waits for them
      volatile int never = 0;
      for (int y = max(0, kn - Lay::ks); y < kn; ++y)
        tc::mbar_wait(&sm.k_land[y % Lay::ks], (y / Lay::ks) & 1, &never, 400000000LL);
      for (int y = max(0, vn - Lay::vs); y < vn; ++y)
        tc::mbar_wait(&sm.v_land[y % Lay::vs], (y / Lay::vs) & 1, &never, 400000000LL);
    } else if (warp == kKWarp) {
      // ---------------- K tiles handed on ----------------
      bool ok;
      int n = 0;
      for (int x = 0; const Item* it = item_at(x, ok); ++x) {
        const int end = n + it->T;
        for (; n < end && (ok = wait_warp(&sm.k_land[n % Lay::ks], (n / Lay::ks) & 1, abort)); ++n)
          if (lane == 0) arrive_issuer<kCta>(&sm.k_full[n % Lay::ks]);
        if (!ok) break;
        if (lane == 0) tc::mbar_arrive(&sm.item_free[x % paged::kItems]);
      }
    } else if (warp == kVWarp) {
      // ---------------- V tiles looked into and handed on ----------------
      bool ok;
      int n = 0, nth = 0;                                   // tiles, items with tiles so far, this one among them
      for (int x = 0; const Item* item = item_at(x, ok); ++x) {
        const Item& it = *item;
        nth += it.T > 0;
        for (int i = 0; i < it.T; ++i, ++n) {
          const int st = n % Lay::vs, key0 = it.tiles.key(it.j0 + i);
          if (!(ok = wait_warp(&sm.v_land[st], (n / Lay::vs) & 1, abort))) break;
          if (!it.tiles.all(key0)) {
            uint8_t* tile = base + Lay::v + st * Lay::v_tile;
            // 8 chunks of 8 channels of a row on their way at once
            uint32_t big = 0;
#pragma unroll 1
            for (int r = lane; r < kKT * (Lay::VC / 64); r += 32) {
              const uint8_t* line = tile + (r >> 7) * Lay::v_blk;
              uint4 u[8];
#pragma unroll
              for (int c = 0; c < 8; ++c) u[c] = *reinterpret_cast<const uint4*>(line + tc::sw128_off(r & 127, c));
#pragma unroll
              for (int c = 0; c < 8; ++c)
                big = __vmaxu2(big, __vmaxu2(__vmaxu2(u[c].x & 0x7fff7fffu, u[c].y & 0x7fff7fffu),
                                             __vmaxu2(u[c].z & 0x7fff7fffu, u[c].w & 0x7fff7fffu)));
            }
            bool found = false;
            if (__any_sync(0xffffffffu, (big & 0xffffu) >= 0x7f80u || (big >> 16) >= 0x7f80u)) {
#pragma unroll 1
              for (int r = lane; r < kKT; r += 32) {
                const bool any = it.tiles.any(key0 + r);
#pragma unroll 1
                for (int c = 0; c < Lay::VC / 8; ++c) {
                  uint4* p = reinterpret_cast<uint4*>(tile + (c >> 3) * Lay::v_blk + tc::sw128_off(r, c & 7));
                  if (any) found |= paged::take_out(p);
                  else *p = make_uint4(0, 0, 0, 0);
                }
              }
            }
            tc::fence_proxy_async();
            if (__any_sync(0xffffffffu, found) && lane == 0) {
              int* mark = &sm.poison[(nth - 1) % paged::kItems];
              *(volatile int*)mark = nth;
              if (kCta == 2) {               // the other CTA's rows see these channels too
                asm volatile(
                    "{\n .reg .b32 p;\n mapa.shared::cluster.u32 p, %0, %1;\n st.shared::cluster.u32 [p], %2;\n}\n" ::"r"(
                        tc::smem_u32(mark)),
                    "r"(rank ^ 1), "r"(nth)
                    : "memory");
                asm volatile("fence.acq_rel.cluster;" ::: "memory");
              }
            }
          }
          __syncwarp();
          if (lane == 0) arrive_issuer<kCta>(&sm.v_full[st]);
        }
        if (!ok) break;
        if (lane == 0) tc::mbar_arrive(&sm.item_free[x % paged::kItems]);
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
      uint32_t tiles = 0, qn[2] = {0, 0}, pn[2] = {0, 0};  // key tiles, query and P tiles by row tile, so far
      uint32_t items = 0;
#pragma unroll 1
      for (int x = 0; ok; ++x) {
        ok = tc::mbar_wait(&sm.item_full[x % paged::kItems], (x / paged::kItems) & 1, abort);
        if (!ok || sm.item[x % paged::kItems].nt == 0) break;
        const int T = sm.item[x % paged::kItems].T;
        const bool both = sm.item[x % paged::kItems].nt == 1;
        tc::mbar_arrive(&sm.item_free[x % paged::kItems]);     // all that is read of it
        if (T == 0) continue;
        const int step = both ? 2 : 1;
        int kst[2], vst[2], count[2];                     // stages of K and V, key tiles by row tile
        uint32_t kph[2], vph[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t first = tiles + (both ? w : 0);
          kst[w] = (int)(first % Lay::ks), kph[w] = first / Lay::ks & 1;
          vst[w] = (int)(first % Lay::vs), vph[w] = first / Lay::vs & 1;
          count[w] = both ? (T - w + 1) >> 1 : T;
        }
#pragma unroll 1
        for (int i = -1; i < count[0] && ok; ++i) {       // P V of tile i (from 0 on), Q K^T of tile i + 1
#pragma unroll
          for (int w = 0; w < 2; ++w) {                   // unrolled: columns are constants
            if (i >= 0 && i < count[w]) {
              ok = tc::mbar_wait(&sm.v_full[vst[w]], vph[w], abort);
              if (!ok) break;
              const uint64_t vd = v_desc + ((vst[w] * Lay::v_tile) >> 4);
#pragma unroll
              for (int c = 0; c < 2; ++c) {               // 32 keys of both halves at a time, as their P lands
                ok = tc::mbar_wait(&sm.p_full[w][c], (pn[w] + i) & 1, abort);
                if (!ok) break;
                tc::tc_fence_after();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const int key = (k >> 1) * 64 + c * 32 + (k & 1) * 16;
                  mma_ts<kCta>(tmem + Lay::o_col + w * 128,
                               tmem + Lay::s_col + w * 128 + (k >> 1) * 64 + c * 16 + (k & 1) * 8, vd + ((key * 128) >> 4),
                               idesc_pv, i > 0 || c > 0 || k > 0 ? 1u : 0u);
                }
              }
              if (!ok) break;
              if (w == 1 || both) commit<kCta>(&sm.v_empty[vst[w]]);
              vst[w] += step;
              if (vst[w] >= Lay::vs) vst[w] -= Lay::vs, vph[w] ^= 1;
            }
            if (i + 1 < count[w]) {
              ok = (i >= 0 || (both && w == 1) || tc::mbar_wait(&sm.q_full[w], qn[w] & 1, abort)) &&
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
        if (!ok) break;
        commit<kCta>(&sm.fin);                            // the item's outputs are complete
        ++items;
        tiles += (uint32_t)T;
        ++qn[0];
        if (!both) ++qn[1];
        pn[0] += (uint32_t)count[0], pn[1] += (uint32_t)count[1];
      }
      // every issued product ends before TMEM is given back
      if (!ok) {
        commit<kCta>(&sm.fin);
        volatile int never = 0;
        tc::mbar_wait(&sm.fin, items & 1, &never, 400000000LL);
      }
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

// ---- joining cut items -----------------------------------------------------------------------
// O = sum_s e^(m_s - m) o_s / sum_s e^(m_s - m) l_s over the parts of an item, m = max_s m_s, in the order of the
// keys.  A warp takes 32 rows and 32 channels, a row a lane (as the partials lie); the outputs go through shared
// memory.  Bound: latency; the maxima, sums and outputs of two parts set out together.
template <int D>
__global__ void __launch_bounds__(256) paged_tc_join_kernel(const PagedAttnArgs a, int per) {
  __shared__ __align__(16) uint8_t stage[8 * 2048];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  const paged::Cut& cut = static_cast<const paged::Cut*>(a.cuts)[blockIdx.x];
  const int n = cut.parts, x = blockIdx.y * 8 + warp;       // (rows, channels) of the item
  const int c = x % (D / 32) * 32, i = x / (D / 32) * 32 + lane;
  const uint32_t r0 = cut.r0, rows = cut.rows;
  const int t0 = cut.t0, h = cut.h;
  // (what another call wrote over the entries, against the rules, leads to wrong outputs, but to no address outside
  // the call's)
  if (n <= 0 || n > a.shares || (uint32_t)h >= (uint32_t)a.Hkv || t0 < 0 || r0 + (uint32_t)(i - lane) >= rows ||
      (int64_t)t0 + (rows - 1) / (uint32_t)a.group >= a.T)
    return;
  const bool has = r0 + (uint32_t)i < rows;
  float m = neg_inf(), l = 0.f, o[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) o[e] = 0.f;
#pragma unroll 1
  for (int s = n - 1; s >= 0; --s) {                        // the parts are listed from the last on
    const int64_t slot = min((uint32_t)cut.slots[s], 2 * (uint32_t)a.shares - 1);
    const float4* p = reinterpret_cast<const float4*>(a.part_o) + (slot * (D / 4) + c / 4) * per + i;
    float2 ml = make_float2(neg_inf(), 0.f);
    float4 v[8];
    if (has) {
      ml = a.part_ml[slot * per + i];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = p[(int64_t)e * per];
    }
    if (ml.y == 0.f) continue;
    const float top = fmaxf(m, ml.x), ref = top == neg_inf() ? 0.f : top, f = expf(m - ref), w = expf(ml.x - ref);
    m = top;
    l = fmaf(w, ml.y, l * f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      o[4 * e] = fmaf(w, v[e].x, o[4 * e] * f), o[4 * e + 1] = fmaf(w, v[e].y, o[4 * e + 1] * f);
      o[4 * e + 2] = fmaf(w, v[e].z, o[4 * e + 2] * f), o[4 * e + 3] = fmaf(w, v[e].w, o[4 * e + 3] * f);
    }
  }
  const bool live = l > 0.f || l != l;
  const float f = live ? 1.f / l : 0.f;
  const uint32_t r = has ? r0 + (uint32_t)i : rows - 1, t = r / (uint32_t)a.group;
  const int64_t tok = t0 + (int)t, head = h * a.group + (int)(r - t * (uint32_t)a.group);
  uint8_t* stg = stage + warp * 2048;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = live ? pack_bf16(o[8 * e + 2 * k] * f, o[8 * e + 2 * k + 1] * f) : 0u;
    *reinterpret_cast<uint4*>(stg + out_off(lane, e)) = make_uint4(y[0], y[1], y[2], y[3]);
  }
  __syncwarp();
  const int64_t off = has ? (head * a.o_hs + tok * a.o_ts) * 2 : -1;
  int64_t to[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) to[k] = __shfl_sync(0xffffffffu, off, k * 8 + (lane >> 2));
  store_rows(static_cast<uint8_t*>(a.out) + c * 2, to, stg, lane);
  if (has && c == 0 && a.lse) a.lse[head * a.T + tok] = live ? m + logf(l) : neg_inf();
}

template <int D, int C>
cudaError_t tc_go(const PagedAttnArgs& a, cudaStream_t s) {
  using Lay = Layout<D, C>;
  constexpr int per = 2 * kRT * Lay::kCta;
  const int page = 1 << a.pool.page_shift;
  CUtensorMap km, vm;
  if (!make_pool_tmap(&km, a, a.pool.k, D, page < Lay::KR ? page : Lay::KR) || !make_pool_tmap(&vm, a, a.pool.v, D, page))
    return cudaErrorInvalidValue;
  cudaError_t e = opt_in_smem((const void*)paged_attn_tc_kernel<D, C>, (int)Lay::bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.shares * Lay::kCta));
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
  e = cudaLaunchKernelEx(&cfg, paged_attn_tc_kernel<D, C>, a, km, vm);
  count_launches(1);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess || !a.part_o) return e;
  e = launch_dependent(paged_tc_join_kernel<D>, dim3((unsigned)a.shares, per / 32 * (D / 32) / 8), dim3(256), 0, s, a, per);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

int paged_tc_rows(int d, bool alone) { return d == 128 && !alone ? 512 : 256; }
size_t paged_tc_cut_bytes() { return sizeof(paged::Cut); }

cudaError_t launch_paged_attn_tc(int d, const PagedAttnArgs& a, bool alone, cudaStream_t s) {
  if (d == 64) return tc_go<64, 1>(a, s);
  return alone ? tc_go<128, 1>(a, s) : tc_go<128, 2>(a, s);
}

}  // namespace fastar
