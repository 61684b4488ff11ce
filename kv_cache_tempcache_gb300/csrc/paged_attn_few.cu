// Softmax attention over a paged cache for few rows, as in single-token steps (bf16): up to 32 (token, query
// head) pairs of a KV head.
//
// Bound: the cache's bytes.  A row tile of the tcgen05 kernel is 128 rows, so with a few it waits from
// product to product; here the rows are the 8 columns (up to four times) of m16n8k16 products
// (mma.sync: its rate is not what bounds this), and each warp runs alone over its share of the
// block's key tiles of 16 rows, several of them on their way by TMA, with its own reference, sums and
// outputs:
//   S^T[16 keys, 8 rows] += K[16, 16 channels] Q^T,   O^T[16 channels, 8 rows] += V^T[16, 16 keys] P^T
// K comes by ldmatrix, V^T by its transposing form, P^T is S^T's registers after an 8 x 8 transpose
// (movmatrix).  A tile lies in one page (pages have 16 rows or more), so a warp needs one table entry a
// tile; it holds 32 of them, a lane each, and asks for the next 32 while it works on these.  The warps'
// results are joined in shared memory, in warp order, at the end, and the blocks' by the join kernel.
// (With the rows moved by cp.async, 16 bytes a lane, 250 of 665 instructions a tile at 32 rows were theirs.)
// Rows of V that no token sees become zeros in shared memory; pages that no token sees, or that are not there,
// come as zeros.
// Measured: one token each of 32 sequences, 32 heads of 8, 8191 + 100 rows 147 to 149 us a call (6.4 TB/s, 0.95 of the measured copy rate); up
// to 28 rows over six sequences of up to 40,000 rows 89 us (5.1 TB/s); one token over 333 rows 6.7 us, a block's start, five
// tiles a warp and the join of its warps, one after the other.
// P is bf16, as V is, or two of them (kSplitGroups): 2^-8 or 2^-15 of itself at every magnitude.  The reference moves only when
// a P would pass 2^kTop.
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

constexpr int kKeys = 16;
constexpr float kTop = 8.f;
// Groups of 8 rows up to which P is two bf16 (2^-15 of itself) and P V two products.  With one bf16 a token's output was up to
// 1.53 times as far from the exact one as fp32 weights leave it after its own rounding to bf16 (12 heads, 333 rows), with
// two 1.00.  The second product is 0 to 0.8 % of a call's time with one group or two (32 sequences of one token 148.6 -> 149.2
// us, 12 rows over six sequences 92.7 -> 93.8), where the bytes are what bounds it; with four 10 % (28 rows 90.0 -> 99.5), for
// outputs that are 1.1 to 1.3 times as far off.
constexpr int kSplitGroups = 2;

// NR: groups of 8 rows.
template <int D, int NR, int W>
struct FewLayout {
  static constexpr int tile = kKeys * D * 2, stage = 2 * tile;      // K, V
  static constexpr int stages = D == 64 ? 6 : 3;
  static constexpr int ring = W * stages * stage;
  static constexpr int ldo = D + 4;                                 // an output row: lanes of 4 rows hit other banks
  static constexpr int red = W * 8 * NR * ldo * 4;                  // the warps' outputs, over the ring
  static constexpr int ctl = ring > red ? ring : red;
  static constexpr int bar = ctl + W * 8 * NR * 8 + 16;
  static constexpr int bytes = bar + W * stages * 8 + 1024;
};

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c = a b
__device__ __forceinline__ void mma16816_first(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, "
      "%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Lane (g, t) holds elements (g, 2t), (g, 2t + 1) of an 8 x 8 matrix of 16-bit values; gets (2t, g), (2t + 1, g).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// Weights as two bf16: their upper halves, and what those leave out.  Nothing but a weight of 0 leaves 0, so that an infinity
// of V stays one.
__device__ __forceinline__ uint32_t upper2(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float left_out(float a) {
  return fmaxf(a - __uint_as_float(__float_as_uint(a) & 0xffff0000u), fminf(a, 0x1p-126f));
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

template <int D, int NR, int W>
__global__ void __launch_bounds__(W * 32)
    paged_attn_few_kernel(const PagedAttnArgs a, const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap) {
  using Lay = FewLayout<D, NR, W>;
  constexpr bool kSplit = NR <= kSplitGroups;             // weights as two bf16
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  float2* sml = reinterpret_cast<float2*>(smem + Lay::ctl);        // [W][8 NR] references and sums
  int* poison = reinterpret_cast<int*>(smem + Lay::ctl + W * 8 * NR * 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (threadIdx.x == 0) {
    tc::tma_prefetch_desc(&kmap);
    tc::tma_prefetch_desc(&vmap);
  }
  pdl_wait();                              // the launch overlaps the end of the kernel before
  if (a.extra > 0) pdl_trigger();          // the join's CTAs may come, find their work and wait
  // heads side by side, then slots
  paged::Work work;
  const int slot = (int)(blockIdx.x / (uint32_t)a.Hkv), h = (int)(blockIdx.x - (uint32_t)slot * (uint32_t)a.Hkv);
  if (!paged::find_work<kKeys>(a, slot, 0, work)) return;
  const int b = work.b;
  const paged::Seq s = paged::sequence(a.cu, a.at, a.B, a.T, a.cap, b, a.status);
  if (s.nq > a.max_q && threadIdx.x == 0) flag_status(a.status, FASTAR_DEV_BAD_LEN);
  const int G = a.group, rows = G * min(s.nq, a.max_q);            // at most 8 NR
  if (rows == 0) return;
  paged::Tiles<kKeys> tiles;
  tiles.set(a, s, 0, (rows - 1) / G);
  const paged::Split part = paged::part_of(tiles.n, work);
  const bool partial = part.used > 1;
  if (threadIdx.x == 0) *poison = 0;
  const int32_t* table = a.table + (int64_t)b * a.max_pages;
  const int shift = a.pool.page_shift;
  // this warp's tiles: j0 + warp, + W, ...; the pages of 32 of them, a lane each
  const int count = part.j1 - part.j0 > warp ? (part.j1 - part.j0 - warp + W - 1) / W : 0;
  auto pages_from = [&](int i) {
    i += lane;
    return i < count ? paged::page_of(table, tiles.key(part.j0 + warp + W * i) >> shift, a.pool.pages, a.status) : -1;
  };
  int pages = pages_from(0), next = pages_from(32);
  // tile i into its stage, in boxes of 16 rows and 64 channels
  constexpr int NB = D / 64;
  uint8_t* ring = smem + warp * Lay::stages * Lay::stage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::bar) + warp * Lay::stages;
  if (lane == 0) {
    for (int i = 0; i < Lay::stages; ++i) tc::mbar_init(&bars[i], 1);
    tc::mbar_fence_init();
  }
  __syncwarp();
  int asked = 0, to = 0;
  auto ask = [&]() {
    if (asked >= count) return;
    const int key0 = tiles.key(part.j0 + warp + W * asked);
    const int page = __shfl_sync(0xffffffffu, pages, asked & 31);
    if (elect_one()) {
      tc::mbar_arrive_tx(&bars[to], Lay::stage);
      const int row = key0 & ((1 << shift) - 1), pg = page < 0 ? (int)a.pool.pages : page;
#pragma unroll
      for (int c = 0; c < 2 * NB; ++c)
        tc::tma_load_4d(ring + to * Lay::stage + c * (kKeys * 128), c < NB ? &kmap : &vmap, (c & (NB - 1)) * 64, row, h, pg,
                        &bars[to]);
    }
    __syncwarp();
    if ((++asked & 31) == 0) {
      pages = next;
      next = pages_from(asked + 32);
    }
    if (++to == Lay::stages) to = 0;
  };
#pragma unroll 1
  for (int i = 0; i < Lay::stages - 1; ++i) ask();
  __syncthreads();                                       // poison is set up
  // query rows: lane (g, t) holds channels 2t, 2t + 1 and 8 + 2t, 9 + 2t of each 16 of row 8 n + g.  One group's come as they
  // are held, four bytes of eight rows at a time (one token over 333 rows 6.7 us, through a stage 7.0); more groups' by
  // whole rows, through the stage that is not asked for yet (28 rows over six sequences of 1800 25.6 us, as they are held 27.0:
  // each load looks up eight lines)
  uint32_t qb[NR][D / 16][2];
  int tok[NR][2];                                        // tokens of the rows 8 n + 2t, 8 n + 2t + 1
  const uint32_t inv = 65536u / (uint32_t)G + 1;         // r / G of r < 32, G <= 32
  auto token = [&](int r) { return (int)((uint32_t)r * inv >> 16); };
  if (NR == 1) {
    const int tk = token(g);
    const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q.p) +
                                                            (int64_t)(h * G + g - tk * G) * a.q.hs + (int64_t)(s.t0 + tk) * a.q.ts);
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      qb[0][c][0] = g < rows ? src[c * 8 + t] : 0u;
      qb[0][c][1] = g < rows ? src[c * 8 + 4 + t] : 0u;
    }
  } else {
    static_assert(8 * NR * D * 2 <= Lay::stage, "rows that fit a stage");
    constexpr int CH = D / 8, QL = NR * D / 32;          // chunks of a row, of a lane
    uint8_t* qs = ring + (Lay::stages - 1) * Lay::stage;
    uint4 u[QL];
#pragma unroll
    for (int k = 0; k < QL; ++k) {
      const int r = (lane + 32 * k) / CH, tk = token(r);
      u[k] = make_uint4(0, 0, 0, 0);
      if (r < rows)
        u[k] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q.p) + (int64_t)(h * G + r - tk * G) * a.q.hs +
                                               (int64_t)(s.t0 + tk) * a.q.ts + lane % CH * 8);
    }
#pragma unroll
    for (int k = 0; k < QL; ++k) {
      const int r = (lane + 32 * k) / CH;
      *reinterpret_cast<uint4*>(qs + r * (2 * D) + ((lane % CH ^ (r & 7)) << 4)) = u[k];
    }
    __syncwarp();
#pragma unroll
    for (int n = 0; n < NR; ++n) {
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          qb[n][c][e] = *reinterpret_cast<const uint32_t*>(qs + (8 * n + g) * (2 * D) + (((2 * c + e) ^ g) << 4) + t * 4);
    }
    tc::fence_proxy_async();                             // the stage is written by TMA next
    __syncwarp();
  }
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) tok[n][e] = token(min(8 * n + 2 * t + e, rows - 1));
  float sl2 = a.scale * 1.4426950408889634f;
  sl2 = fminf(fmaxf(sl2, 1.2e-38f), 3.0e38f);
  // minus the references, in log2 units; 0 while a row has seen no key (isset, a bit a row)
  float nm[NR][2], l[NR][2], o[NR][D / 16][4];
  uint32_t isset = 0;
  bool all_set = false;
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    nm[n][0] = nm[n][1] = 0.f;
    l[n][0] = l[n][1] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][c][e] = 0.f;
  }
  // ldmatrix addresses in a tile, by 16 channels mod 64: rows keys 0-15, chunks 0 and 1 of K; V transposed
  uint32_t ldk[4], ldv[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    ldk[c] = tc::smem_u32(ring) + tc::sw128_off(lane & 15, 2 * c + (lane >> 4));
    ldv[c] = tc::smem_u32(ring) + Lay::tile + tc::sw128_off((lane & 7) + ((lane >> 4) << 3), 2 * c + (lane >> 3 & 1));
  }
  volatile int never = 0;
  bool ok = true;
  int st = 0;
  uint32_t ph = 0;
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    ask();
    ok = __all_sync(0xffffffffu, tc::mbar_wait(&bars[st], ph, &never)) && ok;
    if (!ok) break;
    const uint32_t at = st * Lay::stage;
    const int key0 = tiles.key(part.j0 + warp + W * i);
    float x[NR][4], x2[4];                               // one group alone: two chains of products
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      uint32_t k[4];
      ldsm4(ldk[c & 3] + at + (c >> 2) * (kKeys * 128), k);
      if (NR == 1 && (c & 1)) {
        if (c == 1) mma16816_first(x2, k, qb[0][c][0], qb[0][c][1]);
        else mma16816(x2, k, qb[0][c][0], qb[0][c][1]);
      } else {
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          if (c == 0) mma16816_first(x[n], k, qb[n][c][0], qb[n][c][1]);
          else mma16816(x[n], k, qb[n][c][0], qb[n][c][1]);
        }
      }
    }
    if (NR == 1) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[0][e] += x2[e];
    }
    if (__builtin_expect(!tiles.all(key0), 0)) {
      // lane (g, t): keys g (x[0], x[1]) and 8 + g (x[2], x[3]) of rows 2t and 2t + 1
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t bits = paged::seen32(paged::sees(a, s, tok[n][e]), key0);
          if (!(bits >> g & 1)) x[n][e] = neg_inf();
          if (!(bits >> (8 + g) & 1)) x[n][2 + e] = neg_inf();
        }
      bool found = false;
#pragma unroll 1
      for (int y = lane; y < kKeys * (D / 8); y += 32) {
        const int row = y / (D / 8), c = y % (D / 8);
        uint4* p = reinterpret_cast<uint4*>(ring + at + Lay::tile + (c >> 3) * (kKeys * 128) + tc::sw128_off(row, c & 7));
        if (tiles.any(key0 + row)) found |= paged::take_out(p);
        else *p = make_uint4(0, 0, 0, 0);
      }
      if (found) *(volatile int*)poison = 1;
      tc::fence_proxy_async();                           // before the stage is written by TMA again
      __syncwarp();
    }
    float over = neg_inf();
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) over = fmaxf(over, fmaf(fmaxf(x[n][e], x[n][2 + e]), sl2, nm[n][e]));
    if (__any_sync(0xffffffffu, over > kTop) || !all_set) {
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool set = isset >> (2 * n + e) & 1;
          const float mt = group_max(fmaxf(x[n][e], x[n][2 + e])) * sl2;
          if (set ? mt + nm[n][e] > kTop : mt > neg_inf()) {         // only the rows that need it
            const float f = set ? ex2f(-nm[n][e] - mt) : 0.f;
            nm[n][e] = -mt;
            isset |= 1u << (2 * n + e);
            l[n][e] *= f;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) o[n][c][e] *= f, o[n][c][2 + e] *= f;
          }
        }
      all_set = __all_sync(0xffffffffu, isset == (1u << (2 * NR)) - 1);
    }
    uint32_t pb[NR][2], pl[kSplit ? NR : 1][2];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const float p0 = ex2f(fmaf(x[n][0], sl2, nm[n][0])), p1 = ex2f(fmaf(x[n][1], sl2, nm[n][1]));
      const float p2 = ex2f(fmaf(x[n][2], sl2, nm[n][0])), p3 = ex2f(fmaf(x[n][3], sl2, nm[n][1]));
      l[n][0] += p0 + p2;
      l[n][1] += p1 + p3;
      pb[n][0] = transpose8(kSplit ? upper2(p0, p1) : pack_bf16(p0, p1));
      pb[n][1] = transpose8(kSplit ? upper2(p2, p3) : pack_bf16(p2, p3));
      if (kSplit) {
        pl[n][0] = transpose8(pack_bf16(left_out(p0), left_out(p1)));
        pl[n][1] = transpose8(pack_bf16(left_out(p2), left_out(p3)));
      }
    }
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      uint32_t v[4];
      ldsm4t(ldv[c & 3] + at + (c >> 2) * (kKeys * 128), v);
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        mma16816(o[n][c], v, pb[n][0], pb[n][1]);
        if (kSplit) mma16816(o[n][c], v, pl[n][0], pl[n][1]);
      }
    }
    __syncwarp();                                        // the stage is asked for again
    if (++st == Lay::stages) st = 0, ph ^= 1;
  }
  if (!ok) {                                             // what is on its way lands before the block leaves
    flag_status(a.status, FASTAR_DEV_TIMEOUT);
    for (int i = 0; i < Lay::stages; ++i) tc::mbar_wait(&bars[i], ph ^ (i < st), &never, 400000000LL);
  }
  __syncthreads();                                       // the ring is free in every warp
  // the warps' results side by side, then joined in warp order
  float* so = reinterpret_cast<float*>(smem) + warp * 8 * NR * Lay::ldo;
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * n + 2 * t + e;
      const float sum = group_sum(l[n][e]);
      if (g == 0) sml[warp * 8 * NR + r] = make_float2(-nm[n][e], sum);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        so[r * Lay::ldo + c * 16 + g] = o[n][c][e];
        so[r * Lay::ldo + c * 16 + 8 + g] = o[n][c][2 + e];
      }
    }
  __syncthreads();
  // a row's weights of the warps (-1: a warp that saw none of its keys) and one over its sum (-1: no key), a thread a row, in
  // place
  if ((int)threadIdx.x < rows) {
    float2* ml = sml + threadIdx.x;
    float top = neg_inf(), sum = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w)
      if (ml[w * 8 * NR].y != 0.f) top = fmaxf(top, ml[w * 8 * NR].x);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 x = ml[w * 8 * NR];
      const float f = x.y != 0.f ? ex2f(x.x - top) : -1.f;
      if (x.y != 0.f) sum = fmaf(f, x.y, sum);
      ml[w * 8 * NR].x = f;
    }
    const int r = (int)threadIdx.x, tk = token(r), head = h * G + r - tk * G;
    const bool live = sum > 0.f || sum != sum;
    const float mn = top * 0.6931471805599453f;
    if (partial) a.part_ml[paged::partial_row(a, slot, h, r)] = make_float2(live ? mn : neg_inf(), sum);
    if (!partial && a.lse) a.lse[head * a.T + s.t0 + tk] = live ? mn + logf(sum) : neg_inf();
    ml[0].y = live ? 1.f / sum : -1.f;
  }
  __syncthreads();
#pragma unroll 2
  for (int y = threadIdx.x; y < rows * (D / 4); y += W * 32) {
    const int r = y / (D / 4), c = y % (D / 4) * 4, tk = token(r);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = sml[w * 8 * NR + r].x;
      if (f < 0.f) continue;
      const float4 q = *reinterpret_cast<const float4*>(reinterpret_cast<float*>(smem) + (w * 8 * NR + r) * Lay::ldo + c);
      v[0] = fmaf(f, q.x, v[0]), v[1] = fmaf(f, q.y, v[1]), v[2] = fmaf(f, q.z, v[2]), v[3] = fmaf(f, q.w, v[3]);
    }
    if (__builtin_expect(*(volatile int*)poison, 0))
      paged::add_taken_out<kKeys, 4>(a, tiles, part, b, h, paged::sees(a, s, tk), c, v);
    if (partial) {
      *reinterpret_cast<float4*>(a.part_o + paged::partial_row(a, slot, h, r) * D + c) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      const float f = sml[r].y;
      uint2 w2 = make_uint2(pack_bf16(v[0] * f, v[1] * f), pack_bf16(v[2] * f, v[3] * f));
      if (f < 0.f) w2 = make_uint2(0u, 0u);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + (int64_t)(h * G + r - tk * G) * a.o_hs +
                                (int64_t)(s.t0 + tk) * a.o_ts + c) = w2;
    }
  }
}

template <int D, int NR>
cudaError_t few_go(const PagedAttnArgs& a, cudaStream_t s) {
  constexpr int W = kFewWarps;
  const int64_t blocks = (int64_t)a.Hkv * (a.B + a.extra);
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  CUtensorMap km, vm;
  if (!make_pool_tmap(&km, a, a.pool.k, D, kKeys) || !make_pool_tmap(&vm, a, a.pool.v, D, kKeys))
    return cudaErrorInvalidValue;
  cudaError_t e = opt_in_smem((const void*)paged_attn_few_kernel<D, NR, W>, FewLayout<D, NR, W>::bytes);
  if (e != cudaSuccess) return e;
  e = launch_dependent(paged_attn_few_kernel<D, NR, W>, dim3((unsigned)blocks), dim3(W * 32), FewLayout<D, NR, W>::bytes, s,
                       a, km, vm);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_attn_few(int d, const PagedAttnArgs& a, cudaStream_t s) {
  const int64_t rows = (int64_t)a.group * a.max_q;
  if (rows <= 8) return d == 128 ? few_go<128, 1>(a, s) : few_go<64, 1>(a, s);
  if (rows <= 16) return d == 128 ? few_go<128, 2>(a, s) : few_go<64, 2>(a, s);
  return d == 128 ? few_go<128, 4>(a, s) : few_go<64, 4>(a, s);
}

}  // namespace fastar
