// Writing rows of K and V into the 4-bit cache, and reading rows back as the values they
// stand for.  Both are bound by HBM in their bytes (2 read and 0.56 written a value, or the other
// way round), and near it by the integer operations of the conversions.
// Writing: a lane takes the 16 channels of a scale, d / 16 lanes a row, so a warp's codes and
// scales leave as contiguous runs of 256 and 32 bytes.  4680 rows of K and V of 12 heads of 128
// take 8.2 us with the inputs partly in L2 (10.4 with the rounding by integer
// operations and a check a channel for infinities; with 8 channels a lane, whose scales two lanes form twice,
// 13.4).
// Reading: 8 channels a lane, four rows at once, so that a warp's stores of 16-bit rows are runs
// of 512 bytes.  14,033 rows of 12 heads back take 19.5 us (5.7 TB/s of 6.8 for a copy); with 16
// channels a lane, whose 16-byte stores lie 32 bytes apart, 23.4.  (fp32 rows, whose stores lie so with 8
// channels: 46 us, 4.2 TB/s.  fp32 rows written, compared with seven middles a value: 4680 rows 21 us.)
//
// The scale is s = e4m3(max|x| / 6), the code e2m1(x / s), both rounded to nearest with ties
// to even and held to the largest finite value.  Both roundings are exact decisions:
//  - max|x| / 6 is formed rounded to odd (towards zero, the last bit set when inexact),
//    which a second rounding to 4 bits cannot send to the wrong side of a middle;
//  - a bf16 x has 8 significant bits and the middle of two codes times s at most 7, so x/s
//    is the middle itself or at least 2^-8 away from it (relative), 2^-10 at the least.  x * (1/s)
//    is within 2^-21 of x/s (up to 8; above 6 the code is 6 whatever it is), and added to 1536 it
//    is rounded to a multiple of 2^-13: to the middle exactly when x/s is it (a multiple of
//    2^-2), else to its own side; the conversion then breaks the tie as the definition does.
//    Adding and taking 1536 away run beside the integer operations, which bound this kernel;
//  - an fp32 x is compared with the seven middles themselves (exact in fp32).
// A NaN or an infinity has no 4-bit value: it is stored as 0, takes no part in the maximum
// and sets a status bit, so the cache never holds one.
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"
#include "tmap.h"

namespace fastar {

namespace {

// Both kernels are launched while the one before them ends and wait in the kernel, before anything
// else (so no pointer is __restrict__: that would promise that nothing writes the cache while a read
// runs, and let its loads pass the wait): two reads of 14,033 rows 20.1 -> 19.5 us, an append and two reads of a token 7.1 -> 5.9.
constexpr int kThreadsQ = 256;
constexpr int kRowsR = 4;            // rows a thread reads at once (fastar_kv4_read)

struct Kv4AppendDev {
  int H;
  int64_t n, cap;
  const void *k, *v;
  int64_t k_hs, k_ts, v_hs, v_ts;
  const int32_t *k_exp, *v_exp, *at;
  uint8_t *kc, *ks, *vc, *vs;
  int32_t* len_out;
  int32_t* status;
};

// 16 channels as they lie in memory.
template <typename T>
struct Row16 {
  uint4 u[sizeof(T)];
};
template <typename T>
__device__ __forceinline__ Row16<T> load16(const T* p) {
  Row16<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); ++i) r.u[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}

// e4m3 of a / 6 (a >= 0, finite), as its byte.
__device__ __forceinline__ uint32_t scale_byte(float a) {
  a = fminf(a, 3.0e38f);   // 2^-e may have carried a finite value to infinity
  float r = __fdiv_rz(a, 6.0f);
  if (fmaf(r, 6.0f, -a) != 0.f) r = __int_as_float(__float_as_int(r) | 1);
  uint16_t b;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(0.f), "f"(r));
  return b & 0xffu;
}

// Codes of two values a (low nibble) and b, already divided by the scale.
__device__ __forceinline__ uint32_t pair_code(float a, float b) {
  uint32_t r;
  asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n cvt.u32.u8 %0, t;\n}\n" : "=r"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float scale_of(uint32_t sb) {
  return __half2float(__ushort_as_half((uint16_t)(kv4::scale_f16x2(sb) & 0xffffu)));
}

// The 16 codes of a row's share (two words) and the scale's byte; down = 2^-e.
__device__ __forceinline__ uint32_t quantise16(const Row16<__nv_bfloat16>& r, float down, uint2& codes, bool& bad) {
  uint32_t x[8] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w, r.u[1].x, r.u[1].y, r.u[1].z, r.u[1].w};
  auto largest = [&]() {                     // the largest magnitude's bits, two channels at a time
    uint32_t b = x[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 8; ++i) b = __vmaxu2(b, x[i] & 0x7fff7fffu);
    return max(b & 0xffffu, b >> 16);
  };
  uint32_t big = largest();
  if (big >= 0x7f80u) {                      // a value that is not finite
    bad = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if ((x[i] & 0x7f80u) == 0x7f80u) x[i] &= 0xffff0000u;
      if ((x[i] & 0x7f800000u) == 0x7f800000u) x[i] &= 0xffffu;
    }
    big = largest();
  }
  const uint32_t sb = scale_byte(__uint_as_float(big << 16) * down);
  const float s = scale_of(sb), inv = s > 0.f ? 1.0f / s * down : 0.f;
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float lo = __uint_as_float(x[i] << 16), hi = __uint_as_float(x[i] & 0xffff0000u);
    const float a = fmaf(lo, inv, 1536.f) - 1536.f, b = fmaf(hi, inv, 1536.f) - 1536.f;
    // the sign of what became 0 too (in the low half, bit 15 of x[i], and of its float)
    w[i >> 2] |= pair_code(__uint_as_float(__float_as_uint(a) | (__float_as_uint(lo) & 0x80000000u)),
                           __uint_as_float(__float_as_uint(b) | (x[i] & 0x80000000u)))
                 << (8 * (i & 3));
  }
  codes = make_uint2(w[0], w[1]);
  return sb;
}
__device__ __forceinline__ uint32_t quantise16(const Row16<float>& r, float down, uint2& codes, bool& bad) {
  float x[16], a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint4& u = r.u[i >> 2];
    const uint32_t v = (i & 3) == 0 ? u.x : (i & 3) == 1 ? u.y : (i & 3) == 2 ? u.z : u.w;
    const bool fin = (v & 0x7f800000u) != 0x7f800000u;
    bad |= !fin;
    x[i] = fin ? __uint_as_float(v) * down : 0.f;
    a = fmaxf(a, fabsf(x[i]));
  }
  const uint32_t sb = scale_byte(a);
  const float s = scale_of(sb);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float m = fabsf(x[i]);
    uint32_t c = __float_as_uint(x[i]) >> 31 << 3;
    if (s > 0.f)
      c += (m > 0.25f * s) + (m >= 0.75f * s) + (m > 1.25f * s) + (m >= 1.75f * s) + (m > 2.5f * s) +
           (m >= 3.5f * s) + (m > 5.0f * s);
    w[i >> 3] |= c << (4 * (i & 7));
  }
  codes = make_uint2(w[0], w[1]);
  return sb;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreadsQ) kv4_append_kernel(const Kv4AppendDev a) {
  constexpr int LPR = D / 16;                 // lanes of a row
  constexpr int RB = kThreadsQ / LPR;         // rows of a block
  pdl_wait();
  const int64_t per = (a.n + RB - 1) / RB > 0 ? (a.n + RB - 1) / RB : 1;   // blocks of a head
  const int h = (int)(blockIdx.x / per);
  const int64_t t = (int64_t)(blockIdx.x % per) * RB + threadIdx.x / LPR;
  const int li = threadIdx.x % LPR;
  const int64_t at = a.at ? a.at[h] : 0;
  const bool sane = at >= 0 && at <= a.cap;
  if (blockIdx.x % per == 0 && threadIdx.x == 0) {
    if (!sane || at + a.n > a.cap) flag_status(a.status, FASTAR_DEV_BAD_LEN);
    if (a.len_out) {
      const int64_t end = sane ? at + a.n : at < 0 ? 0 : a.cap;
      a.len_out[h] = (int32_t)(end < a.cap ? end : a.cap);
    }
  }
  if (t >= a.n || !sane || at + t >= a.cap) return;
  const Row16<T> k = load16(static_cast<const T*>(a.k) + h * a.k_hs + t * a.k_ts + li * 16);
  const Row16<T> v = load16(static_cast<const T*>(a.v) + h * a.v_hs + t * a.v_ts + li * 16);
  const int64_t row = (int64_t)h * a.cap + at + t;
  bool bad = false;
  uint2 c;
  uint32_t sb = quantise16(k, kv4::pow2i(-kv4::head_exp(a.k_exp, h)), c, bad);
  reinterpret_cast<uint2*>(a.kc)[row * LPR + li] = c;
  a.ks[row * LPR + li] = (uint8_t)sb;
  sb = quantise16(v, kv4::pow2i(-kv4::head_exp(a.v_exp, h)), c, bad);
  reinterpret_cast<uint2*>(a.vc)[row * LPR + li] = c;
  a.vs[row * LPR + li] = (uint8_t)sb;
  if (bad) flag_status(a.status, FASTAR_DEV_NONFINITE);
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* f) {
  uint4 u;
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
    w[e] = *reinterpret_cast<uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = u;
}
__device__ __forceinline__ void store8(float* p, const float* f) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreadsQ)
    kv4_read_kernel(const uint8_t* codes, const uint8_t* scales, const int32_t* exps, int64_t cap, int64_t first,
                    int64_t n, T* out, int64_t hs, int64_t ts) {
  constexpr int LPR = D / 8;
  constexpr int RB = kThreadsQ / LPR;
  pdl_wait();
  const int64_t per = (n + RB * kRowsR - 1) / (RB * kRowsR);
  const int h = (int)(blockIdx.x / per);
  const int64_t t0 = (int64_t)(blockIdx.x % per) * RB * kRowsR + threadIdx.x / LPR;
  const int li = threadIdx.x % LPR;
  const int64_t row = (int64_t)h * cap + first + t0;
  uint32_t c[kRowsR], s[kRowsR];
#pragma unroll
  for (int i = 0; i < kRowsR; ++i) {
    const bool in = t0 + i * RB < n;
    c[i] = in ? reinterpret_cast<const uint32_t*>(codes)[(row + i * RB) * LPR + li] : 0u;
    s[i] = in ? scales[((row + i * RB) * LPR + li) >> 1] : 0u;
  }
  const float up = kv4::pow2i(kv4::head_exp(exps, h));
#pragma unroll
  for (int i = 0; i < kRowsR; ++i) {
    if (t0 + i * RB >= n) break;
    uint32_t p[4];
    kv4::unpack8(c[i], kv4::scale_f16x2(s[i]), p);
    float f[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 x = kv4::f16x2_to_f32(p[e]);
      f[2 * e] = x.x * up;
      f[2 * e + 1] = x.y * up;
    }
    store8(out + h * hs + (t0 + i * RB) * ts + li * 8, f);
  }
}

template <typename T, int D>
cudaError_t append_go(const Kv4AppendDev& a, cudaStream_t s) {
  constexpr int RB = kThreadsQ / (D / 16);
  const int64_t per = a.n > 0 ? (a.n + RB - 1) / RB : 1;
  if (per * a.H > INT_MAX) return cudaErrorInvalidConfiguration;
  const cudaError_t e = launch_dependent(kv4_append_kernel<T, D>, dim3((unsigned)(per * a.H)), dim3(kThreadsQ), 0, s, a);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int D>
cudaError_t read_go(int H, const uint8_t* codes, const uint8_t* scales, const int32_t* exps, int64_t cap, int64_t first,
                    int64_t n, void* out, int64_t hs, int64_t ts, cudaStream_t s) {
  constexpr int RB = kThreadsQ / (D / 8);
  const int64_t blocks = (n + RB * kRowsR - 1) / (RB * kRowsR) * H;
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  const cudaError_t e = launch_dependent(kv4_read_kernel<T, D>, dim3((unsigned)blocks), dim3(kThreadsQ), 0, s, codes,
                                         scales, exps, cap, first, n, static_cast<T*>(out), hs, ts);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_append(int dtype, int d, int H, int64_t n, TokView k, TokView v, const int32_t* k_exp,
                              const int32_t* v_exp, const int32_t* at, uint8_t* kc, uint8_t* ks, uint8_t* vc,
                              uint8_t* vs, int64_t cap, int32_t* len_out, int32_t* status, cudaStream_t s) {
  Kv4AppendDev a{H, n, cap, k.p, v.p, k.hs, k.ts, v.hs, v.ts, k_exp, v_exp, at, kc, ks, vc, vs, len_out, status};
  if (dtype == FASTAR_BF16) return d == 128 ? append_go<__nv_bfloat16, 128>(a, s) : append_go<__nv_bfloat16, 64>(a, s);
  return d == 128 ? append_go<float, 128>(a, s) : append_go<float, 64>(a, s);
}

cudaError_t launch_kv4_read(int dtype, int d, int H, const uint8_t* codes, const uint8_t* scales, const int32_t* exps,
                            int64_t cap, int64_t first, int64_t n, void* out, int64_t hs, int64_t ts, cudaStream_t s) {
  if (dtype == FASTAR_BF16)
    return d == 128 ? read_go<__nv_bfloat16, 128>(H, codes, scales, exps, cap, first, n, out, hs, ts, s)
                    : read_go<__nv_bfloat16, 64>(H, codes, scales, exps, cap, first, n, out, hs, ts, s);
  return d == 128 ? read_go<float, 128>(H, codes, scales, exps, cap, first, n, out, hs, ts, s)
                  : read_go<float, 64>(H, codes, scales, exps, cap, first, n, out, hs, ts, s);
}

}  // namespace fastar
