// The 4-bit form of a cache row, shared by the kernels that write and read it: 16
// consecutive channels share a scale s (e4m3, one byte); a value is a 4-bit e2m1 number
// (0 0.5 1 1.5 2 3 4 6 and a sign) times s, times 2^e with a per-head exponent e.  Two
// channels to a byte, the even one in the low nibble.
//
// e2m1 has 2 significant bits and e4m3 4, so a product code * s has at most 6 and lies in
// [2^-10, 2688]: it is exact in fp16, in bf16 and in fp32.  The matrix products therefore
// work on fp16 rows that ARE the cache's values; nothing is rounded by unpacking them.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"

namespace fastar {
namespace kv4 {

// The scale byte (e4m3) in both halves of an fp16 pair.
__device__ __forceinline__ uint32_t scale_f16x2(uint32_t byte) {
  uint32_t r;
  const uint16_t b = (uint16_t)((byte & 0xffu) | ((byte & 0xffu) << 8));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(b));
  return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight codes (channels 0..7 from the low nibble up) times the scale: four fp16 pairs.
__device__ __forceinline__ void unpack8(uint32_t codes, uint32_t s2, uint32_t* out) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
      : "r"(codes));
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = mul_f16x2(out[i], s2);
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// A head's exponent, held to the range in which every product stays a normal fp32.
__device__ __forceinline__ int head_exp(const int32_t* e, int h) {
  return e ? max(-64, min(64, e[h])) : 0;
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// A bf16 call holds P = 2^(logit - reference) in fp16.  The reference is set so that the row's largest P
// is then 2^kLift, and moved when a P would pass 2^kTop (fp16 ends at 65,504).  A P is off by 2^-11 of
// itself from 2^-14 up, and by 2^-25 below that, where fp16 is subnormal: by at most 2^-35 of the row's
// largest exponential, so that keys 16 nats below one that takes nearly all of the weight are as exact as
// the others, and at 18 nats more exact than in bf16.  (Without the lift 2^-25: keys 17 nats below were lost or
// doubled, and where the strong key's V is 0 they are all of the output.)  More lift is less room before
// the reference moves: 4680 tokens over 93,600 rows take 1789 us without it and 1807 at 10, each bit
// more 1 %; the first chunk in frames 96.3 and 98.0, at 11 99.9; few rows the same time at each.
constexpr float kLift = 10.f;
constexpr float kTop = 15.98f;
constexpr float kUnlift = 1.0f / (float)(1 << (int)kLift);

// A head's length, held to [0, cap].
__device__ __forceinline__ int64_t held_len(int64_t n, int64_t cap, int32_t* status) {
  if (n < 0 || n > cap) {
    flag_status(status, FASTAR_DEV_BAD_LEN);
    return n < 0 ? 0 : cap;
  }
  return n;
}
__device__ __forceinline__ int64_t head_len(const int32_t* len, int h, int64_t cap, int32_t* status) {
  return held_len(len[h], cap, status);
}

// How many of a head's `len` rows token t of a call's nq sees: all of them, or with blocks
// of `block` tokens those up to the end of the token's own block, where the nq tokens are
// the cache's last nq rows.  May be 0 (a cache shorter than the call).
__device__ __forceinline__ int64_t visible(int64_t len, int64_t nq, int64_t t, int64_t block) {
  if (block <= 0) return len;
  int64_t end = (int64_t)((uint32_t)t / (uint32_t)block + 1) * block;   // both fit 31 bits
  end = end < nq ? end : nq;
  const int64_t v = len - nq + end;
  return v < 0 ? 0 : v;
}

// What the rows r0 .. rlast of a KV head with `len` cached rows work on: the last key
// that any of them sees (rows of two query heads include a last token, which sees all), and the
// splits of the keys in use.  The launch's splits were chosen for a full cache; a shorter one
// takes fewer, none under min_tiles tiles of 128 keys.
struct ItemKeys {
  int64_t most;
  uint32_t tiles, splits;
};
__device__ __forceinline__ ItemKeys item_keys(int64_t len, uint32_t nq, int64_t block, uint32_t r0, uint32_t rlast,
                                              int splits, int min_tiles) {
  ItemKeys k;
  k.most = len;
  k.splits = 1;
  if (block > 0) {
    const uint32_t g = rlast / nq, first = g * nq;                 // the last row's query head, its first row
    if (r0 >= first) k.most = visible(len, nq, rlast - first, block);
  }
  k.tiles = (uint32_t)((k.most + 127) / 128);
  if (splits > 1) {
    const uint32_t s = k.tiles / (uint32_t)min_tiles;
    k.splits = s < 1 ? 1u : s < (uint32_t)splits ? s : (uint32_t)splits;
  }
  return k;
}

}  // namespace kv4
}  // namespace fastar
