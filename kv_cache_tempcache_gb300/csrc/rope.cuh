// What the kernels with rotary positions share: the table of angles and rows of 16 channels a lane.
//
// Angles: the step theta^(-2j/width) / 2 pi, in turns, is a 64-bit binary fraction (formed on
// the host in double), and position * step is taken modulo one turn by the wrap-around of
// the 64-bit product.  So a far position costs no accuracy: the top 32 bits of the turn go to fp32,
// which rounds them by 2^-26 turns at the most wherever the token is (2^24 positions away the
// step's own error adds some 2^-30), where the fp32 product pos * step loses a bit of the angle with every
// doubling of the position; no 64-bit float arithmetic runs on the device.
#pragma once

#include <cmath>

#include "common.cuh"

namespace fastar {

struct RopeTable {
  uint64_t step[64];   // turns per position as a fraction of 2^64, one per pair
  uint8_t axis[64];    // 0 frame, 1 row, 2 column, 3: the pair does not turn
};

// The table of three axes' widths; *all: every pair of the d channels turns.
inline RopeTable rope_table(int d, const int* axes, float theta, bool* all) {
  RopeTable tab;
  int j = 0;
  for (int a = 0; a < 3; ++a) {
    // the steps of an axis as a geometric sequence: at most 63 products, which add 2^-46 to the relative error
    const double ratio = axes[a] > 0 ? std::pow((double)theta, -2.0 / axes[a]) : 1.0;
    double f = 0.15915494309189535;   // 1 / 2 pi turns
    for (int i = 0; i < axes[a] / 2; ++i, ++j, f *= ratio) {
      tab.step[j] = (uint64_t)(f * 18446744073709551616.0);
      tab.axis[j] = (uint8_t)a;
    }
  }
  *all = 2 * j == d;
  for (; j < 64; ++j) {
    tab.step[j] = 0;
    tab.axis[j] = 3;
  }
  return tab;
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

// 16 channels of a row as they lie in memory, and as fp32.
template <typename T>
struct Raw {
  uint4 u[sizeof(T)];
};
__device__ __forceinline__ void expand(const Raw<__nv_bfloat16>& r, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {r.u[i].x, r.u[i].y, r.u[i].z, r.u[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[8 * i + 2 * e] = __uint_as_float(w[e] << 16);
      f[8 * i + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ void expand(const Raw<float>& r, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[4 * i] = __uint_as_float(r.u[i].x), f[4 * i + 1] = __uint_as_float(r.u[i].y);
    f[4 * i + 2] = __uint_as_float(r.u[i].z), f[4 * i + 3] = __uint_as_float(r.u[i].w);
  }
}

// The sine and cosine of position p times the step.
__device__ __forceinline__ void rope_turn(int p, uint64_t step, float& sn, float& cs) {
  const uint64_t turn = (uint64_t)(int64_t)p * step;               // modulo one turn
  sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn, &cs);
}

// 1 / sqrt(mean x^2 + eps) of a row of D channels, of which each of its D / 16 lanes holds 16.
template <int D>
__device__ __forceinline__ float rms_scale(const float* f, float eps) {
  float q0 = 0.f, q1 = 0.f;
#pragma unroll
  for (int e = 0; e < 16; e += 2) q0 = fmaf(f[e], f[e], q0), q1 = fmaf(f[e + 1], f[e + 1], q1);
  float q = q0 + q1;
#pragma unroll
  for (int o = D / 32; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
  // 1 / sqrt to an ulp: the approximate one and a Newton step
  const float z = q * (1.0f / D) + eps, y0 = rsqrtf(z);
  // (of an infinite sum of squares 0, not 0 * infinity; of a NaN, NaN in the whole row)
  return y0 == 0.f ? 0.f : y0 * fmaf(-0.5f * z * y0, y0, 1.5f);
}

// Eight pairs turned: r (A x0 - B x1), r (C x0 + E x1), the rotations times the weights.  turns: a bit a pair.
template <bool kAll>
__device__ __forceinline__ void turn16(float* f, const float* A, const float* B, const float* C, const float* E, float r,
                                       uint32_t turns) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float a0 = f[2 * e], a1 = f[2 * e + 1];
    // a pair that does not turn is not multiplied by (1, 0): its neighbour may be infinite
    const bool on = kAll || (turns >> e & 1);
    f[2 * e] = (on ? A[e] * a0 - B[e] * a1 : A[e] * a0) * r;
    f[2 * e + 1] = (on ? C[e] * a0 + E[e] * a1 : E[e] * a1) * r;
  }
}

}  // namespace fastar
