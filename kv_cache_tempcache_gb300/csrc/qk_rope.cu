// RMS norm of every head of q and k with rotary positions of three axes in the same pass.
//
//   y_c = x_c * w_c / sqrt(mean_c x_c^2 + eps)                       (w null: y = x)
//   (y_2j, y_2j+1) of axis a's part turns by p_a * theta^(-2j / width_a)
//
// Bound: HBM (each element read and written once; some seven operations an element).  A warp
// takes a token, or with few tokens a part of its heads: d / 16 lanes hold a head's row, 16
// channels (eight pairs) each, and the next rows are on their way while these are worked on.  A
// lane holds the same channels of every head, so a token's rotations are formed once for all its
// rows (two pairs a lane, passed round by shuffles), and multiplied with the weights: a pair is
// then r (A v0 - B v1), r (C v0 + D v1) with r = 1 / |row|'s root mean square.
//
// Angles: the step theta^(-2j/width) / 2 pi, in turns, is a 64-bit binary fraction (formed on
// the host in double), and position * step is taken modulo one turn by the wrap-around of
// the 64-bit product.  So a far position costs no accuracy: the top 32 bits of the turn go to fp32,
// which rounds them by 2^-26 turns at the most wherever the token is (2^24 positions away the
// step's own error adds some 2^-30), where the fp32 product pos * step loses a bit of the angle with every
// doubling of the position; no 64-bit float arithmetic runs on the device.
#include <climits>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "tmap.h"

namespace fastar {

namespace {

constexpr int kWarpsR = 4;

struct RopeTable {
  uint64_t step[64];   // turns per position as a fraction of 2^64, one per pair
  uint8_t axis[64];    // 0 frame, 1 row, 2 column, 3: the pair does not turn
};

struct RopeDev {
  int Hq, Hk;
  int64_t n;
  const void *q, *k;
  void *qo, *ko;
  int64_t q_hs, q_ts, k_hs, k_ts, qo_hs, qo_ts, ko_hs, ko_ts;
  const float *wq, *wk;
  float eps;
  const int32_t* pos;      // [n, 3] or null: grid positions
  int t0;
  const int32_t* t0_dev;
  int gh, gw;
  int part_shift;          // log2 of the warps per token
};

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

// Inputs and outputs may be the same tensor: every lane reads its channels before it writes
// them and no other lane does.  kAll: every pair turns.
template <typename T, int D, bool kAll, int kAhead>
__global__ void __launch_bounds__(kWarpsR * 32)
    qk_norm_rope_kernel(const RopeDev a, const __grid_constant__ RopeTable tab) {
  // steps and weights in shared memory: read by lane from the kernel's parameters (a lane each
  // another address, one after the other) they took 3 of 15 us
  pdl_wait();                      // the launch overlaps the end of the kernel before
  __shared__ __align__(16) uint64_t steps[64];
  __shared__ uint8_t axes[64];
  __shared__ __align__(16) float ws[2][D];
  if (threadIdx.x < D / 2) {
    steps[threadIdx.x] = tab.step[threadIdx.x];
    axes[threadIdx.x] = tab.axis[threadIdx.x];
  }
  for (int c = threadIdx.x; c < D; c += kWarpsR * 32) {
    ws[0][c] = a.wq ? a.wq[c] : 1.f;
    ws[1][c] = a.wk ? a.wk[c] : 1.f;
  }
  constexpr int LPR = D / 16;      // lanes of a row
  constexpr int RW = 32 / LPR;     // rows of a warp side by side
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, li = lane % LPR;
  const uint32_t parts = 1u << a.part_shift;
  const int64_t items = a.n << a.part_shift;
  const int64_t stride = (int64_t)gridDim.x * kWarpsR;
  const int gq = (a.Hq + RW - 1) / RW, gk = (a.Hk + RW - 1) / RW;   // groups of rows: of q, then of k
  bool first = true;
  const int64_t u0 = (int64_t)blockIdx.x * kWarpsR + (threadIdx.x >> 5);
  if (u0 >= items) {                         // a last block's spare warps
    __syncthreads();
    return;
  }
  for (int64_t u = u0; u < items; u += stride) {
    const uint32_t tok = (uint32_t)(u >> a.part_shift), part = (uint32_t)u & (parts - 1);   // n fits 31 bits
    // the token's rotations: lane l forms those of pairs 2 l and 2 l + 1 (d = 64: l and no other)
    float sn0 = 0.f, cs0 = 1.f, sn1 = 0.f, cs1 = 1.f;
    auto rotations = [&]() {
      int p3[3];
      if (a.pos) {
        p3[0] = a.pos[(int64_t)tok * 3];
        p3[1] = a.pos[(int64_t)tok * 3 + 1];
        p3[2] = a.pos[(int64_t)tok * 3 + 2];
      } else {
        const uint32_t rowi = tok / (uint32_t)a.gw, fr = rowi / (uint32_t)a.gh;
        p3[0] = a.t0 + (a.t0_dev ? a.t0_dev[0] : 0) + (int)fr;
        p3[1] = (int)(rowi - fr * (uint32_t)a.gh);
        p3[2] = (int)(tok - rowi * (uint32_t)a.gw);
      }
      auto one = [&](int j, float& sn, float& cs) {
        const int ax = axes[j];
        const int p = ax == 0 ? p3[0] : ax == 1 ? p3[1] : p3[2];
        const uint64_t turn = (uint64_t)(int64_t)p * steps[j];       // modulo one turn
        sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn, &cs);
      };
      if (D == 128) {
        one(2 * lane, sn0, cs0);
        one(2 * lane + 1, sn1, cs1);
      } else {
        one(lane, sn0, cs0);
      }
    };
    // group x of q's rows, then k's; kAhead of them are on their way
    Raw<T> v[kAhead];
    auto load = [&](Raw<T>& r, int x) {
      const bool isk = x >= gq;
      const int h = (isk ? x - gq : x) * RW + sub;
      const bool in = x < gq + gk && h < (isk ? a.Hk : a.Hq);
      const T* p = isk ? static_cast<const T*>(a.k) + h * a.k_hs + (int64_t)tok * a.k_ts
                       : static_cast<const T*>(a.q) + h * a.q_hs + (int64_t)tok * a.q_ts;
#pragma unroll
      for (int i = 0; i < (int)sizeof(T); ++i)
        r.u[i] = in ? reinterpret_cast<const uint4*>(p + li * 16)[i] : make_uint4(0, 0, 0, 0);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(v[i], (int)(part + i * parts));
    if (first) __syncthreads();              // the tables; after the first loads are on their way
    first = false;
    rotations();
    float A[8], B[8], C[8], E[8];
    bool norm = false;
    int side = -1;
#pragma unroll 1
    for (int x0 = (int)part; x0 < gq + gk; x0 += kAhead * (int)parts) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int x = x0 + i * (int)parts;
        if (x >= gq + gk) break;
        const bool isk = x >= gq;
        if (side != (int)isk) {              // once for q, once for k: rotations times weights
          side = isk;
          norm = isk ? a.wk != nullptr : a.wq != nullptr;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int src = D == 128 ? li * 4 + (e >> 1) : li * 8 + e;
            const float sn = __shfl_sync(0xffffffffu, D == 128 && (e & 1) ? sn1 : sn0, src);
            const float cs = __shfl_sync(0xffffffffu, D == 128 && (e & 1) ? cs1 : cs0, src);
            const float2 w2 = reinterpret_cast<const float2*>(&ws[side][li * 16])[e];
            A[e] = cs * w2.x, B[e] = sn * w2.y, C[e] = sn * w2.x, E[e] = cs * w2.y;
          }
        }
        float f[16];
        expand(v[i], f);
        if (kAhead > 1) load(v[i], x + kAhead * (int)parts);
        float r = 1.f;
        if (norm) {
          float q0 = 0.f, q1 = 0.f;
#pragma unroll
          for (int e = 0; e < 16; e += 2) q0 = fmaf(f[e], f[e], q0), q1 = fmaf(f[e + 1], f[e + 1], q1);
          float q = q0 + q1;
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
          // 1 / sqrt to an ulp: the approximate one and a Newton step
          const float z = q * (1.0f / D) + a.eps, y0 = rsqrtf(z);
          // (of an infinite sum of squares 0, not 0 * infinity; of a NaN, NaN in the whole row)
          r = y0 == 0.f ? 0.f : y0 * fmaf(-0.5f * z * y0, y0, 1.5f);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a0 = f[2 * e], a1 = f[2 * e + 1];
          // a pair that does not turn is not multiplied by (1, 0): its neighbour may be infinite
          const bool turns = kAll || axes[li * 8 + e] < 3;
          f[2 * e] = (turns ? A[e] * a0 - B[e] * a1 : A[e] * a0) * r;
          f[2 * e + 1] = (turns ? C[e] * a0 + E[e] * a1 : E[e] * a1) * r;
        }
        const int h = (isk ? x - gq : x) * RW + sub;
        if (h < (isk ? a.Hk : a.Hq)) {
          T* p = (isk ? static_cast<T*>(a.ko) + h * a.ko_hs + (int64_t)tok * a.ko_ts
                      : static_cast<T*>(a.qo) + h * a.qo_hs + (int64_t)tok * a.qo_ts) + li * 16;
          store8(p, f);
          store8(p + 8, f + 8);
        }
      }
    }
  }
}

template <typename T, int D>
cudaError_t rope_go(RopeDev a, const RopeTable& tab, bool all, cudaStream_t s) {
  // a warp a token, or while that leaves warp schedulers with few warps, several, down to a warp
  // for each group of rows side by side
  constexpr int RW = 32 / (D / 16);
  const int groups = (a.Hq + RW - 1) / RW + (a.Hk + RW - 1) / RW;
  const int64_t sms = sm_count();
  a.part_shift = 0;
  while ((1 << a.part_shift) < groups && (a.n << a.part_shift) < 16 * sms) ++a.part_shift;
  const int64_t blocks = ((a.n << a.part_shift) + kWarpsR - 1) / kWarpsR;
  // one group a warp: as many warps as there are groups, with few registers; else four resident
  // blocks a multiprocessor, which go on to their next tokens
  const bool one = (1 << a.part_shift) >= groups;
  const int64_t most = one ? 0x7fffffff : 4 * sms;
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  constexpr int kAhead = sizeof(T) == 2 ? 3 : 2;
  const auto kernel = one ? all ? qk_norm_rope_kernel<T, D, true, 1> : qk_norm_rope_kernel<T, D, false, 1>
                      : all ? qk_norm_rope_kernel<T, D, true, kAhead>
                            : qk_norm_rope_kernel<T, D, false, kAhead>;
  const cudaError_t e = launch_dependent(kernel, dim3(grid), dim3(kWarpsR * 32), 0, s, a, tab);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(int dtype, int d, int64_t n, int Hq, TokView q, void* qo, int64_t qo_hs, int64_t qo_ts,
                                int Hk, TokView k, void* ko, int64_t ko_hs, int64_t ko_ts, const float* wq,
                                const float* wk, float eps, const int* axes, const int32_t* pos, int t0,
                                const int32_t* t0_dev, int gh, int gw, float theta, cudaStream_t s) {
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
  const bool all = 2 * j == d;
  for (; j < 64; ++j) {
    tab.step[j] = 0;
    tab.axis[j] = 3;
  }
  RopeDev a{};
  a.Hq = Hq, a.Hk = Hk, a.n = n;
  a.q = q.p, a.q_hs = q.hs, a.q_ts = q.ts;
  a.k = k.p, a.k_hs = k.hs, a.k_ts = k.ts;
  a.qo = qo, a.qo_hs = qo_hs, a.qo_ts = qo_ts;
  a.ko = ko, a.ko_hs = ko_hs, a.ko_ts = ko_ts;
  a.wq = wq, a.wk = wk, a.eps = eps;
  a.pos = pos, a.t0 = t0, a.t0_dev = t0_dev, a.gh = gh, a.gw = gw;
  if (dtype == FASTAR_BF16)
    return d == 128 ? rope_go<__nv_bfloat16, 128>(a, tab, all, s) : rope_go<__nv_bfloat16, 64>(a, tab, all, s);
  return d == 128 ? rope_go<float, 128>(a, tab, all, s) : rope_go<float, 64>(a, tab, all, s);
}

}  // namespace fastar
