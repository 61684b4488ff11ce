// RMS norm of every head of q and k with rotary positions of three axes in the same pass.
//
//   y_c = x_c * w_c / sqrt(mean_c x_c^2 + eps)                       (w null: y = x)
//   (y_2j, y_2j+1) of axis a's part turns by p_a * theta^(-2j / width_a)
//
// Bound: HBM (each element read and written once; some ten operations an element).  One
// warp takes one token and a few heads: d / 8 lanes hold a head's row, 8 channels (four
// pairs) each, and kIt rows are loaded before the first is used.  A lane holds the same
// four pairs of every head, so the four rotations of a token are computed once for all the
// heads of the warp, and the four angular steps once for the life of the thread.
//
// Angles: the step theta^(-2j/width) / 2 pi, in turns, is a 64-bit binary fraction (formed on
// the host in double), and position * step is taken modulo one turn by the wrap-around of
// the 64-bit product.  So a far position costs no accuracy (2^24 positions away the error is
// 2^-31 turns), where the fp32 product pos * step loses a bit of the angle with every
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
  int chunks;              // warps per token
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

// kIt: rows (heads) a lane group takes of its token.  Inputs and outputs may be the same
// tensor: every lane reads its channels before it writes them and no other lane does.
template <typename T, int D, int kIt>
__global__ void __launch_bounds__(kWarpsR * 32)
    qk_norm_rope_kernel(const RopeDev a, const __grid_constant__ RopeTable tab) {
  constexpr int LPR = D / 8;       // lanes of a row
  constexpr int RW = 32 / LPR;     // rows of a warp side by side
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, li = lane % LPR;
  uint64_t step[4];
  int axis[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    step[e] = tab.step[li * 4 + e];
    axis[e] = tab.axis[li * 4 + e];
  }
  const int Ht = a.Hq + a.Hk;
  const int64_t items = a.n * a.chunks;
  const int64_t stride = (int64_t)gridDim.x * kWarpsR;
  const int f0 = a.pos ? 0 : a.t0 + (a.t0_dev ? a.t0_dev[0] : 0);
  for (int64_t u = (int64_t)blockIdx.x * kWarpsR + (threadIdx.x >> 5); u < items; u += stride) {
    const int64_t tok = u / a.chunks;
    const int h0 = (int)(u % a.chunks) * (RW * kIt) + sub;
    float v[kIt][8];
#pragma unroll
    for (int i = 0; i < kIt; ++i) {
      const int h = h0 + i * RW;
      if (h < Ht) {
        const T* p = h < a.Hq ? static_cast<const T*>(a.q) + h * a.q_hs + tok * a.q_ts
                              : static_cast<const T*>(a.k) + (h - a.Hq) * a.k_hs + tok * a.k_ts;
        load8(p + li * 8, v[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
      }
    }
    int p3[3];
    if (a.pos) {
      p3[0] = a.pos[tok * 3];
      p3[1] = a.pos[tok * 3 + 1];
      p3[2] = a.pos[tok * 3 + 2];
    } else {
      const int64_t rowi = tok / a.gw;
      p3[0] = f0 + (int)(rowi / a.gh);
      p3[1] = (int)(rowi % a.gh);
      p3[2] = (int)(tok - rowi * a.gw);
    }
    float sn[4], cs[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int p = axis[e] == 0 ? p3[0] : axis[e] == 1 ? p3[1] : p3[2];
      const uint64_t turn = (uint64_t)(int64_t)p * step[e];            // modulo one turn
      sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn[e], &cs[e]);
    }
#pragma unroll
    for (int i = 0; i < kIt; ++i) {
      const int h = h0 + i * RW;
      const bool isq = h < a.Hq;
      const float* w = isq ? a.wq : a.wk;
      float q = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) q = fmaf(v[i][e], v[i][e], q);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
      if (h >= Ht) continue;
      float y[8];
      if (w) {
        const float r = 1.0f / sqrtf(q / (float)D + a.eps);
        float wv[8];
        load8(w + li * 8, wv);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = v[i][e] * r * wv[e];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = v[i][e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a0 = y[2 * e], a1 = y[2 * e + 1];
        // a pair that does not turn is passed on, not multiplied by (1, 0): its neighbour
        // may be infinite
        y[2 * e] = axis[e] < 3 ? a0 * cs[e] - a1 * sn[e] : a0;
        y[2 * e + 1] = axis[e] < 3 ? a0 * sn[e] + a1 * cs[e] : a1;
      }
      T* p = isq ? static_cast<T*>(a.qo) + h * a.qo_hs + tok * a.qo_ts
                 : static_cast<T*>(a.ko) + (h - a.Hq) * a.ko_hs + tok * a.ko_ts;
      store8(p + li * 8, y);
    }
  }
}

template <typename T, int D, int kIt>
cudaError_t rope_go(RopeDev a, const RopeTable& tab, cudaStream_t s) {
  constexpr int per = (32 / (D / 8)) * kIt;
  a.chunks = (a.Hq + a.Hk + per - 1) / per;
  const int64_t blocks = (a.n * a.chunks + kWarpsR - 1) / kWarpsR;
  const int64_t most = (int64_t)sm_count() * 64;
  qk_norm_rope_kernel<T, D, kIt><<<(unsigned)(blocks < most ? blocks : most), kWarpsR * 32, 0, s>>>(a, tab);
  count_launches(1);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t rope_pick(const RopeDev& a, const RopeTable& tab, cudaStream_t s) {
  // one row per lane group while that leaves warp schedulers without a warp, else four
  const int64_t rows = a.n * (a.Hq + a.Hk) / (32 / (D / 8));
  if (rows < (int64_t)sm_count() * 16) return rope_go<T, D, 1>(a, tab, s);
  return rope_go<T, D, 4>(a, tab, s);
}

}  // namespace

cudaError_t launch_qk_norm_rope(int dtype, int d, int64_t n, int Hq, TokView q, void* qo, int64_t qo_hs, int64_t qo_ts,
                                int Hk, TokView k, void* ko, int64_t ko_hs, int64_t ko_ts, const float* wq,
                                const float* wk, float eps, const int* axes, const int32_t* pos, int t0,
                                const int32_t* t0_dev, int gh, int gw, float theta, cudaStream_t s) {
  RopeTable tab;
  int j = 0;
  for (int a = 0; a < 3; ++a) {
    // the steps of an axis as a geometric sequence: 32 products add 2^-48 to the relative error
    const double ratio = axes[a] > 0 ? std::pow((double)theta, -2.0 / axes[a]) : 1.0;
    double f = 0.15915494309189535;   // 1 / 2 pi turns
    for (int i = 0; i < axes[a] / 2; ++i, ++j, f *= ratio) {
      tab.step[j] = (uint64_t)(f * 18446744073709551616.0);
      tab.axis[j] = (uint8_t)a;
    }
  }
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
    return d == 128 ? rope_pick<__nv_bfloat16, 128>(a, tab, s) : rope_pick<__nv_bfloat16, 64>(a, tab, s);
  return d == 128 ? rope_pick<float, 128>(a, tab, s) : rope_pick<float, 64>(a, tab, s);
}

}  // namespace fastar
