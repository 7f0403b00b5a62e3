// dsa3d_ffn_any.cuh -- the gated feed-forward block on CUDA cores, for every size, both I/O types:
//
//   g = x Wg, u = x Wu, h = act(g) u, y = h Wd (+ add)                      (Wg, Wu [C][hidden], Wd [hidden][C])
//   dh = dy Wd^T, dg = dh u act'(g), du = dh act(g), dx = dg Wg^T + du Wu^T,
//   dWg = x^T dg, dWu = x^T du, dWd = h^T dy
//
// Tiles of 64 x 64 outputs, 16 along the summed axis, 256 threads with 4 x 4 fp32 sums each.  The
// products of one tile that the same outputs need (gate, up and dh) are formed one after another by
// the same block, and the activation, its derivative and the element-wise products are the epilogue,
// so g, u and dh never reach memory.  h, dg and du are kept in the I/O type: they are operands of the
// next product, which reads that type.
#pragma once

#include <stdint.h>

#include "dsa3d_vec.cuh"

namespace dsa3d {

constexpr int kActSilu = 0, kActGelu = 1;

// Activation and derivative.  silu: g s(g), s the logistic function; gelu: g Phi(g), Phi the normal
// distribution (the exact form, with erf).  T float: expf; bf16 results take __expf, whose relative
// error (2^-21 and up to 2^-18 at |g| = 10) is far below their rounding of 2^-9.
template <typename T>
__device__ __forceinline__ float ffn_exp(float x) {
  return sizeof(T) == 4 ? expf(x) : __expf(x);
}
template <typename T>
__device__ __forceinline__ void ffn_act(int act, float g, float& a, float& da) {
  if (act == kActSilu) {
    const float s = 1.f / (1.f + ffn_exp<T>(-g));
    a = g * s;
    da = s * fmaf(g, 1.f - s, 1.f);
  } else {
    const float cdf = 0.5f * (1.f + erff(g * 0.70710678118654752f));
    a = g * cdf;
    da = fmaf(g * 0.39894228040143268f, ffn_exp<T>(-0.5f * g * g), cdf);
  }
}
template <typename T>
__device__ __forceinline__ float ffn_act_only(int act, float g) {
  if (act == kActSilu) return g / (1.f + ffn_exp<T>(-g));
  return g * 0.5f * (1.f + erff(g * 0.70710678118654752f));
}

constexpr int kAnyTile = 64, kAnyK = 16, kAnyThreads = 256;

struct AnyOperand {  // element (i, k) of an operand at p[i * si + k * sk]
  const void* p;
  int64_t si, sk;
};

struct AnySmem {
  float a[kAnyK][kAnyTile + 1], b[kAnyK][kAnyTile + 1];
};

template <typename T>
__device__ __forceinline__ void any_load(float (&dst)[kAnyK][kAnyTile + 1], const AnyOperand& o, int64_t i0,
                                         int64_t ni, int64_t k0, int64_t k1) {
  const T* p = static_cast<const T*>(o.p);
#pragma unroll
  for (int j = 0; j < kAnyTile * kAnyK / kAnyThreads; j++) {
    const int e = threadIdx.x + j * kAnyThreads;
    // consecutive threads along the operand's contiguous axis
    const int i = o.sk == 1 ? e / kAnyK : e % kAnyTile;
    const int k = o.sk == 1 ? e % kAnyK : e / kAnyTile;
    const bool in = i0 + i < ni && k0 + k < k1;
    dst[k][i] = in ? to_f32(p[(i0 + i) * o.si + (k0 + k) * o.sk]) : 0.f;
  }
}

// acc += A[m0.., k0..k1) . B[n0.., k0..k1)
template <typename T>
__device__ __forceinline__ void any_product(float (&acc)[4][4], const AnyOperand& A, const AnyOperand& B,
                                            int64_t m0, int64_t M, int64_t n0, int64_t N, int64_t k0, int64_t k1,
                                            AnySmem& sm) {
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  for (int64_t k = k0; k < k1; k += kAnyK) {
    __syncthreads();
    any_load<T>(sm.a, A, m0, M, k, k1);
    any_load<T>(sm.b, B, n0, N, k, k1);
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kAnyK; kk++) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; i++) a[i] = sm.a[kk][ty + 16 * i];
#pragma unroll
      for (int j = 0; j < 4; j++) b[j] = sm.b[kk][tx + 16 * j];
#pragma unroll
      for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
  }
}

enum AnyMode {
  kAnyHidden,     // out0 = h
  kAnyHiddenBwd,  // out0 = dg, out1 = du, out2 = h
  kAnyOut,        // out0 = sum of up to two products (+ add)
  kAnyPartial     // out0 (fp32, one [M][N] per split) = the product over this split's part of K
};

struct AnyArgs {
  AnyOperand A[3], B[3];  // the products' operands; B's rows are output columns
  const void* add;        // [M][N] or null
  void* out[3];           // [M][N]
  int64_t M, N, K;
  int products, act;
  bool accumulate;  // kAnyPartial: add to what out0 holds
};

template <typename T, int MODE>
__global__ void __launch_bounds__(kAnyThreads) dsa3d_ffn_any_kernel(const __grid_constant__ AnyArgs g) {
  __shared__ AnySmem sm;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const int64_t tiles_n = (g.N + kAnyTile - 1) / kAnyTile;
  const int64_t m0 = blockIdx.x / tiles_n * kAnyTile, n0 = blockIdx.x % tiles_n * kAnyTile;
  constexpr int NA = MODE == kAnyHidden ? 2 : (MODE == kAnyHiddenBwd ? 3 : 1);
  float acc[NA][4][4] = {};
  if (MODE == kAnyHidden || MODE == kAnyHiddenBwd) {
#pragma unroll
    for (int p = 0; p < NA; p++) any_product<T>(acc[p], g.A[p], g.B[p], m0, g.M, n0, g.N, 0, g.K, sm);
  } else if (MODE == kAnyOut) {
    for (int p = 0; p < g.products; p++) any_product<T>(acc[0], g.A[p], g.B[p], m0, g.M, n0, g.N, 0, g.K, sm);
  } else {
    const int64_t len = ((g.K + gridDim.y - 1) / gridDim.y + kAnyK - 1) / kAnyK * kAnyK;
    const int64_t k0 = blockIdx.y * len, k1 = k0 + len < g.K ? k0 + len : g.K;
    any_product<T>(acc[0], g.A[0], g.B[0], m0, g.M, n0, g.N, k0, k1, sm);
  }
#pragma unroll
  for (int i = 0; i < 4; i++) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= g.M || n >= g.N) continue;
      const int64_t at = m * g.N + n;
      if (MODE == kAnyHidden) {
        static_cast<T*>(g.out[0])[at] = from_f32<T>(ffn_act_only<T>(g.act, acc[0][i][j]) * acc[NA > 1 ? 1 : 0][i][j]);
      } else if (MODE == kAnyHiddenBwd) {
        float a, da;
        ffn_act<T>(g.act, acc[0][i][j], a, da);
        const float u = acc[NA > 1 ? 1 : 0][i][j], dh = acc[NA > 2 ? 2 : 0][i][j];
        static_cast<T*>(g.out[0])[at] = from_f32<T>(dh * u * da);
        static_cast<T*>(g.out[1])[at] = from_f32<T>(dh * a);
        static_cast<T*>(g.out[2])[at] = from_f32<T>(a * u);
      } else if (MODE == kAnyOut) {
        float v = acc[0][i][j];
        if (g.add) v += to_f32(static_cast<const T*>(g.add)[at]);
        static_cast<T*>(g.out[0])[at] = from_f32<T>(v);
      } else {
        float* o = static_cast<float*>(g.out[0]) + (int64_t)blockIdx.y * g.M * g.N + at;
        *o = g.accumulate ? *o + acc[0][i][j] : acc[0][i][j];
      }
    }
  }
}

// out[i] = sum_s partial[s * stride + i] (+ add[i]), in order of s: the joining of split sums.
template <typename T>
__global__ void __launch_bounds__(256) dsa3d_ffn_reduce_kernel(const float* __restrict__ partial, int splits,
                                                               int64_t stride, const T* add, T* out, int64_t n) {
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) {
    float v = 0.f;
    for (int s = 0; s < splits; s++) v += partial[s * stride + i];
    if (add) v += to_f32(add[i]);
    out[i] = from_f32<T>(v);
  }
}

}  // namespace dsa3d
