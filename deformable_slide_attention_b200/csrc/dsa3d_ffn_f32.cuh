// dsa3d_ffn_f32.cuh -- the gated feed-forward block for fp32 tensors, on CUDA cores:
//
//   g = x Wg, u = x Wu, h = act(g) u, y = h Wd (+ add)                      (Wg, Wu [C][hidden], Wd [hidden][C])
//   dh = dy Wd^T, dg = dh u act'(g), du = dh act(g), dx = dg Wg^T + du Wu^T,
//   dWg = x^T dg, dWu = x^T du, dWd = h^T dy
//
// fp32 products stay fp32 here: the tensor cores' tf32 keeps 11 bits of each factor, and sums of split
// bf16 factors are cut, not rounded, at every step of the accumulator.  The kernel is bound by the fp32
// FMA pipes, or, at a few hundred tokens, by how many of them the tiles reach (backward of 1001 x 258 x
// 685: 160 us, 18 TFLOP/s; 178 with tiles of 64 rows everywhere).  Tiles of 64 x 64 outputs (32 x 64 where
// those would leave SMs idle), 16 along the summed axis, 4 x 4 sums per thread (8 x 4 leave a scheduler one
// warp: 253 us).  The next 16 are loaded into registers while these are multiplied, by pointers that only
// move on, and two shared buffers make one barrier per step enough.  The products of one tile that the
// same outputs need are formed by the same block (gate and up, and dWg and dWu, from one read of x; dh
// after them), and the activation, its derivative and the element-wise products are the epilogue, so g, u
// and dh never reach memory.
#pragma once

#include <stdint.h>

#include "dsa3d_vec.cuh"

namespace dsa3d {

constexpr int kActSilu = 0, kActGelu = 1;

// Activation and derivative.  silu: g s(g), s the logistic function; gelu: g Phi(g), Phi the normal
// distribution (the exact form, with erf).
__device__ __forceinline__ void f32_act(int act, float g, float& a, float& da) {
  if (act == kActSilu) {
    const float s = 1.f / (1.f + expf(-g));
    a = g * s;
    da = s * fmaf(g, 1.f - s, 1.f);
  } else {
    const float cdf = 0.5f * erfcf(g * -0.70710678118654752f);
    a = g * cdf;
    da = fmaf(g * 0.39894228040143268f, expf(-0.5f * g * g), cdf);
  }
}

constexpr int kF32Cols = 64, kF32K = 16;
constexpr int f32_threads(int TM) { return TM * kF32Cols / 16; }  // 4 x 4 sums each

struct F32Operand {  // element (i, k) of an operand at p[i * si + k * sk]; si or sk is 1
  const float* p;
  int64_t si, sk;
};

template <int TM>
struct F32Smem {
  float a[2][kF32K][TM + 4], b[2][2][kF32K][kF32Cols + 4];  // [buffer], [product][buffer]
};

// One thread's share of an operand's steps (ROWS x 16 of them over T threads): consecutive threads along
// the contiguous axis, the j-th element `apart` behind the first; the pointer moves on by 16 of the
// summed axis per step.
template <int ROWS, int T>
struct F32Loader {
  static constexpr int kLoads = ROWS * kF32K / T;
  const float* p;
  int64_t apart, step;
  int i, k, di, dk;    // position in the tile, and from element to element
  unsigned inside;     // bit j: element j's row lies inside the operand
  __device__ __forceinline__ F32Loader(const F32Operand& o, int64_t i0, int64_t ni, int64_t k0) {
    const bool along_k = o.sk == 1;
    i = along_k ? threadIdx.x / kF32K : threadIdx.x % ROWS;
    k = along_k ? threadIdx.x % kF32K : threadIdx.x / ROWS;
    di = along_k ? T / kF32K : 0;
    dk = along_k ? 0 : T / ROWS;
    apart = di * o.si + dk * o.sk;
    step = kF32K * o.sk;
    p = o.p + (i0 + i) * o.si + (k0 + k) * o.sk;
    inside = 0;
#pragma unroll
    for (int j = 0; j < kLoads; j++) inside |= (i0 + i + j * di < ni ? 1u : 0u) << j;
  }
  // left: elements of the summed axis from this step on
  __device__ __forceinline__ void fetch(float (&r)[kLoads], int left) {
#pragma unroll
    for (int j = 0; j < kLoads; j++)
      r[j] = ((inside >> j) & 1u) && k + j * dk < left ? __ldg(p + j * apart) : 0.f;
    p += step;
  }
  __device__ __forceinline__ void stash(float (&dst)[kF32K][ROWS + 4], const float (&r)[kLoads]) const {
#pragma unroll
    for (int j = 0; j < kLoads; j++) dst[k + j * dk][i + j * di] = r[j];
  }
};

// acc[q] += A[m0.., k0..k1) . B[q][n0.., k0..k1) for NB products that share A; thread (ty, tx) holds rows
// 4 ty.., columns 4 tx...
template <int NB, int TM>
__device__ __forceinline__ void f32_product(float (*acc)[4][4], const F32Operand& A, const F32Operand* B, int64_t m0,
                                            int64_t M, int64_t n0, int64_t N, int64_t k0, int64_t k1, F32Smem<TM>& sm) {
  if (k0 >= k1) return;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  F32Loader<TM, f32_threads(TM)> la(A, m0, M, k0);
  F32Loader<kF32Cols, f32_threads(TM)> lb(B[0], n0, N, k0), lc(B[NB - 1], n0, N, k0);
  int left = (int)(k1 - k0), buf = 0;
  float ra[decltype(la)::kLoads], rb[decltype(lb)::kLoads], rc[decltype(lc)::kLoads];
  auto fetch = [&](int n) {
    la.fetch(ra, n);
    lb.fetch(rb, n);
    if (NB == 2) lc.fetch(rc, n);
  };
  auto stash = [&](int to) {
    la.stash(sm.a[to], ra);
    lb.stash(sm.b[0][to], rb);
    if (NB == 2) lc.stash(sm.b[1][to], rc);
  };
  fetch(left);
  __syncthreads();  // the buffers' last readers (of an earlier product) are done
  stash(0);
  __syncthreads();
  for (; left > 0; left -= kF32K, buf ^= 1) {
    const bool more = left > kF32K;
    if (more) fetch(left - kF32K);
#pragma unroll
    for (int kk = 0; kk < kF32K; kk++) {
      const float4 a0 = *reinterpret_cast<const float4*>(&sm.a[buf][kk][4 * ty]);
      const float a[4] = {a0.x, a0.y, a0.z, a0.w};
#pragma unroll
      for (int q = 0; q < NB; q++) {
        const float4 b0 = *reinterpret_cast<const float4*>(&sm.b[q][buf][kk][4 * tx]);
        const float b[4] = {b0.x, b0.y, b0.z, b0.w};
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
          for (int j = 0; j < 4; j++) acc[q][i][j] = fmaf(a[i], b[j], acc[q][i][j]);
      }
    }
    if (more) stash(buf ^ 1);
    __syncthreads();
  }
}

enum F32Mode {
  kF32Hidden,     // out[0] = h
  kF32HiddenBwd,  // out[0] = dg, out[1] = du, out[2] = h
  kF32Sum         // out[0] = the sum of up to two products (+ add), or this part's share of it; with `pair`
                  // out[0] and out[1] = two products that share A[0]
};

struct F32Args {
  F32Operand A[3], B[3];  // the products' operands; B's rows are output columns
  const float* add;       // [M][N] or null
  float* out[3];          // [M][N]; kF32Sum with parts: [part][M][N]
  int64_t M, N, K;
  int products, parts, act;
  bool accumulate;        // kF32Sum: add to what out holds
  bool pair;
};
struct F32Batch {  // blockIdx.z picks one
  F32Args p[3];
};

template <int MODE, int TM>
__global__ void __launch_bounds__(f32_threads(TM)) dsa3d_ffn_f32_kernel(const __grid_constant__ F32Batch batch) {
  __shared__ __align__(16) F32Smem<TM> sm;
  const F32Args& g = batch.p[MODE == kF32Sum ? blockIdx.z : 0];
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const int64_t tiles_n = (g.N + kF32Cols - 1) / kF32Cols;
  const int64_t m0 = blockIdx.x / tiles_n * TM, n0 = blockIdx.x % tiles_n * kF32Cols;
  if (m0 >= g.M) return;  // a batch's other problem has more tiles
  constexpr int NA = MODE == kF32HiddenBwd ? 3 : 2;
  float acc[NA][4][4] = {};
  if (MODE != kF32Sum) {
    f32_product<2>(acc, g.A[0], g.B, m0, g.M, n0, g.N, 0, g.K, sm);
    if (MODE == kF32HiddenBwd) f32_product<1>(acc + NA - 1, g.A[2], g.B + 2, m0, g.M, n0, g.N, 0, g.K, sm);
  } else {
    const int64_t len = ((g.K + g.parts - 1) / g.parts + kF32K - 1) / kF32K * kF32K;
    const int64_t k0 = blockIdx.y * len, k1 = k0 + len < g.K ? k0 + len : g.K;
    if (g.pair)
      f32_product<2>(acc, g.A[0], g.B, m0, g.M, n0, g.N, k0, k1, sm);
    else
      for (int p = 0; p < g.products; p++) f32_product<1>(acc, g.A[p], g.B + p, m0, g.M, n0, g.N, k0, k1, sm);
  }
#pragma unroll
  for (int i = 0; i < 4; i++) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int64_t m = m0 + 4 * ty + i, n = n0 + 4 * tx + j;
      if (m >= g.M || n >= g.N) continue;
      const int64_t at = m * g.N + n;
      if (MODE == kF32Hidden) {
        float a, da;
        f32_act(g.act, acc[0][i][j], a, da);
        g.out[0][at] = a * acc[1][i][j];
      } else if (MODE == kF32HiddenBwd) {
        float a, da;
        f32_act(g.act, acc[0][i][j], a, da);
        const float u = acc[1][i][j], dh = acc[NA - 1][i][j];
        g.out[0][at] = dh * u * da;
        g.out[1][at] = dh * a;
        g.out[2][at] = a * u;
      } else {
#pragma unroll
        for (int q = 0; q < 2; q++) {
          if (q == 1 && !g.pair) break;
          float* o = g.out[q] + (int64_t)blockIdx.y * g.M * g.N + at;
          float v = acc[q][i][j];
          if (g.add) v += g.add[at];
          *o = g.accumulate ? *o + v : v;
        }
      }
    }
  }
}

// out[p][i] = sum_s partial[p][s][i] (+ add), in order of s: joins the parts of split sums.
// blockIdx.y picks one of up to three outputs.
struct F32Join {
  const float* partial[3];  // [parts][n]
  const float* add;         // [n] or null
  float* out[3];            // [n]
  int64_t n[3];
  int parts;
};
__global__ void __launch_bounds__(256) dsa3d_ffn_join_kernel(const __grid_constant__ F32Join r) {
  prior_kernel_done();
  const int p = blockIdx.y;
  const int64_t n = r.n[p], step = (int64_t)gridDim.x * blockDim.x;
  const float* from = r.partial[p];
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) {
    float v = 0.f;
#pragma unroll 4
    for (int s = 0; s < r.parts; s++) v += from[s * n + i];
    if (r.add) v += r.add[i];
    r.out[p][i] = v;
  }
}

// Rows of n elements copied into rows of ld (a multiple of 8, so that TMA's 16-byte strides fit):
// up to four tensors, blockIdx.y picks one.
struct FfnPad {
  const __nv_bfloat16* from[4];
  __nv_bfloat16* to[4];
  int64_t rows[4], n[4], ld[4];
};
__global__ void __launch_bounds__(256) dsa3d_ffn_pad_kernel(const __grid_constant__ FfnPad a) {
  const int p = blockIdx.y;
  const int64_t n = a.n[p], ld = a.ld[p];
  for (int64_t row = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; row < a.rows[p]; row += (int64_t)gridDim.x * 8)
    for (int64_t c = threadIdx.x % 32; c < n; c += 32) a.to[p][row * ld + c] = a.from[p][row * n + c];
}

}  // namespace dsa3d
