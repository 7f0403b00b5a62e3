// dsa3d_ffn_rows.cuh -- the gated feed-forward block for one token (bf16) or one to eight (fp32): three
// matrix-vector products that read each weight once, so HBM (or L2) binds and the tensor cores' tiles of
// 128 rows have nothing to offer.  A block owns a strip of 32 vectors of columns (512 bytes of each
// weight row) and a part of the summed axis, its eight warps take every eighth row, and each thread
// keeps eight 16-byte loads in flight while it multiplies the eight before; the parts' fp32 sums go
// through the workspace (the strips alone would leave most SMs idle).  Rows of g and u are joined,
// activated and multiplied by the blocks of the second product that need them, whose first weights are
// loading meanwhile, and y's parts are joined by a last small launch.
// One bf16 token at C 4096, hidden 10,944: 269 MB of weights in 57 us (4.7 TB/s over the three launches, of
// which the later two start early; 63 us without that, three or more blocks per SM 70 us and more).

#pragma once

#include <stdint.h>

#include "dsa3d_ffn_f32.cuh"
#include "dsa3d_vec.cuh"

namespace dsa3d {

constexpr int kRowsMaxBf16 = 1, kRowsMaxF32 = 8;  // tokens
constexpr int kRowsThreads = 256, kRowsWarps = 8;
constexpr int kRowsPart = 1024;      // longest part of the summed axis

struct RowsArgs {
  const void* w[2];       // [K][N] weights: gate and up, or down
  const void* x;          // [rows][K] (first products)
  const float* in;        // [in_parts][2][rows][K]: g's and u's parts (second product)
  float* out;             // [parts][weights][rows][N]
  int K, N, rows, per_part, in_parts, act;
};

// NW weights share the row operand; R rows.  GATED: the operand is act(g) * u from the first launch's parts.
template <typename T, int R, int NW, bool GATED>
__global__ void __launch_bounds__(kRowsThreads) dsa3d_ffn_rows_kernel(const __grid_constant__ RowsArgs a) {
  constexpr int V = vec_width<T>();
  constexpr int UNROLL = 8 / NW;
  __shared__ float xs[R][kRowsPart];
  __shared__ float red[kRowsWarps][32 * V];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int k0 = blockIdx.y * a.per_part, len = min(a.per_part, a.K - k0);
  const int64_t col = ((int64_t)blockIdx.x * 32 + lane) * V;
  // This warp's rows of the part are warp, warp + 8, ...; a batch is UNROLL of them.
  const T* w[NW];
#pragma unroll
  for (int j = 0; j < NW; j++) w[j] = static_cast<const T*>(a.w[j]) + (int64_t)(k0 + warp) * a.N + col;
  const int64_t step = (int64_t)kRowsWarps * a.N;
  auto load = [&](Vec<T, V> (&v)[UNROLL][NW], int k) {
#pragma unroll
    for (int q = 0; q < UNROLL; q++) {
#pragma unroll
      for (int j = 0; j < NW; j++) {
        if (col < a.N && k + q * kRowsWarps < len)
          v[q][j].load(w[j]);
        else
          v[q][j].zero();
        w[j] += step;
      }
    }
  };
  Vec<T, V> cur[UNROLL][NW];
  load(cur, warp);  // on its way while the row operand is formed (and, of the second product, while the
                    // first launch ends: the weights do not depend on it)
  next_kernel_may_start();
  if (GATED) prior_kernel_done();
  for (int i = threadIdx.x; i < len; i += kRowsThreads) {
#pragma unroll
    for (int r = 0; r < R; r++) {
      float v = 0.f;
      if (r < a.rows) {
        if (GATED) {
          float g = 0.f, u = 0.f;
          const float* p = a.in + (int64_t)r * a.K + k0 + i;
          const int64_t up = (int64_t)a.rows * a.K;
#pragma unroll 8
          for (int s = 0; s < a.in_parts; s++, p += 2 * up) {
            g += p[0];
            u += p[up];
          }
          float act, unused;
          f32_act(a.act, g, act, unused);
          v = to_f32(from_f32<T>(act * u));  // rounded as the operand of the second product
        } else {
          v = to_f32(static_cast<const T*>(a.x)[(int64_t)r * a.K + k0 + i]);
        }
      }
      xs[r][i] = v;
    }
  }
  __syncthreads();
  float acc[NW][R][V] = {};
  for (int k = warp; k < len; k += UNROLL * kRowsWarps) {
    Vec<T, V> next[UNROLL][NW];
    load(next, k + UNROLL * kRowsWarps);
#pragma unroll
    for (int q = 0; q < UNROLL; q++) {
      const int at = min(k + q * kRowsWarps, len - 1);  // past the part the weights are zero
#pragma unroll
      for (int j = 0; j < NW; j++) {
        float x[V];
        cur[q][j].get(x);
        const bool in = k + q * kRowsWarps < len;
#pragma unroll
        for (int r = 0; r < R; r++) {
          const float f = in ? xs[r][at] : 0.f;
#pragma unroll
          for (int e = 0; e < V; e++) acc[j][r][e] = fmaf(f, x[e], acc[j][r][e]);
        }
        cur[q][j] = next[q][j];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NW; j++) {
#pragma unroll
    for (int r = 0; r < R; r++) {
      if (r >= a.rows) break;
      __syncthreads();
#pragma unroll
      for (int e = 0; e < V; e++) red[warp][lane * V + e] = acc[j][r][e];
      __syncthreads();
      for (int c = threadIdx.x; c < 32 * V; c += kRowsThreads) {
        const int64_t n = (int64_t)blockIdx.x * 32 * V + c;
        float v = 0.f;
#pragma unroll
        for (int q = 0; q < kRowsWarps; q++) v += red[q][c];
        if (n < a.N) a.out[(((int64_t)blockIdx.y * NW + j) * a.rows + r) * a.N + n] = v;
      }
    }
  }
}

// y[i] = sum_s partial[s][i] (+ add[i]), rounded once.
template <typename T>
__global__ void __launch_bounds__(256) dsa3d_ffn_rows_join_kernel(const float* partial, int parts,
                                                                  const T* add, T* y, int n) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  prior_kernel_done();
  if (i >= n) return;
  float v = 0.f;
#pragma unroll 8
  for (int s = 0; s < parts; s++) v += partial[(int64_t)s * n + i];
  if (add) v += to_f32(add[i]);
  y[i] = from_f32<T>(v);
}

}  // namespace dsa3d
