// dsa3d_norm.cuh -- layer norm over the channels of each token, forward and backward.
//
//   h = x (+ add, rounded to the I/O type)      m = mean_c h      r = (mean_c (h - m)^2 + eps)^(-1/2)
//   y = (h - m) r w + b
// and for the upstream gradient dy, with xh = (h - m) r and g = dy w:
//   dx = r (g - mean_c g - xh mean_c(g xh)) (+ add)      dw = sum_n dy xh      db = sum_n dy
//
// Both passes are bound by HBM: a forward reads x (and add) and writes y (and h) once, a backward
// reads h, dy (and add) and writes dx once.  A group of TX threads owns one row at a time, each
// thread the same columns of every row it meets, so that a row is held in registers between its
// reductions, the weights are read once per block and the weight gradient's sums stay in registers
// (one partial row per block, added in a fixed order by dsa3d_norm_reduce_kernel: the result does
// not depend on scheduling).  The variance is the centred sum of squares of the row in registers,
// not E[h^2] - m^2.  All sums are fp32.
#pragma once

#include <stdint.h>

#include "dsa3d_vec.cuh"

namespace dsa3d {

constexpr int kNormMaxThreads = 512;
constexpr int kNormMaxWarps = kNormMaxThreads / 32;

// Sum v[0..R) over the TX threads of the caller's group: every thread of the group gets the sums.
// TX is a power of two up to 32, or a multiple of 32; the whole block calls it.  buf is one of two
// shared buffers that consecutive calls alternate between, so one barrier per call is enough: a
// buffer is written again only after the other buffer's barrier, which every reader has passed.
template <int R>
__device__ __forceinline__ void group_sum(float (&v)[R], int TX, float (*buf)[R]) {
  if (TX < 32) {
    for (int o = TX >> 1; o > 0; o >>= 1) {
#pragma unroll
      for (int i = 0; i < R; i++) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
    return;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
    for (int i = 0; i < R; i++) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  }
  if (TX == 32) return;
  const int warp = threadIdx.x >> 5, nw = TX >> 5;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < R; i++) buf[warp][i] = v[i];
  }
  __syncthreads();
  const int w0 = warp / nw * nw;
#pragma unroll
  for (int i = 0; i < R; i++) v[i] = 0.f;
  for (int w = 0; w < nw; w++) {
#pragma unroll
    for (int i = 0; i < R; i++) v[i] += buf[w0 + w][i];
  }
}

// Block: TX * TY threads; group ty takes R consecutive rows per step.  nv = C / V vectors per row,
// nv <= TX * PER.
template <typename T, int V, int PER, int R>
__global__ void __launch_bounds__(kNormMaxThreads) dsa3d_layer_norm_kernel(
    const T* x, const T* add, const float* __restrict__ weight, const float* __restrict__ bias,
    T* __restrict__ y, T* h, float* __restrict__ stats,  // h may be x or add itself
    int64_t N, int C, float eps, int TX) {
  __shared__ float red[2][kNormMaxWarps][R];
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX, TY = blockDim.x / TX;
  const int nv = C / V;
  const float inv_c = 1.f / (float)C;
  constexpr bool kKeep = PER * V <= 16;  // weights in registers, else read again for every row (L1)
  float wr[kKeep ? PER : 1][V], br[kKeep ? PER : 1][V];
  auto load_affine = [&](int c, float (&w)[V], float (&b)[V]) {
#pragma unroll
    for (int e = 0; e < V; e++) {
      w[e] = weight ? __ldg(weight + (int64_t)c * V + e) : 1.f;
      b[e] = bias ? __ldg(bias + (int64_t)c * V + e) : 0.f;
    }
  };
  if (kKeep) {
#pragma unroll
    for (int p = 0; p < PER; p++) {
      const int c = tx + p * TX;
      if (c < nv) load_affine(c, wr[p], br[p]);
    }
  }
  for (int64_t row0 = (int64_t)blockIdx.x * TY * R; row0 < N; row0 += (int64_t)gridDim.x * TY * R) {
    const int64_t base = row0 + (int64_t)ty * R;
    Vec<T, V> xv[R][PER];
#pragma unroll
    for (int r = 0; r < R; r++) {
#pragma unroll
      for (int p = 0; p < PER; p++) {
        const int c = tx + p * TX;
        if (c < nv && base + r < N)
          xv[r][p].load(x + (base + r) * C + (int64_t)c * V);
        else
          xv[r][p].zero();
      }
    }
    if (add) {
      Vec<T, V> av[R][PER];
#pragma unroll
      for (int r = 0; r < R; r++) {
#pragma unroll
        for (int p = 0; p < PER; p++) {
          const int c = tx + p * TX;
          if (c < nv && base + r < N) av[r][p].load(add + (base + r) * C + (int64_t)c * V);
        }
      }
#pragma unroll
      for (int r = 0; r < R; r++) {
#pragma unroll
        for (int p = 0; p < PER; p++) {
          const int c = tx + p * TX;
          if (c < nv && base + r < N) {
            float a[V], b[V];
            xv[r][p].get(a);
            av[r][p].get(b);
#pragma unroll
            for (int e = 0; e < V; e++) a[e] += b[e];
            xv[r][p].set(a);  // the sum is rounded to the I/O type: h, not x + add, is normalised
            xv[r][p].store(h + (base + r) * C + (int64_t)c * V);
          }
        }
      }
    }
    float s[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
      s[r] = 0.f;
#pragma unroll
      for (int p = 0; p < PER; p++) {
        float a[V];
        xv[r][p].get(a);
#pragma unroll
        for (int e = 0; e < V; e++) s[r] += a[e];
      }
    }
    group_sum<R>(s, TX, red[0]);
    float mean[R], q[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
      mean[r] = s[r] / (float)C;  // a division: a constant row's mean is its value, whatever C is
      q[r] = 0.f;
#pragma unroll
      for (int p = 0; p < PER; p++) {
        if (tx + p * TX < nv) {
          float a[V];
          xv[r][p].get(a);
#pragma unroll
          for (int e = 0; e < V; e++) {
            const float d = a[e] - mean[r];
            q[r] = fmaf(d, d, q[r]);
          }
        }
      }
    }
    group_sum<R>(q, TX, red[1]);
#pragma unroll
    for (int r = 0; r < R; r++) {
      if (base + r >= N) continue;
      const float rstd = 1.f / sqrtf(fmaf(q[r], inv_c, eps));
      if (stats && tx == 0) {
        stats[base + r] = mean[r];
        stats[N + base + r] = rstd;
      }
#pragma unroll
      for (int p = 0; p < PER; p++) {
        const int c = tx + p * TX;
        if (c < nv) {
          float a[V], w[V], b[V];
          xv[r][p].get(a);
          if (!kKeep) load_affine(c, w, b);
#pragma unroll
          for (int e = 0; e < V; e++)
            a[e] = fmaf((a[e] - mean[r]) * rstd, kKeep ? wr[kKeep ? p : 0][e] : w[e],
                        kKeep ? br[kKeep ? p : 0][e] : b[e]);
          Vec<T, V> o;
          o.set(a);
          o.store(y + (base + r) * C + (int64_t)c * V);
        }
      }
    }
  }
}

// dx, and per block one row of partial sums [2][C] (dw, db) at partial + blockIdx.x * 2 * C when
// weight is not null.
template <typename T, int V, int PER, int R>
__global__ void __launch_bounds__(kNormMaxThreads) dsa3d_layer_norm_bwd_kernel(
    const T* __restrict__ h, const float* __restrict__ weight, const float* __restrict__ stats,
    const T* __restrict__ dy, const T* add, T* dx, float* __restrict__ partial,  // dx may be add itself
    int64_t N, int C, int TX) {
  __shared__ float red[2][kNormMaxWarps][2 * R];
  __shared__ float comb[kNormMaxThreads];
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX, TY = blockDim.x / TX;
  const int nv = C / V;
  const float inv_c = 1.f / (float)C;
  float wr[PER][V], aw[PER][V], ab[PER][V];
#pragma unroll
  for (int p = 0; p < PER; p++) {
    const int c = tx + p * TX;
#pragma unroll
    for (int e = 0; e < V; e++) {
      wr[p][e] = (weight && c < nv) ? __ldg(weight + (int64_t)c * V + e) : 1.f;
      aw[p][e] = ab[p][e] = 0.f;
    }
  }
  int flip = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * TY * R; row0 < N; row0 += (int64_t)gridDim.x * TY * R) {
    const int64_t base = row0 + (int64_t)ty * R;
    Vec<T, V> hv[R][PER], gv[R][PER];
    float mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
      const bool in = base + r < N;
      mean[r] = in ? __ldg(stats + base + r) : 0.f;
      rstd[r] = in ? __ldg(stats + N + base + r) : 0.f;
#pragma unroll
      for (int p = 0; p < PER; p++) {
        const int c = tx + p * TX;
        if (c < nv && in) {
          hv[r][p].load(h + (base + r) * C + (int64_t)c * V);
          gv[r][p].load(dy + (base + r) * C + (int64_t)c * V);
        } else {
          hv[r][p].zero();
          gv[r][p].zero();
        }
      }
    }
    float s[2 * R];
#pragma unroll
    for (int r = 0; r < R; r++) {
      s[2 * r] = s[2 * r + 1] = 0.f;
#pragma unroll
      for (int p = 0; p < PER; p++) {
        if (tx + p * TX < nv && base + r < N) {
          float a[V], d[V];
          hv[r][p].get(a);
          gv[r][p].get(d);
#pragma unroll
          for (int e = 0; e < V; e++) {
            const float xh = (a[e] - mean[r]) * rstd[r], g = d[e] * wr[p][e];
            s[2 * r] += g;
            s[2 * r + 1] = fmaf(g, xh, s[2 * r + 1]);
            aw[p][e] = fmaf(d[e], xh, aw[p][e]);
            ab[p][e] += d[e];
          }
        }
      }
    }
    group_sum<2 * R>(s, TX, red[flip]);
    flip ^= 1;
#pragma unroll
    for (int r = 0; r < R; r++) {
      if (base + r >= N) continue;
      const float c1 = s[2 * r] * inv_c, c2 = s[2 * r + 1] * inv_c;
#pragma unroll
      for (int p = 0; p < PER; p++) {
        const int c = tx + p * TX;
        if (c < nv) {
          const int64_t at = (base + r) * C + (int64_t)c * V;
          float a[V], d[V], o[V];
          hv[r][p].get(a);
          gv[r][p].get(d);
#pragma unroll
          for (int e = 0; e < V; e++) {
            const float xh = (a[e] - mean[r]) * rstd[r], g = d[e] * wr[p][e];
            o[e] = rstd[r] * (g - c1 - xh * c2);
          }
          if (add) {
            Vec<T, V> av;
            av.load(add + at);
            av.get(a);
#pragma unroll
            for (int e = 0; e < V; e++) o[e] += a[e];
          }
          Vec<T, V> ov;
          ov.set(o);
          ov.store(dx + at);
        }
      }
    }
  }
  if (!partial) return;
  float* out = partial + (int64_t)blockIdx.x * 2 * C;
#pragma unroll
  for (int p = 0; p < PER; p++) {
    const int c = tx + p * TX;
#pragma unroll
    for (int e = 0; e < V; e++) {
#pragma unroll
      for (int k = 0; k < 2; k++) {
        float v = k ? ab[p][e] : aw[p][e];
        if (TY > 1) {  // add the groups' sums in order
          __syncthreads();
          comb[threadIdx.x] = v;
          __syncthreads();
          v = 0.f;
          if (ty == 0)
            for (int j = 0; j < TY; j++) v += comb[j * TX + tx];
        }
        if (ty == 0 && c < nv) out[(int64_t)k * C + (int64_t)c * V + e] = v;
      }
    }
  }
}

// dw and db (each [C]) = the sum of P partial rows [2 C], in a fixed order.  Block 32 x 32: 32 columns.
__global__ void __launch_bounds__(1024) dsa3d_norm_reduce_kernel(const float* __restrict__ partial, int P,
                                                                 int C, float* __restrict__ dw,
                                                                 float* __restrict__ db) {
  __shared__ float s[32][33];
  const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.x;
  const int64_t width = 2 * (int64_t)C;
  float v = 0.f;
  if (col < width) {
#pragma unroll 4
    for (int p = threadIdx.y; p < P; p += 32) v += partial[p * width + col];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = s[threadIdx.x][threadIdx.y];  // warp y holds column y's 32 sums
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && c < width) {
    if (c < C)
      dw[c] = v;
    else
      db[c - C] = v;
  }
}

}  // namespace dsa3d
