// dsa3d_rotary.cuh -- rotary positions with three axes (frame, row, column) for q and k.
//
// A head's first R = at + ay + ax dims are R/2 pairs; the pairs are shared out to the axes in order.
// Pair j of axis a turns by theta = (start_a + step_a * index_a) * base^(-2 j / axis size):
//   (x0, x1) -> (x0 cos - x1 sin, x0 sin + x1 cos),  the backward pass by -theta.
// Pair i is dims (2i, 2i+1), or (i, i + R/2) in the halves layout; dims from R on are copied.
//
// The operation is bound by HBM (q and k read and written once).  A thread computes the sines and
// cosines of one 16-byte vector's pairs for one token and uses them for several heads of q and k,
// whose loads it issues together.  The angle is formed and reduced to [-pi, pi] in fp64, since fp32
// loses a position of 10^5 to 10^-2 of a radian; the sine and cosine of the reduced angle are fp32.
#pragma once

#include <stdint.h>

#include "dsa3d_vec.cuh"

namespace dsa3d {

constexpr int kRotMaxDh = 256;
constexpr int kRotThreads = 256;

struct RotArgs {
  double freq[kRotMaxDh / 2];  // angular frequency of each pair, in units of pi (negated: backward)
  double start[3], step[3];
  int64_t ld[4];  // token strides in elements: q, k, q_out, k_out
  int64_t rows, first;
  int HW, Wp, heads, dh;
  int half;        // R / 2
  int end0, end1;  // first pair of the second and of the third axis
  bool has_k;
};

__device__ __forceinline__ void rot_position(const RotArgs& a, int64_t row, double (&pos)[3]) {
  const uint32_t n = (uint32_t)(a.first + row);
  const uint32_t t = n / (uint32_t)a.HW, in = n - t * (uint32_t)a.HW;
  const uint32_t y = in / (uint32_t)a.Wp, x = in - y * (uint32_t)a.Wp;
  pos[0] = fma(a.step[0], (double)t, a.start[0]);
  pos[1] = fma(a.step[1], (double)y, a.start[1]);
  pos[2] = fma(a.step[2], (double)x, a.start[2]);
}

__device__ __forceinline__ void rot_angle(const RotArgs& a, const double (&pos)[3], int i, float& c, float& s) {
  if (i >= a.half) {  // past the rotated dims
    c = 1.f;
    s = 0.f;
    return;
  }
  const double p = i < a.end0 ? pos[0] : (i < a.end1 ? pos[1] : pos[2]);
  double t = p * a.freq[i];
  t = fma(-2.0, rint(0.5 * t), t);  // in units of pi, reduced to [-1, 1]
  sincospif((float)t, &s, &c);
}

// 16-byte vectors; HG heads per thread.  Units of a token: (group of heads, vector of the head);
// interleaved: dh / V vectors of V/2 pairs; halves: half / V pairs of vectors, then the copied ones.
template <typename T, bool INTER, int HG>
__global__ void __launch_bounds__(kRotThreads) dsa3d_rotary_kernel(const T* q, const T* k, T* qo, T* ko,
                                                                  const __grid_constant__ RotArgs a) {
  constexpr int V = vec_width<T>();
  constexpr int NP = INTER ? V / 2 : V;  // pairs per unit
  const int pair_units = INTER ? a.dh / V : a.half / V;
  const int upr = INTER ? pair_units : pair_units + (a.dh - 2 * a.half) / V;
  const int groups = (a.heads + HG - 1) / HG;
  const int per_token = upr * groups;
  const int64_t total = a.rows * per_token;
  for (int64_t unit = (int64_t)blockIdx.x * kRotThreads + threadIdx.x; unit < total;
       unit += (int64_t)gridDim.x * kRotThreads) {
    const int64_t row = unit / per_token;
    const int in = (int)(unit - row * per_token);
    const int g = in / upr, u = in - g * upr;
    const bool pair = u < pair_units;
    const int d0 = INTER ? u * V : (pair ? u * V : 2 * a.half + (u - pair_units) * V);
    Vec<T, V> v0[2][HG], v1[INTER ? 1 : 2][INTER ? 1 : HG];
#pragma unroll
    for (int t = 0; t < 2; t++) {
      if (t == 1 && !a.has_k) break;
      const T* src = (t ? k : q) + row * a.ld[t] + d0;
#pragma unroll
      for (int i = 0; i < HG; i++) {
        const int hd = g + i * groups;  // heads of a group are `groups` apart: neighbours read on
        if (hd < a.heads) {
          v0[t][i].load(src + (int64_t)hd * a.dh);
          if (!INTER && pair) v1[INTER ? 0 : t][INTER ? 0 : i].load(src + (int64_t)hd * a.dh + a.half);
        }
      }
    }
    float c[NP], s[NP];
    if (INTER || pair) {
      double pos[3];
      rot_position(a, row, pos);
#pragma unroll
      for (int e = 0; e < NP; e++) rot_angle(a, pos, u * NP + e, c[e], s[e]);
    }
#pragma unroll
    for (int t = 0; t < 2; t++) {
      if (t == 1 && !a.has_k) break;
      T* dst = (t ? ko : qo) + row * a.ld[2 + t] + d0;
#pragma unroll
      for (int i = 0; i < HG; i++) {
        const int hd = g + i * groups;
        if (hd >= a.heads) continue;
        T* to = dst + (int64_t)hd * a.dh;
        float x[V];
        if (INTER) {
          const Vec<T, V> was = v0[t][i];
          was.get(x);
#pragma unroll
          for (int e = 0; e < V / 2; e++) {
            const float x0 = x[2 * e], x1 = x[2 * e + 1];
            x[2 * e] = x0 * c[e] - x1 * s[e];
            x[2 * e + 1] = x0 * s[e] + x1 * c[e];
          }
          v0[t][i].set(x);
          if ((u + 1) * NP > a.half) {  // copied dims keep their bits, an infinity's and a NaN's too
#pragma unroll
            for (int e = 0; e < V / 2; e++)
              if (u * NP + e >= a.half) v0[t][i].copy_pair(e, was);
          }
          v0[t][i].store(to);
        } else if (pair) {
          float z[V];
          v0[t][i].get(x);
          v1[INTER ? 0 : t][INTER ? 0 : i].get(z);
#pragma unroll
          for (int e = 0; e < V; e++) {
            const float x0 = x[e], x1 = z[e];
            x[e] = x0 * c[INTER ? 0 : e] - x1 * s[INTER ? 0 : e];
            z[e] = x0 * s[INTER ? 0 : e] + x1 * c[INTER ? 0 : e];
          }
          v0[t][i].set(x);
          v0[t][i].store(to);
          v0[t][i].set(z);
          v0[t][i].store(to + a.half);
        } else {
          v0[t][i].store(to);
        }
      }
    }
  }
}

// Any even dh, any alignment, halves that are no whole vectors: one pair, or one copied dim, of HG heads
// per unit (35,546 x 29 x 64 bf16 with halves of 31: 387 us with one head per unit, whose fp64 angle then
// binds).
template <typename T, bool INTER, int HG>
__global__ void __launch_bounds__(kRotThreads) dsa3d_rotary_any_kernel(const T* q, const T* k, T* qo, T* ko,
                                                                      const __grid_constant__ RotArgs a) {
  const int upr = a.half + (a.dh - 2 * a.half);
  const int groups = (a.heads + HG - 1) / HG;
  const int per_token = upr * groups;
  const int64_t total = a.rows * per_token;
  for (int64_t unit = (int64_t)blockIdx.x * kRotThreads + threadIdx.x; unit < total;
       unit += (int64_t)gridDim.x * kRotThreads) {
    const int64_t row = unit / per_token;
    const int in = (int)(unit - row * per_token);
    const int g = in / upr, u = in - g * upr;
    const bool pair = u < a.half;
    const int d0 = pair ? (INTER ? 2 * u : u) : 2 * a.half + (u - a.half);
    const int apart = pair ? (INTER ? 1 : a.half) : 0;
    T x0[2][HG], x1[2][HG];
#pragma unroll
    for (int t = 0; t < 2; t++) {
      if (t == 1 && !a.has_k) break;
      const T* src = (t ? k : q) + row * a.ld[t] + d0;
#pragma unroll
      for (int i = 0; i < HG; i++) {
        const int hd = g + i * groups;
        if (hd < a.heads) {
          x0[t][i] = src[(int64_t)hd * a.dh];
          x1[t][i] = src[(int64_t)hd * a.dh + apart];
        }
      }
    }
    float c = 1.f, s = 0.f;
    if (pair) {
      double pos[3];
      rot_position(a, row, pos);
      rot_angle(a, pos, u, c, s);
    }
#pragma unroll
    for (int t = 0; t < 2; t++) {
      if (t == 1 && !a.has_k) break;
      T* dst = (t ? ko : qo) + row * a.ld[2 + t] + d0;
#pragma unroll
      for (int i = 0; i < HG; i++) {
        const int hd = g + i * groups;
        if (hd >= a.heads) continue;
        T* to = dst + (int64_t)hd * a.dh;
        if (pair) {
          const float y0 = to_f32(x0[t][i]), y1 = to_f32(x1[t][i]);
          to[0] = from_f32<T>(y0 * c - y1 * s);
          to[apart] = from_f32<T>(y0 * s + y1 * c);
        } else {
          to[0] = x0[t][i];
        }
      }
    }
  }
}

}  // namespace dsa3d
