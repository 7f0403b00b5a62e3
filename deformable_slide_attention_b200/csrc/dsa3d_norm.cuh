// dsa3d_norm.cuh -- layer norm over the channels of each token, forward and backward.
//
//   h = x (+ add, rounded to the I/O type)      m = mean_c h      r = (mean_c (h - m)^2 + eps)^(-1/2)
//   y = (h - m) r w + b
// and for the upstream gradient dy, with xh = (h - m) r and g = dy w:
//   dx = r (g - mean_c g - xh mean_c(g xh)) (+ add)      dw = sum_n dy xh      db = sum_n dy
//
// Both passes are bound by HBM: a forward reads x (and add) and writes y (and h) once, a backward
// reads h, dy (and add) and writes dx once.  A group of TX threads owns R rows at a time, each
// thread the same columns of every row it meets, so that a row is held in registers between its
// reductions, the weights are read once per block and the weight gradient's sums stay in registers
// (one partial row per block, added in a fixed order by dsa3d_norm_reduce_kernel: the result does
// not depend on scheduling).  The variance is the centred sum of squares of the row in registers,
// not E[h^2] - m^2.  All sums are fp32.
#pragma once

#include <stdint.h>

#include "dsa3d_tc.cuh"
#include "dsa3d_vec.cuh"

namespace dsa3d {

// Threads of a block: 256, or up to 512 for rows that need them at two vectors per thread (more vectors
// than that and the weights no longer fit in registers).
constexpr int kNormThreads = 256, kNormWideThreads = 512;
constexpr int kNormMaxWarps = kNormWideThreads / 32;
constexpr int norm_max_threads(int per, int r) { return per == 2 && r == 1 ? kNormWideThreads : kNormThreads; }

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

// ---- fp32 vectors in packed pairs: one instruction for two sums or products (V = 1: plain ones) ------
template <int V>
struct F32s {
  uint64_t p[V / 2];
  __device__ __forceinline__ void set(const float (&x)[V]) {
#pragma unroll
    for (int i = 0; i < V / 2; i++) p[i] = pack2(x[2 * i], x[2 * i + 1]);
  }
  __device__ __forceinline__ void get(float (&x)[V]) const {
#pragma unroll
    for (int i = 0; i < V / 2; i++) unpack2(p[i], x[2 * i], x[2 * i + 1]);
  }
  __device__ __forceinline__ void fill(float v) {
#pragma unroll
    for (int i = 0; i < V / 2; i++) p[i] = pack2(v, v);
  }
  // the sum of the elements
  __device__ __forceinline__ float total() const {
    uint64_t t = p[0];
#pragma unroll
    for (int i = 1; i < V / 2; i++) t = add2(t, p[i]);
    float a, b;
    unpack2(t, a, b);
    return a + b;
  }
};
template <>
struct F32s<1> {
  float p[1];
  __device__ __forceinline__ void set(const float (&x)[1]) { p[0] = x[0]; }
  __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = p[0]; }
  __device__ __forceinline__ void fill(float v) { p[0] = v; }
  __device__ __forceinline__ float total() const { return p[0]; }
};
template <int V>
__device__ __forceinline__ F32s<V> padd(const F32s<V>& a, const F32s<V>& b) {
  F32s<V> r;
#pragma unroll
  for (int i = 0; i < V / 2; i++) r.p[i] = add2(a.p[i], b.p[i]);
  return r;
}
template <int V>
__device__ __forceinline__ F32s<V> pmul(const F32s<V>& a, const F32s<V>& b) {
  F32s<V> r;
#pragma unroll
  for (int i = 0; i < V / 2; i++) r.p[i] = mul2(a.p[i], b.p[i]);
  return r;
}
template <int V>
__device__ __forceinline__ F32s<V> pfma(const F32s<V>& a, const F32s<V>& b, const F32s<V>& c) {
  F32s<V> r;
#pragma unroll
  for (int i = 0; i < V / 2; i++) r.p[i] = fma2(a.p[i], b.p[i], c.p[i]);
  return r;
}
template <>
__device__ __forceinline__ F32s<1> padd<1>(const F32s<1>& a, const F32s<1>& b) { return {{a.p[0] + b.p[0]}}; }
template <>
__device__ __forceinline__ F32s<1> pmul<1>(const F32s<1>& a, const F32s<1>& b) { return {{a.p[0] * b.p[0]}}; }
template <>
__device__ __forceinline__ F32s<1> pfma<1>(const F32s<1>& a, const F32s<1>& b, const F32s<1>& c) {
  return {{fmaf(a.p[0], b.p[0], c.p[0])}};
}
template <int V>
__device__ __forceinline__ F32s<V> splat(float v) {
  F32s<V> r;
  r.fill(v);
  return r;
}
template <typename T, int V>
__device__ __forceinline__ F32s<V> widen(const Vec<T, V>& v) {
  float x[V];
  v.get(x);
  F32s<V> r;
  r.set(x);
  return r;
}
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> narrow(const F32s<V>& v) {
  float x[V];
  v.get(x);
  Vec<T, V> r;
  r.set(x);
  return r;
}

// V consecutive fp32 weights of vector c; 16-byte loads where the weights are aligned to them.
template <int V>
__device__ __forceinline__ void load_weights(const float* p, int c, bool vec, float (&w)[V]) {
  if (V % 4 == 0 && vec) {
#pragma unroll
    for (int e = 0; e < V / 4; e++) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(p + (int64_t)c * V) + e);
      w[4 * e] = x.x;
      w[(4 * e + 1) % V] = x.y;
      w[(4 * e + 2) % V] = x.z;
      w[(4 * e + 3) % V] = x.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; e++) w[e] = __ldg(p + (int64_t)c * V + e);
  }
}

// Rows base .. base + R - 1 of a tensor: this thread's vectors, zero past the row's end or row N.
template <typename T, int V, int PER, int R>
__device__ __forceinline__ void load_rows(Vec<T, V> (&v)[R][PER], const T* p, int64_t base, int64_t N, int C, int nv,
                                          int tx, int TX) {
#pragma unroll
  for (int r = 0; r < R; r++) {
#pragma unroll
    for (int q = 0; q < PER; q++) {
      const int c = tx + q * TX;
      if (c < nv && base + r < N)
        v[r][q].load(p + (base + r) * C + (int64_t)c * V);
      else
        v[r][q].zero();
    }
  }
}

// A ring of shared-memory stages that one thread fills with whole rows by bulk copies (the rows of a step
// are contiguous), kRing - 1 steps ahead: the bytes in flight then cost no registers, and the reductions'
// barriers no longer leave HBM idle.  NT tensors per stage; rows of whole 16-byte units.
constexpr int kRing = 3;
template <int NT>
struct RowRing {
  uint32_t base, bars;
  uint32_t tensor_bytes;  // of one tensor's rows in a stage
  uint32_t row_bytes;
  int64_t N, first, step;  // rows; this block's first row; rows from one step to its next
  int rows;                // of a step
  const void* p[NT];
  volatile int* abort_flag;

  __device__ __forceinline__ void issue(int64_t it) const {  // one thread
    const int64_t row = first + it * step;
    if (row >= N) return;
    const uint32_t s = (uint32_t)(it % kRing), bytes = (uint32_t)min((int64_t)rows, N - row) * row_bytes;
    const uint32_t bar = bars + 8 * s;
    mbar_arrive_expect_tx(bar, NT * bytes);
#pragma unroll
    for (int k = 0; k < NT; k++)
      asm volatile(
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
              base + (s * NT + k) * tensor_bytes),
          "l"(static_cast<const char*>(p[k]) + row * row_bytes), "r"(bytes), "r"(bar)
          : "memory");
  }
  __device__ __forceinline__ void start() const {
    if (threadIdx.x == 0) {
      for (int s = 0; s < kRing; s++) mbar_init(bars + 8 * s, 1);
      *abort_flag = 0;
      mbar_fence_init();
      for (int s = 0; s < kRing; s++) issue(s);
    }
    __syncthreads();
  }
  __device__ __forceinline__ void wait(int64_t it) const {
    mbar_wait(bars + 8 * (uint32_t)(it % kRing), (uint32_t)(it / kRing) & 1u, abort_flag);
  }
  // After a wait that ran out (every step is issued and waited for all the same): the copies still in
  // flight end before the block's shared memory is released.  steps: all of the block's.
  __device__ __forceinline__ void finish(int64_t steps) const {
    if (threadIdx.x != 0 || *abort_flag == 0) return;
    for (int s = 0; s < kRing; s++) {
      const int64_t uses = steps > s ? (steps - s + kRing - 1) / kRing : 0;
      if (uses) mbar_drain(bars + 8 * s, (uint32_t)(uses - 1) & 1u, abort_flag);
    }
  }
};

// This thread's vectors of R rows of tensor k of stage it % kRing; zero past the row's end or row N.
template <typename T, int V, int PER, int R, int NT>
__device__ __forceinline__ void ring_rows(Vec<T, V> (&v)[R][PER], const RowRing<NT>& ring, const uint8_t* mem, int k,
                                          int64_t it, int64_t base, int64_t N, int C, int nv, int tx, int ty, int TX) {
  const T* from = reinterpret_cast<const T*>(mem + ((it % kRing) * NT + k) * ring.tensor_bytes) + (int64_t)ty * R * C;
#pragma unroll
  for (int r = 0; r < R; r++) {
#pragma unroll
    for (int q = 0; q < PER; q++) {
      const int c = tx + q * TX;
      if (c < nv && base + r < N)
        v[r][q].load(from + r * C + c * V);
      else
        v[r][q].zero();
    }
  }
}

// Block: TX * TY threads; group ty takes R consecutive rows per step.  nv = C / V vectors per row,
// nv <= TX * PER.  The next step's rows are loaded into registers before this step's are reduced: the
// two reductions and their barriers would otherwise leave HBM idle.  Bound by HBM where rows are wide:
// 115,200 x 2048 bf16, residual sum included, 299 to 312 us (6.0 to 6.3 TB/s, 92 to 96% of a copy's rate;
// without the sum 178 to 182 us, 80%: the element-wise work, halved by packed pairs, is then half the issue slots).
template <typename T, int V, int PER, int R, bool ADD>
__global__ void __launch_bounds__(norm_max_threads(PER, R)) dsa3d_layer_norm_kernel(
    const T* x, const T* add_to, const float* __restrict__ weight, const float* __restrict__ bias,
    T* __restrict__ y, T* h, float* __restrict__ stats,  // h may be x or add_to itself
    int64_t N, int C, float eps, int TX, bool vec) {     // vec: 16-byte aligned weights
  __shared__ float red[2][kNormMaxWarps][R];
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX, TY = blockDim.x / TX;
  const int nv = C / V;
  const float inv_c = 1.f / (float)C;
  constexpr bool kKeep = PER * V <= 16;  // weights in registers, else read again for every row (L1)
  F32s<V> wr[kKeep ? PER : 1], br[kKeep ? PER : 1];
  auto load_affine = [&](int c, F32s<V>& w, F32s<V>& b) {
    float wv[V], bv[V];
#pragma unroll
    for (int e = 0; e < V; e++) {
      wv[e] = 1.f;
      bv[e] = 0.f;
    }
    if (weight) load_weights<V>(weight, c, vec, wv);
    if (bias) load_weights<V>(bias, c, vec, bv);
    w.set(wv);
    b.set(bv);
  };
  if (kKeep) {
#pragma unroll
    for (int p = 0; p < PER; p++) {
      const int c = tx + p * TX;
      if (c < nv) load_affine(c, wr[p], br[p]);
    }
  }
  const int64_t step = (int64_t)gridDim.x * TY * R;
  int64_t base = ((int64_t)blockIdx.x * TY + ty) * R;
  Vec<T, V> xn[R][PER], an[ADD ? R : 1][PER];
  load_rows(xn, x, base, N, C, nv, tx, TX);
  if constexpr (ADD) load_rows(an, add_to, base, N, C, nv, tx, TX);
  for (int64_t row0 = (int64_t)blockIdx.x * TY * R; row0 < N; row0 += step, base += step) {
    F32s<V> xv[R][PER];
    float s[R], q[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
#pragma unroll
      for (int p = 0; p < PER; p++) {
        xv[r][p] = widen(xn[r][p]);
        if constexpr (ADD) {
          const int c = tx + p * TX;
          // the sum is rounded to the I/O type: h, not x + add, is normalised
          const Vec<T, V> sum = narrow<T>(padd(xv[r][p], widen(an[r][p])));
          xv[r][p] = widen(sum);
          if (c < nv && base + r < N) sum.store(h + (base + r) * C + (int64_t)c * V);
        }
      }
      F32s<V> t = xv[r][0];
#pragma unroll
      for (int p = 1; p < PER; p++) t = padd(t, xv[r][p]);
      s[r] = t.total();
    }
    load_rows(xn, x, base + step, N, C, nv, tx, TX);
    if constexpr (ADD) load_rows(an, add_to, base + step, N, C, nv, tx, TX);
    group_sum<R>(s, TX, red[0]);
#pragma unroll
    for (int r = 0; r < R; r++) {
      s[r] = s[r] / (float)C;  // a division: a constant row's mean is its value, whatever C is
      const F32s<V> less = splat<V>(-s[r]);
      F32s<V> t = splat<V>(0.f);
#pragma unroll
      for (int p = 0; p < PER; p++) {
        xv[r][p] = padd(xv[r][p], less);
        if (tx + p * TX < nv) t = pfma(xv[r][p], xv[r][p], t);
      }
      q[r] = t.total();
    }
    group_sum<R>(q, TX, red[1]);
#pragma unroll
    for (int r = 0; r < R; r++) {
      if (base + r >= N) continue;
      const float rstd = 1.f / sqrtf(fmaf(q[r], inv_c, eps));
      if (stats && tx == 0) {
        stats[base + r] = s[r];
        stats[N + base + r] = rstd;
      }
      const F32s<V> rs = splat<V>(rstd);
#pragma unroll
      for (int p = 0; p < PER; p++) {
        const int c = tx + p * TX;
        if (c < nv) {
          F32s<V> w, b;
          if (kKeep) {
            w = wr[kKeep ? p : 0];
            b = br[kKeep ? p : 0];
          } else {
            load_affine(c, w, b);
          }
          narrow<T>(pfma(pmul(xv[r][p], rs), w, b)).store(y + (base + r) * C + (int64_t)c * V);
        }
      }
    }
  }
}

// dx, and per block one row of partial sums [2][C] (dw, db) at partial + blockIdx.x * 2 * C when
// weight is not null.  RING: rows come through a RowRing (the column sums leave no registers for rows in
// flight); else plain loads, for odd widths and rows too wide for it.  115,200 x 2048 bf16 with the
// residual gradient: 308 to 318 us (5.9 to 6.1 TB/s, 90 to 93% of a copy's rate); plain loads 332 us at best.
template <typename T, int V, int PER, int R, bool ADD, bool RING>
__global__ void __launch_bounds__(norm_max_threads(PER, R)) dsa3d_layer_norm_bwd_kernel(
    const T* __restrict__ h, const float* __restrict__ weight, const float* __restrict__ stats,
    const T* __restrict__ dy, const T* add_to, T* dx, float* __restrict__ partial,  // dx may be add_to itself
    int64_t N, int C, int TX, bool vec) {
  extern __shared__ __align__(128) uint8_t norm_ring[];
  __shared__ uint64_t ring_bars[kRing];
  __shared__ int ring_abort;
  __shared__ float red[2][kNormMaxWarps][2 * R];
  __shared__ float comb[kNormWideThreads];
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX, TY = blockDim.x / TX;
  const int nv = C / V;
  const float inv_c = 1.f / (float)C;
  constexpr bool kKeep = PER * V <= 16;  // the weight in registers, else read again for every row (L1)
  F32s<V> wr[kKeep ? PER : 1], aw[PER], ab[PER];
  auto load_weight = [&](int c) {
    float w[V];
#pragma unroll
    for (int e = 0; e < V; e++) w[e] = 1.f;
    if (weight && c < nv) load_weights<V>(weight, c, vec, w);
    F32s<V> r;
    r.set(w);
    return r;
  };
#pragma unroll
  for (int p = 0; p < PER; p++) {
    if (kKeep) wr[kKeep ? p : 0] = load_weight(tx + p * TX);
    aw[p].fill(0.f);
    ab[p].fill(0.f);
  }
  const int64_t step = (int64_t)gridDim.x * TY * R;
  int64_t base = ((int64_t)blockIdx.x * TY + ty) * R, it = 0;
  constexpr int NT = ADD ? 3 : 2;
  RowRing<NT> ring;
  if constexpr (RING) {
    ring.base = smem_u32(norm_ring);
    ring.bars = smem_u32(ring_bars);
    ring.abort_flag = &ring_abort;
    ring.row_bytes = C * (uint32_t)sizeof(T);
    ring.rows = TY * R;
    ring.tensor_bytes = ring.rows * ring.row_bytes;
    ring.N = N;
    ring.first = (int64_t)blockIdx.x * TY * R;
    ring.step = step;
    ring.p[0] = h;
    ring.p[1] = dy;
    if constexpr (ADD) ring.p[2] = add_to;
    ring.start();
  }
  int flip = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * TY * R; row0 < N; row0 += step, base += step, it++) {
    Vec<T, V> hv[R][PER], gv[R][PER], av[RING && ADD ? R : 1][PER];
    float mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
      const bool in = base + r < N;
      mean[r] = in ? __ldg(stats + base + r) : 0.f;
      rstd[r] = in ? __ldg(stats + N + base + r) : 0.f;
    }
    if constexpr (RING) {
      ring.wait(it);
      ring_rows(hv, ring, norm_ring, 0, it, base, N, C, nv, tx, ty, TX);
      ring_rows(gv, ring, norm_ring, 1, it, base, N, C, nv, tx, ty, TX);
      if constexpr (ADD) ring_rows(av, ring, norm_ring, 2, it, base, N, C, nv, tx, ty, TX);
    } else {
      load_rows(hv, h, base, N, C, nv, tx, TX);
      load_rows(gv, dy, base, N, C, nv, tx, TX);
    }
    float s[2 * R];
#pragma unroll
    for (int r = 0; r < R; r++) {
      const F32s<V> less = splat<V>(-mean[r]), rs = splat<V>(rstd[r]);
      F32s<V> t1 = splat<V>(0.f), t2 = t1;
#pragma unroll
      for (int p = 0; p < PER; p++) {
        // past the row's end or the last row: dy is zero there, and xh is made so
        const bool in = tx + p * TX < nv && base + r < N;
        const F32s<V> d = widen(gv[r][p]);
        const F32s<V> xh = in ? pmul(padd(widen(hv[r][p]), less), rs) : splat<V>(0.f);
        const F32s<V> g = pmul(d, kKeep ? wr[kKeep ? p : 0] : load_weight(tx + p * TX));
        t1 = padd(t1, g);
        t2 = pfma(g, xh, t2);
        aw[p] = pfma(d, xh, aw[p]);
        ab[p] = padd(ab[p], d);
      }
      s[2 * r] = t1.total();
      s[2 * r + 1] = t2.total();
    }
    group_sum<2 * R>(s, TX, red[flip]);
    flip ^= 1;
    if constexpr (RING) {
      if (TX <= 32) __syncthreads();  // (a wider row's sum has just passed a barrier)
      if (threadIdx.x == 0) ring.issue(it + kRing);  // every thread has read its part of this stage
    }
#pragma unroll
    for (int r = 0; r < R; r++) {
      if (base + r >= N) continue;
      const F32s<V> c1 = splat<V>(-s[2 * r] * inv_c), c2 = splat<V>(-s[2 * r + 1] * inv_c), rs = splat<V>(rstd[r]);
      const F32s<V> less = splat<V>(-mean[r]);
#pragma unroll
      for (int p = 0; p < PER; p++) {
        const int c = tx + p * TX;
        if (c < nv) {
          // xh and g again from the row as it was loaded: half the registers of keeping them
          const int64_t at = (base + r) * C + (int64_t)c * V;
          const F32s<V> xh = pmul(padd(widen(hv[r][p]), less), rs);
          const F32s<V> g = pmul(widen(gv[r][p]), kKeep ? wr[kKeep ? p : 0] : load_weight(c));
          const F32s<V> t = pfma(xh, c2, padd(g, c1));
          F32s<V> o;
          if constexpr (ADD && RING) {
            o = pfma(t, rs, widen(av[r][p]));
          } else if constexpr (ADD) {
            Vec<T, V> a;
            a.load(add_to + at);
            o = pfma(t, rs, widen(a));
          } else {
            o = pmul(t, rs);
          }
          narrow<T>(o).store(dx + at);
        }
      }
    }
  }
  if constexpr (RING) ring.finish(it);
  next_kernel_may_start();
  if (!partial) return;
  float* out = partial + (int64_t)blockIdx.x * 2 * C;
#pragma unroll
  for (int p = 0; p < PER; p++) {
    const int c = tx + p * TX;
    float sw[V], sb[V];
    aw[p].get(sw);
    ab[p].get(sb);
#pragma unroll
    for (int e = 0; e < V; e++) {
#pragma unroll
      for (int k = 0; k < 2; k++) {
        float v = k ? sb[e] : sw[e];
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
__global__ void __launch_bounds__(1024) dsa3d_norm_reduce_kernel(const float* partial, int P, int C, float* dw,
                                                                 float* db) {
  __shared__ float s[32][33];
  const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.x;
  const int64_t width = 2 * (int64_t)C;
  float v = 0.f;
  prior_kernel_done();
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
