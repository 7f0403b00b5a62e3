// dsa3d_vec.cuh -- vectors of I/O-type elements as raw bits (16 bytes, or one element where rows or
// pointers are not 16-byte aligned) and their fp32 values, for the element-wise kernels of the
// transformer block (layer norm, rotary positions, the feed-forward block's helpers).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace dsa3d {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// For kernels launched early (launch_early): waits until the stream's previous kernel is complete and its
// writes are visible; and, in that previous kernel, allows the next one's blocks to start.  What the previous
// kernel writes is not read-only for the life of one that starts early: it is read by ordinary loads after
// the wait, never through __ldg or a const __restrict__ pointer (such loads may be moved over the wait).
__device__ __forceinline__ void prior_kernel_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void next_kernel_may_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Two fp32 values in 64 bits: one instruction for two sums, products or multiply-adds.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// V elements of T: V * sizeof(T) == 16, or V == 1.
template <typename T, int V>
struct Vec;

template <typename T>
struct Vec<T, 1> {
  T raw;
  __device__ __forceinline__ void load(const T* p) { raw = *p; }
  __device__ __forceinline__ void store(T* p) const { *p = raw; }
  __device__ __forceinline__ void zero() { raw = from_f32<T>(0.f); }
  __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = to_f32(raw); }
  __device__ __forceinline__ void set(const float (&x)[1]) { raw = from_f32<T>(x[0]); }
};

template <>
struct Vec<float, 4> {
  float4 raw;
  __device__ __forceinline__ void load(const float* p) { raw = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = raw; }
  __device__ __forceinline__ void zero() { raw = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&x)[4]) const {
    x[0] = raw.x; x[1] = raw.y; x[2] = raw.z; x[3] = raw.w;
  }
  __device__ __forceinline__ void set(const float (&x)[4]) { raw = make_float4(x[0], x[1], x[2], x[3]); }
  // elements 2 e and 2 e + 1 (e a constant) from another vector, bit for bit
  __device__ __forceinline__ void copy_pair(int e, const Vec& o) {
    if (e == 0) { raw.x = o.raw.x; raw.y = o.raw.y; } else { raw.z = o.raw.z; raw.w = o.raw.w; }
  }
};

template <>
struct Vec<__nv_bfloat16, 8> {
  uint4 raw;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { raw = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = raw; }
  __device__ __forceinline__ void zero() { raw = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const unsigned w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const unsigned*>(&b);
    }
    raw = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void copy_pair(int e, const Vec& o) {
    if (e == 0) raw.x = o.raw.x;
    if (e == 1) raw.y = o.raw.y;
    if (e == 2) raw.z = o.raw.z;
    if (e == 3) raw.w = o.raw.w;
  }
};

// Elements of a 16-byte vector of T.
template <typename T>
constexpr int vec_width() { return 16 / (int)sizeof(T); }

}  // namespace dsa3d
