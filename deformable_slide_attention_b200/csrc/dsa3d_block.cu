// dsa3d_block.cu -- C ABI of layer norm and of the three-axis rotary positions (include/dsa3d.h):
// argument validation and launch configuration; the kernels are in dsa3d_norm.cuh and
// dsa3d_rotary.cuh.  This file allocates no device memory.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "dsa3d.h"
#include "dsa3d_host.cuh"
#include "dsa3d_norm.cuh"
#include "dsa3d_rotary.cuh"

namespace dsa3d {
namespace {

using namespace host;

constexpr int kNormMaxChannels = 16384;

// How rows are spread over threads: TX threads per row (a power of two up to 32, else whole warps),
// PER vectors per thread (a power of two), TY rows side by side in a block, R rows in flight per group
// of TX threads, and the blocks of a launch.
struct NormPlan {
  int v, tx, ty, per, r, blocks;
  bool ring;
  size_t smem;
};
// Two vectors per thread where a row has more than a warp's 32: fewer threads to sum over, and weights
// that still fit in registers.  odd_per: the same for rows read element by element, one number for both
// types.  30,000 x 1001: forward, 8 of them: fp32 62 us (66 and more at 2), bf16 with a sum 109 (111 at 4);
// backward, 4 of them and four blocks per SM: fp32 103 (110 at 2; 91 at 8 with three blocks), bf16 109 (141 to
// 150 at 8).
NormPlan norm_plan(int C, dsa3d_dtype_t dtype, int odd_per) {
  NormPlan p{};
  const int vec = dtype == DSA3D_F32 ? 4 : 8;
  p.v = (C % vec == 0) ? vec : 1;
  const int nv = C / p.v;
  p.per = nv > 32 ? 2 : 1;
  if (p.v == 1) {  // single elements: rows in flight come from more blocks instead
    while (p.per < odd_per && nv > 32 * p.per) p.per *= 2;
  }
  while (ceil_div(nv, p.per) > (p.per == 2 ? kNormWideThreads : kNormThreads)) p.per *= 2;
  const int need = (int)ceil_div(nv, p.per);
  if (need <= 32) {
    p.tx = 1;
    while (p.tx < need) p.tx *= 2;
  } else {
    p.tx = (need + 31) / 32 * 32;
  }
  p.ty = std::max(1, kNormThreads / p.tx);
  p.r = 1;
  return p;
}
// Blocks: enough to fill the GPU, each then strides over the rest of the rows.
int norm_blocks(const NormPlan& p, int64_t rows, int per_sm) {
  const int64_t steps = ceil_div(rows, (int64_t)p.ty * p.r);
  return (int)std::max<int64_t>(1, std::min<int64_t>(steps, (int64_t)sm_count() * per_sm));
}
NormPlan norm_fwd_plan(int64_t rows, int C, dsa3d_dtype_t dtype) {
  NormPlan p = norm_plan(C, dtype, 8);
  // two rows in flight per group (720p: 305 against 316 us), if that leaves a block for every SM
  if (p.per <= 2 && p.tx <= kNormThreads && ceil_div(rows, 2 * (int64_t)p.ty) >= sm_count()) p.r = 2;
  p.blocks = norm_blocks(p, rows, 8);
  return p;
}
NormPlan norm_bwd_plan(int64_t rows, int C, dsa3d_dtype_t dtype, bool add) {
  NormPlan p = norm_plan(C, dtype, 4);
  const int64_t row = (int64_t)C * elem_size(dtype), sms = sm_count();
  // short rows, several per step: up to four (2,000,000 x 64 bf16: 141 us at four rows, 163 at one), two of three
  // tensors in whole vectors (4 to 8 KB of each per step, and the ring holds three steps)
  const int most = add && p.v > 1 ? 2 : 4;
  while (p.per == 1 && p.r < most && ceil_div(rows, (int64_t)p.ty * p.r * 2) >= sms) p.r *= 2;
  // the ring: whole 16-byte rows, more steps than SMs (a block with one step has nothing to run ahead
  // of), and two blocks on an SM
  p.smem = (size_t)kRing * (add ? 3 : 2) * p.ty * p.r * row;
  p.ring = p.v > 1 && p.per <= 2 && p.smem <= 100 * 1024 && ceil_div(rows, (int64_t)p.ty * p.r) > sms;
  if (!p.ring) p.smem = 0;
  p.blocks = norm_blocks(p, rows, p.v == 1 ? 4 : 2);
  return p;
}

// Calls f with the plan's PER and R (and RING) as constants; V bounds PER (C <= kNormMaxChannels), and whole
// vectors go from two per thread to eight (two reach 1024 of them with the wide blocks).
#define DSA3D_NORM_CASE(PER, R, RING)                                                                       \
  if constexpr (PER <= (V == 1 ? 32 : kNormMaxChannels / (V * kNormThreads)) && (V > 1 ? PER != 4 : !RING)) \
    if (p.per == PER && p.r == R && p.ring == RING)                                                         \
      return f(std::integral_constant<int, PER>(), std::integral_constant<int, R>(), std::integral_constant<bool, RING>());
template <int V, typename F>
dsa3d_status_t norm_fwd_dispatch(const NormPlan& p, F&& f) {
  DSA3D_NORM_CASE(1, 1, false) DSA3D_NORM_CASE(1, 2, false) DSA3D_NORM_CASE(2, 1, false) DSA3D_NORM_CASE(2, 2, false)
  DSA3D_NORM_CASE(4, 1, false) DSA3D_NORM_CASE(8, 1, false) DSA3D_NORM_CASE(16, 1, false) DSA3D_NORM_CASE(32, 1, false)
  return DSA3D_ERR_UNSUPPORTED;
}
template <int V, typename F>
dsa3d_status_t norm_bwd_dispatch(const NormPlan& p, F&& f) {
  DSA3D_NORM_CASE(1, 1, true) DSA3D_NORM_CASE(1, 2, true) DSA3D_NORM_CASE(1, 4, true) DSA3D_NORM_CASE(2, 1, true)
  DSA3D_NORM_CASE(1, 1, false) DSA3D_NORM_CASE(1, 2, false) DSA3D_NORM_CASE(1, 4, false) DSA3D_NORM_CASE(2, 1, false)
  DSA3D_NORM_CASE(4, 1, false) DSA3D_NORM_CASE(8, 1, false) DSA3D_NORM_CASE(16, 1, false) DSA3D_NORM_CASE(32, 1, false)
  return DSA3D_ERR_UNSUPPORTED;
}
#undef DSA3D_NORM_CASE

template <typename K>
bool norm_smem(K* kern, const NormPlan& p) {  // more than the default 48 KB, the static part included
  return p.smem <= 40 * 1024 ||
         cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)p.smem) == cudaSuccess;
}

struct NormFwd {
  const void *x, *add;
  const float *w, *b;
  void *y, *h;
  float* stats;
  int64_t rows;
  int C;
  float eps;
};

template <typename T, int V>
dsa3d_status_t norm_fwd(const NormFwd& a, const NormPlan& p, cudaStream_t st) {
  return norm_fwd_dispatch<V>(p, [&](auto per, auto r, auto) {
    constexpr int PER = decltype(per)::value, R = decltype(r)::value;
    auto* kern = a.add ? dsa3d_layer_norm_kernel<T, V, PER, R, true> : dsa3d_layer_norm_kernel<T, V, PER, R, false>;
    return launch(kKernLayerNorm, st, [&] {
      kern<<<p.blocks, p.tx * p.ty, 0, st>>>(
          static_cast<const T*>(a.x), static_cast<const T*>(a.add), a.w, a.b, static_cast<T*>(a.y),
          static_cast<T*>(a.h), a.stats, a.rows, a.C, a.eps, p.tx, aligned16(a.w) && aligned16(a.b));
    });
  });
}

struct NormBwd {
  const void *h, *dy, *add;
  const float *w, *stats;
  void* dx;
  float* partial;
  int64_t rows;
  int C;
};

template <typename T, int V>
dsa3d_status_t norm_bwd(const NormBwd& a, const NormPlan& p, cudaStream_t st) {
  return norm_bwd_dispatch<V>(p, [&](auto per, auto r, auto ring) {
    constexpr int PER = decltype(per)::value, R = decltype(r)::value;
    constexpr bool RING = decltype(ring)::value;
    auto* kern = dsa3d_layer_norm_bwd_kernel<T, V, PER, R, false, RING>;
    if constexpr (V == 1 || R < 4) {  // four rows of whole vectors: never with an add
      if (a.add) kern = dsa3d_layer_norm_bwd_kernel<T, V, PER, R, true, RING>;
    }
    if (!norm_smem(kern, p)) return DSA3D_ERR_CUDA;
    return launch(kKernLayerNormBwd, st, [&] {
      kern<<<p.blocks, p.tx * p.ty, p.smem, st>>>(
          static_cast<const T*>(a.h), a.w, a.stats, static_cast<const T*>(a.dy), static_cast<const T*>(a.add),
          static_cast<T*>(a.dx), a.partial, a.rows, a.C, p.tx, aligned16(a.w));
    });
  });
}

int norm_vec(dsa3d_dtype_t t) { return t == DSA3D_F32 ? 4 : 8; }

dsa3d_status_t check_norm_shape(long long rows, int C, dsa3d_dtype_t dtype) {
  if (!known(dtype) || rows < 0 || C < 1) return DSA3D_ERR_INVALID_ARGUMENT;
  if (C > kNormMaxChannels || rows >= (1LL << 31)) return DSA3D_ERR_UNSUPPORTED;
  if (C % norm_vec(dtype) && C > kNormMaxChannels / 2) return DSA3D_ERR_UNSUPPORTED;  // 32 elements per thread
  return DSA3D_OK;
}

// Rows of partial sums: of the larger launch of the two, with and without an add.
size_t norm_bwd_ws_bytes(long long rows, int C, dsa3d_dtype_t dtype) {
  const int blocks = std::max(norm_bwd_plan(rows, C, dtype, false).blocks, norm_bwd_plan(rows, C, dtype, true).blocks);
  return (size_t)blocks * 2 * C * sizeof(float);
}

// --- rotary positions ---------------------------------------------------------------------------
// A strided set of token rows: rows of `width` bytes, `ld` bytes apart.
struct Rows {
  const void* p;
  int64_t ld, width, rows;
};
bool rows_overlap(const Rows& a, const Rows& b) {
  const Range ra = range_of(a.p, (size_t)((a.rows - 1) * a.ld + a.width));
  const Range rb = range_of(b.p, (size_t)((b.rows - 1) * b.ld + b.width));
  if (!overlap(ra, rb)) return false;
  if (a.ld != b.ld) return true;
  const int64_t ld = a.ld;  // interleaved rows (q and k of one packed projection) may still be apart
  const int64_t d = ((int64_t)(rb.lo - ra.lo) % ld + ld) % ld;
  return !(d >= a.width && ld - d >= b.width);
}

template <typename T>
dsa3d_status_t rotary_go(const void* q, const void* k, void* qo, void* ko, const RotArgs& a,
                         bool interleaved, cudaStream_t st) {
  constexpr int V = vec_width<T>();
  constexpr int HG = 4;  // heads per thread (halves layout, 65,273 x 32 x 128: 315 us; 334 at 2; interleaved: 336 at 2)
  const T* qt = static_cast<const T*>(q);
  const T* kt = static_cast<const T*>(k);
  T* qot = static_cast<T*>(qo);
  T* kot = static_cast<T*>(ko);
  // whole vectors: 16-byte rows and pointers, and in the halves layout halves of whole vectors
  bool vec = a.dh % V == 0 && (interleaved || a.half % V == 0);
  for (int i = 0; i < 4; i++) vec = vec && a.ld[i] % V == 0;
  vec = vec && aligned16(q) && aligned16(k) && aligned16(qo) && aligned16(ko);
  const int64_t cap = (int64_t)1 << 24;  // blocks; the kernels stride over what is left
  if (vec) {
    const int upr = interleaved ? a.dh / V : a.half / V + (a.dh - 2 * a.half) / V;
    const int64_t units = a.rows * upr * ceil_div(a.heads, HG);
    const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(units, kRotThreads), cap);
    return launch(kKernRotary, st, [&] {
      if (interleaved)
        dsa3d_rotary_kernel<T, true, HG><<<grid, kRotThreads, 0, st>>>(qt, kt, qot, kot, a);
      else
        dsa3d_rotary_kernel<T, false, HG><<<grid, kRotThreads, 0, st>>>(qt, kt, qot, kot, a);
    });
  }
  constexpr int HG_ANY = 8;
  const int64_t units = a.rows * (a.dh - a.half) * ceil_div(a.heads, HG_ANY);
  const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(units, kRotThreads), cap);
  return launch(kKernRotary, st, [&] {
    if (interleaved)
      dsa3d_rotary_any_kernel<T, true, HG_ANY><<<grid, kRotThreads, 0, st>>>(qt, kt, qot, kot, a);
    else
      dsa3d_rotary_any_kernel<T, false, HG_ANY><<<grid, kRotThreads, 0, st>>>(qt, kt, qot, kot, a);
  });
}

dsa3d_status_t rotary(const void* q, const void* k, void* qo, void* ko, long long ldq, long long ldk,
                      long long ldqo, long long ldko, long long first, long long rows, int F, int Hp, int Wp,
                      int heads, int dh, const int* axes, const double* start, const double* step, double base,
                      int interleaved, bool backward, dsa3d_dtype_t dtype, cudaStream_t st) {
  if (!known(dtype) || !axes || !start || !step) return DSA3D_ERR_INVALID_ARGUMENT;
  if (F < 1 || Hp < 1 || Wp < 1 || heads < 1 || dh < 2 || rows < 0 || first < 0)
    return DSA3D_ERR_INVALID_ARGUMENT;
  if ((dh & 1) || dh > kRotMaxDh) return DSA3D_ERR_UNSUPPORTED;
  if ((int64_t)Hp * Wp >= (int64_t(1) << 31) || (int64_t)F >= (int64_t(1) << 31) / ((int64_t)Hp * Wp) + 1 ||
      (int64_t)F * Hp * Wp >= (int64_t(1) << 31) || (int64_t)heads * dh >= (int64_t(1) << 24))
    return DSA3D_ERR_UNSUPPORTED;
  const int64_t N = (int64_t)F * Hp * Wp, width = (int64_t)heads * dh;
  if (first > N || rows > N - first) return DSA3D_ERR_INVALID_ARGUMENT;
  int R = 0;
  for (int i = 0; i < 3; i++) {
    if (axes[i] < 0 || (axes[i] & 1) || axes[i] > dh) return DSA3D_ERR_INVALID_ARGUMENT;
    R += axes[i];
  }
  if (R < 2 || R > dh) return DSA3D_ERR_INVALID_ARGUMENT;
  if (!(base > 0.0) || !std::isfinite(base)) return DSA3D_ERR_INVALID_ARGUMENT;
  const int dims[3] = {F, Hp, Wp};
  for (int i = 0; i < 3; i++) {  // angles that fp64 can reduce; below a base of 1 the last pair turns fastest
    const double most = std::fabs(start[i]) + std::fabs(step[i]) * dims[i];
    const double fastest = base < 1.0 && axes[i] > 2 ? std::pow(base, -(axes[i] - 2.0) / axes[i]) : 1.0;
    if (!(most <= 1099511627776.0) || !(most * fastest <= 1099511627776.0)) return DSA3D_ERR_INVALID_ARGUMENT;
  }
  if (rows == 0) return DSA3D_OK;
  if (!q || !qo || (k == nullptr) != (ko == nullptr)) return DSA3D_ERR_INVALID_ARGUMENT;
  const size_t es = elem_size(dtype);
  if (ldq < width || ldqo < width || (k && (ldk < width || ldko < width))) return DSA3D_ERR_INVALID_ARGUMENT;
  // token strides whose product with the rows is an offset of 64 bits, in bytes too
  const long long most = std::min<long long>(1LL << 40, (1LL << 60) / rows);
  if (ldq > most || ldqo > most || (k && (ldk > most || ldko > most))) return DSA3D_ERR_UNSUPPORTED;
  const void* al[4] = {q, k, qo, ko};
  for (const void* p : al)
    if (!aligned(p, (unsigned)es)) return DSA3D_ERR_INVALID_ARGUMENT;
  const int64_t e = (int64_t)es;
  const Rows in[2] = {{q, ldq * e, width * e, rows}, {k, ldk * e, width * e, rows}};
  const Rows out[2] = {{qo, ldqo * e, width * e, rows}, {ko, ldko * e, width * e, rows}};
  for (int i = 0; i < (k ? 2 : 1); i++)
    for (int j = 0; j < (k ? 2 : 1); j++) {
      const bool same = i == j && in[i].p == out[j].p && in[i].ld == out[j].ld;  // in place
      if (!same && rows_overlap(in[i], out[j])) return DSA3D_ERR_INVALID_ARGUMENT;
    }
  if (k && rows_overlap(out[0], out[1])) return DSA3D_ERR_INVALID_ARGUMENT;

  RotArgs a;
  int i = 0;
  for (int ax = 0; ax < 3; ax++) {
    a.start[ax] = start[ax];
    a.step[ax] = step[ax];
    const int pairs = axes[ax] / 2;
    // base^(-2j / size) by repeated products: j of them, an error of j half steps of fp64
    const double ratio = pairs > 1 ? std::pow(base, -2.0 / axes[ax]) : 1.0;
    double f = 0.31830988618379067154 * (backward ? -1.0 : 1.0);  // 1 / pi
    for (int j = 0; j < pairs; j++, f *= ratio) a.freq[i++] = f;
  }
  for (; i < kRotMaxDh / 2; i++) a.freq[i] = 0.0;
  a.ld[0] = ldq; a.ld[1] = k ? ldk : ldq; a.ld[2] = ldqo; a.ld[3] = k ? ldko : ldqo;
  a.rows = rows; a.first = first;
  a.HW = Hp * Wp; a.Wp = Wp; a.heads = heads; a.dh = dh;
  a.half = R / 2; a.end0 = axes[0] / 2; a.end1 = (axes[0] + axes[1]) / 2;
  a.has_k = k != nullptr;
  if (dtype == DSA3D_F32) return rotary_go<float>(q, k, qo, ko, a, interleaved != 0, st);
  return rotary_go<__nv_bfloat16>(q, k, qo, ko, a, interleaved != 0, st);
}

}  // namespace

// As ffn_device_check (dsa3d_ffn.cu), for this translation unit's record.
bool block_device_check(int* flag) {
  if (cudaMemcpyFromSymbol(flag, g_dsa3d_check, sizeof(int)) != cudaSuccess) return false;
  const int zero = 0;
  return *flag == 0 || cudaMemcpyToSymbol(g_dsa3d_check, &zero, sizeof(int)) == cudaSuccess;
}

}  // namespace dsa3d

using namespace dsa3d;

extern "C" {

dsa3d_status_t dsa3d_layer_norm(const void* x, const void* add, const float* weight, const float* bias, void* y,
                                void* h, float* stats, long long rows, int C, float eps, dsa3d_dtype_t dtype,
                                cudaStream_t stream) {
  const dsa3d_status_t rc = check_norm_shape(rows, C, dtype);
  if (rc != DSA3D_OK) return rc;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return DSA3D_ERR_INVALID_ARGUMENT;
  if (rows == 0) return DSA3D_OK;
  if (!x || !y || (add == nullptr) != (h == nullptr) || (bias && !weight)) return DSA3D_ERR_INVALID_ARGUMENT;
  const unsigned al = row_alignment(C, dtype);
  if (!aligned(x, al) || !aligned(add, al) || !aligned(y, al) || !aligned(h, al) || !aligned(weight, 4) ||
      !aligned(bias, 4) || !aligned(stats, 4))
    return DSA3D_ERR_INVALID_ARGUMENT;
  const size_t tb = (size_t)rows * C * elem_size(dtype), wb = (size_t)C * 4;
  const Range ry = range_of(y, tb), rh = range_of(h, tb), rs = range_of(stats, (size_t)rows * 8);
  const Range ins[] = {range_of(x, tb), range_of(add, tb), range_of(weight, wb), range_of(bias, wb)};
  for (const Range& r : ins)
    if (overlap(r, ry) || overlap(r, rs)) return DSA3D_ERR_INVALID_ARGUMENT;
  if (overlap(ry, rh) || overlap(ry, rs) || overlap(rh, rs)) return DSA3D_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < 4; i++)  // h may be x or add itself: each element is read before it is written
    if (overlap(ins[i], rh) && !(i < 2 && ins[i].lo == rh.lo)) return DSA3D_ERR_INVALID_ARGUMENT;
  const NormFwd a{x, add, weight, bias, y, h, stats, rows, C, eps};
  const NormPlan p = norm_fwd_plan(rows, C, dtype);
  if (dtype == DSA3D_F32) return p.v == 4 ? norm_fwd<float, 4>(a, p, stream) : norm_fwd<float, 1>(a, p, stream);
  return p.v == 8 ? norm_fwd<__nv_bfloat16, 8>(a, p, stream) : norm_fwd<__nv_bfloat16, 1>(a, p, stream);
}

size_t dsa3d_layer_norm_backward_workspace_bytes(long long rows, int C, dsa3d_dtype_t dtype) {
  if (check_norm_shape(rows, C, dtype) != DSA3D_OK || rows == 0) return 0;
  return norm_bwd_ws_bytes(rows, C, dtype);
}

dsa3d_status_t dsa3d_layer_norm_backward(const void* h, const float* weight, const float* stats, const void* dy,
                                         const void* add, void* dx, float* dweight, float* dbias,
                                         void* workspace, size_t workspace_bytes, long long rows, int C,
                                         dsa3d_dtype_t dtype, cudaStream_t stream) {
  const dsa3d_status_t rc = check_norm_shape(rows, C, dtype);
  if (rc != DSA3D_OK) return rc;
  // the weight and its two gradients come together
  if ((weight == nullptr) != (dweight == nullptr) || (weight == nullptr) != (dbias == nullptr))
    return DSA3D_ERR_INVALID_ARGUMENT;
  if (!aligned(weight, 4) || !aligned(dweight, 4) || !aligned(dbias, 4)) return DSA3D_ERR_INVALID_ARGUMENT;
  const size_t tb = (size_t)rows * C * elem_size(dtype), wb = (size_t)C * 4;
  const Range rdw = range_of(dweight, wb), rdb = range_of(dbias, wb);
  if (overlap(rdw, rdb) || overlap(range_of(weight, wb), rdw) || overlap(range_of(weight, wb), rdb))
    return DSA3D_ERR_INVALID_ARGUMENT;
  if (rows == 0) {
    if (weight && (cudaMemsetAsync(dweight, 0, wb, stream) != cudaSuccess ||
                   cudaMemsetAsync(dbias, 0, wb, stream) != cudaSuccess))
      return DSA3D_ERR_CUDA;
    return DSA3D_OK;
  }
  if (!h || !stats || !dy || !dx) return DSA3D_ERR_INVALID_ARGUMENT;
  const unsigned al = row_alignment(C, dtype);
  if (!aligned(h, al) || !aligned(dy, al) || !aligned(add, al) || !aligned(dx, al) || !aligned(stats, 4) ||
      !aligned16(workspace))
    return DSA3D_ERR_INVALID_ARGUMENT;
  const size_t need = weight ? norm_bwd_ws_bytes(rows, C, dtype) : 0;
  if (weight && !workspace) return DSA3D_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < need) return DSA3D_ERR_WORKSPACE_TOO_SMALL;
  const Range rdx = range_of(dx, tb), rw = range_of(workspace, need);
  const Range ins[] = {range_of(add, tb), range_of(h, tb), range_of(dy, tb), range_of(weight, wb),
                       range_of(stats, (size_t)rows * 8)};
  for (int i = 0; i < 5; i++) {  // dx may be add itself
    if (overlap(ins[i], rdx) && !(i == 0 && ins[i].lo == rdx.lo)) return DSA3D_ERR_INVALID_ARGUMENT;
    if (overlap(ins[i], rdw) || overlap(ins[i], rdb) || overlap(ins[i], rw)) return DSA3D_ERR_INVALID_ARGUMENT;
  }
  const Range outs[] = {rdx, rdw, rdb, rw};
  for (int i = 0; i < 4; i++)
    for (int j = i + 1; j < 4; j++)
      if (overlap(outs[i], outs[j])) return DSA3D_ERR_INVALID_ARGUMENT;

  const NormPlan p = norm_bwd_plan(rows, C, dtype, add != nullptr);
  float* partial = weight ? static_cast<float*>(workspace) : nullptr;
  const NormBwd a{h, dy, add, weight, stats, dx, partial, rows, C};
  dsa3d_status_t st;
  if (dtype == DSA3D_F32)
    st = p.v == 4 ? norm_bwd<float, 4>(a, p, stream) : norm_bwd<float, 1>(a, p, stream);
  else
    st = p.v == 8 ? norm_bwd<__nv_bfloat16, 8>(a, p, stream)
                  : norm_bwd<__nv_bfloat16, 1>(a, p, stream);
  if (st != DSA3D_OK || !weight) return st;
  return launch_early(kKernNormReduce, stream, dsa3d_norm_reduce_kernel, dim3((unsigned)ceil_div(2 * (int64_t)C, 32)),
                      dim3(32, 32), partial, p.blocks, C, dweight, dbias);
}

dsa3d_status_t dsa3d_rotary3d(const void* q, const void* k, void* q_out, void* k_out, long long ldq,
                              long long ldk, long long ldqo, long long ldko, long long first, long long rows,
                              int F, int Hp, int Wp, int heads, int dh, const int* axes, const double* start,
                              const double* step, double base, int interleaved, dsa3d_dtype_t dtype,
                              cudaStream_t stream) {
  return rotary(q, k, q_out, k_out, ldq, ldk, ldqo, ldko, first, rows, F, Hp, Wp, heads, dh, axes, start, step,
                base, interleaved, false, dtype, stream);
}

dsa3d_status_t dsa3d_rotary3d_backward(const void* dq_out, const void* dk_out, void* dq, void* dk,
                                       long long lddqo, long long lddko, long long lddq, long long lddk,
                                       long long first, long long rows, int F, int Hp, int Wp, int heads, int dh,
                                       const int* axes, const double* start, const double* step, double base,
                                       int interleaved, dsa3d_dtype_t dtype, cudaStream_t stream) {
  return rotary(dq_out, dk_out, dq, dk, lddqo, lddko, lddq, lddk, first, rows, F, Hp, Wp, heads, dh, axes, start,
                step, base, interleaved, true, dtype, stream);
}

}  // extern "C"
