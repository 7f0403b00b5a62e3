// dsa3d_ffn.cu -- C ABI of the gated feed-forward block (include/dsa3d.h): argument validation, the
// plan of a call (tokens per chunk, splits, workspace) and the launches.  The kernels are in
// dsa3d_ffn_any.cuh.  This file allocates no device memory.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "dsa3d.h"
#include "dsa3d_ffn_any.cuh"
#include "dsa3d_host.cuh"

namespace dsa3d {
namespace {

using namespace host;

constexpr int64_t kFfnChunk = 65536;    // tokens per chunk of a full-size workspace
constexpr int64_t kFfnMinChunk = 256;   // and of the smallest one
constexpr int kFfnMaxSplits = 32;

size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

struct Ffn {
  int64_t rows;
  int C, hidden, act;
  dsa3d_dtype_t dtype;
  size_t es() const { return elem_size(dtype); }
};

dsa3d_status_t check_ffn_shape(long long rows, int C, int hidden, dsa3d_dtype_t dtype) {
  if (!known(dtype) || rows < 0 || C < 1 || hidden < 1) return DSA3D_ERR_INVALID_ARGUMENT;
  if (rows >= (1LL << 31) || C > (1 << 20) || hidden > (1 << 20)) return DSA3D_ERR_UNSUPPORTED;
  return DSA3D_OK;
}

// Parts of the summed axis for a weight gradient [C][hidden] summed over `tokens`: enough blocks for
// two per SM, each with 256 tokens or more.
int any_splits(const Ffn& f, int64_t tokens) {
  const int64_t tiles = ceil_div(f.C, kAnyTile) * ceil_div(f.hidden, kAnyTile);
  const int64_t want = ceil_div(296, tiles);
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, tokens / 256, (int64_t)kFfnMaxSplits}));
}

size_t fwd_bytes(const Ffn& f, int64_t chunk) { return align256((size_t)chunk * f.hidden * f.es()); }
size_t bwd_bytes(const Ffn& f, int64_t chunk) {
  return 3 * align256((size_t)chunk * f.hidden * f.es()) +
         align256((size_t)any_splits(f, chunk) * 3 * f.C * f.hidden * 4);
}

// The largest chunk whose workspace fits: all rows, or a multiple of kFfnMinChunk; 0 when none does.
template <typename Bytes>
int64_t fit_chunk(const Ffn& f, size_t have, Bytes bytes) {
  if (f.rows <= kFfnChunk && bytes(f, f.rows) <= have) return f.rows;
  int64_t lo = 0, hi = std::min(f.rows, kFfnChunk) / kFfnMinChunk;  // in units of kFfnMinChunk
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) / 2;
    if (bytes(f, mid * kFfnMinChunk) <= have)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo * kFfnMinChunk;
}

template <typename T>
const T* at_row(const void* p, int64_t row, int64_t width) {
  return static_cast<const T*>(p) + row * width;
}

template <typename T, int MODE>
dsa3d_status_t any_launch(const AnyArgs& a, int splits, cudaStream_t st) {
  const int64_t tiles = ceil_div(a.M, kAnyTile) * ceil_div(a.N, kAnyTile);
  if (tiles > INT_MAX) return DSA3D_ERR_UNSUPPORTED;
  return launch(kKernFfnAny, st, [&] {
    dsa3d_ffn_any_kernel<T, MODE><<<dim3((unsigned)tiles, (unsigned)splits), kAnyThreads, 0, st>>>(a);
  });
}

template <typename T>
dsa3d_status_t reduce_launch(const float* partial, int splits, int64_t stride, const void* add, void* out,
                             int64_t n, cudaStream_t st) {
  const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(n, 256), (int64_t)sm_count() * 8);
  return launch(kKernFfnReduce, st, [&] {
    dsa3d_ffn_reduce_kernel<T><<<grid, 256, 0, st>>>(partial, splits, stride, static_cast<const T*>(add),
                                                     static_cast<T*>(out), n);
  });
}

struct FfnFwd {
  const void *x, *wg, *wu, *wd, *add;
  void *y, *ws;
};

template <typename T>
dsa3d_status_t any_forward(const Ffn& f, const FfnFwd& p, int64_t chunk, cudaStream_t st) {
  for (int64_t r0 = 0; r0 < f.rows; r0 += chunk) {
    const int64_t n = std::min(chunk, f.rows - r0);
    const T* x = at_row<T>(p.x, r0, f.C);
    AnyArgs a{};
    a.A[0] = a.A[1] = {x, f.C, 1};
    a.B[0] = {p.wg, 1, f.hidden};
    a.B[1] = {p.wu, 1, f.hidden};
    a.out[0] = p.ws;
    a.M = n; a.N = f.hidden; a.K = f.C;
    a.act = f.act;
    dsa3d_status_t rc = any_launch<T, kAnyHidden>(a, 1, st);
    if (rc != DSA3D_OK) return rc;
    AnyArgs b{};
    b.A[0] = {p.ws, f.hidden, 1};
    b.B[0] = {p.wd, 1, f.C};
    b.add = p.add ? at_row<T>(p.add, r0, f.C) : nullptr;
    b.out[0] = const_cast<T*>(at_row<T>(p.y, r0, f.C));
    b.M = n; b.N = f.C; b.K = f.hidden;
    b.products = 1;
    if ((rc = any_launch<T, kAnyOut>(b, 1, st)) != DSA3D_OK) return rc;
  }
  return DSA3D_OK;
}

struct FfnBwd {
  const void *x, *wg, *wu, *wd, *dy;
  void *dx, *dwg, *dwu, *dwd, *ws;
};

template <typename T>
dsa3d_status_t any_backward(const Ffn& f, const FfnBwd& p, int64_t chunk, cudaStream_t st) {
  const int splits = any_splits(f, chunk);
  const size_t hb = align256((size_t)chunk * f.hidden * sizeof(T));
  char* ws = static_cast<char*>(p.ws);
  T *dg = reinterpret_cast<T*>(ws), *du = reinterpret_cast<T*>(ws + hb), *h = reinterpret_cast<T*>(ws + 2 * hb);
  float* partial = reinterpret_cast<float*>(ws + 3 * hb);
  const int64_t wn = (int64_t)f.C * f.hidden;
  dsa3d_status_t rc;
  for (int64_t r0 = 0; r0 < f.rows; r0 += chunk) {
    const int64_t n = std::min(chunk, f.rows - r0);
    const T *x = at_row<T>(p.x, r0, f.C), *dy = at_row<T>(p.dy, r0, f.C);
    AnyArgs a{};
    a.A[0] = a.A[1] = {x, f.C, 1};
    a.A[2] = {dy, f.C, 1};
    a.B[0] = {p.wg, 1, f.hidden};
    a.B[1] = {p.wu, 1, f.hidden};
    a.B[2] = {p.wd, f.C, 1};
    a.out[0] = dg; a.out[1] = du; a.out[2] = h;
    a.M = n; a.N = f.hidden; a.K = f.C;
    a.act = f.act;
    if ((rc = any_launch<T, kAnyHiddenBwd>(a, 1, st)) != DSA3D_OK) return rc;
    AnyArgs b{};
    b.A[0] = {dg, f.hidden, 1};
    b.A[1] = {du, f.hidden, 1};
    b.B[0] = {p.wg, f.hidden, 1};
    b.B[1] = {p.wu, f.hidden, 1};
    b.out[0] = const_cast<T*>(at_row<T>(p.dx, r0, f.C));
    b.M = n; b.N = f.C; b.K = f.hidden;
    b.products = 2;
    if ((rc = any_launch<T, kAnyOut>(b, 1, st)) != DSA3D_OK) return rc;
    // weight gradients, summed over the chunk's tokens and added to the earlier chunks'
    struct { const T *a, *b; int64_t m, n; } w[3] = {
        {x, dg, f.C, f.hidden}, {x, du, f.C, f.hidden}, {h, dy, f.hidden, f.C}};
    for (int i = 0; i < 3; i++) {
      AnyArgs c{};
      c.A[0] = {w[i].a, 1, w[i].m};
      c.B[0] = {w[i].b, 1, w[i].n};
      c.out[0] = partial + (int64_t)i * splits * wn;
      c.M = w[i].m; c.N = w[i].n; c.K = n;
      c.accumulate = r0 > 0;
      if ((rc = any_launch<T, kAnyPartial>(c, splits, st)) != DSA3D_OK) return rc;
    }
  }
  void* outs[3] = {p.dwg, p.dwu, p.dwd};
  for (int i = 0; i < 3; i++)
    if ((rc = reduce_launch<T>(partial + (int64_t)i * splits * wn, splits, wn, nullptr, outs[i], wn, st)) != DSA3D_OK)
      return rc;
  return DSA3D_OK;
}

}  // namespace
}  // namespace dsa3d

using namespace dsa3d;

extern "C" {

size_t dsa3d_gated_ffn_workspace_bytes(long long rows, int C, int hidden, dsa3d_dtype_t dtype) {
  if (check_ffn_shape(rows, C, hidden, dtype) != DSA3D_OK || rows == 0) return 0;
  const Ffn f{rows, C, hidden, 0, dtype};
  return fwd_bytes(f, std::min<int64_t>(rows, kFfnChunk));
}

dsa3d_status_t dsa3d_gated_ffn(const void* x, const void* gate_weight, const void* up_weight,
                               const void* down_weight, const void* add, void* y, void* workspace,
                               size_t workspace_bytes, long long rows, int C, int hidden,
                               dsa3d_activation_t activation, dsa3d_dtype_t dtype, cudaStream_t stream) {
  const dsa3d_status_t rc = check_ffn_shape(rows, C, hidden, dtype);
  if (rc != DSA3D_OK) return rc;
  if (activation != DSA3D_SILU && activation != DSA3D_GELU) return DSA3D_ERR_INVALID_ARGUMENT;
  if (rows == 0) return DSA3D_OK;
  if (!x || !gate_weight || !up_weight || !down_weight || !y || !workspace) return DSA3D_ERR_INVALID_ARGUMENT;
  const void* al[] = {x, gate_weight, up_weight, down_weight, add, y, workspace};
  for (const void* p : al)
    if (!aligned16(p)) return DSA3D_ERR_INVALID_ARGUMENT;
  const Ffn f{rows, C, hidden, activation == DSA3D_SILU ? kActSilu : kActGelu, dtype};
  const size_t tb = (size_t)rows * C * f.es(), wb = (size_t)C * hidden * f.es();
  const Range ry = range_of(y, tb), rw = range_of(workspace, workspace_bytes);
  const Range ins[] = {range_of(add, tb), range_of(x, tb), range_of(gate_weight, wb), range_of(up_weight, wb),
                       range_of(down_weight, wb)};
  for (int i = 0; i < 5; i++) {  // y may be add itself
    if (overlap(ins[i], ry) && !(i == 0 && ins[i].lo == ry.lo)) return DSA3D_ERR_INVALID_ARGUMENT;
    if (overlap(ins[i], rw)) return DSA3D_ERR_INVALID_ARGUMENT;
  }
  if (overlap(ry, rw)) return DSA3D_ERR_INVALID_ARGUMENT;
  const int64_t chunk = fit_chunk(f, workspace_bytes, fwd_bytes);
  if (chunk == 0) return DSA3D_ERR_WORKSPACE_TOO_SMALL;
  const FfnFwd p{x, gate_weight, up_weight, down_weight, add, y, workspace};
  if (dtype == DSA3D_F32) return any_forward<float>(f, p, chunk, stream);
  return any_forward<__nv_bfloat16>(f, p, chunk, stream);
}

size_t dsa3d_gated_ffn_backward_workspace_bytes(long long rows, int C, int hidden, dsa3d_dtype_t dtype) {
  if (check_ffn_shape(rows, C, hidden, dtype) != DSA3D_OK || rows == 0) return 0;
  const Ffn f{rows, C, hidden, 0, dtype};
  return bwd_bytes(f, std::min<int64_t>(rows, kFfnChunk));
}

dsa3d_status_t dsa3d_gated_ffn_backward(const void* x, const void* gate_weight, const void* up_weight,
                                        const void* down_weight, const void* dy, void* dx, void* dgate_weight,
                                        void* dup_weight, void* ddown_weight, void* workspace,
                                        size_t workspace_bytes, long long rows, int C, int hidden,
                                        dsa3d_activation_t activation, dsa3d_dtype_t dtype,
                                        cudaStream_t stream) {
  const dsa3d_status_t rc = check_ffn_shape(rows, C, hidden, dtype);
  if (rc != DSA3D_OK) return rc;
  if (activation != DSA3D_SILU && activation != DSA3D_GELU) return DSA3D_ERR_INVALID_ARGUMENT;
  const Ffn f{rows, C, hidden, activation == DSA3D_SILU ? kActSilu : kActGelu, dtype};
  const size_t tb = (size_t)rows * C * f.es(), wb = (size_t)C * hidden * f.es();
  if (!gate_weight || !up_weight || !down_weight || !dgate_weight || !dup_weight || !ddown_weight)
    return DSA3D_ERR_INVALID_ARGUMENT;
  if (rows > 0 && (!x || !dy || !dx || !workspace)) return DSA3D_ERR_INVALID_ARGUMENT;
  const void* al[] = {x, gate_weight, up_weight, down_weight, dy, dx, dgate_weight, dup_weight, ddown_weight, workspace};
  for (const void* p : al)
    if (!aligned16(p)) return DSA3D_ERR_INVALID_ARGUMENT;
  const Range ins[] = {range_of(x, tb), range_of(dy, tb), range_of(gate_weight, wb), range_of(up_weight, wb),
                       range_of(down_weight, wb)};
  const Range outs[] = {range_of(dx, tb), range_of(dgate_weight, wb), range_of(dup_weight, wb),
                        range_of(ddown_weight, wb), range_of(workspace, workspace_bytes)};
  for (int i = 0; i < 5; i++) {
    for (const Range& r : ins)
      if (overlap(r, outs[i])) return DSA3D_ERR_INVALID_ARGUMENT;
    for (int j = i + 1; j < 5; j++)
      if (overlap(outs[i], outs[j])) return DSA3D_ERR_INVALID_ARGUMENT;
  }
  if (rows == 0) {
    void* dw[] = {dgate_weight, dup_weight, ddown_weight};
    for (void* p : dw)
      if (cudaMemsetAsync(p, 0, wb, stream) != cudaSuccess) return DSA3D_ERR_CUDA;
    return DSA3D_OK;
  }
  const int64_t chunk = fit_chunk(f, workspace_bytes, bwd_bytes);
  if (chunk == 0) return DSA3D_ERR_WORKSPACE_TOO_SMALL;
  const FfnBwd p{x, gate_weight, up_weight, down_weight, dy, dx, dgate_weight, dup_weight, ddown_weight, workspace};
  if (dtype == DSA3D_F32) return any_backward<float>(f, p, chunk, stream);
  return any_backward<__nv_bfloat16>(f, p, chunk, stream);
}

}  // extern "C"
