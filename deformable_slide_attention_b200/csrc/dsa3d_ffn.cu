// dsa3d_ffn.cu -- C ABI of the gated feed-forward block (include/dsa3d.h): argument validation, the
// plan of a call (tokens per chunk, splits, workspace) and the launches.  The kernels are in
// dsa3d_ffn_tc.cuh (tensor cores: bf16, C and hidden multiples of 8) and dsa3d_ffn_any.cuh (CUDA cores:
// everything else).  This file allocates no device memory.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <mutex>

#include "dsa3d.h"
#include "dsa3d_ffn_any.cuh"
#include "dsa3d_ffn_tc.cuh"
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

// The tensor-core path: bf16 rows of whole 16-byte units, which TMA's strides need.
bool use_tc(const Ffn& f) { return f.dtype == DSA3D_BF16 && f.C % 8 == 0 && f.hidden % 8 == 0; }

// CTAs per tile: pairs, unless the rows fill no more than one CTA's 128.
int tc_pair(int64_t rows) { return rows > 128 ? 2 : 1; }

int64_t tc_tiles(int64_t m, int64_t n, int cg, int tile_n) { return ceil_div(m, 128 * cg) * ceil_div(n, tile_n); }

// Parts of the summed axis (k-blocks of 64): as many as keep every CTA (pair) busy when the tiles alone
// do not, each of 4 k-blocks or more (a part's sums cross memory in fp32 once more).
int tc_parts(int64_t tiles, int64_t kblocks, int cg) {
  const int64_t slots = std::max(1, sm_count() / cg);
  if (tiles >= slots) return 1;
  const int64_t p = std::max<int64_t>(1, std::min<int64_t>({slots / tiles, kblocks / 4, (int64_t)kFfnMaxSplits}));
  return (int)ceil_div(kblocks, ceil_div(kblocks, p));  // no empty part
}
int tc_out_parts(const Ffn& f, int64_t rows) {  // y, and dx, [rows][C] summed over hidden
  const int cg = tc_pair(rows);
  return tc_parts(tc_tiles(rows, f.C, cg, 256), ceil_div(f.hidden, kFtK), cg);
}
int64_t tc_dw_tiles(const Ffn& f) {
  return 2 * tc_tiles(f.C, f.hidden, 2, 256) + tc_tiles(f.hidden, f.C, 2, 256);
}
int tc_dw_parts(const Ffn& f, int64_t rows) { return tc_parts(tc_dw_tiles(f), ceil_div(rows, kFtK), 2); }

size_t out_partial_bytes(const Ffn& f, int64_t rows) {
  const int parts = tc_out_parts(f, rows);
  return parts > 1 ? align256((size_t)parts * rows * f.C * 4) : 0;
}
size_t fwd_bytes(const Ffn& f, int64_t chunk) {
  size_t b = align256((size_t)chunk * f.hidden * f.es());
  if (use_tc(f)) b += out_partial_bytes(f, chunk);
  return b;
}
size_t bwd_bytes(const Ffn& f, int64_t chunk) {
  const size_t hid = 3 * align256((size_t)chunk * f.hidden * f.es()), w = (size_t)3 * f.C * f.hidden * 4;
  if (!use_tc(f)) return hid + align256((size_t)any_splits(f, chunk) * w);
  // weight-gradient sums in fp32 when tokens come in parts or chunks; dx's parts use the space after them,
  // since the sums live on from chunk to chunk
  const int parts = tc_dw_parts(f, chunk);
  return hid + ((parts > 1 || chunk < f.rows) ? align256(parts * w) : 0) + out_partial_bytes(f, chunk);
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

// --- tensor cores -----------------------------------------------------------------------------------
// cuTensorMapEncodeTiled through the runtime's driver entry point (no link to the driver library).
PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// A [rows][cols] bf16 tensor in boxes of box_cols (64: 128-byte swizzle, operands; 32: 64-byte swizzle,
// results) by box_rows.
bool matrix_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int box_cols, int box_rows) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)cols * 2};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  const cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool k_major_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int box_rows) {
  return matrix_map(m, p, rows, cols, 64, box_rows);
}
bool mn_major_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols) {
  return matrix_map(m, p, rows, cols, 64, kFtK);
}
bool result_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols) { return matrix_map(m, p, rows, cols, 32, 32); }

template <int MODE, int CG>
dsa3d_status_t tc_launch_cg(FtArgs& a, cudaStream_t st) {
  using Cf = FtCfg<MODE, CG>;
  auto* kern = dsa3d_ffn_tc_kernel<MODE, CG>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cf::SMEM) != cudaSuccess)
    return DSA3D_ERR_CUDA;
  a.tiles = 0;
  for (int p = 0; p < a.problems; p++) {
    a.tiles_m[p] = (int)ceil_div(a.M[p], Cf::TILE_M);
    const int64_t n = a.tiles_m[p] * ceil_div(a.N[p], Cf::TILE_N);
    if (n > INT_MAX) return DSA3D_ERR_UNSUPPORTED;
    a.tiles_of[p] = (int)n;
    a.tiles += n * a.parts;
  }
  a.per_part = (int)ceil_div(a.kblocks, a.parts);
  a.group = 16 / CG;
  const unsigned grid = (unsigned)(CG * std::min<int64_t>(a.tiles, std::max(1, sm_count() / CG)));
  return launch(kKernFfnTc, st, [&] {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kFtThreads);
    cfg.dynamicSmemBytes = Cf::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CG;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = CG > 1 ? 1 : 0;
    cudaLaunchKernelEx(&cfg, kern, a);
  });
}
template <int MODE>
dsa3d_status_t tc_launch(FtArgs& a, int cg, cudaStream_t st) {
  return cg == 2 ? tc_launch_cg<MODE, 2>(a, st) : tc_launch_cg<MODE, 1>(a, st);
}

using bf16 = __nv_bfloat16;

dsa3d_status_t tc_forward(const Ffn& f, const FfnFwd& p, int64_t chunk, cudaStream_t st) {
  const int64_t C = f.C, H = f.hidden;
  float* partial = reinterpret_cast<float*>(static_cast<char*>(p.ws) + align256((size_t)chunk * H * 2));
  const int out_parts = tc_out_parts(f, chunk);  // of every chunk, the last and shorter one too
  dsa3d_status_t rc;
  for (int64_t r0 = 0; r0 < f.rows; r0 += chunk) {
    const int64_t n = std::min(chunk, f.rows - r0);
    const int cg = tc_pair(n);
    FtArgs a{};
    if (!k_major_map(&a.a[0], at_row<bf16>(p.x, r0, C), n, C, 128) || !mn_major_map(&a.b[0], p.wg, C, H) ||
        !mn_major_map(&a.b[1], p.wu, C, H) || !result_map(&a.o[0], p.ws, n, H))
      return DSA3D_ERR_CUDA;
    a.M[0] = n; a.N[0] = H;
    a.problems = 1; a.parts = 1; a.act = f.act;
    a.kblocks = (int)ceil_div(C, kFtK);
    if ((rc = tc_launch<kTcHidden>(a, cg, st)) != DSA3D_OK) return rc;
    FtArgs b{};
    bf16* y = const_cast<bf16*>(at_row<bf16>(p.y, r0, C));
    const bf16* add = p.add ? at_row<bf16>(p.add, r0, C) : nullptr;
    if (!k_major_map(&b.a[0], p.ws, n, H, 128) || !mn_major_map(&b.b[0], p.wd, H, C) || !result_map(&b.o[0], y, n, C))
      return DSA3D_ERR_CUDA;
    b.M[0] = n; b.N[0] = C;
    b.problems = 1;
    b.parts = out_parts;
    b.kblocks = (int)ceil_div(H, kFtK);
    b.add = add;
    if (b.parts > 1) b.partial = partial;
    if ((rc = tc_launch<kTcOut>(b, cg, st)) != DSA3D_OK) return rc;
    if (b.parts > 1 && (rc = reduce_launch<bf16>(partial, b.parts, n * C, add, y, n * C, st)) != DSA3D_OK) return rc;
  }
  return DSA3D_OK;
}

dsa3d_status_t tc_backward(const Ffn& f, const FfnBwd& p, int64_t chunk, cudaStream_t st) {
  const int64_t C = f.C, H = f.hidden, wn = C * H;
  const size_t hb = align256((size_t)chunk * H * 2);
  char* ws = static_cast<char*>(p.ws);
  void *dg = ws, *du = ws + hb, *h = ws + 2 * hb;
  const int parts = tc_dw_parts(f, chunk);
  const int out_parts = tc_out_parts(f, chunk);
  const bool whole = parts == 1 && chunk >= f.rows;  // the weight gradients are written once, in bf16
  float* dw_sum = reinterpret_cast<float*>(ws + 3 * hb);
  float* dx_sum = reinterpret_cast<float*>(ws + 3 * hb + (whole ? 0 : align256((size_t)parts * 3 * wn * 4)));
  dsa3d_status_t rc;
  for (int64_t r0 = 0; r0 < f.rows; r0 += chunk) {
    const int64_t n = std::min(chunk, f.rows - r0);
    const int cg = tc_pair(n);
    const bf16 *x = at_row<bf16>(p.x, r0, C), *dy = at_row<bf16>(p.dy, r0, C);
    bf16* dx = const_cast<bf16*>(at_row<bf16>(p.dx, r0, C));
    FtArgs a{};
    if (!k_major_map(&a.a[0], dy, n, C, 128) || !k_major_map(&a.a[1], x, n, C, 128) ||
        !mn_major_map(&a.b[0], p.wg, C, H) || !mn_major_map(&a.b[1], p.wu, C, H) ||
        !k_major_map(&a.b[2], p.wd, H, C, 128 / cg) || !result_map(&a.o[0], dg, n, H) ||
        !result_map(&a.o[1], du, n, H) || !result_map(&a.o[2], h, n, H))
      return DSA3D_ERR_CUDA;
    a.M[0] = n; a.N[0] = H;
    a.problems = 1; a.parts = 1; a.act = f.act;
    a.kblocks = (int)ceil_div(C, kFtK);
    if ((rc = tc_launch<kTcHiddenBwd>(a, cg, st)) != DSA3D_OK) return rc;
    FtArgs b{};
    if (!k_major_map(&b.a[0], dg, n, H, 128) || !k_major_map(&b.a[1], du, n, H, 128) ||
        !k_major_map(&b.b[0], p.wg, C, H, 256 / cg) || !k_major_map(&b.b[1], p.wu, C, H, 256 / cg) ||
        !result_map(&b.o[0], dx, n, C))
      return DSA3D_ERR_CUDA;
    b.M[0] = n; b.N[0] = C;
    b.problems = 1;
    b.parts = out_parts;
    b.kblocks = (int)ceil_div(H, kFtK);
    if (b.parts > 1) b.partial = dx_sum;
    if ((rc = tc_launch<kTcDx>(b, cg, st)) != DSA3D_OK) return rc;
    if (b.parts > 1 && (rc = reduce_launch<bf16>(dx_sum, b.parts, n * C, nullptr, dx, n * C, st)) != DSA3D_OK) return rc;
    FtArgs w{};
    if (!mn_major_map(&w.a[0], x, n, C) || !mn_major_map(&w.a[2], h, n, H) || !mn_major_map(&w.b[0], dg, n, H) ||
        !mn_major_map(&w.b[1], du, n, H) || !mn_major_map(&w.b[2], dy, n, C) || !result_map(&w.o[0], p.dwg, C, H) ||
        !result_map(&w.o[1], p.dwu, C, H) || !result_map(&w.o[2], p.dwd, H, C))
      return DSA3D_ERR_CUDA;
    w.a[1] = w.a[0];
    w.M[0] = w.M[1] = C; w.N[0] = w.N[1] = H;
    w.M[2] = H; w.N[2] = C;
    w.problems = 3;
    w.kblocks = (int)ceil_div(n, kFtK);
    w.parts = parts;
    w.partial = whole ? nullptr : dw_sum;
    w.accumulate = r0 > 0;
    if ((rc = tc_launch<kTcDw>(w, 2, st)) != DSA3D_OK) return rc;
  }
  if (whole) return DSA3D_OK;
  void* outs[3] = {p.dwg, p.dwu, p.dwd};
  for (int i = 0; i < 3; i++)
    if ((rc = reduce_launch<bf16>(dw_sum + (int64_t)i * parts * wn, parts, wn, nullptr, outs[i], wn, st)) != DSA3D_OK)
      return rc;
  return DSA3D_OK;
}

}  // namespace

// Reads and clears this translation unit's device check record (a wait that ran out); returns false
// on a CUDA error.  dsa3d_check_device reports it with the attention's.
bool ffn_device_check(int* flag) {
  if (cudaMemcpyFromSymbol(flag, g_dsa3d_check, sizeof(int)) != cudaSuccess) return false;
  const int zero = 0;
  return *flag == 0 || cudaMemcpyToSymbol(g_dsa3d_check, &zero, sizeof(int)) == cudaSuccess;
}

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
  if (use_tc(f)) return tc_forward(f, p, chunk, stream);
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
  if (use_tc(f)) return tc_backward(f, p, chunk, stream);
  if (dtype == DSA3D_F32) return any_backward<float>(f, p, chunk, stream);
  return any_backward<__nv_bfloat16>(f, p, chunk, stream);
}

}  // extern "C"
