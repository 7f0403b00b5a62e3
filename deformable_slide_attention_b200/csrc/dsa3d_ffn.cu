// dsa3d_ffn.cu -- C ABI of the gated feed-forward block (include/dsa3d.h): argument validation, the
// plan of a call (tokens per chunk, splits, workspace) and the launches.  The kernels are in
// dsa3d_ffn_tc.cuh (bf16, tensor cores), dsa3d_ffn_f32.cuh (fp32, CUDA cores) and dsa3d_ffn_rows.cuh (a
// forward of a few tokens).  This file allocates no device memory.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <mutex>

#include "dsa3d.h"
#include "dsa3d_ffn_f32.cuh"
#include "dsa3d_ffn_rows.cuh"
#include "dsa3d_ffn_tc.cuh"
#include "dsa3d_host.cuh"

namespace dsa3d {
namespace {

using namespace host;

using bf16 = __nv_bfloat16;

constexpr int64_t kFfnChunk = 65536;    // tokens per chunk of a full-size workspace
constexpr int64_t kFfnMinChunk = 256;   // and of the smallest one
constexpr int kFfnMaxParts = 32;
// Rounds of CTAs that the parts of a split tail may make (the costs below choose at most eight of their own
// accord): the bound of the workspace for their sums.
constexpr int kFfnTailRounds = 8;

size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

struct Ffn {
  int64_t rows;
  int C, hidden, act;
  dsa3d_dtype_t dtype;
  bool f32() const { return dtype == DSA3D_F32; }
  size_t es() const { return elem_size(dtype); }
  // Row strides of the bf16 tensors that TMA reads: multiples of 16 bytes.  Tensors whose rows are not
  // are copied into the workspace first.
  int64_t ldc() const { return f32() ? C : (C + 7) / 8 * 8; }
  int64_t ldh() const { return f32() ? hidden : (hidden + 7) / 8 * 8; }
  // Row stride of the hidden values in the workspace: whole 128-byte lines (the products' boxes are 128
  // bytes wide; at hidden = 5464 rows of 10,928 bytes cost dx's product a quarter more L2 sectors).
  int64_t ldw() const { return f32() ? hidden : ((int64_t)hidden + 63) / 64 * 64; }
};

dsa3d_status_t check_ffn_shape(long long rows, int C, int hidden, dsa3d_dtype_t dtype) {
  if (!known(dtype) || rows < 0 || C < 1 || hidden < 1) return DSA3D_ERR_INVALID_ARGUMENT;
  if (rows >= (1LL << 31) || C > (1 << 20) || hidden > (1 << 20)) return DSA3D_ERR_UNSUPPORTED;
  return DSA3D_OK;
}

// Tensors whose rows have n elements.
template <size_t K>
bool rows_aligned(const void* const (&tensors)[K], int64_t n, dsa3d_dtype_t dtype) {
  for (const void* p : tensors)
    if (!aligned(p, row_alignment(n, dtype))) return false;
  return true;
}

// --- plan: parts of a summed axis, and the workspace -------------------------------------------------
int64_t tiles_for(int64_t m, int64_t n, int tile_m, int tile_n) { return ceil_div(m, tile_m) * ceil_div(n, tile_n); }

// fp32.  Parts: as many as keep four blocks per SM busy when the tiles alone do not, each of 128 of the
// summed axis or more, none empty.
int f32_parts(int64_t tiles, int64_t len) {
  const int64_t slots = 4 * sm_count(), steps = ceil_div(len, kF32K);
  if (tiles >= slots) return 1;
  const int64_t p = std::max<int64_t>(1, std::min<int64_t>({slots / tiles, steps / 8, (int64_t)kFfnMaxParts}));
  return (int)ceil_div(steps, ceil_div(steps, p));
}
int f32_out_parts(const Ffn& f, int64_t rows) { return f32_parts(tiles_for(rows, f.C, 64, kF32Cols), f.hidden); }
int f32_dw_parts(const Ffn& f, int64_t rows) {
  return f32_parts(2 * tiles_for(f.C, f.hidden, 64, kF32Cols), rows);
}
// Bounds of the split sums that no shorter call passes: the parts go down where the tiles fill the SMs,
// and a workspace for many tokens has to be enough for few.  y and dx: parts * tiles stay within the slots.
int64_t f32_out_sums(const Ffn& f, int64_t rows) {
  const int64_t p = std::min<int64_t>(ceil_div(f.hidden, kF32K) / 8, kFfnMaxParts);
  return p > 1 ? std::min(p * rows * f.C, 4 * (int64_t)sm_count() * 64 * kF32Cols) : 0;
}
int64_t f32_dw_max_parts(const Ffn& f, int64_t rows) {
  const int64_t room = 4 * (int64_t)sm_count() / (2 * tiles_for(f.C, f.hidden, 64, kF32Cols));
  return std::max<int64_t>(1, std::min<int64_t>({room, ceil_div(rows, kF32K) / 8, (int64_t)kFfnMaxParts}));
}

// CTAs per tensor-core tile: pairs, unless the rows fill no more than one CTA's 128.
int tc_pair(int64_t rows) { return rows > 128 ? 2 : 1; }

// Numbers the tiles of M x N outputs and chooses the tail (FtTiles): the tiles of the last, partly empty
// round of CTAs, cut into the number of parts that shortens that round most.  A k-block of a 256-wide
// tile takes about 0.3 us; the joining launch about 6.
FtTiles tc_tiles(int problems, const int64_t (&M)[3], const int64_t (&N)[3], int cg, int64_t kblocks, int products,
                 bool all_tail) {
  FtTiles t{};
  int64_t tiles = 0;
  for (int p = 0; p < problems; p++) {
    t.M[p] = M[p];
    t.N[p] = N[p];
    t.tiles_m[p] = (int)ceil_div(M[p], 128 * cg);
    t.tiles_of[p] = t.tiles_m[p] * (int)ceil_div(N[p], 256);
    tiles += t.tiles_of[p];
  }
  t.problems = problems;
  t.group = 16 / cg;
  t.kblocks = (int)kblocks;
  const int64_t slots = std::max(1, sm_count() / cg);
  const int64_t tail = all_tail ? tiles : tiles % slots;
  const double rounds = (double)ceil_div(tail, slots);
  double best = rounds;
  int64_t parts = 1;
  for (int64_t p = 2; p <= kFfnMaxParts && p <= kblocks / 4 && tail < slots && tail * p <= kFfnTailRounds * slots; p++) {
    if (ceil_div(kblocks, ceil_div(kblocks, p)) != p) continue;  // an empty part
    const double r = (double)ceil_div(tail * p, slots) / p + 0.01 * p;  // the parts' sums cross memory
    if (r < best) {
      best = r;
      parts = p;
    }
  }
  if (!all_tail && (rounds - best) * kblocks * products * 0.3 < 6.0) parts = 1;
  t.full = (all_tail || parts > 1) ? tiles - tail : tiles;
  t.parts = (int)parts;
  t.per_part = (int)ceil_div(kblocks, parts);
  t.units = t.full + (tiles - t.full) * parts;
  return t;
}
// A bound of the split sums of up to `tiles` tail tiles, which grows with the tiles and with the k-blocks.
int64_t tc_sums(int64_t tiles, int64_t kblocks, int cg, bool all_tail) {
  const int64_t tile = 128 * cg * 256, parts = std::min<int64_t>(kFfnMaxParts, kblocks / 4);
  const int64_t split =
      parts > 1 ? std::min(tiles * parts * tile, (int64_t)kFfnTailRounds * sm_count() * 128 * 256) : 0;
  return all_tail ? std::max(split, tiles * tile) : split;
}

// y (one product) and dx (two): [rows][C] summed over hidden.
FtTiles tc_out_tiles(const Ffn& f, int64_t rows, int products) {
  const int64_t M[3] = {rows}, N[3] = {f.C};
  return tc_tiles(1, M, N, tc_pair(rows), ceil_div(f.hidden, kFtK), products, f.ldc() != f.C);
}
int64_t tc_out_sums(const Ffn& f, int64_t rows) {
  const int cg = tc_pair(rows);
  return tc_sums(tiles_for(rows, f.C, 128 * cg, 256), ceil_div(f.hidden, kFtK), cg, f.ldc() != f.C);
}
// The three weight gradients, summed over tokens.
FtTiles tc_dw_tiles(const Ffn& f, int64_t rows, bool all_tail) {
  const int64_t M[3] = {f.C, f.C, f.hidden}, N[3] = {f.hidden, f.hidden, f.C};
  return tc_tiles(3, M, N, 2, ceil_div(rows, kFtK), 1, all_tail);
}
// Their sums in chunks of `chunk` tokens.  Several chunks keep every tile's sums, a call of one chunk those
// of its tail, which may be more: several chunks take the larger.
int64_t tc_dw_sums(const Ffn& f, int64_t chunk) {
  const int64_t tiles = 2 * tiles_for(f.C, f.hidden, 256, 256) + tiles_for(f.hidden, f.C, 256, 256);
  const int64_t kblocks = ceil_div(chunk, kFtK), tail = tiles % std::max(1, sm_count() / 2);
  const bool padded = f.ldc() != f.C || f.ldh() != f.hidden;
  const int64_t all = chunk < f.rows || padded ? tc_sums(tiles, kblocks, 2, true) : 0;
  return padded ? all : std::max(all, tc_sums(tail, kblocks, 2, false));
}
// The hidden values: tiles of tile_n columns, all whole.
FtTiles tc_hidden_tiles(const Ffn& f, int64_t rows, int tile_n) {
  FtTiles t{};
  t.M[0] = rows;
  t.N[0] = f.hidden;
  t.tiles_m[0] = (int)ceil_div(rows, 128 * tc_pair(rows));
  t.tiles_of[0] = t.tiles_m[0] * (int)ceil_div(f.hidden, tile_n);
  t.problems = 1;
  t.group = 16 / tc_pair(rows);
  t.kblocks = (int)ceil_div(f.C, kFtK);
  t.parts = 1;
  t.full = t.units = t.tiles_of[0];
  return t;
}

// Hands out pieces of the workspace in order; with a null base it only counts.
struct Carver {
  char* base;
  size_t used = 0;
  template <typename T>
  T* take(bool wanted, size_t elems) {
    if (!wanted) return nullptr;
    T* p = base ? reinterpret_cast<T*>(base + used) : nullptr;
    used += align256(elems * sizeof(T));
    return p;
  }
};

// A forward of so few tokens that the weights' bytes bind, with rows of whole 16-byte vectors.  bf16, us
// through the vector products against the tensor-core tiles: one token 57 against 70 at C 4096, hidden 10,944,
// 25 against 38 at 2048 x 5464, 20.7 against 22 at 512 x 2048; two tokens 81 against 70, 35 against 38, 20.5
// against 22, so the tiles take two (1024 x 4096: 26 where the vector products need 21).  fp32 at 4096 x
// 10,944: four tokens 136 us against 987 through the tiles of 64 rows.
bool few_rows(const Ffn& f) {
  const int v = f.f32() ? 4 : 8;
  return f.rows <= (f.f32() ? kRowsMaxF32 : kRowsMaxBf16) && f.C % v == 0 && f.hidden % v == 0;
}
// Parts of a summed axis of K for strips over N columns: two blocks per SM, at least 64 of K in each.
int rows_parts(const Ffn& f, int K, int N) {
  const int64_t strips = ceil_div(N, 32 * (f.f32() ? 4 : 8));
  const int64_t want = std::max<int64_t>({ceil_div(2 * sm_count(), strips), ceil_div(K, kRowsPart), (int64_t)1});
  const int64_t most = std::max<int64_t>({ceil_div(K, 64), ceil_div(K, kRowsPart), (int64_t)1});
  return (int)std::min(want, most);
}

struct FwdWs {
  char* h;                     // [chunk][ldw]; of few rows: y's parts (and sums: g's and u's)
  bf16 *x, *wg, *wu, *wd;      // copies with 16-byte rows, where the tensors have none
  float* sums;                 // y's split sums: fp32 [parts][chunk][C], bf16 the tail's tiles
  size_t bytes;
};
FwdWs fwd_ws(const Ffn& f, int64_t chunk, void* base) {
  Carver c{static_cast<char*>(base)};
  FwdWs w{};
  if (few_rows(f)) {
    w.sums = c.take<float>(true, (size_t)rows_parts(f, f.C, f.hidden) * 2 * f.rows * f.hidden);
    w.h = c.take<char>(true, (size_t)rows_parts(f, f.hidden, f.C) * f.rows * f.C * sizeof(float));
    w.bytes = c.used;
    return w;
  }
  const bool padc = f.ldc() != f.C, padh = f.ldh() != f.hidden;
  w.h = c.take<char>(true, (size_t)chunk * f.ldw() * f.es());
  w.x = c.take<bf16>(padc, (size_t)chunk * f.ldc());
  w.wg = c.take<bf16>(padh, (size_t)f.C * f.ldh());
  w.wu = c.take<bf16>(padh, (size_t)f.C * f.ldh());
  w.wd = c.take<bf16>(padc, (size_t)f.hidden * f.ldc());
  const size_t sums = (size_t)(f.f32() ? f32_out_sums(f, chunk) : tc_out_sums(f, chunk));
  w.sums = c.take<float>(sums > 0, sums);
  w.bytes = c.used;
  return w;
}

struct BwdWs {
  char *dg, *du, *h;                // [chunk][ldw]
  bf16 *x, *dy, *wg, *wu, *wd;      // copies with 16-byte rows
  float* dw[3];                     // the weight gradients' split sums (bf16: dw[0], the tail's tiles of all three)
  float* sums;                      // dx's
  size_t bytes;
  bool dw_sums;                     // fp32: the weight gradients go through dw
};
// bf16 weight gradients whose sums all go through the workspace: several chunks, or rows TMA cannot store.
bool dw_all_tail(const Ffn& f, int64_t chunk) {
  return chunk < f.rows || f.ldc() != f.C || f.ldh() != f.hidden;
}
BwdWs bwd_ws(const Ffn& f, int64_t chunk, void* base) {
  Carver c{static_cast<char*>(base)};
  BwdWs w;
  const bool padc = f.ldc() != f.C, padh = f.ldh() != f.hidden;
  const size_t hid = (size_t)chunk * f.ldw() * f.es();
  w.dg = c.take<char>(true, hid);
  w.du = c.take<char>(true, hid);
  w.h = c.take<char>(true, hid);
  w.x = c.take<bf16>(padc, (size_t)chunk * f.ldc());
  w.dy = c.take<bf16>(padc, (size_t)chunk * f.ldc());
  w.wg = c.take<bf16>(padh, (size_t)f.C * f.ldh());
  w.wu = c.take<bf16>(padh, (size_t)f.C * f.ldh());
  w.wd = c.take<bf16>(padc, (size_t)f.hidden * f.ldc());
  w.dw_sums = false;
  w.dw[0] = w.dw[1] = w.dw[2] = nullptr;
  if (f.f32()) {
    w.dw_sums = f32_dw_parts(f, chunk) > 1 || chunk < f.rows;
    const int64_t parts = f32_dw_max_parts(f, chunk);
    const bool room = parts > 1 || chunk < f.rows;
    for (int i = 0; i < 3; i++) w.dw[i] = c.take<float>(room, (size_t)parts * f.C * f.hidden);
  } else {
    const size_t n = (size_t)tc_dw_sums(f, chunk);
    w.dw[0] = c.take<float>(n > 0, n);
  }
  const size_t sums = (size_t)(f.f32() ? f32_out_sums(f, chunk) : tc_out_sums(f, chunk));
  w.sums = c.take<float>(sums > 0, sums);
  w.bytes = c.used;
  return w;
}
// Grows with the chunk; a call past the few-token path asks for no less than that path's longest.
size_t fwd_bytes(const Ffn& f, int64_t chunk) {
  const size_t own = fwd_ws(f, chunk, nullptr).bytes;
  Ffn few = f;
  few.rows = std::min<int64_t>(f.rows, f.f32() ? kRowsMaxF32 : kRowsMaxBf16);
  return few_rows(few) ? std::max(own, fwd_ws(few, few.rows, nullptr).bytes) : own;
}
size_t bwd_bytes(const Ffn& f, int64_t chunk) { return bwd_ws(f, chunk, nullptr).bytes; }

// A chunk whose workspace fits: all rows, or a multiple of kFfnMinChunk; 0 when none does.
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
  return p ? static_cast<const T*>(p) + row * width : nullptr;
}
template <typename T>
T* at_row(void* p, int64_t row, int64_t width) {
  return p ? static_cast<T*>(p) + row * width : nullptr;
}

struct FfnFwd {
  const void *x, *wg, *wu, *wd, *add;
  void *y, *ws;
};
struct FfnBwd {
  const void *x, *wg, *wu, *wd, *dy;
  void *dx, *dwg, *dwu, *dwd, *ws;
};

// --- fp32 -------------------------------------------------------------------------------------------
template <int MODE, int TM>
dsa3d_status_t f32_launch_rows(const F32Batch& b, int problems, cudaStream_t st) {
  int64_t tiles = 0;
  for (int i = 0; i < problems; i++) tiles = std::max(tiles, tiles_for(b.p[i].M, b.p[i].N, TM, kF32Cols));
  if (tiles > INT_MAX) return DSA3D_ERR_UNSUPPORTED;
  return launch(kKernFfnF32, st, [&] {
    dsa3d_ffn_f32_kernel<MODE, TM><<<dim3((unsigned)tiles, b.p[0].parts, problems), f32_threads(TM), 0, st>>>(b);
  });
}
// Tiles of 64 rows, or of 32 where those make fewer than four blocks per SM: finer blocks even out the SMs.
template <int MODE>
dsa3d_status_t f32_launch(const F32Batch& b, int problems, cudaStream_t st) {
  int64_t blocks = 0;
  for (int i = 0; i < problems; i++) blocks += tiles_for(b.p[i].M, b.p[i].N, 64, kF32Cols) * b.p[0].parts;
  return blocks < 4 * (int64_t)sm_count() ? f32_launch_rows<MODE, 32>(b, problems, st)
                                          : f32_launch_rows<MODE, 64>(b, problems, st);
}

dsa3d_status_t f32_join(const F32Join& r, int outputs, cudaStream_t st) {
  int64_t most = 0;
  for (int i = 0; i < outputs; i++) most = std::max(most, r.n[i]);
  const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(most, 256), (int64_t)sm_count() * 8);
  return launch_early(kKernFfnReduce, st, dsa3d_ffn_join_kernel, dim3(grid, outputs), dim3(256), r);
}

// y or dx from up to two products over hidden, in parts where the plan has them.
dsa3d_status_t f32_out(const Ffn& f, F32Batch& b, int64_t n, float* sum, int parts, const float* add, float* out,
                       cudaStream_t st) {
  F32Args& a = b.p[0];
  a.M = n; a.N = f.C; a.K = f.hidden;
  a.parts = parts;
  a.out[0] = parts > 1 ? sum : out;
  a.add = parts > 1 ? nullptr : add;
  const dsa3d_status_t rc = f32_launch<kF32Sum>(b, 1, st);
  if (rc != DSA3D_OK || parts == 1) return rc;
  F32Join r{};
  r.partial[0] = sum; r.add = add; r.out[0] = out;
  r.n[0] = n * f.C;
  r.parts = parts;
  return f32_join(r, 1, st);
}

dsa3d_status_t f32_forward(const Ffn& f, const FfnFwd& p, int64_t chunk, cudaStream_t st) {
  const int64_t C = f.C, H = f.hidden;
  const FwdWs w = fwd_ws(f, chunk, p.ws);
  const int parts = f32_out_parts(f, chunk);  // of every chunk, the last and shorter one too
  float* h = reinterpret_cast<float*>(w.h);
  const float *wg = static_cast<const float*>(p.wg), *wu = static_cast<const float*>(p.wu),
              *wd = static_cast<const float*>(p.wd);
  for (int64_t r0 = 0; r0 < f.rows; r0 += chunk) {
    const int64_t n = std::min(chunk, f.rows - r0);
    const float* x = at_row<float>(p.x, r0, C);
    F32Batch b{};
    F32Args& a = b.p[0];
    a.A[0] = a.A[1] = {x, C, 1};
    a.B[0] = {wg, 1, H};
    a.B[1] = {wu, 1, H};
    a.out[0] = h;
    a.M = n; a.N = H; a.K = C;
    a.parts = 1; a.act = f.act;
    dsa3d_status_t rc = f32_launch<kF32Hidden>(b, 1, st);
    if (rc != DSA3D_OK) return rc;
    F32Batch o{};
    o.p[0].A[0] = {h, H, 1};
    o.p[0].B[0] = {wd, 1, C};
    o.p[0].products = 1;
    rc = f32_out(f, o, n, w.sums, parts, at_row<float>(p.add, r0, C), at_row<float>(p.y, r0, C), st);
    if (rc != DSA3D_OK) return rc;
  }
  return DSA3D_OK;
}

dsa3d_status_t f32_backward(const Ffn& f, const FfnBwd& p, int64_t chunk, cudaStream_t st) {
  const int64_t C = f.C, H = f.hidden;
  const BwdWs w = bwd_ws(f, chunk, p.ws);
  float *dg = reinterpret_cast<float*>(w.dg), *du = reinterpret_cast<float*>(w.du), *h = reinterpret_cast<float*>(w.h);
  const float *wg = static_cast<const float*>(p.wg), *wu = static_cast<const float*>(p.wu),
              *wd = static_cast<const float*>(p.wd);
  const int parts = f32_out_parts(f, chunk), dparts = f32_dw_parts(f, chunk);
  float* outs[3] = {static_cast<float*>(p.dwg), static_cast<float*>(p.dwu), static_cast<float*>(p.dwd)};
  dsa3d_status_t rc;
  for (int64_t r0 = 0; r0 < f.rows; r0 += chunk) {
    const int64_t n = std::min(chunk, f.rows - r0);
    const float *x = at_row<float>(p.x, r0, C), *dy = at_row<float>(p.dy, r0, C);
    F32Batch b{};
    F32Args& a = b.p[0];
    a.A[0] = a.A[1] = {x, C, 1};
    a.A[2] = {dy, C, 1};
    a.B[0] = {wg, 1, H};
    a.B[1] = {wu, 1, H};
    a.B[2] = {wd, C, 1};
    a.out[0] = dg; a.out[1] = du; a.out[2] = h;
    a.M = n; a.N = H; a.K = C;
    a.parts = 1; a.act = f.act;
    if ((rc = f32_launch<kF32HiddenBwd>(b, 1, st)) != DSA3D_OK) return rc;
    F32Batch o{};
    o.p[0].A[0] = {dg, H, 1};
    o.p[0].A[1] = {du, H, 1};
    o.p[0].B[0] = {wg, H, 1};
    o.p[0].B[1] = {wu, H, 1};
    o.p[0].products = 2;
    rc = f32_out(f, o, n, w.sums, parts, nullptr, at_row<float>(p.dx, r0, C), st);
    if (rc != DSA3D_OK) return rc;
    // weight gradients, summed over the chunk's tokens and added to the earlier chunks'
    F32Batch d{};
    F32Args &gu = d.p[0], &dn = d.p[1];  // dWg and dWu, then dWd
    gu.A[0] = {x, 1, C};
    gu.B[0] = {dg, 1, H};
    gu.B[1] = {du, 1, H};
    gu.M = C; gu.N = H;
    gu.pair = true;
    dn.A[0] = {h, 1, H};
    dn.B[0] = {dy, 1, C};
    dn.M = H; dn.N = C;
    gu.out[0] = w.dw_sums ? w.dw[0] : outs[0];
    gu.out[1] = w.dw_sums ? w.dw[1] : outs[1];
    dn.out[0] = w.dw_sums ? w.dw[2] : outs[2];
    for (F32Args* q : {&gu, &dn}) {
      q->K = n;
      q->products = 1;
      q->parts = dparts;
      q->accumulate = r0 > 0;
    }
    if ((rc = f32_launch<kF32Sum>(d, 2, st)) != DSA3D_OK) return rc;
  }
  if (!w.dw_sums) return DSA3D_OK;
  F32Join r{};
  for (int i = 0; i < 3; i++) {
    r.partial[i] = w.dw[i];
    r.out[i] = outs[i];
    r.n[i] = C * H;
  }
  r.parts = dparts;
  return f32_join(r, 3, st);
}

// --- a few tokens -----------------------------------------------------------------------------------
template <typename T, int R>
dsa3d_status_t rows_forward_r(const Ffn& f, const FfnFwd& p, cudaStream_t st) {
  constexpr int V = vec_width<T>();
  const FwdWs w = fwd_ws(f, f.rows, p.ws);
  float* y_parts = reinterpret_cast<float*>(w.h);
  const int rows = (int)f.rows, parts = rows_parts(f, f.C, f.hidden), y_split = rows_parts(f, f.hidden, f.C);
  RowsArgs a{};
  a.w[0] = p.wg; a.w[1] = p.wu;
  a.x = p.x;
  a.out = w.sums;
  a.K = f.C; a.N = f.hidden; a.rows = rows;
  a.per_part = (int)ceil_div(f.C, parts);
  dsa3d_status_t rc = launch(kKernFfnRows, st, [&] {
    dsa3d_ffn_rows_kernel<T, R, 2, false>
        <<<dim3((unsigned)ceil_div(f.hidden, 32 * V), (unsigned)ceil_div(f.C, a.per_part)), kRowsThreads, 0, st>>>(a);
  });
  if (rc != DSA3D_OK) return rc;
  RowsArgs b{};
  b.w[0] = p.wd;
  b.in = w.sums;
  b.in_parts = (int)ceil_div(f.C, a.per_part);
  b.out = y_parts;
  b.K = f.hidden; b.N = f.C; b.rows = rows;
  b.per_part = (int)ceil_div(f.hidden, y_split);
  b.act = f.act;
  const int y_used = (int)ceil_div(f.hidden, b.per_part);
  rc = launch_early(kKernFfnRows, st, dsa3d_ffn_rows_kernel<T, R, 1, true>,
                    dim3((unsigned)ceil_div(f.C, 32 * V), (unsigned)y_used), dim3(kRowsThreads), b);
  if (rc != DSA3D_OK) return rc;
  const int n = rows * f.C;
  return launch_early(kKernFfnReduce, st, dsa3d_ffn_rows_join_kernel<T>, dim3((unsigned)ceil_div(n, 256)), dim3(256),
                      y_parts, y_used, static_cast<const T*>(p.add), static_cast<T*>(p.y), n);
}
dsa3d_status_t rows_forward(const Ffn& f, const FfnFwd& p, cudaStream_t st) {
  if (!f.f32()) return rows_forward_r<bf16, 1>(f, p, st);
  if (f.rows == 1) return rows_forward_r<float, 1>(f, p, st);
  if (f.rows == 2) return rows_forward_r<float, 2>(f, p, st);
  if (f.rows <= 4) return rows_forward_r<float, 4>(f, p, st);
  return rows_forward_r<float, 8>(f, p, st);
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

// A [rows][cols] bf16 tensor, rows ld elements apart, in boxes of box_cols (64: 128-byte swizzle,
// operands; 32: 64-byte swizzle, results) by box_rows.
bool matrix_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_cols, int box_rows) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  const cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool k_major_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  return matrix_map(m, p, rows, cols, ld, 64, box_rows);
}
bool mn_major_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld) {
  return matrix_map(m, p, rows, cols, ld, 64, kFtK);
}
bool result_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld) {
  return matrix_map(m, p, rows, cols, ld, 32, 32);
}

template <int MODE, int CG, int ACT>
dsa3d_status_t tc_launch_cg(FtArgs& a, cudaStream_t st) {
  using Cf = FtCfg<MODE, CG>;
  auto* kern = dsa3d_ffn_tc_kernel<MODE, CG, ACT>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cf::SMEM) != cudaSuccess)
    return DSA3D_ERR_CUDA;
  const unsigned grid = (unsigned)(CG * std::min<int64_t>(a.t.units, std::max(1, sm_count() / CG)));
  return launch(kKernFfnTcHidden + MODE, st, [&] {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(Cf::THREADS);
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
  return cg == 2 ? tc_launch_cg<MODE, 2, 0>(a, st) : tc_launch_cg<MODE, 1, 0>(a, st);
}
template <int MODE>
dsa3d_status_t tc_launch_gated(FtArgs& a, int cg, int act, cudaStream_t st) {
  if (act == kActSilu)
    return cg == 2 ? tc_launch_cg<MODE, 2, kActSilu>(a, st) : tc_launch_cg<MODE, 1, kActSilu>(a, st);
  return cg == 2 ? tc_launch_cg<MODE, 2, kActGelu>(a, st) : tc_launch_cg<MODE, 1, kActGelu>(a, st);
}

// Copies into 16-byte rows for those of the tensors that need it; a tensor's own pointer otherwise.
struct Padder {
  FfnPad a{};
  int count = 0;
  const bf16* use(const void* from, bf16* to, int64_t rows, int64_t n, int64_t ld) {
    const bf16* p = static_cast<const bf16*>(from);
    if (!to) return p;
    a.from[count] = p; a.to[count] = to;
    a.rows[count] = rows; a.n[count] = n; a.ld[count] = ld;
    count++;
    return to;
  }
  dsa3d_status_t run(cudaStream_t st) {
    if (count == 0) return DSA3D_OK;
    int64_t most = 0;
    for (int i = 0; i < count; i++) most = std::max(most, a.rows[i]);
    const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(most, 8), (int64_t)sm_count() * 8);
    const int n = count;
    count = 0;
    return launch(kKernFfnPad, st, [&] { dsa3d_ffn_pad_kernel<<<dim3(grid, n), 256, 0, st>>>(a); });
  }
};

dsa3d_status_t tc_join(const FtTiles& t, int cg, const bf16* add, void* o0, void* o1, void* o2, cudaStream_t st) {
  FtTail a{};
  a.t = t;
  a.add = add;
  a.out[0] = static_cast<bf16*>(o0);
  a.out[1] = static_cast<bf16*>(o1);
  a.out[2] = static_cast<bf16*>(o2);
  a.tile_m = 128 * cg;
  int64_t tiles = 0, rows = 0;
  for (int p = 0; p < t.problems; p++) {
    tiles += t.tiles_of[p];
    rows = std::max(rows, std::min<int64_t>(t.M[p], a.tile_m));
  }
  // about eight blocks per SM over the tail's tiles, of four rows or more
  const int64_t tail = tiles - t.full;
  const unsigned by = (unsigned)std::max<int64_t>(1, std::min(ceil_div(rows, 4), (int64_t)sm_count() * 8 / tail));
  return launch_early(kKernFfnReduce, st, dsa3d_ffn_tail_kernel, dim3((unsigned)tail, by), dim3(256), a);
}

// y or dx: one launch, and the joining of its tail where it has one.
template <int MODE>
dsa3d_status_t tc_out(const Ffn& f, FtArgs& a, int64_t n, float* sums, const bf16* add, bf16* out, cudaStream_t st) {
  const int cg = tc_pair(n);
  a.t = tc_out_tiles(f, n, MODE == kTcDx ? 2 : 1);
  a.t.sums = sums;  // room for a whole chunk's (tc_out_sums), and so for a shorter one's
  a.add = add;
  if (a.t.full > 0 && !result_map(&a.o[0], out, n, f.C, f.C)) return DSA3D_ERR_CUDA;
  const dsa3d_status_t rc = tc_launch<MODE>(a, cg, st);
  if (rc != DSA3D_OK || a.t.units == a.t.full) return rc;
  return tc_join(a.t, cg, add, out, nullptr, nullptr, st);
}

dsa3d_status_t tc_forward(const Ffn& f, const FfnFwd& p, int64_t chunk, cudaStream_t st) {
  const int64_t C = f.C, H = f.hidden, lc = f.ldc(), lh = f.ldh(), lw = f.ldw();
  const FwdWs w = fwd_ws(f, chunk, p.ws);
  Padder pad;
  const bf16 *wg = pad.use(p.wg, w.wg, C, H, lh), *wu = pad.use(p.wu, w.wu, C, H, lh),
             *wd = pad.use(p.wd, w.wd, H, C, lc);
  dsa3d_status_t rc;
  for (int64_t r0 = 0; r0 < f.rows; r0 += chunk) {
    const int64_t n = std::min(chunk, f.rows - r0);
    const bf16* x = pad.use(at_row<bf16>(p.x, r0, C), w.x, n, C, lc);
    if ((rc = pad.run(st)) != DSA3D_OK) return rc;
    FtArgs a{};
    if (!k_major_map(&a.a[0], x, n, C, lc, 128) || !mn_major_map(&a.b[0], wg, C, H, lh) ||
        !mn_major_map(&a.b[1], wu, C, H, lh) || !result_map(&a.o[0], w.h, n, H, lw))
      return DSA3D_ERR_CUDA;
    a.t = tc_hidden_tiles(f, n, 128);
    if ((rc = tc_launch_gated<kTcHidden>(a, tc_pair(n), f.act, st)) != DSA3D_OK) return rc;
    FtArgs b{};
    if (!k_major_map(&b.a[0], w.h, n, H, lw, 128) || !mn_major_map(&b.b[0], wd, H, C, lc)) return DSA3D_ERR_CUDA;
    rc = tc_out<kTcOut>(f, b, n, w.sums, at_row<bf16>(p.add, r0, C), at_row<bf16>(p.y, r0, C), st);
    if (rc != DSA3D_OK) return rc;
  }
  return DSA3D_OK;
}

dsa3d_status_t tc_backward(const Ffn& f, const FfnBwd& p, int64_t chunk, cudaStream_t st) {
  const int64_t C = f.C, H = f.hidden, lc = f.ldc(), lh = f.ldh(), lw = f.ldw();
  const BwdWs w = bwd_ws(f, chunk, p.ws);
  FtTiles dw = tc_dw_tiles(f, chunk, dw_all_tail(f, chunk));  // the same tiles for every chunk
  dw.sums = w.dw[0];
  Padder pad;
  const bf16 *wg = pad.use(p.wg, w.wg, C, H, lh), *wu = pad.use(p.wu, w.wu, C, H, lh),
             *wd = pad.use(p.wd, w.wd, H, C, lc);
  dsa3d_status_t rc;
  if ((rc = pad.run(st)) != DSA3D_OK) return rc;
  for (int64_t r0 = 0; r0 < f.rows; r0 += chunk) {
    const int64_t n = std::min(chunk, f.rows - r0);
    const int cg = tc_pair(n);
    const bf16 *x = pad.use(at_row<bf16>(p.x, r0, C), w.x, n, C, lc),
               *dy = pad.use(at_row<bf16>(p.dy, r0, C), w.dy, n, C, lc);
    if ((rc = pad.run(st)) != DSA3D_OK) return rc;
    FtArgs a{};
    if (!k_major_map(&a.a[0], dy, n, C, lc, 128) || !k_major_map(&a.a[1], x, n, C, lc, 128) ||
        !mn_major_map(&a.b[0], wg, C, H, lh) || !mn_major_map(&a.b[1], wu, C, H, lh) ||
        !k_major_map(&a.b[2], wd, H, C, lc, 256 / cg) || !result_map(&a.o[0], w.dg, n, H, lw) ||
        !result_map(&a.o[1], w.du, n, H, lw) || !result_map(&a.o[2], w.h, n, H, lw))
      return DSA3D_ERR_CUDA;
    a.t = tc_hidden_tiles(f, n, 256);
    if ((rc = tc_launch_gated<kTcHiddenBwd>(a, cg, f.act, st)) != DSA3D_OK) return rc;
    FtArgs b{};
    if (!k_major_map(&b.a[0], w.dg, n, H, lw, 128) || !k_major_map(&b.a[1], w.du, n, H, lw, 128) ||
        !k_major_map(&b.b[0], wg, C, H, lh, 256 / cg) || !k_major_map(&b.b[1], wu, C, H, lh, 256 / cg))
      return DSA3D_ERR_CUDA;
    rc = tc_out<kTcDx>(f, b, n, w.sums, nullptr, at_row<bf16>(p.dx, r0, C), st);
    if (rc != DSA3D_OK) return rc;
    FtArgs d{};
    d.t = dw;
    d.t.kblocks = (int)ceil_div(n, kFtK);
    d.t.per_part = (int)ceil_div(d.t.kblocks, d.t.parts);  // a short last chunk may leave parts empty
    d.t.accumulate = r0 > 0;
    if (!mn_major_map(&d.a[0], x, n, C, lc) || !mn_major_map(&d.a[2], w.h, n, H, lw) ||
        !mn_major_map(&d.b[0], w.dg, n, H, lw) || !mn_major_map(&d.b[1], w.du, n, H, lw) ||
        !mn_major_map(&d.b[2], dy, n, C, lc))
      return DSA3D_ERR_CUDA;
    if (dw.full > 0 && (!result_map(&d.o[0], p.dwg, C, H, H) || !result_map(&d.o[1], p.dwu, C, H, H) ||
                        !result_map(&d.o[2], p.dwd, H, C, C)))
      return DSA3D_ERR_CUDA;
    d.a[1] = d.a[0];
    if ((rc = tc_launch_cg<kTcDw, 2, 0>(d, st)) != DSA3D_OK) return rc;
  }
  return dw.units > dw.full ? tc_join(dw, 2, nullptr, p.dwg, p.dwu, p.dwd, st) : DSA3D_OK;
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
  const void *by_c[] = {x, down_weight, add, y}, *by_hidden[] = {gate_weight, up_weight};
  if (!rows_aligned(by_c, C, dtype) || !rows_aligned(by_hidden, hidden, dtype) || !aligned16(workspace))
    return DSA3D_ERR_INVALID_ARGUMENT;
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
  if (few_rows(f)) return rows_forward(f, p, stream);
  return f.f32() ? f32_forward(f, p, chunk, stream) : tc_forward(f, p, chunk, stream);
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
  const void *by_c[] = {x, down_weight, dy, dx, ddown_weight};
  const void* by_hidden[] = {gate_weight, up_weight, dgate_weight, dup_weight};
  if (!rows_aligned(by_c, C, dtype) || !rows_aligned(by_hidden, hidden, dtype) || !aligned16(workspace))
    return DSA3D_ERR_INVALID_ARGUMENT;
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
  return f.f32() ? f32_backward(f, p, chunk, stream) : tc_backward(f, p, chunk, stream);
}

}  // extern "C"
