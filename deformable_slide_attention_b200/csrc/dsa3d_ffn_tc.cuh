// dsa3d_ffn_tc.cuh -- the gated feed-forward block's products on the tensor cores (bf16, sm_100a):
//
//   kTcHidden     h = act(x Wg) * (x Wu)                                one tile: 128 columns of g and of u
//   kTcHiddenBwd  dh = dy Wd^T for 256 columns, g and u for each of their halves: dg = dh u act'(g),
//                 du = dh act(g), h = act(g) u
//   kTcOut        y = h Wd (+ add), whole or in parts of the summed axis
//   kTcDx         dx = dg Wg^T + du Wu^T                                one accumulator over both products
//   kTcDw         dWg = x^T dg, dWu = x^T du, dWd = h^T dy               summed over tokens, whole or in parts
//
// Every operand is read where it lies: TMA brings 64-wide boxes of row-major tensors into shared
// memory with the 128-byte swizzle, and the tcgen05 descriptors read them K-major (x, h, dy against a
// weight's rows) or MN-major (a weight [C][hidden] as B, tokens-by-channels tensors as both operands of
// a weight gradient), so nothing is transposed in memory.
//
// A persistent kernel with one CTA per SM, in pairs (CG = 2, cta_group::2): the pair's tile is 256 rows
// x 256 columns of products, each CTA holds 128 rows of A and half of B, so each operand byte that
// crosses from L2 feeds twice the products of a single CTA's tile.  The first warp issues the TMA loads,
// the second (of the pair's first CTA) the MMAs, 8 or 16 warps the epilogue: accumulators leave tensor
// memory 32 columns at a time, the activation and its derivative are formed in registers in fp32, and
// the results are rounded once and leave through shared memory by TMA, which also clips them to the
// tensors' edges.  Tensor memory holds two tiles' accumulators, so that the epilogue of a tile overlaps
// the products of the next.  kTcHiddenBwd fills it with one tile's (dh, and g and u of one half): its 16
// warps take g and u into registers at once, and a tile's dh follows its first half's g and u, so that
// those are read while dh's products run and the columns of dh are not waited for.  (All its products are
// 256 columns wide: dh in tiles of 128 read shared memory for A as often as for B, and a step took 658
// cycles instead of 256, whatever the number of stages.)
//
// The products are bound by the tensor cores (6 or 16 rows C hidden operations against a few bytes per
// element).  Four 720p frames (14,400 x 2048), hidden 5464, TFLOP/s over a long run under the power cap:
// hidden values 1300, y 1260, their backward 980, dx 1280, weight gradients 1290; a library product of
// these sizes 1150 to 1200 and 1430 at 8192^3.  The tensor pipe is busy 80 to 88% of the cycles, 64% in
// kTcHiddenBwd.  Waits are bounded (dsa3d_tc.cuh); no load is multicast.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <climits>

#include "dsa3d_ffn_f32.cuh"
#include "dsa3d_tc.cuh"

namespace dsa3d {

enum TcMode { kTcHidden, kTcHiddenBwd, kTcOut, kTcDx, kTcDw };

constexpr int kFtK = 64;                 // summed-axis elements per stage
constexpr uint32_t kFtABytes = 128 * kFtK * 2;
constexpr uint32_t kFtOutBox = 32 * 32 * 2;  // an epilogue store: 32 rows x 32 columns of bf16

template <int MODE, int CG>
struct FtCfg {
  static constexpr bool kGated = MODE == kTcHidden || MODE == kTcHiddenBwd;
  static constexpr int TILE_M = 128 * CG;
  // output columns per tile; kTcHiddenBwd's epilogue takes them in halves of 128
  static constexpr int TILE_N = MODE == kTcHidden ? 128 : 256;
  static constexpr int EPI_WARPS = MODE == kTcHiddenBwd ? 16 : 8;
  static constexpr int THREADS = 32 * (2 + EPI_WARPS);
  static constexpr int PRODUCTS = MODE == kTcHiddenBwd ? 3 : (MODE == kTcDx ? 2 : 1);  // steps per k-block
  static constexpr uint32_t B_BYTES = 256 / CG * kFtK * 2;
  static constexpr uint32_t STAGE = kFtABytes + B_BYTES;
  static constexpr int OUT_BUFS = 2;
  static constexpr uint32_t OUT_BYTES = EPI_WARPS * OUT_BUFS * kFtOutBox;
  static constexpr int STAGES = CG == 2 ? (MODE == kTcHiddenBwd ? 5 : 6) : (MODE == kTcHiddenBwd ? 3 : 4);
  static constexpr uint32_t SMEM = 1024 + STAGES * STAGE + OUT_BYTES + 256;
};

// The numbering of tiles over up to three outputs (kTcDw has three, the others one).  Tiles from `full`
// on are the tail: each is cut into `parts` along the summed axis, and every part writes its fp32 sums
// to sums[(tile - full) * parts + part] ([rows of a tile][256]) for dsa3d_ffn_tail_kernel to join.  The
// tail is what the CTAs' last, partly empty round would hold; all tiles, when the results' rows are no
// multiple of 16 bytes (TMA cannot store them) or sums go on over chunks of tokens.
struct FtTiles {
  int64_t M[3], N[3];
  int tiles_of[3], tiles_m[3];
  int problems, group;  // group: row tiles walked together
  int kblocks;          // of one product's summed axis
  int parts, per_part;  // of a tail tile; k-blocks in each part but the last
  int64_t full, units;  // whole tiles; units of work: full + parts * tail tiles
  float* sums;
  bool accumulate;      // add to what sums holds
};

struct FtArgs {
  CUtensorMap a[3], b[3], o[3];
  const __nv_bfloat16* add;  // kTcOut
  FtTiles t;
};

// ---- cluster helpers ------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t .reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

template <int CG>
__device__ __forceinline__ void mbar_arrive_cluster_or_local(uint32_t addr) {
  if (CG == 1)
    mbar_arrive(addr);
  else
    mbar_arrive_cluster(addr);
}

template <int CG>
__device__ __forceinline__ void ft_tma_load(uint32_t dst, const void* map, uint32_t bar, int c0, int c1) {
  if (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
        "[%2];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
  else  // the barrier may be the pair's first CTA's
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%3, %4}], [%2];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void ft_tma_store(const void* map, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

template <int CG>
__device__ __forceinline__ void ft_tmem_alloc(uint32_t slot) {
  if (CG == 1) {
    tmem_alloc(slot, 512);
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(slot) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void ft_tmem_dealloc(uint32_t taddr) {
  if (CG == 1)
    tmem_dealloc(taddr, 512);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(taddr) : "memory");
}
template <int CG>
__device__ __forceinline__ void ft_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (CG == 1) {
    umma_ss(d, a, b, idesc, acc);
  } else {
    asm volatile(
        "{\n\t .reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  }
}
// Arrive on the barrier at this offset (of both CTAs of a pair) when the MMAs issued so far are done.
template <int CG>
__device__ __forceinline__ void ft_commit(uint32_t bar) {
  if (CG == 1)
    umma_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

// ---- tiles ------------------------------------------------------------------------------------------
struct FtTile {
  int problem, kb0, kb1;
  int64_t m0, n0;
  float* sums;  // a tail part's, else null
};
// Position of tile i of its problem: groups of `group` row tiles whose columns are walked together, so
// that the tiles in flight share their operands in L2.
__device__ __forceinline__ void ft_place(const FtTiles& g, int64_t tile, int tile_m, int tile_n, int& problem,
                                         int64_t& m0, int64_t& n0) {
  problem = 0;
  while (problem + 1 < g.problems && tile >= g.tiles_of[problem]) tile -= g.tiles_of[problem++];
  const int i = (int)tile, tm = g.tiles_m[problem], tn = g.tiles_of[problem] / tm;
  const int gi = i / (g.group * tn), in = i - gi * g.group * tn;
  const int rows = min(g.group, tm - gi * g.group);
  m0 = (int64_t)(gi * g.group + in % rows) * tile_m;
  n0 = (int64_t)(in / rows) * tile_n;
}
// Halves of a kTcHiddenBwd tile that lie inside the output.
__device__ __forceinline__ int ft_halves(const FtTiles& g, int64_t n0) { return n0 + 128 < g.N[0] ? 2 : 1; }

template <int MODE, int CG>
__device__ __forceinline__ FtTile ft_tile(const FtTiles& g, int64_t unit) {
  using C = FtCfg<MODE, CG>;
  FtTile r;
  int64_t tile = unit;
  r.kb0 = 0;
  r.kb1 = g.kblocks;
  r.sums = nullptr;
  if (!C::kGated && unit >= g.full) {
    const int64_t u = unit - g.full;
    const int part = (int)(u % g.parts);
    tile = g.full + u / g.parts;
    r.kb0 = part * g.per_part;
    r.kb1 = min(r.kb0 + g.per_part, g.kblocks);
    r.sums = g.sums + u * (C::TILE_M * 256);
  }
  ft_place(g, tile, C::TILE_M, C::TILE_N, r.problem, r.m0, r.n0);
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t pack_bf16(uint64_t v) {
  float a, b;
  unpack2(v, a, b);
  return pack_bf16(a, b);
}
__device__ __forceinline__ uint64_t pair_of(uint32_t a, uint32_t b) {
  return pack2(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ void bits_of(uint64_t v, uint32_t& a, uint32_t& b) {
  float x, y;
  unpack2(v, x, y);
  a = __float_as_uint(x);
  b = __float_as_uint(y);
}
// Waits for the loads so far, the loaded registers tied to the wait.
__device__ __forceinline__ void tmem_ld_wait16(uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
        "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
      :
      : "memory");
}
__device__ __forceinline__ uint64_t both(float v) { return pack2(v, v); }
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint64_t ex2_both(uint64_t v) {
  float a, b;
  unpack2(v, a, b);
  return pack2(ex2_approx(a), ex2_approx(b));
}
__device__ __forceinline__ uint64_t rcp_both(uint64_t v) {
  float a, b;
  unpack2(v, a, b);
  return pack2(rcp_approx(a), rcp_approx(b));
}

// Activation (and derivative) of two values, for results in bf16: packed pairs halve the issue slots,
// after which the exponentials and reciprocals bind.  silu: s = 1 / (1 + e^-g).  gelu: the normal
// distribution from erfc by the Chebyshev fit of Press et al., Numerical Recipes (erfcc), whose
// relative error is below 1.2e-7 everywhere, so that small values keep their digits too; no branches.
template <int ACT, bool DERIV>
__device__ __forceinline__ void ft_act(uint64_t g, uint64_t& a, uint64_t& da) {
  const uint64_t one = both(1.f);
  if (ACT == kActSilu) {
    const uint64_t s = rcp_both(add2(one, ex2_both(mul2(g, both(-kLog2e)))));
    a = mul2(g, s);
    if (DERIV) da = mul2(s, fma2(g, fma2(s, both(-1.f), one), one));
  } else {
    float g0, g1;
    unpack2(g, g0, g1);
    const uint64_t z = pack2(fabsf(g0) * 0.70710678118654752f, fabsf(g1) * 0.70710678118654752f);
    const uint64_t t = rcp_both(fma2(z, both(0.5f), one));
    uint64_t p = both(0.17087277f);
    p = fma2(p, t, both(-0.82215223f));
    p = fma2(p, t, both(1.48851587f));
    p = fma2(p, t, both(-1.13520398f));
    p = fma2(p, t, both(0.27886807f));
    p = fma2(p, t, both(-0.18628806f));
    p = fma2(p, t, both(0.09678418f));
    p = fma2(p, t, both(0.37409196f));
    p = fma2(p, t, both(1.00002368f));
    p = fma2(p, t, both(-1.26551223f));
    const uint64_t mzz = mul2(mul2(z, both(-1.f)), z);
    const uint64_t half_erfc = mul2(mul2(t, both(0.5f)), ex2_both(mul2(add2(mzz, p), both(kLog2e))));
    float h0, h1, c0, c1;  // of |g|'s upper tail: the distribution is 1 - it for positive g
    unpack2(half_erfc, h0, h1);
    unpack2(fma2(half_erfc, both(-1.f), one), c0, c1);
    const uint64_t cdf = pack2(g0 > 0.f ? c0 : h0, g1 > 0.f ? c1 : h1);
    a = mul2(g, cdf);
    if (DERIV) da = fma2(mul2(g, both(0.39894228040143268f)), ex2_both(mul2(mzz, both(kLog2e))), cdf);
  }
}

// ACT (kTcHidden, kTcHiddenBwd): a constant, so that the epilogue's elements are independent instruction
// streams; a branch per element on the activation held the chain of each exp and reciprocal open.
template <int MODE, int CG, int ACT>
__global__ void __launch_bounds__(FtCfg<MODE, CG>::THREADS, 1) dsa3d_ffn_tc_kernel(const __grid_constant__ FtArgs g) {
  using C = FtCfg<MODE, CG>;
  extern __shared__ uint8_t ft_smem_raw[];
  const uint32_t raw = smem_u32(ft_smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* const gen = ft_smem_raw + (base - raw);
  const uint32_t out_base = base + C::STAGES * C::STAGE;
  const uint32_t bars = out_base + C::OUT_BYTES;
  const uint32_t full = bars, empty = full + 8 * C::STAGES, tfull = empty + 8 * C::STAGES, tempty = tfull + 16;
  uint8_t* const tail = gen + C::STAGES * C::STAGE + C::OUT_BYTES;
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tail + 16 * C::STAGES + 32);
  uint32_t* const tslot = reinterpret_cast<uint32_t*>(tail + 16 * C::STAGES + 40);

  const int warp = __shfl_sync(kFull, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const int64_t first = blockIdx.x / CG, stride = gridDim.x / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; s++) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; s++) {
      mbar_init(tfull + 8 * s, 1);
      mbar_init(tempty + 8 * s, C::EPI_WARPS * CG);  // kTcHiddenBwd: [0] g and u, [1] dh
    }
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 1) ft_tmem_alloc<CG>(smem_u32(tslot));
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tslot;

  if (warp == 0) {
    // ---- TMA producer: each CTA loads its own operands; the pair's bytes complete on the first CTA's
    // barrier, which its producer arms for both.
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int64_t t = first; ok && t < g.t.units; t += stride) {
        const FtTile tl = ft_tile<MODE, CG>(g.t, t);
        const int m = (int)tl.m0 + (int)rank * 128, n = (int)tl.n0;
        const int nkb = tl.kb1 - tl.kb0;
        const int steps = (MODE == kTcHiddenBwd ? 1 + ft_halves(g.t, tl.n0) : C::PRODUCTS) * nkb;
        for (int i = 0; ok && i < steps; i++, it++) {
          {
            // which product: kTcHiddenBwd g and u of the first half, dh, g and u of the second; kTcDx both
            // gradients in turn
            int seg = 0, kb = tl.kb0 + i;
            if (C::PRODUCTS > 1)
              while (kb >= tl.kb0 + nkb) {
                seg++;
                kb -= nkb;
              }
            const bool dh = MODE == kTcHiddenBwd && seg == 1;
            const int which = MODE == kTcDw ? tl.problem : (MODE == kTcHiddenBwd ? (dh ? 0 : 1) : seg);
            const void* ma = &g.a[which];
            const int s = it % C::STAGES;
            if (it >= C::STAGES) ok = mbar_wait(empty + 8 * s, (it / C::STAGES - 1) & 1, abort_flag);
            if (!ok) break;
            const uint32_t sa = base + s * C::STAGE, sb = sa + kFtABytes;
            const uint32_t local = full + 8 * s;
            const uint32_t bar = CG == 2 ? map_to_rank(local, 0) : local;
            if (rank == 0) mbar_arrive_expect_tx(local, CG * kFtABytes + 256 * kFtK * 2);
            const int k = kb * kFtK;
            if (MODE == kTcDw) {  // MN-major A: two boxes of 64 rows
              ft_tma_load<CG>(sa, ma, bar, m, k);
              ft_tma_load<CG>(sa + 8192, ma, bar, m + 64, k);
            } else {
              ft_tma_load<CG>(sa, ma, bar, k, m);
            }
            if (dh) {  // Wd's rows n.. as B, K-major
              ft_tma_load<CG>(sb, &g.b[2], bar, k, n + (int)rank * 128);
            } else if (C::kGated) {  // Wg's and Wu's columns, MN-major: gate for the first half of B
              const int c = n + (MODE == kTcHiddenBwd ? 64 * seg : 0);
              if (CG == 1) {
                for (int j = 0; j < 4; j++) ft_tma_load<CG>(sb + 8192 * j, &g.b[j >> 1], bar, c + (j & 1) * 64, k);
              } else {
                for (int j = 0; j < 2; j++) ft_tma_load<CG>(sb + 8192 * j, &g.b[rank], bar, c + j * 64, k);
              }
            } else if (MODE == kTcDx) {
              ft_tma_load<CG>(sb, &g.b[seg], bar, k, n + (int)rank * 128);
            } else {
              for (int j = 0; j < 4 / CG; j++)
                ft_tma_load<CG>(sb + 8192 * j, &g.b[which], bar, n + (int)rank * 128 + j * 64, k);
            }
          }
        }
      }
      // the last loads of this CTA are consumed before its memory is released: the empty barrier's last
      // phase of each stage used completes after the MMAs that read it
      for (int s = 0; s < C::STAGES; s++) {
        const uint32_t uses = it > (uint32_t)s ? (it - s + C::STAGES - 1) / C::STAGES : 0;
        if (uses) mbar_drain(empty + 8 * s, (uses - 1) & 1, abort_flag);
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer: one warp of the pair's first CTA.  The warp stays converged and only the MMAs and
    // commits are one lane's: descriptors and barrier addresses then live in uniform registers, which
    // the instructions take.  (With the whole loop inside one lane's branch a step of four MMAs took
    // 600 cycles to issue, more than the 512 they run.)
    if (rank == 0) {
      constexpr uint32_t ID = umma_idesc_bf16(128 * CG, 256, MODE == kTcDw, MODE != kTcDx);
      constexpr uint32_t ID_DH = umma_idesc_bf16(128 * CG, 256, false, false);
      constexpr uint32_t A_STEP = MODE == kTcDw ? 2048 : 32;  // bytes per 16 of the summed axis
      constexpr uint32_t B_STEP = MODE == kTcDx ? 32 : 2048;
      const uint64_t da0 = umma_sdesc_sw128(base, MODE == kTcDw ? 8192 : 16, 1024);
      const uint64_t db0 = umma_sdesc_sw128(base + kFtABytes, MODE == kTcDx ? 16 : 8192, 1024);
      const uint64_t db0_dh = umma_sdesc_sw128(base + kFtABytes, 16, 1024);
      constexpr uint32_t kAccBufs = MODE == kTcHiddenBwd ? 1 : 2;  // of 256 columns
      uint32_t stage = 0, phase = 0, n_tile = 0, n_acc = 0;  // n_acc: accumulators handed to the epilogue so far
      bool ok = true;
      for (int64_t t = first; ok && t < g.t.units; t += stride, n_tile++) {
        int nkb, halves;
        {
          const FtTile tl = ft_tile<MODE, CG>(g.t, t);
          nkb = tl.kb1 - tl.kb0;
          halves = MODE == kTcHiddenBwd ? ft_halves(g.t, tl.n0) : 1;
        }
        for (int half = 0; ok && half < halves; half++, n_acc++) {
          const uint32_t buf = MODE == kTcHiddenBwd ? 0 : (n_acc & 1);
          // the columns' previous contents have been read
          if (n_acc >= kAccBufs)
            ok = __all_sync(kFull, mbar_wait(tempty + 8 * buf, (n_acc / kAccBufs - 1) & 1, abort_flag));
          const int dh_from = (MODE == kTcHiddenBwd && half == 0) ? nkb : INT_MAX;  // dh's steps follow g and u's
          const int steps = (MODE == kTcDx || (MODE == kTcHiddenBwd && half == 0) ? 2 : 1) * nkb;
          for (int i = 0; ok && i < steps; i++) {
            const bool dh = MODE == kTcHiddenBwd && i >= dh_from;
            if (MODE == kTcHiddenBwd && i == dh_from) {
              if (elect_one()) ft_commit<CG>(tfull);  // g and u: the epilogue reads them during dh's products
              __syncwarp();
              if (n_tile > 0) ok = __all_sync(kFull, mbar_wait(tempty + 8, (n_tile - 1) & 1, abort_flag));
              if (!ok) break;
            }
            ok = __all_sync(kFull, mbar_wait(full + 8 * stage, phase, abort_flag));
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem + (dh ? 256 : 256 * buf);
            const uint64_t da = da0 + (uint64_t)(stage * (C::STAGE >> 4));
            const uint64_t db = (dh ? db0_dh : db0) + (uint64_t)(stage * (C::STAGE >> 4));
            const uint32_t more = i != 0 && i != dh_from;  // a later step of a product adds
            if (elect_one()) {
              if (MODE == kTcHiddenBwd && dh) {
#pragma unroll
                for (int k = 0; k < kFtK / 16; k++)
                  ft_mma<CG>(d, da + (uint64_t)(k * A_STEP >> 4), db + (uint64_t)(k * 32 >> 4), ID_DH,
                           k > 0 ? 1u : more);
              } else {
#pragma unroll
                for (int k = 0; k < kFtK / 16; k++)
                  ft_mma<CG>(d, da + (uint64_t)(k * A_STEP >> 4), db + (uint64_t)(k * B_STEP >> 4), ID,
                           k > 0 ? 1u : more);
              }
              ft_commit<CG>(empty + 8 * stage);
            }
            __syncwarp();
            if (++stage == C::STAGES) {
              stage = 0;
              phase ^= 1;
            }
          }
          // kTcHiddenBwd: [0] g and u of a half, [1] dh of a tile; else the two buffers in turn
          const uint32_t done = MODE == kTcHiddenBwd ? (half == 0 ? 1u : 0u) : (n_acc & 1);
          if (ok && elect_one()) ft_commit<CG>(tfull + 8 * done);
          __syncwarp();
        }
      }
    }
  } else {
    // ---- epilogue: a warp reads tensor-memory lanes 32 (warp % 4).., and its share of the columns
    const int quarter = warp & 3, share = (warp - 2) >> 2;
    const uint32_t lane_base = (uint32_t)(32 * quarter) << 16;
    const uint32_t obuf = out_base + (uint32_t)(warp - 2) * C::OUT_BUFS * kFtOutBox;
    const uint32_t free_bar = CG == 2 ? map_to_rank(tempty, 0) : tempty;
    uint32_t n_acc = 0, n_store = 0, tiles_done = 0;
    // 32 columns of this lane's row into a staging box (64-byte rows, 64-byte swizzle) and out by TMA
    auto put = [&](const void* map, const uint32_t (&v)[16], int col, int row) {
      if (lane == 0) bulk_wait_read<C::OUT_BUFS - 1>();
      __syncwarp();
      const uint32_t box = obuf + n_store % C::OUT_BUFS * kFtOutBox;
      n_store++;
#pragma unroll
      for (int c = 0; c < 4; c++) {
        const uint32_t at = box + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[4 * c]), "r"(v[4 * c + 1]),
                     "r"(v[4 * c + 2]), "r"(v[4 * c + 3])
                     : "memory");
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ft_tma_store(map, box, col, row);
    };
    auto acc_ready = [&](uint32_t which, uint32_t parity) -> bool {
      const bool ok = __all_sync(kFull, mbar_wait(tfull + 8 * which, parity, abort_flag));
      tc_fence_after();
      return ok;
    };
    auto acc_release = [&](uint32_t buf) {  // this warp's loads from tensor memory are complete
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_or_local<CG>(free_bar + 8 * buf);
    };
    bool alive = true;
    for (int64_t t = first; alive && t < g.t.units; t += stride) {
      const FtTile tl = ft_tile<MODE, CG>(g.t, t);
      const int64_t M = g.t.M[tl.problem], N = g.t.N[tl.problem];
      const int row0 = (int)tl.m0 + (int)rank * 128 + 32 * quarter;
      if (MODE == kTcHiddenBwd) {
        const int halves = ft_halves(g.t, tl.n0);
        const uint32_t n_tile = tiles_done++;
        for (int half = 0; half < halves; half++, n_acc++) {
          if (!acc_ready(0, n_acc & 1)) {
            alive = false;
            break;
          }
          const int col = 32 * share, n = (int)tl.n0 + 128 * half + col;
          const uint32_t at = tmem + lane_base + col;
          // g and u leave tensor memory at once (the next products wait for their columns); what they
          // give takes their registers' place, and dh is read 16 columns at a time after that
          uint32_t gv[32], uv[32], o[16], o1[16];
          tmem_ld32(at, gv);
          tmem_ld32(at + 128, uv);
          tmem_ld_wait(gv);
          tmem_ld_wait(uv);
          acc_release(0);
          const bool in = row0 < M && n < N;
#pragma unroll
          for (int i = 0; i < 16; i++) {
            const uint64_t uu = pair_of(uv[2 * i], uv[2 * i + 1]);
            uint64_t a, da;
            ft_act<ACT, true>(pair_of(gv[2 * i], gv[2 * i + 1]), a, da);
            bits_of(mul2(uu, da), gv[2 * i], gv[2 * i + 1]);
            bits_of(a, uv[2 * i], uv[2 * i + 1]);
            o[i] = pack_bf16(mul2(a, uu));
          }
          if (in) put(&g.o[2], o, n, row0);
          if (half == 0 && !acc_ready(1, n_tile & 1)) {
            alive = false;
            break;
          }
#pragma unroll
          for (int c = 0; c < 2; c++) {
            uint32_t dv[16];
            tmem_ld16(at + 256 + 128 * half + 16 * c, dv);
            tmem_ld_wait16(dv);
#pragma unroll
            for (int i = 0; i < 8; i++) {
              const uint64_t dd = pair_of(dv[2 * i], dv[2 * i + 1]);
              const int j = 8 * c + i;
              o[j] = pack_bf16(mul2(dd, pair_of(gv[2 * j], gv[2 * j + 1])));
              o1[j] = pack_bf16(mul2(dd, pair_of(uv[2 * j], uv[2 * j + 1])));
            }
          }
          if (half + 1 == halves) acc_release(1);
          if (in) {
            put(&g.o[0], o, n, row0);
            put(&g.o[1], o1, n, row0);
          }
        }
        continue;
      }
      if (!acc_ready(n_acc & 1, (n_acc >> 1) & 1)) break;
      const uint32_t buf = n_acc & 1;
      n_acc++;
      const uint32_t acc = tmem + lane_base + 256 * buf;
      if (MODE == kTcHidden) {
#pragma unroll 1
        for (int c = 0; c < 2; c++) {
          const int col = share * 64 + c * 32;
          uint32_t gv[32], uv[32], o[16];
          tmem_ld32(acc + col, gv);
          tmem_ld32(acc + 128 + col, uv);
          tmem_ld_wait(gv);
          tmem_ld_wait(uv);
          if (c == 1) acc_release(buf);
          if (row0 >= M || tl.n0 + col >= N) continue;
#pragma unroll
          for (int i = 0; i < 16; i++) {
            uint64_t a, da;
            ft_act<ACT, false>(pair_of(gv[2 * i], gv[2 * i + 1]), a, da);
            o[i] = pack_bf16(mul2(a, pair_of(uv[2 * i], uv[2 * i + 1])));
          }
          put(&g.o[0], o, (int)tl.n0 + col, row0);
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < 4; c++) {
          const int col = share * 128 + c * 32;
          uint32_t v[32];
          tmem_ld32(acc + col, v);
          tmem_ld_wait(v);
          if (tl.kb0 >= tl.kb1) {  // a part that a short last chunk leaves empty: no product was formed
#pragma unroll
            for (int i = 0; i < 32; i++) v[i] = 0u;
          }
          if (c == 3) acc_release(buf);
          if (row0 >= M || tl.n0 + col >= N) continue;
          const int64_t row = row0 + lane, n = tl.n0 + col;
          if (tl.sums) {
            if (row < M) {
              float* to = tl.sums + (int64_t)((int)rank * 128 + 32 * quarter + lane) * 256 + col;
#pragma unroll
              for (int j = 0; j < 8; j++) {
                float4 x = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                       __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
                if (g.t.accumulate) {
                  const float4 old = *reinterpret_cast<const float4*>(to + 4 * j);
                  x.x += old.x; x.y += old.y; x.z += old.z; x.w += old.w;
                }
                *reinterpret_cast<float4*>(to + 4 * j) = x;
              }
            }
          } else {
            uint32_t o[16];
            if (MODE == kTcOut && g.add) {
              uint32_t ad[16];
#pragma unroll
              for (int j = 0; j < 4; j++) {
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (row < M && n + 8 * j < N) x = *reinterpret_cast<const uint4*>(g.add + row * N + n + 8 * j);
                ad[4 * j] = x.x; ad[4 * j + 1] = x.y; ad[4 * j + 2] = x.z; ad[4 * j + 3] = x.w;
              }
#pragma unroll
              for (int i = 0; i < 16; i++)
                o[i] = pack_bf16(__uint_as_float(v[2 * i]) + __uint_as_float(ad[i] << 16),
                                 __uint_as_float(v[2 * i + 1]) + __uint_as_float(ad[i] & 0xffff0000u));
            } else {
#pragma unroll
              for (int i = 0; i < 16; i++) o[i] = pack_bf16(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
            }
            put(&g.o[tl.problem], o, (int)n, row0);
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();  // the pair's barriers and tensor memory stay until both are done
  tc_fence_after();
  if (warp == 1) ft_tmem_dealloc<CG>(tmem);
}

// Joins the parts of the tail's tiles: out = sum of the parts, in order, (+ add), rounded once.  Block:
// 64 groups of four columns by four rows; blockIdx.x a tail tile, blockIdx.y a share of its rows.
struct FtTail {
  FtTiles t;
  const __nv_bfloat16* add;
  __nv_bfloat16* out[3];
  int tile_m;
};
__global__ void __launch_bounds__(256) dsa3d_ffn_tail_kernel(const __grid_constant__ FtTail a) {
  int problem;
  int64_t m0, n0;
  ft_place(a.t, a.t.full + blockIdx.x, a.tile_m, 256, problem, m0, n0);
  prior_kernel_done();
  const int64_t M = a.t.M[problem], N = a.t.N[problem];
  const int c = 4 * (threadIdx.x & 63);
  const int64_t n = n0 + c;
  if (n >= N) return;
  const float* from = a.t.sums + (int64_t)blockIdx.x * a.t.parts * a.tile_m * 256 + c;
  __nv_bfloat16* out = a.out[problem];
  for (int r = blockIdx.y * 4 + (threadIdx.x >> 6); r < a.tile_m && m0 + r < M; r += gridDim.y * 4) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = 0; p < a.t.parts; p++) {
      const float4 x = *reinterpret_cast<const float4*>(from + ((int64_t)p * a.tile_m + r) * 256);
      v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
    }
    const int64_t at = (m0 + r) * N + n;
    float o[4] = {v.x, v.y, v.z, v.w};
    if (N % 4 == 0) {
      if (a.add) {
        const uint2 x = *reinterpret_cast<const uint2*>(a.add + at);
        o[0] += __uint_as_float(x.x << 16);
        o[1] += __uint_as_float(x.x & 0xffff0000u);
        o[2] += __uint_as_float(x.y << 16);
        o[3] += __uint_as_float(x.y & 0xffff0000u);
      }
      *reinterpret_cast<uint2*>(out + at) = make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
    } else {
#pragma unroll
      for (int e = 0; e < 4; e++)
        if (n + e < N) out[at + e] = __float2bfloat16_rn(o[e] + (a.add ? __bfloat162float(a.add[at + e]) : 0.f));
    }
  }
}

}  // namespace dsa3d
