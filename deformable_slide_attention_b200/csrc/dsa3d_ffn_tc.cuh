// dsa3d_ffn_tc.cuh -- the gated feed-forward block's products on the tensor cores (bf16, sm_100a):
//
//   kTcHidden     h = act(x Wg) * (x Wu)                                one tile: 128 columns of g and of u
//   kTcHiddenBwd  g, u as above and dh = dy Wd^T, then dg = dh u act'(g), du = dh act(g), h = act(g) u
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
// the second (of the pair's first CTA) the MMAs, eight warps the epilogue: accumulators leave tensor
// memory 32 columns at a time, the activation and its derivative are formed in registers in fp32, and
// the results are rounded once and leave through shared memory by TMA, which also clips them to the
// tensors' edges.  Tensor memory holds two tiles' accumulators (kTcHiddenBwd: g and u once, dh twice,
// its next tile's dh product running while the epilogue still reads), so that the epilogue of a tile
// overlaps the products of the next.
//
// The products are bound by the tensor cores (6 or 16 rows C hidden operations against a few bytes per
// element).  Waits are bounded (dsa3d_tc.cuh); no load is multicast.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "dsa3d_ffn_any.cuh"
#include "dsa3d_tc.cuh"

namespace dsa3d {

enum TcMode { kTcHidden, kTcHiddenBwd, kTcOut, kTcDx, kTcDw };

constexpr int kFtEpiWarps = 8;
constexpr int kFtThreads = 32 * (2 + kFtEpiWarps);
constexpr int kFtK = 64;                 // summed-axis elements per stage
constexpr uint32_t kFtABytes = 128 * kFtK * 2;
constexpr uint32_t kFtOutBox = 32 * 32 * 2;  // an epilogue store: 32 rows x 32 columns of bf16

template <int MODE, int CG>
struct FtCfg {
  static constexpr bool kGated = MODE == kTcHidden || MODE == kTcHiddenBwd;
  static constexpr int TILE_M = 128 * CG;
  static constexpr int TILE_N = kGated ? 128 : 256;  // output columns per tile
  static constexpr uint32_t B_BYTES = 256 / CG * kFtK * 2;
  static constexpr uint32_t STAGE = kFtABytes + B_BYTES;
  static constexpr int OUT_BUFS = MODE == kTcHiddenBwd ? 3 : 2;
  static constexpr uint32_t OUT_BYTES = kFtEpiWarps * OUT_BUFS * kFtOutBox;
  static constexpr int STAGES = CG == 2 ? (MODE == kTcHiddenBwd ? 5 : 6) : (MODE == kTcHiddenBwd ? 3 : 4);
  static constexpr uint32_t SMEM = 1024 + STAGES * STAGE + OUT_BYTES + 256;
};

struct FtArgs {
  CUtensorMap a[3], b[3], o[3];
  const __nv_bfloat16* add;  // kTcOut
  float* partial;            // parts of the summed axis: [part][M][N] per problem, instead of o
  int64_t M[3], N[3];        // outputs' sizes per problem (kTcDw: three problems, else one)
  int64_t tiles;             // over all problems and parts
  int tiles_of[3];           // per problem and part
  int tiles_m[3];
  int kblocks;               // of one product's summed axis
  int parts, per_part;       // parts of it, k-blocks in each but the last
  int problems, act, group;  // group: row tiles walked together
  bool accumulate;           // add to what partial holds
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
  int problem, part, kb0, kb1;
  int64_t m0, n0;
};
// Tiles are numbered problem by problem, part by part, in groups of `group` row tiles whose columns
// are walked together, so that the tiles in flight share their operands in L2.
template <int MODE, int CG>
__device__ __forceinline__ FtTile ft_tile(const FtArgs& g, int64_t t) {
  using C = FtCfg<MODE, CG>;
  FtTile r;
  r.problem = 0;
  if (MODE == kTcDw) {
    while (r.problem < 2 && t >= (int64_t)g.tiles_of[r.problem] * g.parts) {
      t -= (int64_t)g.tiles_of[r.problem] * g.parts;
      r.problem++;
    }
  }
  const int per = g.tiles_of[r.problem], tm = g.tiles_m[r.problem];
  r.part = (int)(t / per);
  const int i = (int)(t - (int64_t)r.part * per), tn = per / tm;
  const int gi = i / (g.group * tn), in = i - gi * g.group * tn;
  const int rows = min(g.group, tm - gi * g.group);
  r.m0 = (int64_t)(gi * g.group + in % rows) * C::TILE_M;
  r.n0 = (int64_t)(in / rows) * C::TILE_N;
  r.kb0 = r.part * g.per_part;
  r.kb1 = min(r.kb0 + g.per_part, g.kblocks);
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float ft_silu_sig(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }

template <int MODE, int CG>
__global__ void __launch_bounds__(kFtThreads, 1) dsa3d_ffn_tc_kernel(const __grid_constant__ FtArgs g) {
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

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const int64_t first = blockIdx.x / CG, stride = gridDim.x / CG;
  constexpr int kAccBufs = MODE == kTcHiddenBwd ? 1 : 2;  // of 256 columns that the epilogue releases

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; s++) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; s++) {
      mbar_init(tfull + 8 * s, 1);
      mbar_init(tempty + 8 * s, kFtEpiWarps * CG);
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
      for (int64_t t = first; ok && t < g.tiles; t += stride) {
        const FtTile tl = ft_tile<MODE, CG>(g, t);
        const int m = (int)tl.m0 + (int)rank * 128, n = (int)tl.n0;
        constexpr int SEGS = (MODE == kTcHiddenBwd || MODE == kTcDx) ? 2 : 1;
#pragma unroll
        for (int seg = 0; seg < SEGS; seg++) {
          const bool dh = MODE == kTcHiddenBwd && seg == 0;
          const int which = MODE == kTcDw ? tl.problem : seg;
          const void* ma = &g.a[which];
          for (int kb = tl.kb0; ok && kb < tl.kb1; kb++, it++) {
            const int s = it % C::STAGES;
            if (it >= C::STAGES) ok = mbar_wait(empty + 8 * s, (it / C::STAGES - 1) & 1, abort_flag);
            if (!ok) break;
            const uint32_t sa = base + s * C::STAGE, sb = sa + kFtABytes;
            const uint32_t local = full + 8 * s;
            const uint32_t bar = CG == 2 ? map_to_rank(local, 0) : local;
            if (rank == 0) mbar_arrive_expect_tx(local, CG * kFtABytes + (dh ? 128 : 256) * kFtK * 2);
            const int k = kb * kFtK;
            if (MODE == kTcDw) {  // MN-major A: two boxes of 64 rows
              ft_tma_load<CG>(sa, ma, bar, m, k);
              ft_tma_load<CG>(sa + 8192, ma, bar, m + 64, k);
            } else {
              ft_tma_load<CG>(sa, ma, bar, k, m);
            }
            if (dh) {  // Wd's rows n.. as B, K-major
              ft_tma_load<CG>(sb, &g.b[2], bar, k, n + (int)rank * 64);
            } else if (C::kGated) {  // Wg's and Wu's columns, MN-major: gate for the first half of B
              if (CG == 1) {
                for (int j = 0; j < 4; j++) ft_tma_load<CG>(sb + 8192 * j, &g.b[j >> 1], bar, n + (j & 1) * 64, k);
              } else {
                for (int j = 0; j < 2; j++) ft_tma_load<CG>(sb + 8192 * j, &g.b[rank], bar, n + j * 64, k);
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
    // ---- MMA issuer: one thread, of the pair's first CTA
    if (lane == 0 && rank == 0) {
      constexpr uint32_t ID = umma_idesc_bf16(128 * CG, 256, MODE == kTcDw, MODE != kTcDx);
      constexpr uint32_t ID_DH = umma_idesc_bf16(128 * CG, 128, false, false);
      constexpr uint32_t A_STEP = MODE == kTcDw ? 2048 : 32;  // bytes per 16 of the summed axis
      constexpr uint32_t B_STEP = MODE == kTcDx ? 32 : 2048;
      uint32_t it = 0, n_tile = 0;
      bool ok = true;
      for (int64_t t = first; ok && t < g.tiles; t += stride, n_tile++) {
        const FtTile tl = ft_tile<MODE, CG>(g, t);
        const int nkb = tl.kb1 - tl.kb0;
        const uint32_t buf = kAccBufs == 2 ? (n_tile & 1) : 0;
        constexpr int SEGS = (MODE == kTcHiddenBwd || MODE == kTcDx) ? 2 : 1;
#pragma unroll
        for (int seg = 0; seg < SEGS; seg++) {
          const bool dh = MODE == kTcHiddenBwd && seg == 0;
          const uint32_t d = tmem + (dh ? 256 + 128 * (n_tile & 1) : 256 * buf);
          // the columns' previous tile has been read (dh's: known since the last tile's wait for g, u)
          if (!dh && (MODE != kTcDx || seg == 0)) {
            if (n_tile >= (uint32_t)kAccBufs)
              ok = ok && mbar_wait(tempty + 8 * buf, (n_tile / kAccBufs - 1) & 1, abort_flag);
          }
          for (int kb = 0; ok && kb < nkb; kb++, it++) {
            const int s = it % C::STAGES;
            ok = mbar_wait(full + 8 * s, (it / C::STAGES) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sa = base + s * C::STAGE, sb = sa + kFtABytes;
            const uint64_t da = umma_sdesc_sw128(sa, MODE == kTcDw ? 8192 : 16, 1024);
            const uint64_t db = umma_sdesc_sw128(sb, (dh || MODE == kTcDx) ? 16 : 8192, 1024);
#pragma unroll
            for (int k = 0; k < kFtK / 16; k++) {
              const uint32_t acc = (kb > 0 || k > 0 || (MODE == kTcDx && seg > 0)) ? 1u : 0u;
              ft_mma<CG>(d, da + (uint64_t)(k * A_STEP >> 4), db + (uint64_t)(k * (dh ? 32 : B_STEP) >> 4),
                         dh ? ID_DH : ID, acc);
            }
            ft_commit<CG>(empty + 8 * s);
          }
        }
        if (ok) ft_commit<CG>(tfull + 8 * (n_tile & 1));
      }
    }
  } else {
    // ---- epilogue: warp e reads tensor-memory lanes 32 (warp % 4).., half the tile's columns
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lane_base = (uint32_t)(32 * quarter) << 16;
    const uint32_t obuf = out_base + (uint32_t)(warp - 2) * C::OUT_BUFS * kFtOutBox;
    const uint32_t free_bar = CG == 2 ? map_to_rank(tempty, 0) : tempty;
    uint32_t n_tile = 0, n_store = 0;
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
    for (int64_t t = first; t < g.tiles; t += stride, n_tile++) {
      const FtTile tl = ft_tile<MODE, CG>(g, t);
      if (!__all_sync(kFull, mbar_wait(tfull + 8 * (n_tile & 1), (n_tile >> 1) & 1, abort_flag))) break;
      tc_fence_after();
      const uint32_t buf = kAccBufs == 2 ? (n_tile & 1) : 0;
      const uint32_t acc = tmem + lane_base + 256 * buf;
      const int64_t M = g.M[tl.problem], N = g.N[tl.problem];
      const int row0 = (int)tl.m0 + (int)rank * 128 + 32 * quarter;
      if (C::kGated) {
#pragma unroll 1
        for (int c = 0; c < 2; c++) {
          const int col = half * 64 + c * 32;
          uint32_t gv[32], uv[32], o[16];
          tmem_ld32(acc + col, gv);
          tmem_ld32(acc + 128 + col, uv);
          const bool in = row0 < M && tl.n0 + col < N;
          if (MODE == kTcHidden) {
            tmem_ld_wait(gv);
            tmem_ld_wait(uv);
            if (c == 1) {
              tc_fence_before();
              if (lane == 0) mbar_arrive_cluster_or_local<CG>(free_bar + 8 * buf);
            }
            if (!in) continue;
#pragma unroll
            for (int i = 0; i < 16; i++) {
              float h[2];
#pragma unroll
              for (int e = 0; e < 2; e++) {
                const float gg = __uint_as_float(gv[2 * i + e]), uu = __uint_as_float(uv[2 * i + e]);
                h[e] = (g.act == kActSilu ? gg * ft_silu_sig(gg) : ffn_act_only<__nv_bfloat16>(kActGelu, gg)) * uu;
              }
              o[i] = pack_bf16(h[0], h[1]);
            }
            put(&g.o[0], o, (int)tl.n0 + col, row0);
          } else {
            uint32_t dv[32];
            tmem_ld32(tmem + lane_base + 256 + 128 * (n_tile & 1) + col, dv);
            tmem_ld_wait(gv);
            tmem_ld_wait(uv);
            tmem_ld_wait(dv);
            if (c == 1) {
              tc_fence_before();
              if (lane == 0) mbar_arrive_cluster_or_local<CG>(free_bar);
            }
            if (!in) continue;
            uint32_t o1[16], o2[16];
#pragma unroll
            for (int i = 0; i < 16; i++) {
              float r0[2], r1[2], r2[2];
#pragma unroll
              for (int e = 0; e < 2; e++) {
                const float gg = __uint_as_float(gv[2 * i + e]), uu = __uint_as_float(uv[2 * i + e]);
                const float dd = __uint_as_float(dv[2 * i + e]);
                float a, da;
                if (g.act == kActSilu) {
                  const float s = ft_silu_sig(gg);
                  a = gg * s;
                  da = s * fmaf(gg, 1.f - s, 1.f);
                } else {
                  ffn_act<__nv_bfloat16>(kActGelu, gg, a, da);
                }
                r0[e] = dd * uu * da;
                r1[e] = dd * a;
                r2[e] = a * uu;
              }
              o[i] = pack_bf16(r0[0], r0[1]);
              o1[i] = pack_bf16(r1[0], r1[1]);
              o2[i] = pack_bf16(r2[0], r2[1]);
            }
            put(&g.o[0], o, (int)tl.n0 + col, row0);
            put(&g.o[1], o1, (int)tl.n0 + col, row0);
            put(&g.o[2], o2, (int)tl.n0 + col, row0);
          }
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < 4; c++) {
          const int col = half * 128 + c * 32;
          uint32_t v[32];
          tmem_ld32(acc + col, v);
          tmem_ld_wait(v);
          if (tl.kb0 >= tl.kb1) {  // a part that a short last chunk leaves empty: no product was formed
#pragma unroll
            for (int i = 0; i < 32; i++) v[i] = 0u;
          }
          if (c == 3) {
            tc_fence_before();
            if (lane == 0) mbar_arrive_cluster_or_local<CG>(free_bar + 8 * buf);
          }
          if (row0 >= M || tl.n0 + col >= N) continue;
          const int64_t row = row0 + lane, n = tl.n0 + col;
          if (g.partial) {
            int64_t off = 0;
            for (int p = 0; p < tl.problem; p++) off += g.M[p] * g.N[p] * g.parts;
            float* to = g.partial + off + ((int64_t)tl.part * M + row) * N + n;
            if (row < M) {
#pragma unroll
              for (int j = 0; j < 8; j++) {
                if (n + 4 * j < N) {
                  float4 x = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                         __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
                  if (g.accumulate) {
                    const float4 old = *reinterpret_cast<const float4*>(to + 4 * j);
                    x.x += old.x; x.y += old.y; x.z += old.z; x.w += old.w;
                  }
                  *reinterpret_cast<float4*>(to + 4 * j) = x;
                }
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

}  // namespace dsa3d
