// bi_gemm4.cu — batch-invariant product of two matrices in 4 bits, y = alpha x w^T, for sm_103a (TMA, tcgen05
// block-scaled MMAs, TMEM).  Implements the product of include/bi_fp4.h.
//
//   y[m, n] = alpha * sum over k of (code_x[m, k] scale_x[m, k / block]) (code_w[n, k] scale_w[n, k / block])
//
// Every element of y is summed by one sequence of tcgen05.mma instructions, 64 elements of K each, ascending: a
// function of K alone.  fp32 accumulators in tensor memory; alpha and the rounding to bf16 come once, at the end.
//
// Two forms share the work, with the same bits.  Many rows: CTA pairs take 256 x 256 of y, bound by the tensor pipe:
// 8192 x 4096 x 14336 (M, K, N) in 154 us with nvfp4 (6.2 PFLOP/s) and 149 with mxfp4 (6.4), where four times the
// measured bf16 rate would allow 125 (the rate of these instructions by themselves was not measured, nor that of their
// form of 96 elements); thousands of calls on end, at the power limit and 1770 MHz, 167 and 158.  2048 rows 43 us.  Few
// rows: the operands change places, bound by the latency of one CTA's chain of stages: one row by 4096 x 14336 in 8.1
// us where its bytes take 4.9, 64 rows by 14336 x 4096 (mxfp4) in 13.0.  By a vocabulary, bound by the bytes of w: 1,
// 32 and 128 rows by 4096 x 128256 in 47, 49 and 56 us (0.94, 0.92 and 0.86 of the measured copy).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>

#include "../../include/bi_fp4.h"
#include "attn_ptx.cuh"
#include "fp4.cuh"

#ifndef BI_GEMM_API
#define BI_GEMM_API extern "C" __attribute__((visibility("default")))
#endif

namespace big4 {

namespace ptx = bigemm::ptx;
using biattn_tc::Sync;
using biattn_tc::wait_bar;

constexpr int kStageK = 256;              // elements of K a stage: one 128-byte swizzle row
constexpr uint64_t kTimeoutNs = biattn_tc::kTimeoutNs;

struct Params {
  const uint8_t* sx;
  const uint8_t* sw;
  uint32_t* status;
  int32_t M, N, K;
  int32_t m_tiles, n_tiles, kblocks;
  int32_t tiles;            // scale tiles along K
  int32_t x_rows;           // rows of an x box
  int32_t group_m;          // raster: M tiles of a group (N tiles vary slowest within it)
  float alpha;
  int32_t stall;            // failure injection (test controls only): nothing is loaded
  uint64_t timeout_ns;
};

template <bool kNv>
__device__ __forceinline__ void mma4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                          uint32_t accumulate) {
  if constexpr (kNv)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Instruction descriptor: E2M1 x E2M1, both along K, E8M0 or E4M3 scales.
template <bool kNv>
constexpr __host__ __device__ uint32_t idesc4(int M, int N) {
  return (1u << 7) | (1u << 10) | (uint32_t(N >> 3) << 17) | (kNv ? 0u : 1u << 23) | (uint32_t(M >> 4) << 24);
}

// Matrix descriptor: rows of 128 bytes, 128-byte swizzle, groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_rows(uint32_t a) { return biattn_tc::sdesc_sw128(a, 16, 1024); }
// A tile of scales, 32 rows of 16 bytes, no swizzle: tcgen05.cp makes four columns of it.
__device__ __forceinline__ uint64_t desc_scales(uint32_t a) {
  return uint64_t((a & 0x3FFFFu) >> 4) | (uint64_t(128 >> 4) << 32) | (1ull << 46);
}

template <bool kNv>
__device__ __forceinline__ void mma4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                     uint32_t accumulate) {
  if constexpr (kNv)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Untiled bulk copy global -> shared (16-byte aligned, a multiple of 16 bytes), counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// ------------------------------------------------------------------ the form for many rows
//
// A pair of CTAs, persistent; warp 0 of each loads its half of the codes (128-byte swizzle rows of 256 elements) and
// the scales (tiles as they lie in memory, as boxes of 512-byte rows), the leader's warp 1 moves the scales to tensor
// memory (tcgen05.cp) and issues the products, eight warps store.  One accumulator: 256 columns, and five stages'
// scales behind it; the eight warps read it at once and hand it back before they round and store.  us for 8192 x 4096
// x 14336, nvfp4: 310 with the issuing thread chosen by its lane number, 206 with the scales stored to tensor memory
// by four warps, 157 with the thread named by elect.sync (operands in uniform registers) and the copies back; without
// copies of scales 145, without loads 134.  Waits: every lane polls, backing off by the clock (one lane alone 228,
// suspended waits 210, nanosleep 300); a wait with a cluster-wide acquire in the issuing thread 380.

template <bool kNv_, bool kF32_>
struct Wide {
  static constexpr bool kNv = kNv_, kF32 = kF32_;
  static constexpr int TM = 256, TN = 256;             // of y per CTA pair
  static constexpr int TILES_K = kNv ? 4 : 2;          // scale tiles (of 4 scales) a stage
  static constexpr int A_BYTES = 128 * 128, B_BYTES = 128 * 128;
  static constexpr int SFA_BYTES = TILES_K * 512, SFB_BYTES = 2 * TILES_K * 512;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
  static constexpr int STAGES = 5;
  static constexpr int SF_COLS = TILES_K * 12;         // TMEM columns of a stage's scales: x 4, w 8 a tile
  static constexpr int SF_COL0 = TN;
  static_assert(SF_COL0 + STAGES * SF_COLS <= 512, "tensor memory");
  static constexpr int EPI_WARPS = 8, EPI_WARP0 = 4, THREADS = 384;       // warps: 0 loads, 1 products, 4 .. results
  static constexpr int OUT = kF32 ? 4 : 2;
  static constexpr int STG_BYTES = 32 * 32 * OUT;
  static constexpr int STG_BUFS = kF32 ? 1 : 2;
  static constexpr int OFF_B = STAGES * A_BYTES;
  static constexpr int OFF_SF = OFF_B + STAGES * B_BYTES;
  static constexpr int OFF_STG = OFF_SF + STAGES * (SFA_BYTES + SFB_BYTES);
  static_assert(OFF_STG % 1024 == 0, "swizzle atoms");
  static constexpr int OFF_BAR = OFF_STG + EPI_WARPS * STG_BUFS * STG_BYTES;
  static constexpr int BARS = 2 * STAGES + 3;
  static constexpr int SMEM = OFF_BAR + BARS * 8 + 16 + 1024;
  static_assert(SMEM <= 232448, "shared memory");
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) __cluster_dims__(2, 1, 1)
    wide_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                const __grid_constant__ CUtensorMap msx, const __grid_constant__ CUtensorMap msw,
                const __grid_constant__ CUtensorMap my, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = ptx::smem_u32(smem), bars = base + C::OFF_BAR;
  auto full = [&](int s) { return bars + 8u * s; };                        // the leader's: both CTAs' operands are there
  auto empty = [&](int s) { return bars + 8u * (C::STAGES + s); };         // the stage's products are done
  const uint32_t tfull = bars + 16u * C::STAGES, tempty = tfull + 8, drain = tfull + 16;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + C::BARS * 8);
  volatile uint32_t* gave_up = misc + 1;
  const int warp = __shfl_sync(0xFFFFFFFFu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  // One lane of a warp loads, or issues the products.  elect.sync names it: the compiler then keeps the operands of
  // TMA and MMA instructions in uniform registers (with `lane == 0` a product cost about 180 clocks to issue).
  const bool lead = biattn_tc::elect_one();
  const int group = blockIdx.x / 2, groups = gridDim.x / 2, units = p.m_tiles * p.n_tiles;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      ptx::mbar_init(full(s), 1);
      ptx::mbar_init(empty(s), 1);
    }
    ptx::mbar_init(tfull, 1);
    ptx::mbar_init(tempty, 2 * C::EPI_WARPS);
    ptx::mbar_init(drain, 1);
    *gave_up = 0u;
    ptx::fence_barrier_init();
    ptx::fence_proxy_async_smem();
    for (const CUtensorMap* m : {&mx, &mw, &msx, &msw, &my}) ptx::prefetch_tensormap(m);
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_u32(misc), 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();                   // the peer's barriers are there and its TMEM is allocated
  ptx::tc_fence_after();
  const uint32_t tmem = misc[0];
  const Sync sy{gave_up, p.status, p.timeout_ns};
  auto place = [&](int u, int& m, int& n) {
    // groups of group_m M tiles; within a group N slowest, so that the tiles in work share W
    const int per = p.group_m * p.n_tiles, g = u / per, r = u - g * per;
    const int gm = min(p.group_m, p.m_tiles - g * p.group_m);
    n = r / gm;
    m = g * p.group_m + (r - n * gm);
  };
  if (warp == 0 && lead) {
    // ---------------------------------------------------------------- loads
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    const uint32_t x_bytes = uint32_t(p.x_rows) * 128u + C::SFA_BYTES, w_bytes = C::B_BYTES + C::SFB_BYTES;
    for (int u = group; u < units && ok; u += groups) {
      int m, n;
      place(u, m, n);
      const int row0 = m * C::TM + int(rank) * 128, col0 = n * C::TN;
      const bool mine = row0 < p.M, peers = m * C::TM + 128 < p.M;    // rows past M are not loaded
      for (int kb = 0; kb < p.kblocks; ++kb) {
        if (!wait_bar(empty(s), ph ^ 1u, sy)) {
          ok = false;
          break;
        }
        if (!p.stall) {
          const uint32_t fb = ptx::mapa_shared(full(s), 0);
          if (rank == 0) ptx::mbar_arrive_expect_tx(full(s), x_bytes * (peers ? 2u : 1u) + 2u * w_bytes);
          const uint32_t sf = base + C::OFF_SF + uint32_t(s) * (C::SFA_BYTES + C::SFB_BYTES);
          if (mine) {
            ptx::tma_load_2d_pair(base + uint32_t(s) * C::A_BYTES, &mx, fb, kb * 128, row0);
            ptx::tma_load_2d_pair(sf, &msx, fb, kb * (C::TILES_K * 64), row0 / 128);
          }
          ptx::tma_load_2d_pair(base + C::OFF_B + uint32_t(s) * C::B_BYTES, &mw, fb, kb * 128, col0 + int(rank) * 128);
          ptx::tma_load_2d_pair(sf + C::SFA_BYTES, &msw, fb, kb * (C::TILES_K * 64), col0 / 128);
        }
        if (++s == C::STAGES) s = 0, ph ^= 1u;
      }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  } else if (warp == 1 && lead && rank == 0) {
    // ---------------------------------------------------------------- products (leader)
    int s = 0;
    uint32_t ph = 0, tph = 0;
    bool ok = true, issued = false;
    for (int u = group; u < units && ok; u += groups) {
      if (!wait_bar(tempty, tph ^ 1u, sy)) {
        ok = false;
        break;
      }
      tph ^= 1u;
      ptx::tc_fence_after();
      for (int kb = 0; kb < p.kblocks; ++kb) {
        if (!wait_bar(full(s), ph, sy)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t a = base + uint32_t(s) * C::A_BYTES, b = base + C::OFF_B + uint32_t(s) * C::B_BYTES;
        const uint32_t sf = base + C::OFF_SF + uint32_t(s) * (C::SFA_BYTES + C::SFB_BYTES);
        const uint32_t ta = tmem + C::SF_COL0 + uint32_t(s) * C::SF_COLS, tb = ta + C::TILES_K * 4;
        // scales: x's tiles of each CTA's rows, w's of all 256 columns (a tile's halves side by side)
#pragma unroll
        for (int t = 0; t < C::TILES_K; ++t) {
          ptx::tc_cp_32x128b_x4_pair(ta + 4u * t, desc_scales(sf + 512u * t));
#pragma unroll
          for (int h = 0; h < 2; ++h)
            ptx::tc_cp_32x128b_x4_pair(tb + 8u * t + 4u * h,
                                       desc_scales(sf + C::SFA_BYTES + uint32_t(h * C::TILES_K + t) * 512u));
        }
        const int steps = min(4, (p.K - kb * kStageK) / 64);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k < steps) {
            const int t = C::kNv ? k : k >> 1;
            const uint32_t id = C::kNv ? 0u : uint32_t(k & 1) * 2u;
            mma4_pair<C::kNv>(tmem, desc_rows(a + 32u * k), desc_rows(b + 32u * k),
                              idesc4<C::kNv>(C::TM, C::TN) | (id << 4) | (id << 29), ta + 4u * t, tb + 8u * t,
                              kb != 0 || k != 0 ? 1u : 0u);
          }
        }
        issued = true;
        ptx::tc_commit_pair_mc(empty(s), 0x3);
        if (++s == C::STAGES) s = 0, ph ^= 1u;
      }
      if (ok) ptx::tc_commit_pair_mc(tfull, 0x3);
    }
    if (!ok && issued) {                 // what was issued ends before TMEM is released
      ptx::tc_commit_pair_mc(drain, 0x1);
      volatile uint32_t never = 0;
      wait_bar(drain, 0u, Sync{&never, p.status, p.timeout_ns});
    }
  } else if (warp >= C::EPI_WARP0) {
    // ---------------------------------------------------------------- results
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int e = warp - C::EPI_WARP0, q = warp & 3, half = e >> 2;
    const uint32_t stg = base + C::OFF_STG + uint32_t(e) * (C::STG_BUFS * C::STG_BYTES);
    uint32_t tph = 0;
    int buf = 0;
    for (int u = group; u < units; u += groups) {
      int m, n;
      place(u, m, n);
      if (!__all_sync(0xFFFFFFFFu, wait_bar(tfull, tph, sy))) break;
      tph ^= 1u;
      ptx::tc_fence_after();
      const int row0 = m * C::TM + int(rank) * 128 + q * 32, col0 = n * C::TN + half * 128;
      const int chunks = row0 < p.M ? max(0, min(4, (p.N - col0 + 31) / 32)) : 0;
      const uint32_t from = tmem + (uint32_t(q * 32) << 16) + uint32_t(half * 128);
      auto release = [&]() {             // the accumulator is free (the leader waits for both CTAs)
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          ptx::fence_release_shared();
          ptx::mbar_arrive_remote_relaxed(ptx::mapa_shared(tempty, 0));
        }
      };
      auto store = [&](int c, const uint32_t (&w)[16 * C::OUT / 2]) {
        const uint32_t dst = stg + uint32_t(buf) * C::STG_BYTES;
        if (lane == 0) ptx::bulk_wait_read<C::STG_BUFS - 1>();
        __syncwarp();
#pragma unroll
        for (int v = 0; v < 2 * C::OUT; ++v)              // rows of 128 or 64 bytes in their swizzle
          ptx::st_shared_v4(dst + uint32_t(C::kF32 ? lane * 128 + ((v ^ (lane & 7)) << 4)
                                                   : lane * 64 + ((v ^ ((lane >> 1) & 3)) << 4)),
                            w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::tma_store_2d(&my, dst, col0 + c * 32, row0);
          ptx::bulk_commit();
        }
        if (++buf == C::STG_BUFS) buf = 0;
      };
      if constexpr (C::kF32) {
        if (chunks == 0) release();
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
          uint32_t r[32];
          ptx::tmem_ld_32x32b_x32(from + 32u * c, r);
          ptx::tmem_wait_ld();
          if (c + 1 == chunks) release();
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__fmul_rn(__uint_as_float(r[i]), p.alpha));
          store(c, r);
        }
      } else {
        // the warp's whole share leaves tensor memory, rounded, before any of it is stored
        uint32_t pk[4][16];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c < chunks) {
            uint32_t r[32];
            ptx::tmem_ld_32x32b_x32(from + 32u * c, r);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              pk[c][i] = ptx::pack_bf16x2_ordered(__fmul_rn(__uint_as_float(r[2 * i]), p.alpha),
                                                  __fmul_rn(__uint_as_float(r[2 * i + 1]), p.alpha));
          }
        }
        release();
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < chunks) store(c, pk[c]);
      }
    }
    if (lane == 0) ptx::bulk_wait_read<0>();
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *gave_up) {    // let every copy in flight land before the block leaves
    const uint64_t t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < 2000000ull) {
    }
  }
  __syncwarp();
  ptx::cluster_sync();                   // neither CTA leaves while the pair still works
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------ the form for few rows
//
// The operands change places: rows of w on the 128 rows of the MMA, up to 128 rows of x on its columns, so that a CTA
// alone takes 32, 64 or 128 columns of y and as many of them as there are SMs share the reading of w.  The sums have
// the wide form's bits: an element is the same sequence of 64-element products, and neither the place of its row and
// column in an instruction nor the instruction's extent enters (compared over every shape that the tests run).
//
// A CTA's R rows of w take the MMA's rows that they have in their tile of 128 (so that a tile of scales serves as it
// is); the other rows multiply whatever the neighbouring slots hold, and are not stored.
//
// A stage is two or four slots of 256 elements of K.  A turn of the loading loop costs about 250 clocks besides its
// copies, of 28 each; one of the issuing loop about 160 besides its products, of 40 each (128 rows of 32 bytes from
// shared memory, however few columns meet them), and its scales' copies, of 11: for 1 x 14336 x 4096 these, not the
// loads, take the time (9.7 us without the products, 13.5 with them; two loading warps 8.0 and 13.7).  Four slots are
// taken where three such stages fit: 13.5 -> 12.3 us there, 64 x 14336 x 4096 14.3 -> 13.1 (both mxfp4; nvfp4 takes
// 14.0 and 14.4 with them), 16 x 32768 x 2048 30.8 -> 27.3 (nvfp4); with two stages 64 x 4096 x 14336 9.4 -> 11.0,
// with one 1 x 512 x 4096 2.7 -> 2.9.

constexpr int kFewMaxStages = 8;
constexpr int kFewCols = 128;             // rows of x at most
constexpr int kFewThreads = 256;          // warps: 0 loads, 1 products, 4 .. 7 results

struct FewParams {
  Params p;
  int32_t rows;             // R
  int32_t cols;             // columns of the MMA: rows of x of a tile, a multiple of 16
  int32_t slots, stages;
  int32_t tmem_cols;
  int32_t off_w, off_sf, off_stg, off_bar;   // shared memory: x ring at 0, w ring, scales ring, staging, barriers
};

template <bool kNv, bool kF32, int kSlots_>
struct Few {
  static constexpr int kSlots = kSlots_;                     // of a stage
  static constexpr int TILES_K = kNv ? 4 : 2;                // scale tiles of a slot
  static constexpr int SF_BYTES = kSlots * TILES_K * 512;    // of a stage and operand
  static constexpr int SF_COLS = TILES_K * 8;                // TMEM columns of a slot's scales
  static constexpr int OUT = kF32 ? 4 : 2, STG_BYTES = 32 * 32 * OUT;      // of a warp
};

template <bool kNv, bool kF32, int kSlots>
__global__ void __launch_bounds__(kFewThreads)
    few_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
               const __grid_constant__ CUtensorMap my, const FewParams f) {
  using C = Few<kNv, kF32, kSlots>;
  const Params& p = f.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = ptx::smem_u32(smem), bars = base + uint32_t(f.off_bar);
  const int NS = f.stages;
  auto full = [&](int s) { return bars + 8u * s; };                        // codes and scales are there
  auto empty = [&](int s) { return bars + 8u * (kFewMaxStages + s); };     // the stage's products are done
  const uint32_t tfull = bars + 16u * kFewMaxStages, tempty = tfull + 8, drain = tfull + 16;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + f.off_bar + (2 * kFewMaxStages + 3) * 8);
  volatile uint32_t* gave_up = misc + 1;
  const int warp = __shfl_sync(0xFFFFFFFFu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const bool lead = biattn_tc::elect_one();               // (as above)
  const int units = p.m_tiles * p.n_tiles;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      ptx::mbar_init(full(s), 1);
      ptx::mbar_init(empty(s), 1);
    }
    ptx::mbar_init(tfull, 1);
    ptx::mbar_init(tempty, 4);
    ptx::mbar_init(drain, 1);
    *gave_up = 0u;
    ptx::fence_barrier_init();
    ptx::fence_proxy_async_smem();
    for (const CUtensorMap* m : {&mx, &mw, &my}) ptx::prefetch_tensormap(m);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(misc), uint32_t(f.tmem_cols));
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = misc[0];
  const Sync sy{gave_up, p.status, p.timeout_ns};
  if (warp == 0 && lead) {
    // ---------------------------------------------------------------- loads
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const int n = u / p.m_tiles, row0 = (u - n * p.m_tiles) * f.cols, col0 = n * f.rows;
      const uint8_t* sx = p.sx + int64_t(row0 / 128) * p.tiles * 512;
      const uint8_t* sw = p.sw + int64_t(col0 / 128) * p.tiles * 512;
      for (int kb = 0; kb < p.kblocks; kb += kSlots) {
        if (!wait_bar(empty(s), ph ^ 1u, sy)) {
          ok = false;
          break;
        }
        if (!p.stall) {
          const int t0 = kb * C::TILES_K, slots = min(kSlots, p.kblocks - kb);
          const uint32_t bytes = uint32_t(min(kSlots * C::TILES_K, p.tiles - t0)) * 512u;
          const uint32_t sf = base + uint32_t(f.off_sf) + uint32_t(s) * (2u * C::SF_BYTES);
          ptx::mbar_arrive_expect_tx(full(s), uint32_t((p.x_rows + f.rows) * slots) * 128u + 2u * bytes);
#pragma unroll
          for (int j = 0; j < kSlots; ++j) {
            if (j < slots) {
              const int at = s * kSlots + j;
              ptx::tma_load_2d(base + uint32_t(f.off_w) + uint32_t(at * f.rows) * 128u, &mw, full(s), (kb + j) * 128, col0);
              ptx::tma_load_2d(base + uint32_t(at * f.cols) * 128u, &mx, full(s), (kb + j) * 128, row0);
            }
          }
          bulk_load(sf, sw + int64_t(t0) * 512, bytes, full(s));
          bulk_load(sf + C::SF_BYTES, sx + int64_t(t0) * 512, bytes, full(s));
        }
        if (++s == NS) s = 0, ph ^= 1u;
      }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  } else if (warp == 1 && lead) {
    // ---------------------------------------------------------------- products
    int s = 0;
    uint32_t ph = 0, tph = 0;
    bool ok = true, issued = false;
    const uint32_t id0 = idesc4<kNv>(128, 0) | (uint32_t(f.cols >> 3) << 17);
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const int col0 = u / p.m_tiles * f.rows;
      if (!wait_bar(tempty, tph ^ 1u, sy)) {
        ok = false;
        break;
      }
      tph ^= 1u;
      ptx::tc_fence_after();
      const uint32_t shift = uint32_t(col0 & 127) * 128u;
      for (int kb = 0; kb < p.kblocks; kb += kSlots) {
        if (!wait_bar(full(s), ph, sy)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t sf = base + uint32_t(f.off_sf) + uint32_t(s) * (2u * C::SF_BYTES);
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
          const int at = s * kSlots + j;
          const uint32_t a = base + uint32_t(f.off_w) + uint32_t(at * f.rows) * 128u - shift;
          const uint32_t b = base + uint32_t(at * f.cols) * 128u;
          const uint32_t ta = tmem + uint32_t(f.cols + at * C::SF_COLS), tb = ta + C::TILES_K * 4;
          const int steps = min(4, (p.K - (kb + j) * kStageK) / 64);
          if (steps > 0) {
#pragma unroll
            for (int t = 0; t < C::TILES_K; ++t) {
              ptx::tc_cp_32x128b_x4(ta + 4u * t, desc_scales(sf + uint32_t(j * C::TILES_K + t) * 512u));
              ptx::tc_cp_32x128b_x4(tb + 4u * t, desc_scales(sf + C::SF_BYTES + uint32_t(j * C::TILES_K + t) * 512u));
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k < steps) {
              const int t = kNv ? k : k >> 1;
              const uint32_t id = kNv ? 0u : uint32_t(k & 1) * 2u;
              mma4<kNv>(tmem, desc_rows(a + 32u * k), desc_rows(b + 32u * k), id0 | (id << 4) | (id << 29), ta + 4u * t,
                        tb + 4u * t, kb + j != 0 || k != 0 ? 1u : 0u);
            }
          }
        }
        issued = true;
        ptx::tc_commit(empty(s));
        if (++s == NS) s = 0, ph ^= 1u;
      }
      if (ok) ptx::tc_commit(tfull);
    }
    if (!ok && issued) {                 // what was issued ends before TMEM is released
      ptx::tc_commit(drain);
      volatile uint32_t never = 0;
      wait_bar(drain, 0u, Sync{&never, p.status, p.timeout_ns});
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- results
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int q = warp - 4;
    const uint32_t quarter = uint32_t(q * 32) << 16, stg = base + uint32_t(f.off_stg + q * C::STG_BYTES);
    uint32_t tph = 0;
    bool stored = false;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
      const int n = u / p.m_tiles, row0 = (u - n * p.m_tiles) * f.cols, col0 = n * f.rows;
      if (!__all_sync(0xFFFFFFFFu, wait_bar(tfull, tph, sy))) break;
      tph ^= 1u;
      ptx::tc_fence_after();
      // this warp's 32 rows of the MMA are columns of y where they are the CTA's
      const int col = (col0 & ~127) + q * 32;
      const bool mine = col >= col0 && col < col0 + f.rows && col < p.N;
      const int chunks = mine ? (min(f.cols, p.M - row0) + 31) / 32 : 0;
      for (int c = 0; c < chunks; ++c) {
        uint32_t r[32];
        ptx::tmem_ld_32x32b_x32(tmem + quarter + 32u * c, r);
        ptx::tmem_wait_ld();
        if (lane == 0 && stored) ptx::bulk_wait_read<0>();
        __syncwarp();
        // a lane has a column of y: 32 of its rows
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float v = __fmul_rn(__uint_as_float(r[i]), p.alpha);
          if constexpr (kF32) {
            ptx::st_shared_u32(stg + uint32_t(i * 128 + (((lane >> 2) ^ (i & 7)) << 4) + (lane & 3) * 4), __float_as_uint(v));
          } else {
            const uint16_t h = uint16_t(ptx::pack_bf16x2(v, v));
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(stg + uint32_t(i * 64 + (((lane >> 3) ^ ((i >> 1) & 3)) << 4) + (lane & 7) * 2)),
                         "h"(h)
                         : "memory");
          }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::tma_store_2d(&my, stg, col, row0 + 32 * c);
          ptx::bulk_commit();
        }
        stored = true;
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(tempty);
    }
    if (lane == 0) ptx::bulk_wait_read<0>();
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *gave_up) {    // let every copy in flight land before the block leaves
    const uint64_t t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < 2000000ull) {
    }
  }
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, uint32_t(f.tmem_cols));
  }
}

// ------------------------------------------------------------------ host

// A matrix of `rows` x `cols` elements, rows `pitch` bytes apart, in boxes of box_rows x box_cols.
bool encode(CUtensorMap* m, CUtensorMapDataType type, const void* at, uint64_t rows, uint64_t cols, uint64_t pitch,
            uint32_t box_rows, uint32_t box_cols, CUtensorMapSwizzle swizzle) {
  auto fn = biattn_tc::encode_fn();
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {pitch};
  const cuuint32_t box[2] = {box_cols, box_rows}, ones[2] = {1, 1};
  return fn && fn(m, type, 2, const_cast<void*>(at), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Kernel {
  const void* wide = nullptr;
  const void* few[2] = {nullptr, nullptr};   // two and four slots
  int wide_smem = 0, stages = 0;
};
template <bool kNv, bool kF32>
Kernel kernel() {
  using W = Wide<kNv, kF32>;
  Kernel k;
  k.wide = reinterpret_cast<const void*>(&wide_kernel<W>);
  k.few[0] = reinterpret_cast<const void*>(&few_kernel<kNv, kF32, 2>);
  k.few[1] = reinterpret_cast<const void*>(&few_kernel<kNv, kF32, 4>);
  k.wide_smem = W::SMEM;
  k.stages = W::STAGES;
  return k;
}
inline Kernel select(bool nv, bool f32) {
  if (nv) return f32 ? kernel<true, true>() : kernel<true, false>();
  return f32 ? kernel<false, true>() : kernel<false, false>();
}

constexpr int kSmemSm = 228 * 1024, kSmemBlock = 227 * 1024;

// Layout of the form for few rows with `per_sm` CTAs an SM and stages of n slots: as deep a ring as shared and tensor
// memory hold; its bytes of shared memory, 0 where fewer than `least` stages fit.
int few_layout(FewParams& f, bool nv, bool f32, int per_sm, int n, int least) {
  const int tiles = nv ? 4 : 2, sf = 2 * n * tiles * 512;
  f.slots = n;
  f.tmem_cols = 512 / per_sm;
  const int stg = 4 * 32 * 32 * (f32 ? 4 : 2), bar = (2 * kFewMaxStages + 3) * 8 + 16;
  const int room = std::min(kSmemBlock, kSmemSm / per_sm - 1024) - 1024 - stg - bar;
  // The MMA reads 128 rows around a CTA's own: up to 128 - R before the ring of w (the x ring, filled up to them) and
  // behind it.
  const int margin = (128 - f.rows) * 128;
  f.stages = std::min(kFewMaxStages, (f.tmem_cols - f.cols) / (n * tiles * 8));
  for (; f.stages >= least; --f.stages) {
    const int slots = f.stages * n;
    f.off_w = std::max(slots * f.cols * 128, margin);
    f.off_sf = f.off_w + slots * f.rows * 128;
    f.off_stg = (f.off_sf + std::max(f.stages * sf, margin) + 1023) / 1024 * 1024;
    f.off_bar = f.off_stg + stg;
    if (f.off_stg <= room) return f.off_bar + bar + 1024;
  }
  return 0;
}

}  // namespace big4

struct bi_gemm4 {
  int64_t K = 0, N = 0;
  bool nv = false, f32 = false;
  int device = 0, max_groups = 0, sms = 0;
  big4::Kernel kern;
  uint32_t* d_status = nullptr;
};

BI_GEMM_API int bi_gemm4_create(bi_gemm4_t* out, int64_t K, int64_t N, int32_t format, int32_t out_f32) {
  if (!out) return BI_GEMM_ERR_INVALID_ARG;
  *out = nullptr;
  if (K <= 0 || N <= 0 || (format != BI_MXFP4 && format != BI_NVFP4) || out_f32 < 0 || out_f32 > 1)
    return BI_GEMM_ERR_INVALID_ARG;
  if (K % 128 != 0 || K > (1 << 24) || N % 8 != 0 || N > (1 << 24)) return BI_GEMM_ERR_UNSUPPORTED;
  int dev = 0, sms = 0;
  if (const int rc = bifp4::check_device(&dev)) return rc;
  if (!biattn_tc::encode_fn()) return BI_GEMM_ERR_CUDA;
  const big4::Kernel k = big4::select(format == BI_NVFP4, out_f32 != 0);
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaFuncSetAttribute(k.wide, cudaFuncAttributeMaxDynamicSharedMemorySize, k.wide_smem) != cudaSuccess ||
      cudaFuncSetAttribute(k.few[0], cudaFuncAttributeMaxDynamicSharedMemorySize, big4::kSmemBlock) != cudaSuccess ||
      cudaFuncSetAttribute(k.few[1], cudaFuncAttributeMaxDynamicSharedMemorySize, big4::kSmemBlock) != cudaSuccess) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  bi_gemm4* h = new (std::nothrow) bi_gemm4();
  if (!h) return BI_GEMM_ERR_OOM;
  h->K = K;
  h->N = N;
  h->nv = format == BI_NVFP4;
  h->f32 = out_f32 != 0;
  h->device = dev;
  h->kern = k;
  h->sms = sms;
  // pairs that are resident at once (a pair needs two SMs of one cluster)
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(unsigned(sms / 2 * 2));
  cfg.blockDim = dim3(384);
  cfg.dynamicSmemBytes = size_t(k.wide_smem);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  if (cudaOccupancyMaxActiveClusters(&clusters, k.wide, &cfg) != cudaSuccess || clusters < 1 ||
      cudaMalloc(&h->d_status, sizeof(uint32_t)) != cudaSuccess ||
      cudaMemset(h->d_status, 0, sizeof(uint32_t)) != cudaSuccess) {
    cudaGetLastError();
    if (h->d_status) cudaFree(h->d_status);
    delete h;
    return BI_GEMM_ERR_CUDA;
  }
  h->max_groups = clusters;
  *out = h;
  return BI_GEMM_OK;
}

namespace {

// Whether a call of M rows takes the form for few rows, and its layout.  Both forms give the same bits.  Measured with
// nvfp4 (us; this form, in tiles of 128 rows of x, against pairs of 256 x 256): 256 x 4096 x 4096 (M, K, N) 7.9 against
// 9.8, 512 x 4096 x 4096 8.4 against 9.8, 777 x 2176 x 1000 5.7 against 7.2, 4096 x 1024 x 256 4.5 against 5.5, and
// with more tiles than SMs 256 x 4096 x 14336 14.7 against 11.3, 2048 x 4096 x 14336 69.6 against 42.6: a call takes
// it where its tiles run all at once.  Fewer columns of y a CTA where 128 would leave half the SMs without work: 300
// x 4096 x 1024 7.4 with 128, 7.0 with the rule's; 128 x 4096 x 4096 8.4 and 7.6; 777 x 2176 x 1000 6.0 and 5.7, with
// fp32 results 7.0 and 5.8.  Two CTAs an SM for many columns and a handful of rows: 1 x 4096 x 28672 14.1 with one,
// 13.3 with two.
bool few_choice(const bi_gemm4* h, int64_t M, big4::FewParams& f, int& per_sm, int& smem) {
  f.cols = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  const int64_t m_tiles = (M + f.cols - 1) / f.cols;
  auto units = [&]() { return (h->N + f.rows - 1) / f.rows * m_tiles; };
  f.rows = 128;
  if (M > big4::kFewCols && units() > h->sms) return false;
  while (f.rows > 32 && units() < h->sms / 2) f.rows /= 2;
  // (nvfp4 with fp32 results and 32 columns: two stages of two CTAs an SM do not fit, one CTA is taken.  17 x 4096 x
  // 20480 13.5 us, pairs 17.2; x 128256 50.0 and 57.7)
  per_sm = units() > h->sms && f.cols <= 32 ? 2 : 1;
  for (smem = 0;; per_sm = 1) {
    if (h->K > 4 * big4::kStageK) smem = big4::few_layout(f, h->nv, h->f32, per_sm, 4, 3);
    if (!smem) smem = big4::few_layout(f, h->nv, h->f32, per_sm, 2, 2);
    if (smem || per_sm == 1) break;
  }
  return smem > 0;
}

// bi_gemm4_run with the failure injection of the test controls (stall: nothing is loaded) and the limit of
// the waits.
int gemm4_run(bi_gemm4* h, const void* x, const void* sx, int64_t M, const void* w, const void* sw, float alpha, void* y,
              void* stream, int32_t stall, uint64_t timeout_ns) {
  if (!h || M < 0 || !std::isfinite(alpha)) return BI_GEMM_ERR_INVALID_ARG;
  if (M == 0) return BI_GEMM_OK;
  if (!x || !sx || !w || !sw || !y) return BI_GEMM_ERR_INVALID_ARG;
  if (M >= (int64_t(1) << 31) - 256) return BI_GEMM_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(sx) | reinterpret_cast<uintptr_t>(w) |
       reinterpret_cast<uintptr_t>(sw) | reinterpret_cast<uintptr_t>(y)) & 15u)
    return BI_GEMM_ERR_ALIGNMENT;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  if (dev != h->device) return BI_GEMM_ERR_INVALID_ARG;
  using namespace big4;
  FewParams f;
  std::memset(&f, 0, sizeof(f));
  Params& p = f.p;
  p.sx = static_cast<const uint8_t*>(sx);
  p.sw = static_cast<const uint8_t*>(sw);
  p.status = h->d_status;
  p.M = int32_t(M);
  p.N = int32_t(h->N);
  p.K = int32_t(h->K);
  p.kblocks = int32_t((h->K + kStageK - 1) / kStageK);
  p.tiles = int32_t(h->K / (h->nv ? 64 : 128));
  p.group_m = 16;
  p.alpha = alpha;
  p.stall = stall;
  p.timeout_ns = timeout_ns;
  int per_sm = 0, smem = 0;
  const bool few = few_choice(h, M, f, per_sm, smem);
  const int64_t m_tiles = few ? (M + f.cols - 1) / f.cols : (M + 255) / 256;
  const int64_t n_tiles = few ? (h->N + f.rows - 1) / f.rows : (h->N + 255) / 256;
  if (m_tiles * n_tiles >= (int64_t(1) << 31)) return BI_GEMM_ERR_UNSUPPORTED;
  p.m_tiles = int32_t(m_tiles);
  p.n_tiles = int32_t(n_tiles);
  p.x_rows = int32_t(std::min<int64_t>(few ? f.cols : 128, (M + 7) / 8 * 8));
  CUtensorMap mx, mw, msx, msw, my;
  const uint64_t tiles = uint64_t(p.tiles);
  const uint32_t tiles_k = h->nv ? 4 : 2;
  if (!encode(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, x, uint64_t(M), uint64_t(h->K / 2), uint64_t(h->K / 2),
              uint32_t(p.x_rows), 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, uint64_t(h->N), uint64_t(h->K / 2), uint64_t(h->K / 2),
              few ? uint32_t(f.rows) : 128u, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      (!few && (!encode(&msx, CU_TENSOR_MAP_DATA_TYPE_FLOAT64, sx, uint64_t((M + 127) / 128), tiles * 64, tiles * 512, 1,
                        tiles_k * 64, CU_TENSOR_MAP_SWIZZLE_NONE) ||
                !encode(&msw, CU_TENSOR_MAP_DATA_TYPE_FLOAT64, sw, uint64_t((h->N + 127) / 128), tiles * 64, tiles * 512, 2,
                        tiles_k * 64, CU_TENSOR_MAP_SWIZZLE_NONE))) ||
      !encode(&my, h->f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, y, uint64_t(M),
              uint64_t(h->N), uint64_t(h->N) * (h->f32 ? 4 : 2), 32, 32,
              h->f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
    return BI_GEMM_ERR_CUDA;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(unsigned(few ? std::min<int64_t>(m_tiles * n_tiles, int64_t(per_sm) * h->sms)
                                  : 2 * std::min<int64_t>(m_tiles * n_tiles, h->max_groups)));
  cfg.blockDim = dim3(few ? kFewThreads : 384);
  cfg.dynamicSmemBytes = size_t(few ? smem : h->kern.wide_smem);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* few_args[4] = {&mx, &mw, &my, &f};
  void* wide_args[6] = {&mx, &mw, &msx, &msw, &my, &p};
  if (cudaLaunchKernelExC(&cfg, few ? h->kern.few[f.slots / 4] : h->kern.wide, few ? few_args : wide_args) != cudaSuccess) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  return BI_GEMM_OK;
}

}  // namespace

BI_GEMM_API int bi_gemm4_run(bi_gemm4_t h, const void* x, const void* sx, int64_t M, const void* w, const void* sw,
                             float alpha, void* y, void* stream) {
  return gemm4_run(h, x, sx, M, w, sw, alpha, y, stream, 0, big4::kTimeoutNs);
}

BI_GEMM_API int bi_gemm4_get_device_error(bi_gemm4_t h, void* stream) {
  if (!h) return BI_GEMM_ERR_INVALID_ARG;
  return bifp4::read_status(h->d_status, static_cast<cudaStream_t>(stream), biattn_tc::kErrTimeout);
}

BI_GEMM_API int bi_gemm4_get_config(bi_gemm4_t h, bi_gemm4_config* c) {
  if (!h || !c) return BI_GEMM_ERR_INVALID_ARG;
  std::memset(c, 0, sizeof(*c));
  c->K = int32_t(h->K);
  c->N = int32_t(h->N);
  c->format = h->nv ? BI_NVFP4 : BI_MXFP4;
  c->out_f32 = h->f32;
  c->tile_rows = c->tile_cols = 256;
  c->stages = h->kern.stages;
  c->max_groups = h->max_groups;
  c->few_rows = big4::kFewCols;
  c->smem_bytes = h->kern.wide_smem;
  return BI_GEMM_OK;
}

BI_GEMM_API int bi_gemm4_destroy(bi_gemm4_t h) {
  if (!h) return BI_GEMM_OK;
  if (h->d_status) cudaFree(h->d_status);
  delete h;
  return BI_GEMM_OK;
}
