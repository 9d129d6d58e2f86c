// bi_prompt.cu — batch-invariant causal attention of packed prompts over a paged KV cache, sm_103a.
// Implements include/bi_prompt.h.
//
// Mathematics: per query row, over blocks of 128 keys in ascending order, with s the scores times
// scale log2(e) and m a running reference of their maximum:
//     P = 2^(s - m),   l += sum P,   O += bf16(P) V;     when m rises, l and O shrink by 2^(m_old - m)
// and o = O / l.  One pass over keys and values; scores and weights never leave the SM.  m rises only
// when a block's maximum passes it by more than 8 (a weight is then at most 2^8, and the product's
// relative rounding is the same), so O is rescaled rarely.  The rule looks at the row alone.  P is rounded
// to bf16 for the product because the tensor cores take operands of 16 bits beside bf16 values: a second
// part, as the decode keeps, would be half as many MMAs again in a kernel that they bound.  l sums P as it is, so
// the error against 64 bits is 1.2 to 1.44 times that of weights of 32 bits.
//
// Bound: the tensor cores, 4 D operations per query row and key, beside 16-bit operands that stay on
// chip.  Measured at 32/8 heads of 128: a prompt of 16384 tokens 1366 to 1406 us (1.56 to 1.61
// PFLOP/s, 0.82 to 0.84 of the measured dense peak), 24 prompts of 1 to 2000 tokens 271 to 273 us (1.16
// PFLOP/s); 8192 tokens 344 us, 782 in pages of 12, whose rows are copied one by one; 8192 tokens of 32/8
// heads of 64, with twice the exponentials per operation, 304 us (0.91 PFLOP/s).
// Tile: 128 rows = 128 / G positions x the G query heads of a KV head, so a block of keys is loaded once
// for all its heads and a short chunk still fills rows.  A unit is two tiles (256 / G positions) that
// share every key and value block and take turns: while one tile's softmax runs, the tensor cores work
// for the other.  Tiles and blocks are cut at multiples of their size in the request's own positions, so
// a row's arithmetic never depends on the chunk it came in.
//
// Warps (384 threads, one block per SM; a unit each, or, where there are more, persistent blocks that take
// planned units, longest first, from a counter):
//   0       takes units, loads the tiles' queries (TMA box: 64 dims x G heads x positions) and the
//           key blocks, page by page, into the ring (K0, V0, K1, V1, ...)
//   1       issues the MMAs:  S = Q K^T (both operands in shared memory), O += P V (P in TMEM)
//   2       loads the value blocks (two warps, since a box takes about 48 clocks to issue)
//   3       cleans the value blocks on the diagonal: rows a query must not see meet weights of zero,
//           and zero times a value that is not finite is not zero.  Those values become zeros; for
//           the rows that do see them, the epilogue adds them back (bad_v).  With one query head per
//           KV head the unit's two tiles end in different blocks; both tiles' rows then have the first
//           of them cleaned.  It is the block of the unit's first position, whichever tiles the chunk
//           fills: an infinite value added back is infinite, and one that meets a weight of zero is not
//   4 - 11  softmax, a warpgroup per tile, a thread per row: S from TMEM, P to TMEM over S's columns
// TMEM (512 columns): S0 / P0, S1 / P1 (128 each), O0, O1 (D each).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>

#include "../../include/bi_prompt.h"
#include "attn_ptx.cuh"

#ifndef BI_GEMM_API
#define BI_GEMM_API extern "C" __attribute__((visibility("default")))
#endif

namespace biprompt {

using namespace biattn_tc;

constexpr int kThreads = 384;
constexpr int kUnitRows = 256;            // query rows of a unit: two tiles of 128
constexpr int kBins = 2048;               // plan: units are sorted by key blocks, up to this many
constexpr int kUnitSlots = 2;             // units handed from the producer to the other warps
constexpr int kUnitReaders = 11;          // warps 1 .. 11
constexpr float kSlack = 8.0f;            // how far (log2) a maximum may pass its reference

struct Params {
  const int32_t* q_start;
  const int32_t* q_pos0;
  uint16_t* o;
  int2* rec;                // [tiles] (sequence, tile of its request), longest first
  uint32_t* counter;        // [2]: tiles planned, units taken; NULL: no plan, a block per unit
  uint32_t* status;
  Cache c;
  int64_t T, B;
  int32_t max_pos, Hq;
  int32_t stall;            // failure injection (test controls only): nothing is loaded for this sequence
  uint64_t timeout_ns;
  float scale_log2;
};

// A unit as the roles see it.
struct Unit {
  int32_t row0;        // token row of the unit's position `base` (negative where the chunk starts later)
  int32_t base;        // first position
  int32_t first, last; // positions of the chunk
  int32_t b, kh;
  int32_t nb[2];       // key blocks of each tile (0: none of its rows belong to the chunk)
};

// The block from which a unit's values are cleaned, a function of its place in the request alone.
__device__ __forceinline__ int32_t first_dirty(int32_t base) { return base / kBlockPos; }

template <int D_, int G_>
struct Cfg {
  static constexpr int D = D_, G = G_;
  static constexpr int P = 128 / G;                       // positions per tile
  static constexpr int UP = kUnitRows / G;                // positions per unit
  static constexpr int HALVES = D / 64;
  static constexpr int TILE_BYTES = 128 * D * 2;
  static constexpr int STAGE_BYTES = kBlockPos * D * 2;
  // (five stages and no room for the outputs were 0 to 5 % faster between units, but stores of rows
  // by their threads, 32 lines an instruction, held each unit up for 6000 clocks)
  static constexpr int STAGES = D == 128 ? 4 : 8;
  static constexpr int OFF_RING = 2 * TILE_BYTES;
  static constexpr int OFF_OUT = OFF_RING + STAGES * STAGE_BYTES;   // per tile, 64 of the output's dimensions
  static constexpr int OFF_BAR = OFF_OUT + 2 * 128 * 128;
  // ring full, empty, cleaned; unit full, empty; Q full, empty; S full, P full, O done (per tile); drain
  static constexpr int NUM_BARS = 3 * STAGES + 2 * kUnitSlots + 2 + 6 + 1;
  static constexpr int OFF_UNIT = OFF_BAR + 8 * NUM_BARS;
  static constexpr int OFF_MISC = OFF_UNIT + kUnitSlots * int(sizeof(Unit));
  static constexpr int SMEM = OFF_MISC + 32 + 1024;
  static_assert(SMEM <= 232448, "shared memory");
  static constexpr uint32_t IDESC_QK = idesc_bf16(128, kBlockPos, false, false);
  static constexpr uint32_t IDESC_PV = idesc_bf16(128, D, false, true);
};

// ------------------------------------------------------------------ plan

// Tiles of sequence b: its first tile and how many (0 where its inputs cannot be served).
__device__ __forceinline__ int32_t tiles_of(const Params& p, int64_t b, int32_t up, int32_t* first) {
  const int32_t s = p.q_start[b], e = p.q_start[b + 1], pos0 = p.q_pos0[b];
  const int64_t n = int64_t(e) - s, last = int64_t(pos0) + n - 1;
  *first = 0;
  if (s < 0 || n < 0 || e > p.T || pos0 < 0 || last / p.c.page_size >= p.c.max_pages) {
    if (n != 0 || s < 0 || e > p.T) atomicOr(p.status, kErrInput);
    return 0;
  }
  if (n == 0) return 0;
  if (last > p.max_pos) {
    atomicOr(p.status, kErrBound);
    return 0;
  }
  *first = pos0 / up;
  return int32_t(last / up) - *first + 1;
}

// One block: every tile's record, the sequences sorted by their last position's block (descending), a
// sequence's tiles one after the other from its last: side by side run units of the same keys, and the
// shortest come last.  (The order among sequences of one length is not fixed and decides no bit.)
__global__ void __launch_bounds__(1024) plan_kernel(const Params p, int32_t up) {
  __shared__ int32_t warp_sums[32];
  __shared__ int32_t bins[kBins];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kBins; i += 1024) bins[i] = 0;
  __syncthreads();
  bool descends = false;
  auto bin_of = [&](int32_t tile) { return kBins - 1 - min(kBins - 1, int32_t(int64_t(tile) * up / kBlockPos)); };
  for (int64_t b = tid; b < p.B; b += 1024) {
    int32_t first;
    const int32_t n = tiles_of(p, b, up, &first);
    if (n > 0) atomicAdd(&bins[bin_of(first + n - 1)], n);
    descends |= p.q_start[b + 1] < p.q_start[b];         // (reported by tiles_of)
  }
  // Sequences of an ascending q_start are disjoint and have at most cap_tiles tiles; of one that descends
  // nothing is computed.
  descends = __syncthreads_or(descends) != 0;
  int32_t total;
  {                                           // exclusive scan of the bins, two per thread
    const int32_t a0 = bins[2 * tid], a1 = bins[2 * tid + 1];
    int32_t x = a0 + a1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
      int32_t w = warp_sums[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xFFFFFFFFu, w, o);
        if (lane >= o) w += y;
      }
      warp_sums[lane] = w;
    }
    __syncthreads();
    const int32_t ex = x - a0 - a1 + (warp > 0 ? warp_sums[warp - 1] : 0);
    bins[2 * tid] = ex;
    bins[2 * tid + 1] = ex + a0;
    total = warp_sums[31];
    __syncthreads();
  }
  for (int64_t b = warp; b < p.B && !descends; b += 32) {
    int32_t first, at = 0;
    const int32_t n = tiles_of(p, b, up, &first);
    if (n == 0) continue;
    if (lane == 0) at = atomicAdd(&bins[bin_of(first + n - 1)], n);
    at = __shfl_sync(0xFFFFFFFFu, at, 0);
    for (int32_t k = lane; k < n; k += 32) p.rec[at + k] = make_int2(int32_t(b), first + n - 1 - k);
  }
  if (tid == 0) {
    p.counter[0] = descends ? 0u : uint32_t(total);
    p.counter[1] = 0u;
  }
}

// The record of tile `rank` without a plan (the whole warp): sequences in their order, a sequence's tiles
// from its last; sequence -1 past the last tile, or where q_start descends.
__device__ __forceinline__ int2 find_tile(const Params& p, int32_t up, int32_t rank, int lane) {
  int2 r = make_int2(-1, 0);
  int32_t before = 0;
  bool descends = false;
  for (int64_t b0 = 0; b0 < p.B; b0 += 32) {
    const int64_t b = b0 + lane;
    int32_t n = 0, first = 0;
    if (b < p.B) {
      n = tiles_of(p, b, up, &first);
      descends |= p.q_start[b + 1] < p.q_start[b];
    }
    int32_t x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    const int32_t at = rank - (before + x - n);          // among the tiles of the lane's sequence
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, at >= 0 && at < n);
    if (hit) {
      const int src = __ffs(int(hit)) - 1;
      r.x = int32_t(b0) + src;
      r.y = __shfl_sync(0xFFFFFFFFu, first + n - 1 - at, src);
    }
    before += __shfl_sync(0xFFFFFFFFu, x, 31);
  }
  return __any_sync(0xFFFFFFFFu, descends) ? make_int2(-1, 0) : r;
}

// ------------------------------------------------------------------ attention

template <class C, bool kTma>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmo, const Params p) {
  constexpr int D = C::D, G = C::G, NS = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto full = [&](uint32_t s) { return bar0 + 8 * s; };
  auto empty = [&](uint32_t s) { return bar0 + 8 * (NS + s); };
  auto clean = [&](uint32_t s) { return bar0 + 8 * (2 * NS + s); };
  const uint32_t ubar = bar0 + 8 * (3 * NS);
  auto unit_full = [&](uint32_t s) { return ubar + 8 * s; };
  auto unit_empty = [&](uint32_t s) { return ubar + 8 * (kUnitSlots + s); };
  const uint32_t q_full = ubar + 8 * (2 * kUnitSlots), q_empty = q_full + 8;
  auto s_full = [&](int i) { return q_empty + 8 + 8 * i; };
  auto p_full = [&](int i) { return q_empty + 24 + 8 * i; };
  auto o_done = [&](int i) { return q_empty + 40 + 8 * i; };
  const uint32_t drain = q_empty + 56;
  Unit* units = reinterpret_cast<Unit*>(smem + C::OFF_UNIT);
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  uint32_t* tmem_slot = misc;
  volatile uint32_t* abort = misc + 1;
  // [4]: the number (from 1) of the unit, one in four, that last met values on the diagonal that are
  // not finite; no slot is written again before every warp has left that unit
  volatile uint32_t* bad_v = misc + 2;
  const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      ptx::mbar_init(full(s), 1);
      ptx::mbar_init(empty(s), 2);             // the MMAs' commit and the cleaning warp
      ptx::mbar_init(clean(s), 1);
    }
    for (int s = 0; s < kUnitSlots; ++s) {
      ptx::mbar_init(unit_full(s), 1);
      ptx::mbar_init(unit_empty(s), kUnitReaders);
    }
    ptx::mbar_init(q_full, 1);
    ptx::mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(s_full(i), 1);
      ptx::mbar_init(p_full(i), 4);
      ptx::mbar_init(o_done(i), 1);
    }
    ptx::mbar_init(drain, 1);
    for (int i = 1; i < 6; ++i) misc[i] = 0u;
    ptx::fence_barrier_init();
    ptx::prefetch_tensormap(&tmq);
    ptx::prefetch_tensormap(&tmo);
    if (kTma) {
      ptx::prefetch_tensormap(&tmk);
      ptx::prefetch_tensormap(&tmv);
    }
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ptx::grid_dependency_wait();   // the plan (and what ran before it) is complete and visible
  ptx::launch_dependents();
  const Sync sy{abort, p.status, p.timeout_ns};

  // The next unit, handed over by the producer; false at the end (or after a wait gave up).
  uint32_t un = 0;               // units seen
  auto next_unit = [&](Unit& u) {
    const uint32_t s = un % kUnitSlots, ph = (un / kUnitSlots) & 1u;
    bool ok = true;
    if (lane == 0) ok = wait_bar(unit_full(s), ph, sy);
    ok = __shfl_sync(0xFFFFFFFFu, ok ? 1 : 0, 0) != 0;
    if (!ok) return false;
    (void)ptx::mbar_try_wait(unit_full(s), ph);   // (complete: every lane observes it)
    u = units[s];
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(unit_empty(s));
    ++un;
    return u.b >= 0;
  };

  if (warp < 4) {
    ptx::setmaxnreg_dec<80>();
    bool bad = false;                        // (loading warps) a page outside the cache
    uint32_t late = 0, late_at = 0;          // (row copies) a load not yet announced, its ring number
    auto announce = [&]() {
      if (late) {
        ptx::cp_async_wait<0>();
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(full(late_at % NS));
        late = 0;
      }
    };
    // Block j of a unit's keys or values as load number `n` of the ring; false once a wait gave up.
    auto load = [&](bool values, const Unit& u, const int32_t* trow, int32_t j, uint32_t n) {
      const uint32_t s = n % NS, dst = sbase + uint32_t(C::OFF_RING) + s * uint32_t(C::STAGE_BYTES);
      int32_t box = 0;
      int64_t off[4];
      if constexpr (kTma) box = block_box(p.c, trow, j * kBlockPos, u.last, lane, &bad);
      else block_rows(p.c, trow, j * kBlockPos, u.last, D, lane, off, &bad);
      if (n >= uint32_t(NS)) {
        if constexpr (!kTma) {                 // nothing of ours may hold the wait up
          if (!__all_sync(0xFFFFFFFFu, ptx::mbar_try_wait(empty(s), (n / NS - 1) & 1u))) announce();
        }
        const bool ok = __all_sync(0xFFFFFFFFu, wait_bar(empty(s), (n / NS - 1) & 1u, sy));
        if (!ok) return false;
      }
      if (u.b == p.stall) return true;
      if constexpr (kTma) {
        load_block_tma<D>(dst, full(s), values ? &tmv : &tmk, p.c, box, u.kh, lane);
      } else {
        load_block_rows<D>(dst, values ? p.c.vc : p.c.kc, off, u.kh, lane);
        ptx::cp_async_commit();
        if (late) {                            // (the load before this one has had a block's time)
          ptx::cp_async_wait<1>();
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(full(late_at % NS));
        }
        late = 1, late_at = n;
      }
      return true;
    };
    if (warp == 0) {
      // ------------------------------------------------------------ units, queries, keys
      const bool planned = p.counter != nullptr;
      const int2 only = planned ? make_int2(-1, 0) : find_tile(p, C::UP, int32_t(blockIdx.x) / p.c.Hkv, lane);
      const int32_t total = planned ? int32_t(p.counter[0]) : only.x >= 0 ? int32_t(gridDim.x) : 0;
      bool ok = true;
      uint32_t seq = 0, nun = 0;               // ring loads and units so far
      uint32_t id = blockIdx.x;
      if (planned && lane == 0) id = atomicAdd(p.counter + 1, 1u);
      while (ok) {
        id = __shfl_sync(0xFFFFFFFFu, id, 0);
        Unit u;
        u.b = -1;
        u.row0 = u.base = u.first = u.last = u.kh = u.nb[0] = u.nb[1] = 0;
        const int64_t rank = int64_t(id) / p.c.Hkv;
        if (rank < total) {
          const int2 r = planned ? p.rec[rank] : only;
          u.b = r.x;
          u.kh = int32_t(int64_t(id) - rank * p.c.Hkv);
          const int32_t s = p.q_start[r.x];
          u.first = p.q_pos0[r.x];
          u.last = u.first + (p.q_start[r.x + 1] - s) - 1;
          u.base = r.y * C::UP;
          u.row0 = s + (u.base - u.first);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int32_t t0 = u.base + i * C::P, t1 = t0 + C::P - 1;
            u.nb[i] = t1 >= u.first && t0 <= u.last ? t0 / kBlockPos + 1 : 0;
          }
          if (lane == 0) id = planned ? atomicAdd(p.counter + 1, 1u) : 0xFFFFFFFFu;   // the next one, ahead of its use
        }
        const uint32_t us = nun % kUnitSlots;
        if (nun >= kUnitSlots) {
          ok = __all_sync(0xFFFFFFFFu, wait_bar(unit_empty(us), (nun / kUnitSlots - 1) & 1u, sy));
          if (!ok) break;
        }
        if (lane == 0) {
          units[us] = u;
          ptx::mbar_arrive(unit_full(us));
        }
        if (u.b < 0) break;
        const int32_t nb = max(u.nb[0], u.nb[1]);
        const int32_t* trow = p.c.table + int64_t(u.b) * p.c.max_pages;
        for (int32_t j = 0; j < nb && ok; ++j, seq += 2) {
          ok = load(false, u, trow, j, seq);
          if (ok && j == 0) {                                     // the queries behind the first key block
            if (nun > 0) ok = __all_sync(0xFFFFFFFFu, wait_bar(q_empty, (nun - 1) & 1u, sy));
            if (!ok) break;
            if (lane == 0 && u.b != p.stall) {
              ptx::mbar_arrive_expect_tx(q_full, uint32_t((u.nb[0] > 0) + (u.nb[1] > 0)) * C::TILE_BYTES);
              for (int t = 0; t < 2; ++t)
                if (u.nb[t] > 0)
                  for (int hh = 0; hh < C::HALVES; ++hh)
                    tma_load_3d(sbase + uint32_t(t * C::TILE_BYTES + hh * 128 * 128), &tmq, q_full, hh * 64,
                                u.kh * G, u.row0 + t * C::P);
            }
          }
        }
        announce();
        ++nun;
      }
      if (bad) atomicOr(p.status, kErrPage);
    } else if (warp == 2) {
      // ------------------------------------------------------------ values
      Unit u;
      uint32_t seq = 1;
      bool ok = true;
      while (ok && next_unit(u)) {
        const int32_t nb = max(u.nb[0], u.nb[1]);
        const int32_t* trow = p.c.table + int64_t(u.b) * p.c.max_pages;
        for (int32_t j = 0; j < nb && ok; ++j, seq += 2) ok = load(true, u, trow, j, seq);
        announce();
      }
      if (bad) atomicOr(p.status, kErrPage);
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      // The tensor pipe holds about four MMAs (256 clocks) beside the one that runs, so whatever lies
      // between two batches of eight has to be shorter than that: one lane does it all, ring stages and
      // phases are counted, descriptors are added up from constants, and every wait stands where the
      // pipe has work left (the next block's values are awaited before tile 1's scores are issued, so
      // that only tile 0's weights are awaited at the turn of the loop).
      const bool lead = elect_one();
      bool issued = false;
      if (lead) {
        const uint64_t qd[2] = {sdesc_sw128(sbase, 16, 1024), sdesc_sw128(sbase + C::TILE_BYTES, 16, 1024)};
        const uint64_t kd0 = BlockLayout<D>::by_row(sbase + C::OFF_RING, 0);
        const uint64_t vd0 = BlockLayout<D>::by_dim(sbase + C::OFF_RING, 0);
        constexpr uint64_t kStep = C::STAGE_BYTES >> 4;
        uint32_t st = 0, ph = 0;              // stage and phase of the next load to consume
        uint32_t nu = 0, cleaned = 0, np[2] = {0, 0};
        auto advance = [&]() {
          if (++st == uint32_t(NS)) st = 0, ph ^= 1u;
        };
        auto qk = [&](int i, uint32_t s) {
          const uint64_t kd = kd0 + s * kStep;
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            ptx::mma_bf16(tmem + uint32_t(i * 128), qd[i] + uint64_t(((k >> 2) * 128 * 128 + (k & 3) * 32) >> 4),
                          kd + uint64_t(((k >> 2) * BlockLayout<D>::HALF + (k & 3) * 32) >> 4), C::IDESC_QK, k ? 1u : 0u);
          ptx::tc_commit(s_full(i));
        };
        auto pv = [&](int i, uint32_t s, bool first) {
          const uint64_t vd = vd0 + s * kStep;
#pragma unroll
          for (int k = 0; k < kBlockPos / 16; ++k)
            mma_bf16_ta(tmem + uint32_t(256 + i * D), tmem + uint32_t(i * 128 + k * 8),
                        vd + uint64_t((k * 2 * BlockLayout<D>::GROUP) >> 4), C::IDESC_PV, (first && k == 0) ? 0u : 1u);
        };
        auto values_clean = [&](uint32_t s) {
          if (!wait_bar(clean(s), (cleaned >> s) & 1u, sy)) return false;
          cleaned ^= 1u << s;
          return true;
        };
        // One unit; false once a wait gave up.
        auto unit = [&](const int32_t nb0, const int32_t nb1, const int32_t dirty) {
          const int32_t nb = max(nb0, nb1);
          if (!wait_bar(q_full, nu & 1u, sy) || !wait_bar(full(st), ph, sy)) return false;
          ptx::tc_fence_after();
          issued = true;
          if (nb0 > 0) qk(0, st);
          if (nb1 > 0) qk(1, st);
          ptx::tc_commit(empty(st));
          if (nb == 1) ptx::tc_commit(q_empty);
          advance();
          if (kTma && !wait_bar(full(st), ph, sy)) return false;
          for (int32_t j = 0; j < nb; ++j) {
            const uint32_t vs = st;                                  // this block's values
            if (!kTma && !wait_bar(full(st), ph, sy)) return false;  // (row copies come late)
            advance();
            const uint32_t ks = st, kph = ph;                        // the next block's keys
            const bool more = j + 1 < nb;
            if (more) advance();
            const uint32_t v2 = st, v2ph = ph;                       // and values
            if (j >= dirty && !values_clean(vs)) return false;
            if (j < nb0) {
              if (!wait_bar(p_full(0), np[0]++ & 1u, sy)) return false;
              ptx::tc_fence_after();
              pv(0, vs, j == 0);
              if (j + 1 == nb0) ptx::tc_commit(o_done(0));
              if (j >= nb1) ptx::tc_commit(empty(vs));
            }
            if (more) {
              if (!wait_bar(full(ks), kph, sy)) return false;
              ptx::tc_fence_after();
              if (j + 1 < nb0) qk(0, ks);
            }
            if (j < nb1) {
              if (!wait_bar(p_full(1), np[1]++ & 1u, sy)) return false;
              ptx::tc_fence_after();
              pv(1, vs, j == 0);
              if (j + 1 == nb1) ptx::tc_commit(o_done(1));
              ptx::tc_commit(empty(vs));
            }
            if (more) {
              if (kTma && !wait_bar(full(v2), v2ph, sy)) return false;
              if (j + 1 < nb1) qk(1, ks);
              ptx::tc_commit(empty(ks));
              if (j + 2 == nb) ptx::tc_commit(q_empty);
            }
          }
          ++nu;
          return true;
        };
        while (true) {
          const uint32_t us = un % kUnitSlots;
          if (!wait_bar(unit_full(us), (un / kUnitSlots) & 1u, sy)) break;
          const int32_t b = units[us].b, nb0 = units[us].nb[0], nb1 = units[us].nb[1];
          const int32_t dirty = first_dirty(units[us].base);
          ptx::mbar_arrive(unit_empty(us));
          ++un;
          if (b < 0 || !unit(nb0, nb1, dirty)) break;
        }
      }
      if (lead && issued) {          // no MMA of ours may be in flight when TMEM is released
        volatile uint32_t none = 0;
        const Sync end{&none, p.status, p.timeout_ns};
        ptx::tc_commit(drain);
        wait_bar(drain, 0u, end);
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------ cleaning of the diagonal's values
      Unit u;
      uint32_t seq = 0, nu = 0;
      bool ok = true;
      while (ok && next_unit(u)) {
        const int32_t nb = max(u.nb[0], u.nb[1]);
        const int32_t dirty = first_dirty(u.base);
        // Every load is waited for in turn and released, so that a parity is never a lap off.
        for (int32_t x = 0; x < 2 * nb && ok; ++x) {
          const uint32_t vs = seq + uint32_t(x);
          ok = __all_sync(0xFFFFFFFFu, wait_bar(full(vs % NS), (vs / NS) & 1u, sy));
          if (!ok) break;
          const int32_t j = x >> 1;
          if ((x & 1) == 0 || j < dirty) {
            if (lane == 0) ptx::mbar_arrive(empty(vs % NS));
            continue;
          }
          const uint32_t va = sbase + uint32_t(C::OFF_RING) + (vs % NS) * uint32_t(C::STAGE_BYTES);
          // magnitudes from 0x7F80 on are infinities and NaN
          uint32_t top = 0;
#pragma unroll 8
          for (int e = lane; e < C::STAGE_BYTES / 16; e += 32) {
            uint32_t w[4];
            ld_shared_v4(va + uint32_t(e) * 16, w);
#pragma unroll
            for (int k = 0; k < 4; ++k) top = __vmaxu2(top, w[k] & 0x7FFF7FFFu);
          }
          const bool hit = (top & 0xFFFFu) >= 0x7F80u || (top >> 16) >= 0x7F80u;
          if (__any_sync(0xFFFFFFFFu, hit)) {
            bool found = false;
            for (int e = lane; e < C::STAGE_BYTES / 16; e += 32) {
              uint32_t w[4];
              ld_shared_v4(va + uint32_t(e) * 16, w);
              bool here = false;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if ((w[k] & 0x7F80u) == 0x7F80u) w[k] &= 0xFFFF0000u, here = true;
                if ((w[k] & 0x7F800000u) == 0x7F800000u) w[k] &= 0xFFFFu, here = true;
              }
              if (here) {
                ptx::st_shared_v4(va + uint32_t(e) * 16, w[0], w[1], w[2], w[3]);
                // (the swizzle only moves chunks inside a row; unused slots are seen by nobody)
                found |= j * kBlockPos + e / (64 * C::HALVES) * 8 + (e / 8) % 8 <= u.last;
              }
            }
            if (__any_sync(0xFFFFFFFFu, found) && lane == 0) bad_v[nu & 3u] = nu + 1;
            ptx::fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) {
            ptx::mbar_arrive(clean(vs % NS));
            ptx::mbar_arrive(empty(vs % NS));
          }
        }
        seq += 2 * uint32_t(nb);
        ++nu;
      }
    }
  } else {
    // -------------------------------------------------------------- softmax: a thread per query row
    ptx::setmaxnreg_inc<208>();
    const int i = (warp - 4) >> 2;                 // tile
    const int r = tid - 128 - i * 128;             // row of the tile = TMEM lane
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_base + uint32_t(i * 128), to = tmem + lane_base + uint32_t(256 + i * D);
    const uint32_t out_row = sbase + uint32_t(C::OFF_OUT + i * 128 * 128 + r * 128);
    // (aligned, as the tensor memory instructions are: the warp's lanes have to arrive together, and come
    // from branches and loops of their own length)
    auto tile_sync = [&]() {
      __syncwarp();
      asm volatile("bar.sync %0, 128;" ::"r"(1 + i) : "memory");
    };
    uint32_t ns = 0, nt = 0;                       // blocks and units of this tile
    Unit u;
    bool ok = true;
    // The tile's four warps meet at named barriers, so they start and finish units together or not at all.
    while (true) {
      ok = next_unit(u);
      if (bar_or(1 + i, !ok)) break;
      const int32_t nb = i ? u.nb[1] : u.nb[0];
      if (nb == 0) continue;
      const int32_t pos = u.base + i * C::P + r / G;
      float m = -INFINITY, l = 0.0f;
      for (int32_t j = 0; j < nb; ++j) {
        ok = wait_bar(s_full(i), ns & 1u, sy);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        ++ns;
        ptx::tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) ptx::tmem_ld_32x32b_x32(ts + uint32_t(c * 32), s[c]);
        ptx::tmem_wait_ld();
        if (j + 1 == nb) {                         // the diagonal: keys behind the row's position
          const int32_t lim = pos - j * kBlockPos;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c * 32 + e > lim) s[c][e] = 0xFF800000u;
        }
        // eight chains of three-input maxima
        float mx[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mx[k] = __uint_as_float(s[k >> 1][(k & 1) * 16]);
#pragma unroll
        for (int e = 1; e < 15; e += 2)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mx[k] = max3(mx[k], __uint_as_float(s[k >> 1][(k & 1) * 16 + e]),
                         __uint_as_float(s[k >> 1][(k & 1) * 16 + e + 1]));
#pragma unroll
        for (int k = 0; k < 8; ++k) mx[k] = fmaxf(mx[k], __uint_as_float(s[k >> 1][(k & 1) * 16 + 15]));
        const float mb = __fmul_rn(max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])),
                                   p.scale_log2);
        float f = 1.0f;
        if (mb > m + kSlack || m == -INFINITY) {
          f = m == -INFINITY ? 1.0f : ex2(__fsub_rn(m, mb));      // (nothing to shrink yet)
          m = mb;
          l = __fmul_rn(l, f);
        }
        // P V of the block before is complete: this block's S was issued behind it
        if (__any_sync(0xFFFFFFFFu, f != 1.0f)) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            ptx::tmem_ld_32x32b_x32(to + uint32_t(c), o);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__fmul_rn(__uint_as_float(o[e]), f));
            tmem_st_x32(to + uint32_t(c), o);
          }
        }
        const float ref = m == -INFINITY ? 0.0f : m;   // a row of -infinity so far: weights of zero
        const uint64_t sc2 = pair(p.scale_log2, p.scale_log2), ref2 = pair(-ref, -ref);
        uint64_t ls[4] = {0, 0, 0, 0};             // four pairs of partial sums
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint64_t x = fma2(pair(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])), sc2, ref2);
            float w0, w1;
            unpair(x, w0, w1);
            w0 = ex2(w0);
            w1 = ex2(w1);
            ls[(e >> 1) & 3] = add2(ls[(e >> 1) & 3], pair(w0, w1));
            pk[e >> 1] = ptx::pack_bf16x2(w0, w1);
          }
          tmem_st_x16(ts + uint32_t(c * 16), pk);
        }
        float l0, l1;
        unpair(add2(add2(ls[0], ls[1]), add2(ls[2], ls[3])), l0, l1);
        l = __fadd_rn(l, __fadd_rn(l0, l1));
        tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(p_full(i));
      }
      if (ok) ok = wait_bar(o_done(i), nt & 1u, sy);
      if (bar_or(1 + i, !ok)) break;
      __syncwarp();                                // (the wait lets lanes go one by one)
      ++nt;
      ptx::tc_fence_after();
      const bool store = pos >= u.first && pos <= u.last;
      const bool dirty = bad_v[(un - 1) & 3u] == un;      // (written before the values' MMA)
      uint16_t* orow = p.o + ((int64_t(u.row0) + i * C::P + r / G) * p.Hq + u.kh * G + r % G) * D;
      const float rl = __fdiv_rn(1.0f, l);
      // A whole tile leaves through shared memory as two TMA boxes (64 dims x G heads x positions); the
      // tile at an end of the chunk row by row.
      const int32_t t0 = u.base + i * C::P;
      const bool whole = t0 >= u.first && t0 + C::P - 1 <= u.last;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        ptx::tmem_ld_32x32b_x32(to + uint32_t(c), o);
        ptx::tmem_wait_ld();
        if (dirty && store) {
          // values of the cleaned blocks that are not finite: each counts as itself, as under a positive
          // weight (also where the weight has underflowed to zero)
          for (int32_t k = first_dirty(u.base) * kBlockPos; k <= pos; ++k) {
            const int64_t page = p.c.table[int64_t(u.b) * p.c.max_pages + k / p.c.page_size];
            if (page < 0 || page >= p.c.num_pages) continue;
            const uint16_t* v = p.c.vc + ((page * p.c.page_size + k % p.c.page_size) * p.c.Hkv + u.kh) * D + c;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if ((v[e] & 0x7F80u) == 0x7F80u)
                o[e] = __float_as_uint(__fadd_rn(__uint_as_float(o[e]), __uint_as_float(uint32_t(v[e]) << 16)));
          }
        }
        __syncwarp();                           // (a row's loop ends at its own position)
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 16; ++k)
          w[k] = ptx::pack_bf16x2(__fmul_rn(__uint_as_float(o[2 * k]), rl), __fmul_rn(__uint_as_float(o[2 * k + 1]), rl));
        if (whole) {
          if ((c & 32) == 0) {                  // the box before this one has been read
            if (r == 0) ptx::bulk_wait_read<0>();
            tile_sync();
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            ptx::st_shared_v4(out_row + uint32_t((((c & 32) / 8 + k) ^ (r & 7)) << 4), w[4 * k], w[4 * k + 1],
                              w[4 * k + 2], w[4 * k + 3]);
          if ((c & 32) != 0) {
            ptx::fence_proxy_async_smem();
            tile_sync();
            if (r == 0) {
              tma_store_3d(&tmo, sbase + uint32_t(C::OFF_OUT + i * 128 * 128), c - 32, u.kh * G, u.row0 + i * C::P);
              ptx::bulk_commit();
            }
          }
        } else if (store) {
#pragma unroll
          for (int k = 0; k < 4; ++k) ptx::st_global_v4(orow + c + 8 * k, w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        }
        __syncwarp();
      }
      ptx::tc_fence_before();
    }
    if (r == 0) bulk_wait_all();                   // the outputs are written
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (*abort) {                      // a wait gave up: let every copy in flight land before the block leaves
    const uint64_t t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < 2000000ull) {
    }
    __syncwarp();
  }
  if (warp == 1) ptx::tmem_dealloc(tmem, 512);
}

struct KernelInfo {
  const void* tma = nullptr;
  const void* rows = nullptr;
  int smem = 0, stages = 0, up = 0;
};

template <int D, int G>
KernelInfo info() {
  using C = Cfg<D, G>;
  KernelInfo k;
  k.tma = reinterpret_cast<const void*>(&prompt_kernel<C, true>);
  k.rows = reinterpret_cast<const void*>(&prompt_kernel<C, false>);
  k.smem = C::SMEM;
  k.stages = C::STAGES;
  k.up = C::UP;
  return k;
}

inline KernelInfo select(int D, int G) {
  if (D == 128) {
    switch (G) {
      case 1: return info<128, 1>();
      case 2: return info<128, 2>();
      case 4: return info<128, 4>();
      case 8: return info<128, 8>();
    }
  } else if (D == 64) {
    switch (G) {
      case 1: return info<64, 1>();
      case 2: return info<64, 2>();
      case 4: return info<64, 4>();
      case 8: return info<64, 8>();
    }
  }
  return KernelInfo{};
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace biprompt

struct bi_prompt {
  int Hq = 0, Hkv = 0, D = 0, G = 0, page_size = 0;
  float scale = 0.0f;
  int device = 0, num_sms = 0;
  biprompt::KernelInfo kern;
  uint32_t* d_status = nullptr;
  biattn_tc::Workspace ws;
};

namespace {

struct PromptWs {
  size_t counter, rec, total;
  int64_t cap_tiles;
  bool planned;
};

PromptWs prompt_layout(const bi_prompt* h, int64_t T, int64_t B) {
  PromptWs w;
  w.cap_tiles = T / h->kern.up + 2 * B;     // a sequence of n tokens touches at most n / up + 2 units
  // Where every unit has a block of its own at once, each block finds its unit itself, and the plan's
  // launch and workspace are spared (37 tokens, 32/8 heads of 128: 9.3 us, 11.6 with a plan; 3 chunks of
  // 200 to 700 behind 28000, 16/2 heads of 64: 243 against 247).  With more units than blocks the plan's
  // order pays: the longest units start first and blocks take the next as they end.
  w.planned = w.cap_tiles * h->Hkv > h->num_sms;
  w.counter = 0;
  w.rec = 256;
  w.total = w.planned ? w.rec + biprompt::align256(size_t(w.cap_tiles) * sizeof(int2)) : 0;
  return w;
}

}  // namespace

BI_GEMM_API int bi_prompt_create(bi_prompt_t* out, int64_t num_q_heads, int64_t num_kv_heads, int64_t head_dim,
                                 int64_t page_size, float scale) {
  if (!out) return BI_GEMM_ERR_INVALID_ARG;
  *out = nullptr;
  if (!std::isfinite(scale) || scale <= 0.0f) return BI_GEMM_ERR_INVALID_ARG;
  if (num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || page_size <= 0) return BI_GEMM_ERR_INVALID_ARG;
  if (num_q_heads % num_kv_heads != 0 || num_q_heads > 4096 || page_size > (1 << 20) ||
      (head_dim != 64 && head_dim != 128))
    return BI_GEMM_ERR_UNSUPPORTED;
  const int64_t G = num_q_heads / num_kv_heads;
  if (G > 8) return BI_GEMM_ERR_UNSUPPORTED;
  const biprompt::KernelInfo k = biprompt::select(int(head_dim), int(G));
  if (!k.tma) return BI_GEMM_ERR_UNSUPPORTED;
  int dev = 0, major = 0, minor = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  if (major != 10 || minor != 3) return BI_GEMM_ERR_UNSUPPORTED;
  if (!biattn_tc::encode_fn() ||
      cudaFuncSetAttribute(k.tma, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem) != cudaSuccess ||
      cudaFuncSetAttribute(k.rows, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem) != cudaSuccess) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  bi_prompt* h = new (std::nothrow) bi_prompt();
  if (!h) return BI_GEMM_ERR_OOM;
  h->Hq = int(num_q_heads);
  h->Hkv = int(num_kv_heads);
  h->D = int(head_dim);
  h->G = int(G);
  h->page_size = int(page_size);
  h->scale = scale;
  h->device = dev;
  h->num_sms = sms;
  h->kern = k;
  if (cudaMalloc(&h->d_status, sizeof(uint32_t)) != cudaSuccess ||
      cudaMemset(h->d_status, 0, sizeof(uint32_t)) != cudaSuccess) {
    cudaGetLastError();
    if (h->d_status) cudaFree(h->d_status);
    delete h;
    return BI_GEMM_ERR_CUDA;
  }
  *out = h;
  return BI_GEMM_OK;
}

BI_GEMM_API int bi_prompt_workspace_size(bi_prompt_t h, int64_t T, int64_t num_seqs, uint64_t* bytes) {
  if (!h || !bytes || T < 0 || num_seqs < 0) return BI_GEMM_ERR_INVALID_ARG;
  *bytes = T == 0 || num_seqs == 0 ? 0 : uint64_t(prompt_layout(h, T, num_seqs).total);
  return BI_GEMM_OK;
}

namespace {

// bi_prompt_run with the failure injection of the test controls (stall >= 0: nothing is loaded for that sequence) and
// the limit of the waits.
int prompt_run(bi_prompt* h, const void* q, int64_t T, const int32_t* q_start, const int32_t* q_pos0, int64_t B,
               const void* k_cache, const void* v_cache, int64_t num_pages, const int32_t* page_table,
               int64_t max_pages, int64_t max_pos, void* o, void* stream, int32_t stall, uint64_t timeout_ns) {
  if (!h || T < 0 || B < 0 || num_pages < 0 || max_pages < 0 || max_pos < 0) return BI_GEMM_ERR_INVALID_ARG;
  if (T == 0 || B == 0) return BI_GEMM_OK;
  // row coordinates, unit numbers and positions are 32-bit
  if (T > (int64_t(1) << 28) || B > (int64_t(1) << 24) || max_pos >= (int64_t(1) << 30) ||
      (T / h->kern.up + 2 * B) * h->Hkv >= (int64_t(1) << 31))
    return BI_GEMM_ERR_UNSUPPORTED;
  if (!q || !q_start || !q_pos0 || !k_cache || !v_cache || !page_table || !o) return BI_GEMM_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(o) | reinterpret_cast<uintptr_t>(k_cache) |
       reinterpret_cast<uintptr_t>(v_cache)) & 15u)
    return BI_GEMM_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(q_start) | reinterpret_cast<uintptr_t>(q_pos0) |
       reinterpret_cast<uintptr_t>(page_table)) & 3u)
    return BI_GEMM_ERR_ALIGNMENT;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  if (dev != h->device) return BI_GEMM_ERR_INVALID_ARG;
  CUtensorMap tmq, tmk, tmv, tmo;
  std::memset(&tmk, 0, sizeof(tmk));
  std::memset(&tmv, 0, sizeof(tmv));
  if (!biattn_tc::encode_queries(&tmq, q, T, h->Hq, h->D, h->G, 128 / h->G) ||
      !biattn_tc::encode_queries(&tmo, o, T, h->Hq, h->D, h->G, 128 / h->G))
    return BI_GEMM_ERR_CUDA;
  // TMA boxes need whole pages and row coordinates (one page past the end included) of 32 bits;
  // otherwise rows are copied: the same bits.
  const int64_t rows = num_pages * h->page_size;
  const bool tma = biattn_tc::tma_page_size(h->page_size) && num_pages > 0 &&
                   rows + h->page_size < (int64_t(1) << 31) &&
                   biattn_tc::encode_pages(&tmk, k_cache, rows, h->Hkv, h->D, h->page_size) &&
                   biattn_tc::encode_pages(&tmv, v_cache, rows, h->Hkv, h->D, h->page_size);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const PromptWs w = prompt_layout(h, T, B);
  if (const int rc = h->ws.need(w.total, st)) return rc;
  uint8_t* ws = static_cast<uint8_t*>(h->ws.at);
  biprompt::Params p;
  std::memset(&p, 0, sizeof(p));
  p.q_start = q_start;
  p.q_pos0 = q_pos0;
  p.o = static_cast<uint16_t*>(o);
  p.counter = w.planned ? reinterpret_cast<uint32_t*>(ws + w.counter) : nullptr;
  p.rec = w.planned ? reinterpret_cast<int2*>(ws + w.rec) : nullptr;
  p.status = h->d_status;
  p.c.kc = static_cast<const uint16_t*>(k_cache);
  p.c.vc = static_cast<const uint16_t*>(v_cache);
  p.c.table = page_table;
  p.c.num_pages = num_pages;
  p.c.max_pages = max_pages;
  p.c.Hkv = h->Hkv;
  p.c.page_size = h->page_size;
  p.T = T;
  p.B = B;
  p.max_pos = int32_t(max_pos);
  p.Hq = h->Hq;
  p.stall = stall;
  p.timeout_ns = timeout_ns;
  p.scale_log2 = h->scale * 1.4426950408889634f;   // log2(e)
  int32_t up = h->kern.up;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(1024);
  void* pargs[2] = {&p, &up};
  cudaError_t e = cudaSuccess;
  if (w.planned) e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(&biprompt::plan_kernel), pargs);
  if (e == cudaSuccess) {
    void* args[5] = {&tmq, &tmk, &tmv, &tmo, &p};
    cfg.gridDim = dim3(unsigned(std::min<int64_t>(w.cap_tiles * h->Hkv, h->num_sms)));
    cfg.blockDim = dim3(biprompt::kThreads);
    cfg.dynamicSmemBytes = size_t(h->kern.smem);
    e = cudaLaunchKernelExC(&cfg, tma ? h->kern.tma : h->kern.rows, args);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  return BI_GEMM_OK;
}

}  // namespace

BI_GEMM_API int bi_prompt_run(bi_prompt_t h, const void* q, int64_t T, const int32_t* q_start, const int32_t* q_pos0,
                              int64_t num_seqs, const void* k_cache, const void* v_cache, int64_t num_pages,
                              const int32_t* page_table, int64_t max_pages, int64_t max_pos, void* o, void* stream) {
  return prompt_run(h, q, T, q_start, q_pos0, num_seqs, k_cache, v_cache, num_pages, page_table, max_pages, max_pos, o,
                    stream, -1, biattn_tc::kTimeoutNs);
}

BI_GEMM_API int bi_prompt_get_device_error(bi_prompt_t h, void* stream) {
  if (!h) return BI_GEMM_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint32_t s = 0;
  if (cudaMemcpyAsync(&s, h->d_status, sizeof(s), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  if (s == 0) return BI_GEMM_OK;
  if (cudaMemsetAsync(h->d_status, 0, sizeof(uint32_t), st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  return (s & biattn_tc::kErrTimeout) ? BI_GEMM_ERR_TIMEOUT : BI_GEMM_ERR_INVALID_ARG;
}

BI_GEMM_API int bi_prompt_get_config(bi_prompt_t h, bi_prompt_config* c) {
  if (!h || !c) return BI_GEMM_ERR_INVALID_ARG;
  c->num_q_heads = h->Hq;
  c->num_kv_heads = h->Hkv;
  c->head_dim = h->D;
  c->page_size = h->page_size;
  c->tile_positions = h->kern.up;
  c->block_positions = biattn_tc::kBlockPos;
  c->stages = h->kern.stages;
  c->threads = biprompt::kThreads;
  c->max_ctas = h->num_sms;
  c->tma_pages = biattn_tc::tma_page_size(h->page_size) ? 1 : 0;
  return BI_GEMM_OK;
}

BI_GEMM_API int bi_prompt_destroy(bi_prompt_t h) {
  if (!h) return BI_GEMM_OK;
  h->ws.release(h->device);
  if (h->d_status) cudaFree(h->d_status);
  delete h;
  return BI_GEMM_OK;
}
