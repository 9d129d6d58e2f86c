// bi_attention_shared.cuh — decode attention over groups of tokens that share a prefix (included by
// bi_attention.cu; implements bi_attention_run_shared of include/bi_attention.h), sm_103a.
//
// A split of bi_attention_run whose positions all lie in a group's prefix is the same keys and values
// for every token of the group.  One unit here computes such a split for up to 128 query columns (a
// column is a token's query head of one KV head) from one load of its keys and values; every other
// split stays a unit of attn_kernel / attn_tma_kernel, and merge_kernel joins them all as ever.
//
// The bits are those kernels': per column the same scores (S^T = K Q^T, sixteen dimensions at a time
// in ascending order), maximum, weights, sum (by position modulo 128, butterfly, warp order) and
// values (O^T += V^T P^T, sixteen positions at a time, high then low bf16 part of the weights), here
// by tcgen05.mma (128 positions or dimensions on its rows, the columns on its N) where they use
// mma.sync m16n8k16.  The two instructions accumulate a step of sixteen alike: measured, no bit of
// 6.5 million sums of 64 to 4096 products differed, over normal, wide-range, cancelling and
// denormal inputs, and the tests hold whole calls to it on such inputs.
//
// Bound: for many tokens the tensor cores (6 D operations per query row and key, a third of them for
// the weights' low part) and the softmax's instructions, for few the load of the prefix.  Measured at
// 32/8 heads of 128: 64 tokens behind 8192 positions 61 us for the whole call (bi_attention_run 308), of
// which the groups' units alone 32; 256 tokens behind 16384 350 us (2319), units alone 177.
//
// Warps (640 threads, one block per SM): 0 loads (queries, then K1 .. K(n-1), K0, V0 .. V(n-1)
// through a ring), 1 issues the MMAs, 2 and 3 check that the group's page tables agree, 4 - 19
// softmax: four warpgroups, each a quarter of the columns, a thread per position of a block.  (Two
// warpgroups with half of the columns each issued an instruction in 28 % of the clocks: their phases
// are chains of dependent steps.)
// TMEM: block b's scores at column 128 b (64 b for splits above 512); the value sums take block 0's
// columns once its weights are out, so a unit's block 0 is the last whose scores are computed, and the
// other blocks' scores of the next unit run beside the end of this one.  The weights of a block are
// computed into registers while the block before still feeds the tensor cores from the one buffer.
#pragma once

#include "attn_ptx.cuh"

namespace biattn {

namespace tc = biattn_tc;

constexpr int kSharedGroups = 4;              // softmax warpgroups
constexpr int kSharedThreads = 128 + 128 * kSharedGroups;
constexpr int kSharedStages = 3;
constexpr int kMaxBlocks = 8;                 // blocks of a split: 1024 / 128

struct SharedParams {
  Params a;                    // as bi_attention_run's (part, ml, status, shapes, ...)
  const int32_t* group_start;
  const int32_t* group_len;
  int32_t* nsh;                // [T] leading splits of each token that its group computes
  int4* srec;                  // [cap] (first token, tokens, split, token whose pages are read)
  int32_t* count;              // [1] records
  tc::Cache c;
  int64_t num_groups;
  int32_t stall;               // failure injection (test controls only): this block loads no keys
  int32_t cols;                // columns of a unit at most: 128, or 64 above splits of 512
};

constexpr int kPlanTokens = 1024;             // tokens (and groups) that the plan keeps in shared memory

// One block: per token the splits that its group computes, the units of the groups, then the
// records of all other units in the form that the attention kernels read.  Bound by latency: what the
// first 1024 tokens and groups say is loaded at once, the rest works from shared memory, and a warp
// writes one token's records at a time.  (With groups read when they were met and a token's records
// written by the warp that scanned it, a call of 64 tokens behind a prefix of 8192 took 65.8 us, then 60.9.)
__global__ void __launch_bounds__(1024) plan_shared_kernel(const SharedParams sp) {
  __shared__ int32_t warp_sums[32];
  __shared__ int32_t carry;
  __shared__ int32_t nrec;
  __shared__ int32_t gs[kPlanTokens + 1], gl[kPlanTokens];   // the first groups
  // of 1024 tokens: request, position (-1: cannot be served), shared splits, first own unit, own units
  __shared__ int32_t sb[kPlanTokens], spos[kPlanTokens], snsh[kPlanTokens], sat[kPlanTokens], sn[kPlanTokens];
  const Params& p = sp.a;
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  if (tid == 0) carry = 0, nrec = 0;
  auto served = [&](int32_t b, int32_t pos) {
    return b >= 0 && b < p.B && pos >= 0 && pos <= p.max_pos && int64_t(pos / p.page_size) < p.max_pages;
  };
  auto position = [&](int64_t t) {
    const int32_t pos = p.q_pos[t];
    return served(p.q_seq[t], pos) ? pos : -1;
  };
  const int32_t b0 = tid < p.T ? p.q_seq[tid] : -1, p0 = tid < p.T ? p.q_pos[tid] : -1;
  // Ranges that leave [0, T] or descend may overlap: then nothing is shared, and every token is served
  // by units of its own.
  bool bad = false;
  for (int64_t g = tid; g < sp.num_groups; g += 1024) {
    const int32_t s = sp.group_start[g], e = sp.group_start[g + 1], len = sp.group_len[g];
    bad |= s < 0 || e < s || e > p.T || len < 0;
    if (g < kPlanTokens) {
      gs[g] = s, gl[g] = len;
      if (g + 1 == sp.num_groups || g + 1 == kPlanTokens) gs[g + 1] = e;
    }
  }
  spos[tid] = served(b0, p0) ? p0 : -1;
  snsh[tid] = 0;
  for (int64_t t = tid; t < p.T; t += 1024) sp.nsh[t] = 0;
  bad = __syncthreads_or(bad) != 0;
  if (bad && tid == 0) atomicOr(p.status, kErrInput);
  const int32_t G = p.Hq / p.Hkv, per = sp.cols / G;     // tokens of a unit
  // a warp per group, or 32 / groups warps that share out its rows of units where there are few
  const int wpg = sp.num_groups < 32 ? 32 / int(sp.num_groups) : 1, wi = warp % wpg;
  for (int64_t g = warp / wpg; g < sp.num_groups && !bad; g += 32 / wpg) {
    const bool near = g < kPlanTokens;
    const int32_t s = near ? gs[g] : sp.group_start[g], e = near ? gs[g + 1] : sp.group_start[g + 1];
    const int32_t len = near ? gl[g] : sp.group_len[g];
    if (e - s < 2) continue;                             // (alone: its own units serve it as well)
    for (int32_t t0 = s + wi * per; t0 < e; t0 += wpg * per) {
      const int32_t n = min(per, e - t0);
      int32_t most = 0, first = 0;
      for (int32_t k = lane; k < n; k += 32) {
        const int32_t pos = t0 + k < kPlanTokens ? spos[t0 + k] : position(t0 + k);
        // (the split that holds the token itself is always its own)
        const int32_t x = pos < 0 ? 0 : min(len, pos) / p.split;
        sp.nsh[t0 + k] = x;
        if (t0 + k < kPlanTokens) snsh[t0 + k] = x;
        most = max(most, x);
        if (k == 0) first = x;
      }
      most = int32_t(__reduce_max_sync(0xFFFFFFFFu, unsigned(most)));
      first = __shfl_sync(0xFFFFFFFFu, first, 0);        // the first token's, which mostly shares all
      __syncwarp();
      int32_t at = 0;
      if (lane == 0 && most > 0) at = atomicAdd(&nrec, most);
      at = __shfl_sync(0xFFFFFFFFu, at, 0);
      for (int32_t sx = lane; sx < most; sx += 32) {
        int32_t src = t0;
        if (first <= sx)
          while (sp.nsh[src] <= sx) ++src;               // (ends: a token has `most`)
        sp.srec[at + sx] = make_int4(t0, n, sx, src);
      }
    }
  }
  __syncthreads();
  if (tid == 0) sp.count[0] = nrec;                      // (at most sp.cap: the groups are disjoint)
  for (int64_t base = 0; base < p.T; base += 1024) {
    const int64_t t = base + tid;
    int32_t n = 0;
    if (t < p.T) {
      const int32_t b = base == 0 ? b0 : p.q_seq[t], pos = base == 0 ? p0 : p.q_pos[t];
      if (b < 0 || b >= p.B || pos < 0 || int64_t(pos / p.page_size) >= p.max_pages) {
        atomicOr(p.status, kErrInput);
      } else if (pos > p.max_pos) {
        atomicOr(p.status, kErrBound);
      } else {
        const int32_t sh = base == 0 ? snsh[tid] : sp.nsh[t];
        n = (splits_of(pos, p.split) - sh) * p.Hkv;
        sb[tid] = b, spos[tid] = pos, snsh[tid] = sh;
      }
    }
    int32_t x = n;
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
    const int32_t incl = carry + x + (warp > 0 ? warp_sums[warp - 1] : 0);
    if (t < p.T) p.cum[t] = incl - n;
    sat[tid] = incl - n, sn[tid] = n;
    __syncthreads();
    if (tid == 1023) carry = incl;
    const int here = int(min(int64_t(1024), p.T - base));
    for (int k = warp; k < here; k += 32) {
      const int32_t nk = sn[k], at = sat[k], r0 = snsh[k] * p.Hkv;
      for (int32_t r = lane; r < nk; r += 32) p.urec[at + r] = make_int4(int32_t(base) + k, sb[k], spos[k], r0 + r);
    }
    __syncthreads();
  }
  if (tid == 0) p.cum[p.T] = carry;
}

__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// 32 columns over the warp's 32 lanes: lane c ends with column c combined over the lanes, in the
// order of the xor butterfly 16, 8, 4, 2, 1 (each step adds the same pairs; the operands' order does
// not matter).  31 shuffles instead of 5 per column.
template <class Op>
__device__ __forceinline__ float reduce_columns(float (&v)[32], int lane, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
    for (int k = 0; k < o; ++k) {
      const float send = (lane & o) ? v[k] : v[k + o];
      const float keep = (lane & o) ? v[k + o] : v[k];
      v[k] = op(keep, __shfl_xor_sync(0xFFFFFFFFu, send, o));
    }
  }
  return v[0];
}

template <int D, int G>
struct SharedCfg {
  static constexpr int NS = kSharedStages;
  static constexpr int STAGE_BYTES = tc::kBlockPos * D * 2;
  static constexpr int Q_BYTES = 128 * D * 2;
  static constexpr int ATOM = tc::kBlockPos * 128;            // 128 positions x 64 columns of weights
  static constexpr int OFF_RING = Q_BYTES;
  static constexpr int OFF_P = OFF_RING + NS * STAGE_BYTES;   // high parts of both halves, then low parts
  static constexpr int OFF_M = OFF_P + 4 * ATOM;              // [4][32] the warpgroups' maxima
  static constexpr int OFF_RED = OFF_M + 128 * 4;             // [4][4][32] their warps' maxima, then sums
  static constexpr int OFF_BAR = OFF_RED + 4 * 4 * 32 * 4;
  // ring full, empty; Q full, empty; scores of a block; weights full, free; O free; drain
  static constexpr int NUM_BARS = 2 * NS + 2 + kMaxBlocks + 2 + 2;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NUM_BARS;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static_assert(SMEM <= 232448, "shared memory");
};

template <int D, int G, bool kTma>
__global__ void __launch_bounds__(kSharedThreads, 1)
    shared_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tmv, const SharedParams sp) {
  using C = SharedCfg<D, G>;
  constexpr int NS = C::NS;
  const Params& p = sp.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto full = [&](uint32_t s) { return bar0 + 8 * s; };
  auto empty = [&](uint32_t s) { return bar0 + 8 * (NS + s); };
  const uint32_t q_full = bar0 + 8 * (2 * NS), q_empty = q_full + 8;
  auto s_full = [&](int b) { return q_empty + 8 + 8 * b; };
  const uint32_t p_full = q_empty + 8 + 8 * kMaxBlocks, p_free = p_full + 8, o_free = p_full + 16, drain = p_full + 24;
  float* msm = reinterpret_cast<float*>(smem + C::OFF_M);
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile uint32_t* abort = misc + 1;
  const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      ptx::mbar_init(full(s), 1);
      ptx::mbar_init(empty(s), 1);
    }
    ptx::mbar_init(q_full, 1);
    ptx::mbar_init(q_empty, 1);
    for (int b = 0; b < kMaxBlocks; ++b) ptx::mbar_init(s_full(b), 1);
    ptx::mbar_init(p_full, 4 * kSharedGroups);
    ptx::mbar_init(p_free, 1);
    ptx::mbar_init(o_free, 4 * kSharedGroups);
    ptx::mbar_init(drain, 1);
    misc[1] = 0u;
    ptx::fence_barrier_init();
    ptx::prefetch_tensormap(&tmq);
    if (kTma) {
      ptx::prefetch_tensormap(&tmk);
      ptx::prefetch_tensormap(&tmv);
    }
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(misc), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = misc[0];
  // No wait here: this grid is launched behind the own units' and may start once each of their blocks
  // has passed its wait for the plan, so the plan (and what ran before it) is complete; its results are
  // read from L2.  The two grids' units run side by side where there is room.  The wait at the end makes
  // this grid end after the other, so that the merge, which waits for this one, waits for both.
  ptx::launch_dependents();
  const tc::Sync sy{abort, p.status, p.timeout_ns};
  const int32_t units = __ldcg(sp.count) * p.Hkv;
  const int nblk = p.split / tc::kBlockPos;

  // A unit's record; its columns (a multiple of 16, the MMA's step in N) and how many a warpgroup takes.
  struct U {
    int32_t t0, n, s, src, kh, cols, share;
  };
  auto record = [&](int32_t u) { return u < units ? __ldcg(sp.srec + u / p.Hkv) : make_int4(0, 0, 0, 0); };
  auto unit = [&](const int4 r, int32_t u) {
    U x;
    x.t0 = r.x, x.n = r.y, x.s = r.z, x.src = r.w;
    x.kh = u % p.Hkv;
    x.cols = (x.n * G + 15) & ~15;
    x.share = (x.cols + 16 * kSharedGroups - 1) / (16 * kSharedGroups) * 16;
    return x;
  };

  if (warp < 4) {
    ptx::setmaxnreg_dec<56>();
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      bool ok = true, bad = false;
      uint32_t seq = 0, nu = 0, late = 0, q_issued = 0;
      auto announce = [&](uint32_t keep) {      // (row copies) loads but the last `keep` have landed
        while (late > keep) {
          if (keep == 1) ptx::cp_async_wait<1>();
          else ptx::cp_async_wait<0>();
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(full((seq - late) % NS));
          --late;
        }
      };
      int4 rec = record(int32_t(blockIdx.x));
      for (int32_t u = int32_t(blockIdx.x); u < units && ok; u += int32_t(gridDim.x), ++nu) {
        const U x = unit(rec, u);
        rec = record(u + int32_t(gridDim.x));      // the next one's, ahead of its use
        if (nu > 0) {
          if (lane == 0) ok = tc::wait_bar(q_empty, (nu - 1) & 1u, sy);
          ok = __shfl_sync(0xFFFFFFFFu, ok ? 1 : 0, 0) != 0;
          if (!ok) break;
        }
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(q_full, uint32_t(sp.cols * D * 2));
          for (int hh = 0; hh < D / 64; ++hh)
            tc::tma_load_3d(sbase + uint32_t(hh * 128 * 128), &tmq, q_full, hh * 64, x.kh * G, x.t0);
        }
        ++q_issued;
        const int32_t* trow = p.table + int64_t(__ldcg(p.q_seq + x.src)) * p.max_pages;
        const int32_t base = x.s * p.split, last = base + p.split - 1;
        for (int32_t i = 0; i < 2 * nblk; ++i, ++seq) {
          const int32_t b = i < nblk ? (i + 1 < nblk ? i + 1 : 0) : i - nblk;
          const int32_t pos0 = base + b * tc::kBlockPos;
          const uint32_t s = seq % NS, dst = sbase + uint32_t(C::OFF_RING) + s * uint32_t(C::STAGE_BYTES);
          if (int(blockIdx.x) == sp.stall) {
            ok = __all_sync(0xFFFFFFFFu, tc::wait_bar(full(0), 0u, sy));   // (never)
            break;
          }
          if constexpr (kTma) {
            const int32_t box = tc::block_box(sp.c, trow, pos0, last, lane, &bad);
            if (seq >= uint32_t(NS)) {
              if (lane == 0) ok = tc::wait_bar(empty(s), (seq / NS - 1) & 1u, sy);
              ok = __shfl_sync(0xFFFFFFFFu, ok ? 1 : 0, 0) != 0;
              if (!ok) break;
            }
            tc::load_block_tma<D>(dst, full(s), i < nblk ? &tmk : &tmv, sp.c, box, x.kh, lane);
          } else {
            int64_t off[4];
            tc::block_rows(sp.c, trow, pos0, last, D, lane, off, &bad);
            if (seq >= uint32_t(NS)) {
              announce(0);                     // nothing of ours may hold the wait up
              if (lane == 0) ok = tc::wait_bar(empty(s), (seq / NS - 1) & 1u, sy);
              ok = __shfl_sync(0xFFFFFFFFu, ok ? 1 : 0, 0) != 0;
              if (!ok) break;
            }
            tc::load_block_rows<D>(dst, i < nblk ? sp.c.kc : sp.c.vc, off, x.kh, lane);
            ptx::cp_async_commit();
            ++seq, ++late;
            announce(1);
            --seq;                             // (the loop counts it)
          }
        }
        if (!kTma) announce(0);
      }
      if (bad) atomicOr(p.status, kErrPage);
      if (!kTma) ptx::cp_async_wait<0>();
      if (lane == 0) {                         // no copy of ours may be in flight when the block leaves
        volatile uint32_t none = 0;
        const tc::Sync end{&none, p.status, p.timeout_ns};
        if (kTma)
          for (uint32_t k = 0; k < uint32_t(NS) && k < seq; ++k)
            tc::wait_bar(full((seq - 1 - k) % NS), ((seq - 1 - k) / NS) & 1u, end);
        if (q_issued > 0) tc::wait_bar(q_full, (q_issued - 1) & 1u, end);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      if (lane == 0) {
        uint32_t seq = 0, nu = 0, np = 0;
        bool ok = true, issued = false;
        int4 rec = record(int32_t(blockIdx.x));
        for (int32_t u = int32_t(blockIdx.x); u < units && ok; u += int32_t(gridDim.x), ++nu) {
          const U x = unit(rec, u);
          rec = record(u + int32_t(gridDim.x));      // the next one's, ahead of its use
          const uint32_t id_qk = tc::idesc_bf16(128, x.cols, false, false);
          ok = tc::wait_bar(q_full, nu & 1u, sy);
          for (int32_t i = 0; i < nblk && ok; ++i, ++seq) {
            const int32_t b = i + 1 < nblk ? i + 1 : 0;
            // block 0's columns hold the previous unit's value sums until they are read
            if (b == 0 && nu > 0) ok = tc::wait_bar(o_free, (nu - 1) & 1u, sy);
            ok = ok && tc::wait_bar(full(seq % NS), (seq / NS) & 1u, sy);
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t ka = sbase + uint32_t(C::OFF_RING) + (seq % NS) * uint32_t(C::STAGE_BYTES);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t o = uint32_t((k >> 2) * 128 * 128 + (k & 3) * 32);
              ptx::mma_bf16(tmem + uint32_t(b * sp.cols), tc::BlockLayout<D>::by_row(ka, k),
                            tc::sdesc_sw128(sbase + o, 16, 1024), id_qk, k ? 1u : 0u);
            }
            issued = true;
            ptx::tc_commit(s_full(b));
            ptx::tc_commit(empty(seq % NS));
            if (i + 1 == nblk) ptx::tc_commit(q_empty);
          }
          const uint32_t id_pv = tc::idesc_bf16(128, x.cols, true, true);
          for (int32_t b = 0; b < nblk && ok; ++b, ++seq) {
            ok = tc::wait_bar(full(seq % NS), (seq / NS) & 1u, sy) && tc::wait_bar(p_full, np & 1u, sy);
            if (!ok) break;
            ++np;
            ptx::tc_fence_after();
            const uint32_t va = sbase + uint32_t(C::OFF_RING) + (seq % NS) * uint32_t(C::STAGE_BYTES);
            const uint64_t ph = tc::sdesc_sw128(sbase + C::OFF_P, C::ATOM, 1024);
            const uint64_t pl = tc::sdesc_sw128(sbase + C::OFF_P + 2 * C::ATOM, C::ATOM, 1024);
#pragma unroll
            for (int k = 0; k < tc::kBlockPos / 16; ++k) {
              const uint64_t vd = tc::BlockLayout<D>::by_dim(va, k), o = uint64_t(k * 16 * 128 >> 4);
              ptx::mma_bf16(tmem, vd, ph + o, id_pv, (b | k) ? 1u : 0u);
              ptx::mma_bf16(tmem, vd, pl + o, id_pv, 1u);
            }
            ptx::tc_commit(p_free);
            ptx::tc_commit(empty(seq % NS));
          }
        }
        if (issued) {                          // no MMA of ours may be in flight when TMEM is released
          volatile uint32_t none = 0;
          const tc::Sync end{&none, p.status, p.timeout_ns};
          ptx::tc_commit(drain);
          tc::wait_bar(drain, 0u, end);
        }
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------ the group's tables agree
      const int hid = (warp - 2) * 32 + lane;
      bool differ = false;
      int4 rec = record(int32_t(blockIdx.x));
      for (int32_t u = int32_t(blockIdx.x); u < units; u += int32_t(gridDim.x)) {
        const U x = unit(rec, u);
        rec = record(u + int32_t(gridDim.x));      // the next one's, ahead of its use
        const int32_t* src = p.table + int64_t(__ldcg(p.q_seq + x.src)) * p.max_pages;
        const int32_t pg0 = x.s * p.split / p.page_size, pgs = ((x.s + 1) * p.split - 1) / p.page_size + 1 - pg0;
        for (int32_t k = x.kh; k < x.n; k += p.Hkv) {    // (the KV heads' units share the tokens out)
          if (__ldcg(sp.nsh + x.t0 + k) <= x.s) continue;
          const int32_t* row = p.table + int64_t(__ldcg(p.q_seq + x.t0 + k)) * p.max_pages;
          for (int32_t i = hid; i < pgs; i += 64) differ |= __ldcg(row + pg0 + i) != __ldcg(src + pg0 + i);
        }
      }
      if (differ) atomicOr(p.status, kErrInput);
    }
  } else {
    // -------------------------------------------------------------- softmax: a thread per position
    ptx::setmaxnreg_inc<104>();
    const int i = (warp - 4) >> 2, w4 = warp & 3;
    const int pos = w4 * 32 + lane;                      // position of a block = TMEM lane
    const uint32_t tl = tmem + (uint32_t(w4 * 32) << 16);
    float* mine = msm + 32 * i;
    float* red = reinterpret_cast<float*>(smem + C::OFF_RED) + 128 * i;      // [4][32]
    auto group_sync = [&]() {       // (aligned: the warp's lanes arrive together)
      __syncwarp();
      asm volatile("bar.sync %0, 128;" ::"r"(1 + i) : "memory");
    };
    // this position's row of the weights' buffer
    const uint32_t prow = sbase + uint32_t(C::OFF_P + pos * 128);
    uint32_t nu = 0, np = 0;
    bool ok = true;
    int4 rec = record(int32_t(blockIdx.x));
    for (int32_t u = int32_t(blockIdx.x); u < units && ok; u += int32_t(gridDim.x), ++nu) {
      const U x = unit(rec, u);
      rec = record(u + int32_t(gridDim.x));      // the next one's, ahead of its use
      const int32_t cb = min(i * x.share, x.cols), nc = min(x.share, x.cols - cb);      // its columns: 0, 16 or 32
      const uint32_t atom = prow + uint32_t((cb >> 6) * C::ATOM), ch0 = uint32_t(cb & 63) / 8;
      // pass 1: each column's maximum (of the raw sums: the scaling is monotone)
      {
        float mx[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) mx[k] = -INFINITY;
#pragma unroll 1
        for (int32_t q = 0; q < nblk; ++q) {
          const int32_t b = q + 1 < nblk ? q + 1 : 0;
          ok = __all_sync(0xFFFFFFFFu, tc::wait_bar(s_full(b), nu & 1u, sy));
          if (!ok) break;
          ptx::tc_fence_after();
          // (sixteen at a time: the last block's columns end where tensor memory does)
          if (nc > 0) {
            uint32_t s[16], s2[16];
            tmem_ld_x16(tl + uint32_t(b * sp.cols + cb), s);
            if (nc > 16) tmem_ld_x16(tl + uint32_t(b * sp.cols + cb + 16), s2);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) mx[e] = fmaxf(mx[e], __uint_as_float(s[e]));
            if (nc > 16) {
#pragma unroll
              for (int e = 0; e < 16; ++e) mx[16 + e] = fmaxf(mx[16 + e], __uint_as_float(s2[e]));
            }
          }
        }
        if (ok && nc > 0) red[w4 * 32 + lane] = reduce_columns(mx, lane, [](float a, float b) { return fmaxf(a, b); });
      }
      // (a warp that gave up still walks the barriers)
      group_sync();
      if (pos < nc)
        mine[pos] = __fmul_rn(fmaxf(fmaxf(red[pos], red[32 + pos]), fmaxf(red[64 + pos], red[96 + pos])), p.c);
      group_sync();
      // pass 2: weights, their sums, and their two bf16 parts for the value product
      uint64_t ls[16];                                   // pairs of columns
#pragma unroll
      for (int k = 0; k < 16; ++k) ls[k] = 0;
#pragma unroll 1
      for (int32_t b = 0; b < nblk && ok; ++b) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (k * 16 < nc) {
            uint32_t s[16];
            tmem_ld_x16(tl + uint32_t(b * sp.cols + cb + k * 16), s);
            ptx::tmem_wait_ld();
            float w[16];
            float low = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 m = *reinterpret_cast<const float4*>(mine + k * 16 + e);
              // (mul and add on pairs came out fused, with one rounding where these have two)
              w[e] = __fsub_rn(__fmul_rn(__uint_as_float(s[e]), p.c), m.x);
              w[e + 1] = __fsub_rn(__fmul_rn(__uint_as_float(s[e + 1]), p.c), m.y);
              w[e + 2] = __fsub_rn(__fmul_rn(__uint_as_float(s[e + 2]), p.c), m.z);
              w[e + 3] = __fsub_rn(__fmul_rn(__uint_as_float(s[e + 3]), p.c), m.w);
              low = tc::min3(low, tc::min3(w[e], w[e + 1], w[e + 2]), w[e + 3]);
            }
            // From -126 to 0 the instruction alone gives exp2f's bits (every float of the range was
            // compared); a column past the unit's, with whatever is in it, at worst takes the other way.
            if (__any_sync(0xFFFFFFFFu, low < -126.0f)) {
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = exp2f(w[e]);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = tc::ex2(w[e]);
            }
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const int j = k * 8 + (e >> 1);
              ls[j] = tc::add2(ls[j], tc::pair(w[e], w[e + 1]));
              hi[j] = pack_bf16x2(w[e], w[e + 1]);
              lo[j] = pack_bf16x2(__fsub_rn(w[e], bf16_lo(hi[j])), __fsub_rn(w[e + 1], bf16_hi(hi[j])));
            }
          }
        }
        if (b > 0) {                                     // the block before has been multiplied
          ok = __all_sync(0xFFFFFFFFu, tc::wait_bar(p_free, np & 1u, sy));
          if (!ok) break;
          ++np;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k * 8 < nc) {
            const uint32_t a = atom + (((ch0 + uint32_t(k)) ^ uint32_t(pos & 7)) << 4);
            ptx::st_shared_v4(a, hi[4 * k], hi[4 * k + 1], hi[4 * k + 2], hi[4 * k + 3]);
            ptx::st_shared_v4(a + 2 * C::ATOM, lo[4 * k], lo[4 * k + 1], lo[4 * k + 2], lo[4 * k + 3]);
          }
        }
        ptx::tc_fence_before();
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(p_full);
      }
      if (ok && nc > 0) {                                // the sums, while the last product runs
        float v[32];
#pragma unroll
        for (int k = 0; k < 16; ++k) tc::unpair(ls[k], v[2 * k], v[2 * k + 1]);
        red[w4 * 32 + lane] = reduce_columns(v, lane, [](float a, float b) { return __fadd_rn(a, b); });
      }
      group_sync();
      const int64_t stride_t = int64_t(p.Hkv) * p.max_splits * G;            // rows of part between tokens
      const int64_t row0 = ((int64_t(x.t0) * p.Hkv + x.kh) * p.max_splits + x.s) * G;
      // which of the columns are tokens that share the split
      const int32_t tok = (cb + lane) / G;
      const uint32_t live =
          __ballot_sync(0xFFFFFFFFu, lane < nc && tok < x.n && __ldcg(sp.nsh + x.t0 + min(tok, x.n - 1)) > x.s);
      if (ok && w4 == 0 && ((live >> lane) & 1u)) {
        const float l = __fadd_rn(__fadd_rn(__fadd_rn(red[lane], red[32 + lane]), red[64 + lane]), red[96 + lane]);
        *reinterpret_cast<float2*>(p.ml + (row0 + tok * stride_t + (cb + lane) % G) * 2) = make_float2(mine[lane], l);
      }
      ok = ok && __all_sync(0xFFFFFFFFu, tc::wait_bar(p_free, np & 1u, sy));   // the last block's product
      ++np;
      ptx::tc_fence_after();
      if (ok && nc > 0) {
        // value sums: thread = output dimension, a warp writes 32 of a column's at once, tokens G
        // columns at a time (a token's heads share the split or none does)
        float* dst = p.part + (row0 + (cb / G) * stride_t) * D + pos;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (k * 16 < nc) {
            uint32_t o[16];
            tmem_ld_x16(tl + uint32_t(cb + k * 16), o);
            ptx::tmem_wait_ld();
            if (pos < D) {
#pragma unroll
              for (int e = 0; e < 16; e += G) {
                if ((live >> (k * 16 + e)) & 1u) {
#pragma unroll
                  for (int g = 0; g < G; ++g) dst[g * D] = __uint_as_float(o[e + g]);
                }
                dst += stride_t * D;
              }
            }
          }
        }
      }
      // the warps of a group go on or stop together (they meet at its barrier)
      ok = !tc::bar_or(1 + i, !ok);
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_relaxed(o_free);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) ptx::tmem_dealloc(tmem, 512);
  ptx::grid_dependency_wait();   // (see above)
}

// merge_kernel's arithmetic, output by output the same operations in the same order, for lists of many
// splits: a thread holds an output pair for all four groups, so that a warp reads 256 bytes of a
// split's sums at once (there four lanes share a pair, 64 bytes of each of four splits), and the
// splits' factors are computed once per head, not per output.  256 tokens of 36 splits (32 heads of
// 128, 150 MB of partial sums): 31 us, 86 with merge_kernel.
constexpr int kWideThreads = 256, kWideChunk = 128, kWideBatch = 8;

template <int D, int G>
__global__ void __launch_bounds__(kWideThreads) merge_wide_kernel(const Params p) {
  constexpr int kPairs = G * D / 2;
  constexpr int kSlices = (kPairs + kWideThreads - 1) / kWideThreads;
  __shared__ float fac[kWideChunk * G], wsum[kWideChunk * G], top[G];
  const int64_t job = blockIdx.x / kSlices;              // token * Hkv + KV head
  const int slice = int(blockIdx.x - job * kSlices), tid = int(threadIdx.x);
  const int64_t t = job / p.Hkv;
  const int32_t kh = int32_t(job - t * p.Hkv);
  const int32_t b = __ldcg(p.q_seq + t), pos = __ldcg(p.q_pos + t);
  ptx::grid_dependency_wait();   // every unit's partial results are complete and visible
  if (b < 0 || b >= p.B || pos < 0 || int64_t(pos / p.page_size) >= p.max_pages || pos > p.max_pos) return;
  const int32_t n = splits_of(pos, p.split);
  if (n == 1) return;                                    // written directly
  const int64_t slot0 = job * int64_t(p.max_splits);
  const float2* ml = reinterpret_cast<const float2*>(p.ml) + slot0 * G;
  for (int g = tid >> 5; g < G; g += kWideThreads / 32) {        // M, a warp per head
    float m = -INFINITY;
    for (int32_t s = tid & 31; s < n; s += 32) m = fmaxf(m, ml[int64_t(s) * G + g].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if ((tid & 31) == 0) top[g] = m;
  }
  __syncthreads();
  const int pr = slice * kWideThreads + tid;
  const bool valid = pr < kPairs;
  const int g = valid ? pr / (D / 2) : 0, d = valid ? (pr % (D / 2)) * 2 : 0;
  const float* pp = p.part + (slot0 * G + g) * D + d;
  const int32_t c = (n + 3) / 4;                         // splits per group
  float L = 0.0f, A0 = 0.0f, A1 = 0.0f, Ls = 0.0f, As0 = 0.0f, As1 = 0.0f;
  int32_t left = c, group = 0;                           // of the current group
  auto close = [&]() {                                   // the group's sums join those before it
    Ls = group ? __fadd_rn(Ls, L) : L;
    As0 = group ? __fadd_rn(As0, A0) : A0;
    As1 = group ? __fadd_rn(As1, A1) : A1;
    L = A0 = A1 = 0.0f;
    ++group;
    left = c;
  };
  for (int32_t c0 = 0; c0 < n; c0 += kWideChunk) {
    const int32_t cn = min(kWideChunk, n - c0);
    __syncthreads();
    for (int i = tid; i < cn * G; i += kWideThreads) {
      const float2 x = ml[int64_t(c0) * G + i];
      const float f = exp2f(__fsub_rn(x.x, top[i % G]));
      fac[i] = f;
      wsum[i] = __fmul_rn(x.y, f);
    }
    __syncthreads();
    if (!valid) continue;
    for (int32_t s0 = 0; s0 < cn; s0 += kWideBatch) {
      float2 v[kWideBatch];
#pragma unroll
      for (int k = 0; k < kWideBatch; ++k)
        if (s0 + k < cn) v[k] = *reinterpret_cast<const float2*>(pp + int64_t(c0 + s0 + k) * G * D);
#pragma unroll
      for (int k = 0; k < kWideBatch; ++k) {
        if (s0 + k < cn) {
          const float f = fac[(s0 + k) * G + g];
          L = __fadd_rn(L, wsum[(s0 + k) * G + g]);
          A0 = __fadd_rn(A0, __fmul_rn(v[k].x, f));
          A1 = __fadd_rn(A1, __fmul_rn(v[k].y, f));
          if (--left == 0) close();
        }
      }
    }
  }
  if (!valid) return;
  if (left < c) close();
  *reinterpret_cast<uint32_t*>(p.o + (t * p.Hq + int64_t(kh) * G + g) * D + d) =
      pack_bf16x2(__fdiv_rn(As0, Ls), __fdiv_rn(As1, Ls));
}

struct SharedInfo {
  const void* tma = nullptr;
  const void* rows = nullptr;
  const void* merge = nullptr;
  int smem = 0, merge_slices = 1;
};

template <int D, int G>
SharedInfo shared_info() {
  SharedInfo k;
  k.tma = reinterpret_cast<const void*>(&shared_kernel<D, G, true>);
  k.rows = reinterpret_cast<const void*>(&shared_kernel<D, G, false>);
  k.smem = SharedCfg<D, G>::SMEM;
  k.merge = reinterpret_cast<const void*>(&merge_wide_kernel<D, G>);
  k.merge_slices = (G * D / 2 + kWideThreads - 1) / kWideThreads;
  return k;
}

inline SharedInfo select_shared(int D, int G) {
  if (D == 128) {
    switch (G) {
      case 1: return shared_info<128, 1>();
      case 2: return shared_info<128, 2>();
      case 4: return shared_info<128, 4>();
      case 8: return shared_info<128, 8>();
    }
  } else if (D == 64) {
    switch (G) {
      case 1: return shared_info<64, 1>();
      case 2: return shared_info<64, 2>();
      case 4: return shared_info<64, 4>();
      case 8: return shared_info<64, 8>();
    }
  }
  return SharedInfo{};
}

}  // namespace biattn
