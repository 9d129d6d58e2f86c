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
// denormal inputs, and the tests hold whole calls to it.
//
// Bound: for many tokens the tensor cores (6 D operations per query row and key, a third of them for
// the weights' low part) and the softmax's instructions, for few the load of the prefix.
//
// Warps (384 threads, one block per SM): 0 loads (queries, then K1 .. K(n-1), K0, V0 .. V(n-1)
// through a ring), 1 issues the MMAs, 2 and 3 check that the group's page tables agree, 4 - 11
// softmax: two warpgroups, each half of the columns, a thread per position of a block.
// TMEM: block b's scores at column 128 b (64 b for splits above 512); the value sums take block 0's
// columns once its weights are out, so a unit's block 0 is the last whose scores are computed.
#pragma once

#include "attn_ptx.cuh"

namespace biattn {

namespace tc = biattn_tc;

constexpr int kSharedThreads = 384;
constexpr int kSharedStages = 4;
constexpr int kMaxBlocks = 8;                 // blocks of a split: 1024 / 128

struct SharedParams {
  Params a;                    // as bi_attention_run's (part, ml, status, shapes, ...)
  const int32_t* group_start;
  const int32_t* group_len;
  int32_t* nsh;                // [T] leading splits of each token that its group computes
  int4* srec;                  // [cap] (first token, tokens, split, token whose pages are read)
  int32_t* count;              // [1] records
  tc::Cache c;
  int64_t num_groups, cap;
  int32_t cols;                // columns of a unit at most: 128, or 64 above splits of 512
};

// One block: per token the splits that its group computes, the units of the groups, then the
// records of all other units in the form that the attention kernels read.
__global__ void __launch_bounds__(1024) plan_shared_kernel(const SharedParams sp) {
  __shared__ int32_t warp_sums[32];
  __shared__ int32_t carry;
  __shared__ int32_t nrec;
  const Params& p = sp.a;
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  if (tid == 0) carry = 0, nrec = 0;
  for (int64_t t = tid; t < p.T; t += 1024) sp.nsh[t] = 0;
  __syncthreads();
  const int32_t G = p.Hq / p.Hkv, per = sp.cols / G;     // tokens of a unit
  for (int64_t g = warp; g < sp.num_groups; g += 32) {
    const int32_t s = sp.group_start[g], e = sp.group_start[g + 1], len = sp.group_len[g];
    if (s < 0 || e < s || e > p.T || len < 0) {
      if (lane == 0) atomicOr(p.status, kErrInput);
      continue;
    }
    if (e - s < 2) continue;                             // (alone: its own units serve it as well)
    for (int32_t t0 = s; t0 < e; t0 += per) {
      const int32_t n = min(per, e - t0);
      int32_t most = 0;
      for (int32_t k = lane; k < n; k += 32) {
        const int32_t b = p.q_seq[t0 + k], pos = p.q_pos[t0 + k];
        // (the split that holds the token itself is always its own)
        int32_t x = 0;
        if (b >= 0 && b < p.B && pos >= 0 && pos <= p.max_pos && int64_t(pos / p.page_size) < p.max_pages)
          x = min(len, pos) / p.split;
        sp.nsh[t0 + k] = x;
        most = max(most, x);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
      __syncwarp();
      int32_t at = 0;
      if (lane == 0) at = atomicAdd(&nrec, most);
      at = __shfl_sync(0xFFFFFFFFu, at, 0);
      for (int32_t sx = lane; sx < most; sx += 32) {
        int32_t src = t0;
        while (sp.nsh[src] <= sx) ++src;                 // (ends: a token has `most`)
        if (at + sx < sp.cap) sp.srec[at + sx] = make_int4(t0, n, sx, src);
        else atomicOr(p.status, kErrInput);              // (only from a group_start that descends)
      }
    }
  }
  __syncthreads();
  if (tid == 0) sp.count[0] = int32_t(min(int64_t(nrec), sp.cap));
  for (int64_t base = 0; base < p.T; base += 1024) {
    const int64_t t = base + tid;
    int32_t n = 0, b = 0, pos = 0, sh = 0;
    if (t < p.T) {
      b = p.q_seq[t];
      pos = p.q_pos[t];
      if (b < 0 || b >= p.B || pos < 0 || int64_t(pos / p.page_size) >= p.max_pages) {
        atomicOr(p.status, kErrInput);
      } else if (pos > p.max_pos) {
        atomicOr(p.status, kErrBound);
      } else {
        sh = sp.nsh[t];
        n = (splits_of(pos, p.split) - sh) * p.Hkv;
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
    for (int k = 0; k < 32; ++k) {
      const int32_t nk = __shfl_sync(0xFFFFFFFFu, n, k), sk = __shfl_sync(0xFFFFFFFFu, incl - n, k);
      const int32_t bk = __shfl_sync(0xFFFFFFFFu, b, k), pk = __shfl_sync(0xFFFFFFFFu, pos, k);
      const int32_t hk = __shfl_sync(0xFFFFFFFFu, sh, k);
      const int32_t tk = int32_t(base + warp * 32 + k);
      for (int32_t r = lane; r < nk; r += 32) p.urec[sk + r] = make_int4(tk, bk, pk, hk * p.Hkv + r);
    }
    __syncthreads();
    if (tid == 1023) carry = incl;
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
  static constexpr int P_BYTES = 2 * tc::kBlockPos * 128;     // high and low parts: 128 positions x 64 columns
  static constexpr int OFF_RING = Q_BYTES;
  static constexpr int OFF_P = OFF_RING + NS * STAGE_BYTES;   // [2 warpgroups]
  static constexpr int OFF_M = OFF_P + 2 * P_BYTES;           // [128] maxima
  static constexpr int OFF_BAR = OFF_M + 128 * 4;
  // ring full, empty; Q full, empty; scores of a block; weights full, free (per warpgroup); O free; drain
  static constexpr int NUM_BARS = 2 * NS + 2 + kMaxBlocks + 4 + 2;
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
  auto p_full = [&](int i) { return q_empty + 8 + 8 * (kMaxBlocks + i); };
  auto p_free = [&](int i) { return q_empty + 8 + 8 * (kMaxBlocks + 2 + i); };
  const uint32_t o_free = q_empty + 8 + 8 * (kMaxBlocks + 4), drain = o_free + 8;
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
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(p_full(i), 4);
      ptx::mbar_init(p_free(i), 1);
    }
    ptx::mbar_init(o_free, 8);
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
  ptx::grid_dependency_wait();   // the plan is complete and visible
  ptx::launch_dependents();
  const tc::Sync sy{abort, p.status, p.timeout_ns};
  const int32_t units = sp.count[0] * p.Hkv;
  const int nblk = p.split / tc::kBlockPos;

  // A unit's record; columns and their halves (multiples of 16, the MMA's step in N).
  struct U {
    int32_t t0, n, s, src, kh, cols, c0;
  };
  auto unit = [&](int32_t u) {
    const int4 r = sp.srec[u / p.Hkv];
    U x;
    x.t0 = r.x, x.n = r.y, x.s = r.z, x.src = r.w;
    x.kh = u % p.Hkv;
    x.cols = (x.n * G + 15) & ~15;
    x.c0 = ((x.cols / 16 + 1) / 2) * 16;        // columns of warpgroup 0
    return x;
  };

  if (warp < 4) {
    ptx::setmaxnreg_dec<80>();
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
      for (int32_t u = int32_t(blockIdx.x); u < units && ok; u += int32_t(gridDim.x), ++nu) {
        const U x = unit(u);
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
        const int32_t* trow = p.table + int64_t(p.q_seq[x.src]) * p.max_pages;
        const int32_t base = x.s * p.split, last = base + p.split - 1;
        for (int32_t i = 0; i < 2 * nblk; ++i, ++seq) {
          const int32_t b = i < nblk ? (i + 1 < nblk ? i + 1 : 0) : i - nblk;
          const int32_t pos0 = base + b * tc::kBlockPos;
          const uint32_t s = seq % NS, dst = sbase + uint32_t(C::OFF_RING) + s * uint32_t(C::STAGE_BYTES);
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
        uint32_t seq = 0, nu = 0, np[2] = {0, 0};
        bool ok = true, issued = false;
        for (int32_t u = int32_t(blockIdx.x); u < units && ok; u += int32_t(gridDim.x), ++nu) {
          const U x = unit(u);
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
          for (int32_t b = 0; b < nblk && ok; ++b, ++seq) {
            ok = tc::wait_bar(full(seq % NS), (seq / NS) & 1u, sy);
            const uint32_t va = sbase + uint32_t(C::OFF_RING) + (seq % NS) * uint32_t(C::STAGE_BYTES);
            for (int i = 0; i < 2 && ok; ++i) {
              const int32_t nc = i ? x.cols - x.c0 : x.c0;
              if (nc == 0) continue;
              ok = tc::wait_bar(p_full(i), np[i] & 1u, sy);
              if (!ok) break;
              ++np[i];
              ptx::tc_fence_after();
              const uint32_t id_pv = tc::idesc_bf16(128, nc, true, true);
              const uint32_t ph = sbase + uint32_t(C::OFF_P + i * C::P_BYTES), pl = ph + uint32_t(C::P_BYTES / 2);
              const uint32_t od = tmem + uint32_t(i ? x.c0 : 0);
#pragma unroll
              for (int k = 0; k < tc::kBlockPos / 16; ++k) {
                const uint64_t vd = tc::BlockLayout<D>::by_dim(va, k);
                ptx::mma_bf16(od, vd, tc::sdesc_sw128(ph + uint32_t(k * 16 * 128), 16, 1024), id_pv, (b | k) ? 1u : 0u);
                ptx::mma_bf16(od, vd, tc::sdesc_sw128(pl + uint32_t(k * 16 * 128), 16, 1024), id_pv, 1u);
              }
              ptx::tc_commit(p_free(i));
            }
            if (!ok) break;
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
      for (int32_t u = int32_t(blockIdx.x); u < units; u += int32_t(gridDim.x)) {
        const U x = unit(u);
        const int32_t* src = p.table + int64_t(p.q_seq[x.src]) * p.max_pages;
        const int32_t pg0 = x.s * p.split / p.page_size, pgs = ((x.s + 1) * p.split - 1) / p.page_size + 1 - pg0;
        for (int32_t k = x.kh; k < x.n; k += p.Hkv) {    // (the KV heads' units share the tokens out)
          if (sp.nsh[x.t0 + k] <= x.s) continue;
          const int32_t* row = p.table + int64_t(p.q_seq[x.t0 + k]) * p.max_pages;
          for (int32_t i = hid; i < pgs; i += 64) differ |= row[pg0 + i] != src[pg0 + i];
        }
      }
      if (differ) atomicOr(p.status, kErrInput);
    }
  } else {
    // -------------------------------------------------------------- softmax: a thread per position
    ptx::setmaxnreg_inc<208>();
    const int i = (warp - 4) >> 2, w4 = warp & 3;
    const int pos = w4 * 32 + lane;                      // position of a block = TMEM lane
    const uint32_t tl = tmem + (uint32_t(w4 * 32) << 16);
    uint8_t* pbuf = smem + C::OFF_P + i * C::P_BYTES;
    float* red = reinterpret_cast<float*>(pbuf);         // [4][64], while the weights' buffer is free
    const uint32_t pb = sbase + uint32_t(C::OFF_P + i * C::P_BYTES) + uint32_t(pos * 128);
    auto group_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + i) : "memory"); };
    uint32_t nu = 0, np = 0;
    bool ok = true;
    for (int32_t u = int32_t(blockIdx.x); u < units && ok; u += int32_t(gridDim.x), ++nu) {
      const U x = unit(u);
      const int32_t cb = i ? x.c0 : 0, nc = i ? x.cols - x.c0 : x.c0;
      if (nc == 0) {                                     // the unit's phases still pass one by one
        for (int32_t b = 0; b < nblk && ok; ++b) ok = __all_sync(0xFFFFFFFFu, tc::wait_bar(s_full(b), nu & 1u, sy));
      } else {
        // pass 1: each column's maximum (of the raw sums: the scaling is monotone)
        float mx[2][32];
#pragma unroll
        for (int k = 0; k < 64; ++k) mx[k >> 5][k & 31] = -INFINITY;
        for (int32_t q = 0; q < nblk; ++q) {
          const int32_t b = q + 1 < nblk ? q + 1 : 0;
          ok = tc::wait_bar(s_full(b), nu & 1u, sy);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          ptx::tc_fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k * 16 < nc) {
              uint32_t s[16];
              tmem_ld_x16(tl + uint32_t(b * sp.cols + cb + k * 16), s);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float& m = mx[k >> 1][(k & 1) * 16 + e];
                m = fmaxf(m, __uint_as_float(s[e]));
              }
            }
          }
        }
        if (ok) {
          auto fmx = [](float a, float b) { return fmaxf(a, b); };
          red[w4 * 64 + lane] = reduce_columns(mx[0], lane, fmx);
          if (nc > 32) red[w4 * 64 + 32 + lane] = reduce_columns(mx[1], lane, fmx);
        }
        // (a warp that gave up still walks the barriers)
        group_sync();
        if (pos < nc)
          msm[64 * i + pos] = __fmul_rn(fmaxf(fmaxf(red[pos], red[64 + pos]), fmaxf(red[128 + pos], red[192 + pos])), p.c);
        group_sync();
        // pass 2: weights, their sums, and their two bf16 parts for the value product
        float ls[2][32];
#pragma unroll
        for (int k = 0; k < 64; ++k) ls[k >> 5][k & 31] = 0.0f;
        for (int32_t b = 0; b < nblk && ok; ++b) {
          if (b > 0) {
            ok = tc::wait_bar(p_free(i), np & 1u, sy);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            ++np;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k * 16 < nc) {
              uint32_t s[16], hi[8], lo[8];
              tmem_ld_x16(tl + uint32_t(b * sp.cols + cb + k * 16), s);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                const float2 m = *reinterpret_cast<const float2*>(msm + 64 * i + k * 16 + e);
                const float w0 = exp2f(__fsub_rn(__fmul_rn(__uint_as_float(s[e]), p.c), m.x));
                const float w1 = exp2f(__fsub_rn(__fmul_rn(__uint_as_float(s[e + 1]), p.c), m.y));
                float& l0 = ls[k >> 1][(k & 1) * 16 + e];
                float& l1 = ls[k >> 1][(k & 1) * 16 + e + 1];
                l0 = __fadd_rn(l0, w0);
                l1 = __fadd_rn(l1, w1);
                hi[e >> 1] = pack_bf16x2(w0, w1);
                lo[e >> 1] = pack_bf16x2(__fsub_rn(w0, bf16_lo(hi[e >> 1])), __fsub_rn(w1, bf16_hi(hi[e >> 1])));
              }
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t a = pb + uint32_t(((2 * k + h) ^ (pos & 7)) << 4);
                ptx::st_shared_v4(a, hi[4 * h], hi[4 * h + 1], hi[4 * h + 2], hi[4 * h + 3]);
                ptx::st_shared_v4(a + uint32_t(C::P_BYTES / 2), lo[4 * h], lo[4 * h + 1], lo[4 * h + 2], lo[4 * h + 3]);
              }
            }
          }
          ptx::tc_fence_before();
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(p_full(i));
        }
        if (ok) {
          ok = tc::wait_bar(p_free(i), np & 1u, sy);     // the last block's product: the sums are complete
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (ok) ++np;
        }
        ptx::tc_fence_after();
        if (ok) {
          auto add = [](float a, float b) { return __fadd_rn(a, b); };
          red[w4 * 64 + lane] = reduce_columns(ls[0], lane, add);
          if (nc > 32) red[w4 * 64 + 32 + lane] = reduce_columns(ls[1], lane, add);
        }
        group_sync();
        if (ok) {
          const int32_t col = cb + pos, tok = col / G;
          if (pos < nc && tok < x.n && sp.nsh[x.t0 + tok] > x.s) {
            const float l = __fadd_rn(__fadd_rn(__fadd_rn(red[pos], red[64 + pos]), red[128 + pos]), red[192 + pos]);
            const int64_t slot = (int64_t(x.t0 + tok) * p.Hkv + x.kh) * p.max_splits + x.s;
            float* ml = p.ml + (slot * G + col % G) * 2;
            ml[0] = msm[64 * i + pos];
            ml[1] = l;
          }
          // value sums: thread = output dimension, a warp writes 32 of a column's at once
          for (int32_t k = 0; k < nc; k += 16) {
            uint32_t o[16];
            tmem_ld_x16(tl + uint32_t(cb + k), o);
            ptx::tmem_wait_ld();
            const int32_t c16 = cb + k + (lane & 15);
            const bool mine = c16 / G < x.n && sp.nsh[min(x.t0 + c16 / G, x.t0 + x.n - 1)] > x.s;
            const uint32_t live = __ballot_sync(0xFFFFFFFFu, mine);
            if (pos < D) {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                if ((live >> e) & 1u) {
                  const int32_t col = cb + k + e;
                  const int64_t slot = (int64_t(x.t0 + col / G) * p.Hkv + x.kh) * p.max_splits + x.s;
                  p.part[(slot * G + col % G) * D + pos] = __uint_as_float(o[e]);
                }
              }
            }
          }
        }
      }
      // The scratch is the next unit's weights' buffer; the warps of the group go on or stop together.
      ok = !tc::bar_or(1 + i, !ok);
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(o_free);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) ptx::tmem_dealloc(tmem, 512);
}

struct SharedInfo {
  const void* tma = nullptr;
  const void* rows = nullptr;
  int smem = 0;
};

template <int D, int G>
SharedInfo shared_info() {
  SharedInfo k;
  k.tma = reinterpret_cast<const void*>(&shared_kernel<D, G, true>);
  k.rows = reinterpret_cast<const void*>(&shared_kernel<D, G, false>);
  k.smem = SharedCfg<D, G>::SMEM;
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
