// bi_qkrope.cu — per-head RMSNorm of queries and keys, rotation by position and append of keys and
// values to the paged cache, in one pass over the fused projection's output, for sm_103a.
// Implements include/bi_qkrope.h.
//
// Bound: HBM bandwidth (every element read once, written once) beside the instructions, about eight
// operations an element; one launch's latency for a few tokens.  Measured at 32/8 heads of 128: 1 token
// 3.0 us, 64 tokens 2.9, 8192 tokens 41.3 (206 MB: 5.0 TB/s, 0.74 of a plain copy's rate).  A head of D
// elements belongs to D / 8 lanes, eight elements each: two runs of four that are rotation partners (dimensions 4 j and
// 4 j + rot / 2 on), or eight neighbours for an interleaved handle, so that a rotation needs no other
// lane and its arithmetic goes two values an instruction.  A token has a power of two of such lane
// groups, each with up to kHeads heads at a time in registers: their loads are issued before the
// token's position is known, and its cosines, sines and the norm weights are read once for all of them.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>

#include "../../include/bi_qkrope.h"
#include "attn_ptx.cuh"

#ifndef BI_GEMM_API
#define BI_GEMM_API extern "C" __attribute__((visibility("default")))
#endif

namespace biqkr {

namespace ptx = bigemm::ptx;

// Untiled bulk copy global -> shared (16-byte aligned, a multiple of 16 bytes), counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

constexpr int kThreads = 256;
constexpr int kHeads = 4;                // heads a lane group holds at a time
constexpr int kMaxRing = 16;             // stages of the ring
constexpr int kRingBytes = 54 * 1024;    // shared memory of a block's ring at most: four blocks per SM
constexpr int kRingRows = 40 * 1024;     // bytes of rows that a block of it has to have
constexpr uint32_t kErrInput = 1u;       // q_seq, q_pos or the page table's extent
constexpr uint32_t kErrPage = 2u;        // page outside [0, num_pages)

struct Params {
  const uint16_t* qkv;
  const uint16_t* gq;       // NULL: no norm
  const uint16_t* gk;
  const float* cs;          // [num_positions, rot]
  const int32_t* q_seq;
  const int32_t* q_pos;
  const int32_t* table;
  uint16_t* kc;
  uint16_t* vc;
  uint16_t* q_out;
  uint32_t* status;
  int64_t T, stride, num_positions, num_pages, B, max_pages;
  int32_t Hq, Hkv, page_size, rot;
  int32_t groups_log2;      // lane groups per token
  int32_t ring;             // stages (tokens) of the ring, in the form for many tokens
  int32_t team_log2;        // and its warps per token
  int32_t stall;            // failure injection (test controls only): this block of it loads nothing
  uint64_t timeout_ns;      // limit of its waits
  float eps;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two fp32 values in a register pair, each rounded as by the scalar instruction.
using biattn_tc::fma2;
using biattn_tc::mul2;
using biattn_tc::pair;
using biattn_tc::unpair;
__device__ __forceinline__ uint64_t widen(uint32_t w) { return pair(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ uint32_t narrow(uint64_t v) {
  float lo, hi;
  unpair(v, lo, hi);
  return pack_bf16x2(lo, hi);
}

// What a lane does to the heads of a token: its two runs of four dimensions of the head, whether they
// are rotated, the norm weights, and of the token the cosines and sines of its pairs: of the four pairs
// (a, b) of its runs, or, interleaved, of each two neighbours, both alike and the sine with either sign.
template <int D, bool kInterleaved>
struct Lane {
  static constexpr int LANES = D / 8, PAIRS = kInterleaved ? 4 : 2;
  int l, da, db, half;
  bool turned, norm;
  uint32_t mask;            // the lane group's lanes
  uint2 wqa, wqb, wka, wkb;
  uint64_t co[PAIRS], si[PAIRS];

  __device__ __forceinline__ Lane(const Params& p, int tid) {
    l = tid & (LANES - 1);
    half = p.rot >> 1;
    turned = l < (p.rot >> 3);
    da = kInterleaved || !turned ? 8 * l : 4 * l;
    db = kInterleaved || !turned ? da + 4 : da + half;
    mask = LANES == 16 ? 0xFFFFu << (tid & 16) : 0xFFu << (tid & 24);
    norm = p.gq != nullptr;
    wqa = wqb = wka = wkb = make_uint2(0, 0);
    if (norm) {
      wqa = *reinterpret_cast<const uint2*>(p.gq + da), wqb = *reinterpret_cast<const uint2*>(p.gq + db);
      wka = *reinterpret_cast<const uint2*>(p.gk + da), wkb = *reinterpret_cast<const uint2*>(p.gk + db);
    }
#pragma unroll
    for (int e = 0; e < PAIRS; ++e) co[e] = si[e] = 0;
  }

  // c: the position's cosines, then its sines
  __device__ __forceinline__ void angles(const float* c) {
    if (!turned) return;
    const float4 cv = *reinterpret_cast<const float4*>(c + 4 * l);
    const float4 sv = *reinterpret_cast<const float4*>(c + half + 4 * l);
    if constexpr (kInterleaved) {
      co[0] = pair(cv.x, cv.x), co[1] = pair(cv.y, cv.y), co[2] = pair(cv.z, cv.z), co[3] = pair(cv.w, cv.w);
      si[0] = pair(-sv.x, sv.x), si[1] = pair(-sv.y, sv.y), si[2] = pair(-sv.z, sv.z), si[3] = pair(-sv.w, sv.w);
    } else {
      co[0] = pair(cv.x, cv.y), co[1] = pair(cv.z, cv.w);
      si[0] = pair(sv.x, sv.y), si[1] = pair(sv.z, sv.w);
    }
  }

  // Normalises and rotates the lane's share (a, b) of a query or key head.
  __device__ __forceinline__ void head(const Params& p, bool key, uint2& a, uint2& b) const {
    uint64_t x[4] = {widen(a.x), widen(a.y), widen(b.x), widen(b.y)};
    if (norm) {
      uint64_t q2 = mul2(x[0], x[0]);
      q2 = fma2(x[1], x[1], q2);
      q2 = fma2(x[2], x[2], q2);
      q2 = fma2(x[3], x[3], q2);
      float s0, s1;
      unpair(q2, s0, s1);
      float s = __fadd_rn(s0, s1);
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) s = __fadd_rn(s, __shfl_xor_sync(mask, s, o));
      const float r = __frsqrt_rn(__fmaf_rn(s, 1.0f / D, p.eps));     // (the product with 1 / D is exact)
      const uint64_t r2 = pair(r, r);
      x[0] = mul2(mul2(x[0], r2), widen(key ? wka.x : wqa.x));
      x[1] = mul2(mul2(x[1], r2), widen(key ? wka.y : wqa.y));
      x[2] = mul2(mul2(x[2], r2), widen(key ? wkb.x : wqb.x));
      x[3] = mul2(mul2(x[3], r2), widen(key ? wkb.y : wqb.y));
    }
    if (turned) {
      if constexpr (kInterleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float lo, hi;
          unpair(x[e], lo, hi);
          x[e] = fma2(x[e], co[e], mul2(pair(hi, lo), si[e]));
        }
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint64_t u = x[e], v = x[e + 2];
          float lo, hi;
          unpair(mul2(v, si[e]), lo, hi);
          x[e] = fma2(u, co[e], pair(-lo, -hi));
          x[e + 2] = fma2(v, co[e], mul2(u, si[e]));
        }
      }
    }
    a = make_uint2(narrow(x[0]), narrow(x[1]));
    b = make_uint2(narrow(x[2]), narrow(x[3]));
  }

  // Head h of a token: computed, and stored in q_out (row t) or the token's slot.
  __device__ __forceinline__ void finish(const Params& p, int h, int64_t t, int64_t slot, bool store, uint2 a,
                                         uint2 b) const {
    uint16_t* dst;
    if (h >= p.Hq + p.Hkv) {                            // values: as they are
      dst = p.vc + (slot * p.Hkv + (h - p.Hq - p.Hkv)) * D;
    } else {
      const bool key = h >= p.Hq;
      head(p, key, a, b);
      dst = key ? p.kc + (slot * p.Hkv + (h - p.Hq)) * D : p.q_out + (t * p.Hq + h) * D;
    }
    if (store) {
      *reinterpret_cast<uint2*>(dst + da) = a;
      *reinterpret_cast<uint2*>(dst + db) = b;
    }
  }
};

// The cache slot of a token, -1 (and an error) where it has none.
__device__ __forceinline__ int64_t slot_of(const Params& p, int32_t b, int32_t pos) {
  if (b < 0 || b >= p.B || pos < 0 || pos >= p.num_positions || int64_t(pos / p.page_size) >= p.max_pages) {
    atomicOr(p.status, kErrInput);
    return -1;
  }
  const int64_t page = p.table[int64_t(b) * p.max_pages + pos / p.page_size];
  if (page < 0 || page >= p.num_pages) {
    atomicOr(p.status, kErrPage);
    return -1;
  }
  return page * p.page_size + pos % p.page_size;
}

// A block per token or few: the form for few tokens.
template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 4) qkrope_kernel(const Params p) {
  constexpr int LANES = D / 8;
  // Programmatic dependent launch: the block may start while the previous kernel finishes and
  // waits for it (and its memory) before its first global access.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = int(threadIdx.x);
  const int groups = 1 << p.groups_log2;
  const int g = (tid / LANES) & (groups - 1);           // lane group of the token
  const int per_block = (kThreads / LANES) >> p.groups_log2;
  const int64_t t = int64_t(blockIdx.x) * per_block + ((tid / LANES) >> p.groups_log2);
  if (t >= p.T) return;                                 // (whole lane groups: the shuffles stay inside them)
  const int H = p.Hq + 2 * p.Hkv;
  Lane<D, kInterleaved> ln(p, tid);
  const uint16_t* row = p.qkv + t * p.stride;
  uint2 ra[kHeads], rb[kHeads];
  auto load = [&](int h0) {
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const int h = h0 + k * groups;
      if (h < H) {
        ra[k] = *reinterpret_cast<const uint2*>(row + h * D + ln.da);
        rb[k] = *reinterpret_cast<const uint2*>(row + h * D + ln.db);
      }
    }
  };
  load(g);
  const int32_t pos = p.q_pos[t];
  const int64_t slot = slot_of(p, p.q_seq[t], pos);
  if (slot >= 0) ln.angles(p.cs + int64_t(pos) * p.rot);
  // The loop is uniform over a lane group, not over a warp: a shuffle names its group's lanes.
  for (int h0 = g;; h0 += kHeads * groups) {
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const int h = h0 + k * groups;
      if (h >= H) break;
      ln.finish(p, h, t, slot, slot >= 0, ra[k], rb[k]);
    }
    if (h0 + kHeads * groups >= H) break;
    load(h0 + kHeads * groups);
  }
}

// The form for many tokens: persistent blocks; a warp ahead of the others looks up 32 tokens' slots at a
// time and copies their rows and angles into a ring (cp.async.bulk), so that several rows per block are
// on their way whatever the lookups take.  (A block per token is up for 4 us, a third of it with loads
// in flight: 52 us for 8192 tokens of 32/8 heads of 128, now 42.  With a larger ring and three blocks per SM
// it took 43.5, with five, and registers spilled, 47.)
template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kThreads + 32, 4) qkrope_ring_kernel(const Params p) {
  constexpr int LANES = D / 8;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[2 * kMaxRing];
  __shared__ int64_t slots[kMaxRing];
  __shared__ uint32_t gave_up;
  const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int H = p.Hq + 2 * p.Hkv, NS = p.ring;
  const uint32_t row_bytes = uint32_t(H) * D * 2, stage_bytes = row_bytes + uint32_t(p.rot) * 4;
  const uint32_t sbase = ptx::smem_u32(smem), full = ptx::smem_u32(bars), empty = full + 8 * kMaxRing;
  if (tid == 0) {
    gave_up = 0u;
    for (int s = 0; s < NS; ++s) {
      ptx::mbar_init(full + 8 * s, 1);
      ptx::mbar_init(empty + 8 * s, 1u << p.team_log2);
    }
    ptx::fence_barrier_init();
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const biattn_tc::Sync sy{&gave_up, p.status, p.timeout_ns};      // (every wait is bounded)
  const int64_t step = gridDim.x;
  int s = 0;
  uint32_t ph = 0;                                      // stage and phase of the next token
  bool go = true;
  if (warp == kThreads / 32) {
    for (int64_t t0 = blockIdx.x; t0 < p.T && go; t0 += 32 * step) {
      const int64_t mine = t0 + lane * step;
      int64_t slot = -1;
      int32_t pos = -1;
      if (mine < p.T) {
        pos = p.q_pos[mine];
        slot = slot_of(p, p.q_seq[mine], pos);
      }
      for (int k = 0; k < 32 && t0 + k * step < p.T; ++k) {
        const int64_t t = t0 + k * step, sl = __shfl_sync(0xFFFFFFFFu, slot, k);
        const int32_t at = __shfl_sync(0xFFFFFFFFu, pos, k);
        go = __all_sync(0xFFFFFFFFu, biattn_tc::wait_bar(empty + 8 * s, ph ^ 1u, sy));
        if (!go) break;
        if (lane == 0 && int(blockIdx.x) != p.stall) {
          slots[s] = sl;
          const uint32_t dst = sbase + uint32_t(s) * stage_bytes;
          ptx::mbar_arrive_expect_tx(full + 8 * s, sl >= 0 ? stage_bytes : 0u);
          if (sl >= 0) {
            bulk_load(dst, p.qkv + t * p.stride, row_bytes, full + 8 * s);
            bulk_load(dst + row_bytes, p.cs + int64_t(at) * p.rot, uint32_t(p.rot) * 4, full + 8 * s);
          }
        }
        __syncwarp();
        if (++s == NS) s = 0, ph ^= 1u;
      }
    }
  } else {
    Lane<D, kInterleaved> ln(p, tid);
    // teams of warps take the tokens in turn: a short row is not spread over more lanes than it has work for
    const int team = warp >> p.team_log2, teams = (kThreads / 32) >> p.team_log2;
    const int groups = (32 / LANES) << p.team_log2, g = (tid / LANES) & (groups - 1);
    int turn = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += step) {
      if (turn != team) {
        if (++turn == teams) turn = 0;
        if (++s == NS) s = 0, ph ^= 1u;
        continue;
      }
      if (++turn == teams) turn = 0;
      go = __all_sync(0xFFFFFFFFu, biattn_tc::wait_bar(full + 8 * s, ph, sy));
      if (!go) break;
      const int64_t slot = slots[s];
      const uint8_t* stage = smem + size_t(s) * stage_bytes;
      if (slot >= 0) {
        ln.angles(reinterpret_cast<const float*>(stage + row_bytes));
        const uint16_t* row = reinterpret_cast<const uint16_t*>(stage);
        for (int h = g; h < H; h += groups)
          ln.finish(p, h, t, slot, true, *reinterpret_cast<const uint2*>(row + h * D + ln.da),
                    *reinterpret_cast<const uint2*>(row + h * D + ln.db));
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(empty + 8 * s);
      if (++s == NS) s = 0, ph ^= 1u;
    }
  }
  __syncthreads();
  if (gave_up) {                     // let every copy in flight land before the block leaves
    const uint64_t t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < 2000000ull) {
    }
  }
}

using Kernel = void (*)(const Params);
inline Kernel kernel_of(int D, bool interleaved) {
  if (D == 128) return interleaved ? qkrope_kernel<128, true> : qkrope_kernel<128, false>;
  return interleaved ? qkrope_kernel<64, true> : qkrope_kernel<64, false>;
}
inline Kernel ring_kernel_of(int D, bool interleaved) {
  if (D == 128) return interleaved ? qkrope_ring_kernel<128, true> : qkrope_ring_kernel<128, false>;
  return interleaved ? qkrope_ring_kernel<64, true> : qkrope_ring_kernel<64, false>;
}

}  // namespace biqkr

struct bi_qkrope {
  int Hq = 0, Hkv = 0, D = 0, page_size = 0, rot = 0, interleaved = 0;
  float eps = 0.0f;
  int device = 0, groups_log2 = 0, per_block = 0;
  int ring = 0, ring_ctas = 0;      // stages and resident blocks of the form for many tokens (0: none),
  int team_log2 = 0;                // its warps per token
  int ring_from = 0;                // and the tokens from which it runs
  size_t ring_smem = 0;
  uint32_t* d_status = nullptr;
};

BI_GEMM_API int bi_qkrope_create(bi_qkrope_t* out, int64_t num_q_heads, int64_t num_kv_heads, int64_t head_dim,
                                 int64_t page_size, int64_t rot_dim, int32_t interleaved, float eps) {
  if (!out) return BI_GEMM_ERR_INVALID_ARG;
  *out = nullptr;
  if (!std::isfinite(eps) || eps < 0.0f || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || page_size <= 0 ||
      rot_dim <= 0 || interleaved < 0 || interleaved > 1)
    return BI_GEMM_ERR_INVALID_ARG;
  if ((head_dim != 64 && head_dim != 128) || rot_dim % 16 != 0 || rot_dim > head_dim || page_size > (1 << 20) ||
      num_q_heads > 4096 || num_kv_heads > 4096 || num_q_heads + 2 * num_kv_heads > 4096)
    return BI_GEMM_ERR_UNSUPPORTED;
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  if (major != 10 || minor != 3) return BI_GEMM_ERR_UNSUPPORTED;
  bi_qkrope* h = new (std::nothrow) bi_qkrope();
  if (!h) return BI_GEMM_ERR_OOM;
  h->Hq = int(num_q_heads);
  h->Hkv = int(num_kv_heads);
  h->D = int(head_dim);
  h->page_size = int(page_size);
  h->rot = int(rot_dim);
  h->interleaved = interleaved;
  h->eps = eps;
  h->device = dev;
  // lane groups per token: the power of two that leaves a group kHeads heads or fewer, up to a block
  const int groups = biqkr::kThreads / (h->D / 8), heads = h->Hq + 2 * h->Hkv;
  while ((1 << h->groups_log2) < groups && (biqkr::kHeads << h->groups_log2) < heads) ++h->groups_log2;
  h->per_block = groups >> h->groups_log2;
  // the ring: as many tokens' rows and angles as its room holds, at least three
  const size_t stage = size_t(heads) * h->D * 2 + size_t(h->rot) * 4;
  const int ring = int(std::min<size_t>(biqkr::kMaxRing, biqkr::kRingBytes / stage));
  // warps per token: the power of two that leaves a lane group kHeads heads or fewer
  while (h->team_log2 < 3 && ((32 / (h->D / 8) * biqkr::kHeads) << h->team_log2) < heads) ++h->team_log2;
  if (ring >= 3) {
    int sms = 0, per_sm = 0;
    h->ring = ring;
    h->ring_smem = ring * stage;
    const auto fn = biqkr::ring_kernel_of(h->D, interleaved != 0);
    // (the attribute is the kernel's, shared by every handle: the most any of them needs)
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, biqkr::kRingBytes) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, biqkr::kThreads + 32, h->ring_smem) !=
            cudaSuccess ||
        per_sm < 1) {
      cudaGetLastError();
      delete h;
      return BI_GEMM_ERR_CUDA;
    }
    h->ring_ctas = per_sm * sms;
    const int64_t row = int64_t(heads) * h->D * 2;
    h->ring_from = int((int64_t(biqkr::kRingRows) * h->ring_ctas + row - 1) / row);
  }
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

namespace {

// bi_qkrope_run with the failure injection of the test controls (stall >= 0: that block of the form for
// many tokens loads nothing) and the limit of its waits.
int qkrope_run(bi_qkrope* h, const void* qkv, int64_t T, int64_t qkv_stride, const void* gq, const void* gk,
               const float* cos_sin, int64_t num_positions, const int32_t* q_seq, const int32_t* q_pos, void* k_cache,
               void* v_cache, int64_t num_pages, const int32_t* page_table, int64_t num_seqs, int64_t max_pages,
               void* q_out, void* stream, int32_t stall, uint64_t timeout_ns) {
  if (!h || T < 0 || num_positions < 0 || num_pages < 0 || num_seqs < 0 || max_pages < 0 || !gq != !gk)
    return BI_GEMM_ERR_INVALID_ARG;
  if (T == 0) return BI_GEMM_OK;
  if (!qkv || !cos_sin || !q_seq || !q_pos || !k_cache || !v_cache || !page_table || !q_out)
    return BI_GEMM_ERR_INVALID_ARG;
  if (qkv_stride % 8 != 0 || qkv_stride < int64_t(h->Hq + 2 * h->Hkv) * h->D || T > (int64_t(1) << 30))
    return BI_GEMM_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(qkv) | reinterpret_cast<uintptr_t>(gq) | reinterpret_cast<uintptr_t>(gk) |
       reinterpret_cast<uintptr_t>(cos_sin) | reinterpret_cast<uintptr_t>(k_cache) |
       reinterpret_cast<uintptr_t>(v_cache) | reinterpret_cast<uintptr_t>(q_out)) & 15u)
    return BI_GEMM_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(q_seq) | reinterpret_cast<uintptr_t>(q_pos) |
       reinterpret_cast<uintptr_t>(page_table)) & 3u)
    return BI_GEMM_ERR_ALIGNMENT;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  if (dev != h->device) return BI_GEMM_ERR_INVALID_ARG;
  biqkr::Params p;
  std::memset(&p, 0, sizeof(p));
  p.qkv = static_cast<const uint16_t*>(qkv);
  p.gq = static_cast<const uint16_t*>(gq);
  p.gk = static_cast<const uint16_t*>(gk);
  p.cs = cos_sin;
  p.q_seq = q_seq;
  p.q_pos = q_pos;
  p.table = page_table;
  p.kc = static_cast<uint16_t*>(k_cache);
  p.vc = static_cast<uint16_t*>(v_cache);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.status = h->d_status;
  p.T = T;
  p.stride = qkv_stride;
  p.num_positions = num_positions;
  p.num_pages = num_pages;
  p.B = num_seqs;
  p.max_pages = max_pages;
  p.Hq = h->Hq;
  p.Hkv = h->Hkv;
  p.page_size = h->page_size;
  p.rot = h->rot;
  p.groups_log2 = h->groups_log2;
  p.eps = h->eps;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  // The ring from 40 KB of rows per resident block on, where its start is paid for (us, ring against a
  // block per token or few): 32/8 heads of 128 (12 KB a token), 1216 tokens 9.8 against 9.4, 2432 16.5
  // against 17.7, 8192 42.0 against 52.3; 16/8 of 128, 2432 11.3 against 11.2, 4096 16.9 against 17.8;
  // 16/2 of 64, 8192 15.2 against 14.9, 12000 19.6 against 19.9.
  const bool ring = h->ring_from > 0 && T >= h->ring_from;
  p.ring = h->ring;
  p.team_log2 = h->team_log2;
  p.stall = stall;
  p.timeout_ns = timeout_ns;
  cfg.gridDim = dim3(unsigned(ring ? h->ring_ctas : (T + h->per_block - 1) / h->per_block));
  cfg.blockDim = dim3(biqkr::kThreads + (ring ? 32 : 0));
  cfg.dynamicSmemBytes = ring ? h->ring_smem : 0;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto fn = ring ? biqkr::ring_kernel_of(h->D, h->interleaved != 0) : biqkr::kernel_of(h->D, h->interleaved != 0);
  if (cudaLaunchKernelEx(&cfg, fn, p) != cudaSuccess) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  return BI_GEMM_OK;
}

}  // namespace

BI_GEMM_API int bi_qkrope_run(bi_qkrope_t h, const void* qkv, int64_t T, int64_t qkv_stride, const void* gq,
                              const void* gk, const float* cos_sin, int64_t num_positions, const int32_t* q_seq,
                              const int32_t* q_pos, void* k_cache, void* v_cache, int64_t num_pages,
                              const int32_t* page_table, int64_t num_seqs, int64_t max_pages, void* q_out,
                              void* stream) {
  return qkrope_run(h, qkv, T, qkv_stride, gq, gk, cos_sin, num_positions, q_seq, q_pos, k_cache, v_cache, num_pages,
                    page_table, num_seqs, max_pages, q_out, stream, -1, biattn_tc::kTimeoutNs);
}

BI_GEMM_API int bi_qkrope_get_device_error(bi_qkrope_t h, void* stream) {
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

BI_GEMM_API int bi_qkrope_get_config(bi_qkrope_t h, bi_qkrope_config* c) {
  if (!h || !c) return BI_GEMM_ERR_INVALID_ARG;
  c->num_q_heads = h->Hq;
  c->num_kv_heads = h->Hkv;
  c->head_dim = h->D;
  c->page_size = h->page_size;
  c->rot_dim = h->rot;
  c->interleaved = h->interleaved;
  c->threads = biqkr::kThreads;
  c->tokens_per_block = h->per_block;
  c->ring_tokens = h->ring;
  c->ring_ctas = h->ring_ctas;
  c->ring_from = h->ring_from;
  return BI_GEMM_OK;
}

BI_GEMM_API int bi_qkrope_destroy(bi_qkrope_t h) {
  if (!h) return BI_GEMM_OK;
  if (h->d_status) cudaFree(h->d_status);
  delete h;
  return BI_GEMM_OK;
}
