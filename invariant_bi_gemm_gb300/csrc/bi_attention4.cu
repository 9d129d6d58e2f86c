// bi_attention4.cu — batch-invariant decode attention over a paged KV cache in 4 bits, and the expansion of its
// pages, for sm_103a.  Implements include/bi_attention4.h.
//
// A unit is (token, split) and up to eight KV heads side by side, HB of them; a block of eight computing warps and a
// loading one runs it.  A computing warp has one head and, where HB is below eight, every 8 / HB-th sixteen of the split's
// positions; it keeps a running maximum reference, a sum and the weighted values of its positions, and writes them as one
// of the split's 8 / HB parts: the computing warps never wait for one another.  The loading warp copies whole
// stages (sixteen positions for each of the eight warps, 18 KB at 128 dimensions, all of the HB heads' bytes of a row
// together) into a ring with cp.async, looking its pages up a stage ahead.
//
// Per step of two stages, with g = lane / 4 and t = lane % 4 (mma.sync m16n8k16, f16 in, fp32 accumulate; the G <= 8 query
// heads of the KV head on the columns):
//   scores  S^T = K Q^T: 16 positions on the rows.  The order of the products' dimensions is free as long as both
//           operands agree, so lane t takes a quarter of a row, whole 16-byte chunks: eight codes become four f16
//           pairs by cvt, times their block's scale (exact: 2 + 4 significant bits).
//   weights P = 2^(s - m + 7) in fp32, rounded to f16 and transposed in registers (movmatrix).
//   values  O^T += V^T P^T: 16 dimensions on the rows, 16 positions deep.  Lane g owns D / 8 consecutive
//           dimensions, lane t the positions 2t, 2t + 1, 2t + 8, 2t + 9 of each sixteen: the codes of two
//           positions are interleaved before cvt, so that a pair of f16 is one dimension at two positions.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>

#include "../../include/bi_attention4.h"
#include "attn_ptx.cuh"
#include "fp4.cuh"

#ifndef BI_GEMM_API
#define BI_GEMM_API extern "C" __attribute__((visibility("default")))
#endif

namespace biattn4 {

namespace ptx = bigemm::ptx;
using biattn_tc::ex2;

constexpr int kWarps = 8, kThreads = 32 * (kWarps + 1);
constexpr int kBlocksPerSm = 2;
constexpr int kMaxStages = 8;
constexpr int kTokens = 512;              // of a launch
constexpr int kSplitPerPart = 256;        // a split by default, for each of its parts
constexpr int kMergeWarps = 8;
constexpr float kLift = 7.0f;             // weights are 2^7 at the reference, 2^15 at most
constexpr float kSlack = 8.0f;            // the reference moves when a score passes it by more
constexpr uint32_t kErrInput = 1u, kErrPage = 2u, kErrBound = 4u;      // (8: a wait that timed out)

struct Params {
  const uint16_t* q;
  const int32_t* q_seq;
  const int32_t* q_pos;
  const uint8_t* kc;
  const uint8_t* ks;
  const uint8_t* vc;
  const uint8_t* vs;
  const int32_t* table;
  uint16_t* o;
  float* part;        // [T, Hkv, max_parts, G, D] partial weighted sums
  float* ml;          // [T, Hkv, max_parts, G, 2] (reference, sum; the sum of a part without positions is 0)
  uint32_t* status;
  int64_t num_pages, max_pages, B;
  int32_t T, Hq, Hkv, G, page_size, split, max_pos;
  int32_t parts;      // of a split: 8 / HB
  int32_t max_parts;  // of a token
  uint32_t page_mul;  // pos / page_size = pos * page_mul >> page_shift for pos < 2^30
  int32_t page_shift;
  int32_t stall;      // failure injection (test controls only): this block loads nothing
  uint64_t timeout_ns;
  float c;            // scale * k_scale * log2(e)
  float v_scale;
};

template <int D, int HB>
struct Cfg {
  static constexpr int CODES = D / 2, SCALES = D / 16;           // bytes of a head's row
  static constexpr int GROUPS = kWarps / HB, POS = 16 * GROUPS;  // positions of a stage
  // Rows in shared memory are padded so that the rows a load takes at once (eight apart by one for the keys, four apart
  // by two for the values) are on different banks.
  static constexpr int KROW = HB * CODES + (HB > 1 ? CODES : 0), VROW = HB * CODES + 16, SROW = HB * SCALES;
  static constexpr int OFF_V = POS * KROW, OFF_KS = OFF_V + POS * VROW, OFF_VS = OFF_KS + POS * SROW;
  static constexpr int STAGE = OFF_VS + POS * SROW;
  static constexpr int TABLES = (3 * kTokens + 1 + kWarps + 1) * 4, BARS = 2 * kMaxStages * 8 + 16;
  static constexpr int ROOM = 228 * 1024 / kBlocksPerSm - 1024 - TABLES - BARS;
  static constexpr int STAGES = ROOM / STAGE < kMaxStages ? ROOM / STAGE : kMaxStages;
  static_assert(STAGES >= 4 && STAGE % 16 == 0, "ring");
  static constexpr int OFF_BAR = STAGES * STAGE, OFF_CUM = OFF_BAR + BARS, SMEM = OFF_CUM + TABLES;
  // copies of the codes: chunks of 16 bytes, CH of them a row, ROWS rows an instruction, COPIES of these a stage
  static constexpr int CH = HB * CODES / 16, ROWS = 32 / CH, COPIES = POS / ROWS;
  // and of the scales, in pieces of SU bytes
  static constexpr int SU = SROW < 16 ? SROW : 16, SCH = SROW / SU, SROWS = 32 / SCH, SCOPIES = (POS + SROWS - 1) / SROWS;
  static constexpr int LOOKUPS = (POS + 31) / 32;                // positions a lane looks up
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_zfill(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(bytes), "n"(N) : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
struct Unit {
  int32_t v, t, split, first, last;   // the v-th (token, split) and its positions (last < first: none)
};

// Splits of a token: one for an empty place, none for one that cannot be served (which `report` says).
__device__ __forceinline__ int32_t splits_of(const Params& p, int32_t b, int32_t pos, bool report) {
  if (pos == -1) return 1;
  uint32_t bad = 0;
  if (b < 0 || b >= p.B || pos < 0 || int64_t(pos / p.page_size) >= p.max_pages) bad = kErrInput;
  else if (pos > p.max_pos) bad = kErrBound;
  if (bad && report) atomicOr(p.status, bad);
  return bad ? 0 : pos / p.split + 1;
}

template <int D, int HB>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) attn_kernel(const Params p) {
  using C = Cfg<D, HB>;
  extern __shared__ __align__(128) uint8_t smem[];
  int32_t* cum = reinterpret_cast<int32_t*>(smem + C::OFF_CUM);
  int32_t* seqs = cum + kTokens + 1;                     // the tokens' requests and positions
  int32_t* poss = seqs + kTokens;
  int32_t* sums = poss + kTokens;
  uint32_t* gave_up = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 2 * kMaxStages * 8);
  const uint32_t bars = ptx::smem_u32(smem + C::OFF_BAR);
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kMaxStages + s); };
  const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  if (tid == 0) {
    *gave_up = 0u;
    for (int s = 0; s < C::STAGES; ++s) {
      ptx::mbar_init(full(s), 32);
      ptx::mbar_init(empty(s), kWarps);
    }
    ptx::fence_barrier_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // first split of every token
  int32_t carry = 0;
  for (int base = 0; base < p.T; base += kThreads) {
    const int i = base + tid;
    int32_t n = 0;
    if (i < p.T) {
      seqs[i] = p.q_seq[i];
      poss[i] = p.q_pos[i];
      n = splits_of(p, seqs[i], poss[i], blockIdx.x == 0);
    }
    int32_t x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int32_t before = carry;
#pragma unroll
    for (int w = 0; w <= kWarps; ++w) {
      const int32_t s = sums[w];
      if (w < warp) before += s;
      carry += s;
    }
    if (i < p.T) cum[i] = before + x - n;
    __syncthreads();
  }
  if (tid == 0) cum[p.T] = carry;
  __syncthreads();

  // Block (chain, heads) takes a run of consecutive (token, split) of its heads, so that a token's query is prepared once
  // for its splits there.
  const int32_t blocks = p.Hkv / HB, kh0 = int32_t(blockIdx.x % uint32_t(blocks)) * HB;
  const int32_t chain = int32_t(blockIdx.x / uint32_t(blocks)), chains = int32_t(gridDim.x / uint32_t(blocks));
  const int32_t v_end = int32_t(int64_t(carry) * (chain + 1) / chains);
  auto locate = [&](Unit& r) {                           // t: cum[t] <= v < cum[t + 1]
    for (;;) {
      const int i = r.t + 1 + lane;
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, i >= p.T || cum[i] > r.v);
      if (past) {
        r.t += __ffs(past) - 1;
        break;
      }
      r.t += 32;
    }
    r.split = r.v - cum[r.t];
    r.first = r.split * p.split;
    r.last = min(poss[r.t], r.first + p.split - 1);
  };
  auto start = [&](Unit& r) {
    r.v = int32_t(int64_t(carry) * chain / chains);
    r.t = 0;
    if (r.v < v_end) locate(r);
  };
  auto advance = [&](Unit& r) {
    if (++r.v < v_end) locate(r);
  };
  const biattn_tc::Sync sy{gave_up, p.status, p.timeout_ns};

  if (warp == kWarps) {
    // ---- loads.  A lane looks up positions lane, lane + 32, ... of a stage; a row's place comes from its lane (fewer than
    // 2^32 - 1 rows: the host).
    Unit L;
    int32_t pos = 0, page[C::LOOKUPS], in_page[C::LOOKUPS];
    auto fetch = [&]() {
#pragma unroll
      for (int k = 0; k < C::LOOKUPS; ++k) {
        const int32_t at = min(pos + 32 * k + (C::POS < 32 ? lane & (C::POS - 1) : lane), L.last);
        const int32_t pg = int32_t((uint64_t(uint32_t(at)) * p.page_mul) >> p.page_shift);
        in_page[k] = at - pg * p.page_size;
        page[k] = __ldg(p.table + int64_t(seqs[L.t]) * p.max_pages + pg);
      }
    };
    auto seek = [&]() {                                  // the next unit, from L on, that has positions
      for (; L.v < v_end; advance(L)) {
        pos = L.first;
        if (pos <= L.last) {
          fetch();
          return true;
        }
      }
      return false;
    };
    const uint8_t* kc = p.kc + int64_t(kh0) * C::CODES + (lane % C::CH) * 16;
    const uint8_t* vc = p.vc + int64_t(kh0) * C::CODES + (lane % C::CH) * 16;
    const uint8_t* ks = p.ks + int64_t(kh0) * C::SCALES + (lane % C::SCH) * C::SU;
    const uint8_t* vs = p.vs + int64_t(kh0) * C::SCALES + (lane % C::SCH) * C::SU;
    const int row = lane / C::CH, srow = lane / C::SCH;
    const uint32_t to = ptx::smem_u32(smem), ch = uint32_t(lane % C::CH) * 16, sch = uint32_t(lane % C::SCH) * C::SU;
    const uint32_t pitch = uint32_t(p.Hkv) * C::CODES, spitch = uint32_t(p.Hkv) * C::SCALES;
    int s = 0;
    uint32_t ph = 0;
    start(L);
    for (bool more = seek(); more;) {
      if (!__all_sync(0xFFFFFFFFu, biattn_tc::wait_bar(empty(s), ph ^ 1u, sy))) break;
      uint32_t at[C::LOOKUPS];
      bool whole = true;
#pragma unroll
      for (int k = 0; k < C::LOOKUPS; ++k) {
        const bool here = pos + 32 * k + (C::POS < 32 ? lane & (C::POS - 1) : lane) <= L.last;
        const bool good = page[k] >= 0 && page[k] < p.num_pages;
        if (here && !good) atomicOr(p.status, kErrPage);
        at[k] = here && good ? uint32_t(int64_t(page[k]) * p.page_size + in_page[k]) : 0xFFFFFFFFu;
        whole = whole && here && good;
      }
      const uint32_t dst = to + uint32_t(s) * C::STAGE;
      // a row's number, from the lane that looked it up
      auto of = [&](int r0, int r) { return __shfl_sync(0xFFFFFFFFu, at[r0 / 32], (r0 + r) & 31); };
      if (int(blockIdx.x) == p.stall) {
      } else if (__all_sync(0xFFFFFFFFu, whole)) {
#pragma unroll
        for (int i = 0; i < C::COPIES; ++i) {
          const uint64_t off = uint64_t(of(i * C::ROWS, row)) * pitch;
          const int r = i * C::ROWS + row;
          cp_async_16(dst + uint32_t(r * C::KROW) + ch, kc + off);
          cp_async_16(dst + uint32_t(C::OFF_V + r * C::VROW) + ch, vc + off);
        }
#pragma unroll
        for (int i = 0; i < C::SCOPIES; ++i) {
          const uint64_t off = uint64_t(of(i * C::SROWS, srow)) * spitch;
          const int r = i * C::SROWS + srow;
          if (C::POS >= C::SROWS || r < C::POS) {
            cp_async<C::SU>(dst + uint32_t(C::OFF_KS + r * C::SROW) + sch, ks + off);
            cp_async<C::SU>(dst + uint32_t(C::OFF_VS + r * C::SROW) + sch, vs + off);
          }
        }
      } else {
        // the last stage of a token, or a page that is not there: zeros in its place
#pragma unroll
        for (int i = 0; i < C::COPIES; ++i) {
          const uint32_t x = of(i * C::ROWS, row), n = x != 0xFFFFFFFFu ? 16u : 0u;
          const uint64_t off = n ? uint64_t(x) * pitch : 0;
          const int r = i * C::ROWS + row;
          ptx::cp_async_16(dst + uint32_t(r * C::KROW) + ch, kc + off, n);
          ptx::cp_async_16(dst + uint32_t(C::OFF_V + r * C::VROW) + ch, vc + off, n);
        }
#pragma unroll
        for (int i = 0; i < C::SCOPIES; ++i) {
          const uint32_t x = of(i * C::SROWS, srow), n = x != 0xFFFFFFFFu ? uint32_t(C::SU) : 0u;
          const uint64_t off = n ? uint64_t(x) * spitch : 0;
          const int r = i * C::SROWS + srow;
          if (C::POS >= C::SROWS || r < C::POS) {
            cp_async_zfill<C::SU>(dst + uint32_t(C::OFF_KS + r * C::SROW) + sch, ks + off, n);
            cp_async_zfill<C::SU>(dst + uint32_t(C::OFF_VS + r * C::SROW) + sch, vs + off, n);
          }
        }
      }
      if (int(blockIdx.x) != p.stall)
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full(s)) : "memory");
      if (++s == C::STAGES) s = 0, ph ^= 1u;
      pos += C::POS;
      if (pos <= L.last) {
        fetch();
      } else {
        advance(L);
        more = seek();
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }

  // ---- products
  const int hh = warp % HB, group = warp / HB;
  const int32_t kh = kh0 + hh;
  int s = 0;
  uint32_t ph = 0;
  int32_t token = -1;
  uint32_t qf[D / 8];
  float fac[2] = {0.0f, 0.0f};
  Unit U;
  for (start(U); U.v < v_end; advance(U)) {
    // the query in f16, relative to its head's largest element
    if (U.t != token) {
      token = U.t;
      const uint16_t* src = p.q + (int64_t(U.t) * p.Hq + kh * p.G + g) * D + t4 * (D / 4);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 v = g < p.G ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
        qf[4 * i] = v.x, qf[4 * i + 1] = v.y, qf[4 * i + 2] = v.z, qf[4 * i + 3] = v.w;
      }
      uint32_t most = bifp4::most_of(qf, D / 8);
      most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
      most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
      // times 2^11 / 2^exponent of the largest element (within fp32's range): sizes below 2^12
      const int e = min(max(int(most >> 7), 12), 254);
      const float up = __uint_as_float(uint32_t(265 - e) << 23), down = __uint_as_float(uint32_t(e - 11) << 23);
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        qf[i] = pack_f16x2(__uint_as_float(qf[i] << 16) * up, __uint_as_float(qf[i] & 0xFFFF0000u) * up);
      // the factors of the two heads whose scores this lane has
      // (above zero, so that a hidden position's -inf stays one)
      fac[0] = fmaxf(__fmul_rn(__shfl_sync(0xFFFFFFFFu, down, 8 * t4), p.c), 1e-45f);
      fac[1] = fmaxf(__fmul_rn(__shfl_sync(0xFFFFFFFFu, down, 8 * t4 + 4), p.c), 1e-45f);
    }
    // (the reference m is a product's sum as it comes from the MMA; the difference to it is taken before the factor, so
    // that it is exact near the reference however large the scores are)
    float acc[D / 16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    bool ok = true;
    for (int32_t pos = U.first; pos <= U.last; pos += 2 * C::POS) {
      // two stages, or the unit's last one (then its sixteen positions twice, hidden the second time)
      const bool two = pos + C::POS <= U.last;
      const int s1 = s + 1 == C::STAGES ? 0 : s + 1;
      const uint32_t ph1 = s1 == 0 ? ph ^ 1u : ph;
      ok = __all_sync(0xFFFFFFFFu, biattn_tc::wait_bar(full(s), ph, sy) && (!two || biattn_tc::wait_bar(full(s1), ph1, sy)));
      if (!ok) break;
      const int32_t mine = pos + 16 * group;              // this warp's sixteen of the first stage
      if (mine <= U.last) {
        const uint8_t* src0 = smem + s * C::STAGE;
        const uint8_t* src1 = two ? smem + s1 * C::STAGE : src0;
        // scores: two sixteens of positions side by side, for two chains of products
        constexpr int W = D / 32;                         // words of codes a lane has of a row
        float x2[2][4];
        uint32_t kw[4][W], ksc[4][2];                     // rows g, g + 8 of either
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint8_t* src = r < 2 ? src0 : src1;
          const int at = 16 * group + 8 * (r & 1) + g;
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(src + at * C::KROW + hh * C::CODES + t4 * 16);
            kw[r][0] = v.x, kw[r][1] = v.y, kw[r][2] = v.z, kw[r][3] = v.w;
            const uint32_t b =
                bifp4::e4m3_pair(*reinterpret_cast<const uint16_t*>(src + C::OFF_KS + at * C::SROW + hh * C::SCALES + 2 * t4));
            ksc[r][0] = __byte_perm(b, b, 0x1010), ksc[r][1] = __byte_perm(b, b, 0x3232);
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(src + at * C::KROW + hh * C::CODES + t4 * 8);
            kw[r][0] = v.x, kw[r][1] = v.y;
            const uint32_t b = bifp4::e4m3_pair(src[C::OFF_KS + at * C::SROW + hh * C::SCALES + t4]);
            ksc[r][0] = ksc[r][1] = __byte_perm(b, b, 0x1010);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) x2[h][j] = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t x[4], y[4];
            bifp4::values8(kw[2 * h][i], x);
            bifp4::values8(kw[2 * h + 1][i], y);
            const int k = i * 2 / W;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = mul_f16x2(x[j], ksc[2 * h][k]), y[j] = mul_f16x2(y[j], ksc[2 * h + 1][k]);
            mma(x2[h], x[0], y[0], x[1], y[1], qf[4 * i], qf[4 * i + 1]);
            mma(x2[h], x[2], y[2], x[3], y[3], qf[4 * i + 2], qf[4 * i + 3]);
          }
        }
        if (!two || mine + C::POS + 15 > U.last) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (mine + h * C::POS + 8 * (j >> 1) + g > U.last) x2[h][j] = -INFINITY;
        }
        bool move = false;
        float top[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          top[j] = fmaxf(fmaxf(x2[0][j], x2[0][j + 2]), fmaxf(x2[1][j], x2[1][j + 2]));
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) top[j] = fmaxf(top[j], __shfl_xor_sync(0xFFFFFFFFu, top[j], o));
          move |= __fmul_rn(__fsub_rn(top[j], m[j]), fac[j]) > kSlack;
        }
        if (__any_sync(0xFFFFFFFFu, move)) {              // (a head's rule looks at that head alone)
          float f[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const bool mv = __fmul_rn(__fsub_rn(top[j], m[j]), fac[j]) > kSlack;
            f[j] = mv ? ex2(__fmul_rn(__fsub_rn(m[j], top[j]), fac[j])) : 1.0f;
            if (mv) m[j] = top[j];
            l[j] *= f[j];
          }
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] *= f[j & 1];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* src = h == 0 ? src0 : src1;
#pragma unroll
          for (int j = 0; j < 4; ++j) x2[h][j] = ex2(__fmaf_rn(__fsub_rn(x2[h][j], m[j & 1]), fac[j & 1], kLift));
          l[0] += x2[h][0] + x2[h][2];
          l[1] += x2[h][1] + x2[h][3];
          const uint32_t b0 = transposed(pack_f16x2(x2[h][0], x2[h][1])), b1 = transposed(pack_f16x2(x2[h][2], x2[h][3]));
          constexpr int WV = D / 64;                      // words of codes a lane has of a row
          uint32_t w[4][WV], sc[2];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int at = 16 * group + 2 * t4 + (r & 1) + 8 * (r >> 1);
            const uint8_t* a = src + C::OFF_V + at * C::VROW + hh * C::CODES + g * (C::CODES / 8);
            if constexpr (D == 128) {
              const uint2 v = *reinterpret_cast<const uint2*>(a);
              w[r][0] = v.x, w[r][1] = v.y;
            } else {
              w[r][0] = *reinterpret_cast<const uint32_t*>(a);
            }
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint8_t* a =
                src + C::OFF_VS + (16 * group + 2 * t4 + 8 * r) * C::SROW + hh * C::SCALES + (D == 128 ? g : g >> 1);
            sc[r] = bifp4::e4m3_pair(uint32_t(a[0]) | uint32_t(a[C::SROW]) << 8);
          }
#pragma unroll
          for (int i = 0; i < WV; ++i) {
            // even and odd dimensions of the lane's eight, a pair of positions each
            uint32_t x0[4], x1[4], y0[4], y1[4];
            constexpr uint32_t LO = 0x0F0F0F0Fu;
            bifp4::values8((w[0][i] & LO) | ((w[1][i] << 4) & ~LO), x0);
            bifp4::values8(((w[0][i] >> 4) & LO) | (w[1][i] & ~LO), x1);
            bifp4::values8((w[2][i] & LO) | ((w[3][i] << 4) & ~LO), y0);
            bifp4::values8(((w[2][i] >> 4) & LO) | (w[3][i] & ~LO), y1);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma(acc[4 * i + j], mul_f16x2(x0[j], sc[0]), mul_f16x2(x1[j], sc[0]), mul_f16x2(y0[j], sc[1]),
                  mul_f16x2(y1[j], sc[1]), b0, b1);
          }
        }
      }
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(empty(s));
        if (two) ptx::mbar_arrive(empty(s1));
      }
      s = two ? s1 : s, ph = two ? ph1 : ph;
      if (++s == C::STAGES) s = 0, ph ^= 1u;
    }
    if (!ok) break;
    // ---- the part, or the token's result where it has no other
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[j] = __fadd_rn(l[j], __shfl_xor_sync(0xFFFFFFFFu, l[j], o));
    const bool alone = C::GROUPS == 1 && U.split == 0 && U.last == poss[U.t];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int head = 2 * t4 + j;
      if (head >= p.G) continue;
      if (alone) {
        const bool none = U.last < 0;
        const float f = none ? 0.0f : __fdiv_rn(p.v_scale, l[j]);
        uint16_t* dst = p.o + (int64_t(U.t) * p.Hq + kh * p.G + head) * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          *reinterpret_cast<uint2*>(dst + 4 * i) =
              make_uint2(ptx::pack_bf16x2(__fmul_rn(acc[2 * i][j], f), __fmul_rn(acc[2 * i][j + 2], f)),
                         ptx::pack_bf16x2(__fmul_rn(acc[2 * i + 1][j], f), __fmul_rn(acc[2 * i + 1][j + 2], f)));
      } else {
        const int64_t at =
            ((int64_t(U.t) * p.Hkv + kh) * p.max_parts + U.split * C::GROUPS + group) * p.G + head;
        float* dst = p.part + at * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          *reinterpret_cast<float4*>(dst + 4 * i) =
              make_float4(acc[2 * i][j], acc[2 * i][j + 2], acc[2 * i + 1][j], acc[2 * i + 1][j + 2]);
        if (g == 0) *reinterpret_cast<float2*>(p.ml + at * 2) = make_float2(__fmul_rn(m[j], fac[j]), l[j]);
      }
    }
  }
}

// The parts of a token's query head, a block each: warp w sums the w-th of eight consecutive groups of ceil(n / 8)
// parts, ascending; the groups are added in order.
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_kernel(const Params p) {
  constexpr int PER = D / 32;                             // dimensions a lane
  __shared__ float sums[kMergeWarps][D];
  __shared__ float2 mls[kMergeWarps];
  const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int32_t t = int32_t(blockIdx.x / p.Hq), h = int32_t(blockIdx.x - uint32_t(t) * p.Hq);
  const int32_t pos = p.q_pos[t], n = splits_of(p, p.q_seq[t], pos, false) * p.parts;
  if (n <= 1) return;                                     // written by its unit, or refused
  if (pos < 0) {                                          // an empty place
    if (int(threadIdx.x) < D / 2) *reinterpret_cast<uint32_t*>(p.o + (int64_t(t) * p.Hq + h) * D + 2 * threadIdx.x) = 0u;
    return;
  }
  const int32_t kh = h / p.G, hd = h - kh * p.G;
  const int64_t slot0 = (int64_t(t) * p.Hkv + kh) * p.max_parts * p.G + hd;
  const int32_t c = (n + kMergeWarps - 1) / kMergeWarps, s0 = min(n, warp * c), s1 = min(n, s0 + c);
  const float2* mlp = reinterpret_cast<const float2*>(p.ml) + slot0;
  float M = -INFINITY;
  for (int32_t s = s0 + lane; s < s1; s += 32) M = fmaxf(M, mlp[int64_t(s) * p.G].x);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  float L = 0.0f, A[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) A[i] = 0.0f;
  constexpr int BATCH = 8;
  for (int32_t b = s0; b < s1; b += BATCH) {
    float2 ml[BATCH];
    float v[BATCH][PER];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      if (b + i < s1) {
        ml[i] = mlp[int64_t(b + i) * p.G];
        const float* src = p.part + (slot0 + int64_t(b + i) * p.G) * D + lane * PER;
        if constexpr (PER == 4) {
          const float4 x = *reinterpret_cast<const float4*>(src);
          v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(src);
          v[i][0] = x.x, v[i][1] = x.y;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      if (b + i < s1) {
        const float f = ml[i].y == 0.0f ? 0.0f : ex2(__fsub_rn(ml[i].x, M));   // (a part without positions)
        L = __fmaf_rn(ml[i].y, f, L);
#pragma unroll
        for (int j = 0; j < PER; ++j) A[j] = __fmaf_rn(v[i][j], f, A[j]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) sums[warp][lane * PER + j] = A[j];
  if (lane == 0) mls[warp] = make_float2(M, L);
  __syncthreads();
  if (int(threadIdx.x) < D / 2) {
    float top = -INFINITY, Ls = 0.0f, a0 = 0.0f, a1 = 0.0f;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) top = fmaxf(top, mls[w].x);
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
      if (w * c < n) {                                    // (a group of no parts adds nothing)
        const float f = mls[w].y == 0.0f ? 0.0f : ex2(__fsub_rn(mls[w].x, top));
        Ls = __fmaf_rn(mls[w].y, f, Ls);
        a0 = __fmaf_rn(sums[w][2 * threadIdx.x], f, a0);
        a1 = __fmaf_rn(sums[w][2 * threadIdx.x + 1], f, a1);
      }
    }
    const float f = __fdiv_rn(p.v_scale, Ls);
    *reinterpret_cast<uint32_t*>(p.o + (int64_t(t) * p.Hq + h) * D + 2 * threadIdx.x) =
        ptx::pack_bf16x2(__fmul_rn(a0, f), __fmul_rn(a1, f));
  }
}

struct ExpandParams {
  const uint8_t* kc;
  const uint8_t* ks;
  const uint8_t* vc;
  const uint8_t* vs;
  const int32_t* pages;
  uint16_t* ko;
  uint16_t* vo;
  uint32_t* status;
  int64_t num_pages, blocks;              // blocks of sixteen elements in all
  int64_t per_page;                       // and of a page
  float k_scale, v_scale;
};

__global__ void __launch_bounds__(256) expand_kernel(const ExpandParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= p.blocks) return;
  const int64_t n = i / p.per_page, r = i - n * p.per_page;
  const int64_t page = p.pages[n];
  if (page < 0 || page >= p.num_pages) {
    if (page != -1 && r == 0) atomicOr(p.status, kErrPage);
    return;
  }
  const int64_t at = page * p.per_page + r;
  const uint2 kc = *reinterpret_cast<const uint2*>(p.kc + at * 8), vc = *reinterpret_cast<const uint2*>(p.vc + at * 8);
  const float ks = bifp4::scale_value<true>(p.ks[at], p.k_scale), vs = bifp4::scale_value<true>(p.vs[at], p.v_scale);
  uint32_t out[8];
  bifp4::values_bf16(kc.x, ks, out);
  bifp4::values_bf16(kc.y, ks, out + 4);
  uint4* dst = reinterpret_cast<uint4*>(p.ko + i * 16);
  dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
  dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
  bifp4::values_bf16(vc.x, vs, out);
  bifp4::values_bf16(vc.y, vs, out + 4);
  dst = reinterpret_cast<uint4*>(p.vo + i * 16);
  dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
  dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

struct Kernel {
  const void* fn;
  int smem;
};
template <int D, int HB>
Kernel kernel() {
  return {reinterpret_cast<const void*>(&attn_kernel<D, HB>), Cfg<D, HB>::SMEM};
}
template <int D>
Kernel kernel_of(int heads) {
  return heads == 8 ? kernel<D, 8>() : heads == 4 ? kernel<D, 4>() : heads == 2 ? kernel<D, 2>() : kernel<D, 1>();
}
inline const void* merge_of(int D) {
  return D == 128 ? reinterpret_cast<const void*>(&merge_kernel<128>) : reinterpret_cast<const void*>(&merge_kernel<64>);
}

}  // namespace biattn4

struct bi_attention4 {
  int Hq = 0, Hkv = 0, D = 0, G = 0, page_size = 0, split = 0;
  float scale = 0.0f, k_scale = 1.0f, v_scale = 1.0f;
  int heads = 1;             // KV heads of a block
  int device = 0, max_ctas = 0;
  biattn4::Kernel kern;
  uint32_t* d_status = nullptr;
  biattn_tc::Workspace ws;
};

BI_GEMM_API int bi_attention4_create(bi_attention4_t* out, int64_t num_q_heads, int64_t num_kv_heads, int64_t head_dim,
                                     int64_t page_size, float scale, float k_scale, float v_scale, int64_t split_size) {
  if (!out) return BI_GEMM_ERR_INVALID_ARG;
  *out = nullptr;
  auto fine = [](float s) { return s >= 0x1p-64f && s <= 0x1p64f; };
  if (!std::isfinite(scale) || scale <= 0.0f || !fine(k_scale) || !fine(v_scale)) return BI_GEMM_ERR_INVALID_ARG;
  if (num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || page_size <= 0 || split_size < 0)
    return BI_GEMM_ERR_INVALID_ARG;
  int heads = biattn4::kWarps;
  while (num_kv_heads % heads != 0) heads /= 2;
  const int64_t split = split_size ? split_size : int64_t(biattn4::kSplitPerPart) * (biattn4::kWarps / heads);
  if (num_q_heads % num_kv_heads != 0 || num_q_heads > 4096 || page_size > (1 << 20) || split % 128 != 0 || split > 4096 ||
      (head_dim != 64 && head_dim != 128))
    return BI_GEMM_ERR_UNSUPPORTED;
  const int64_t G = num_q_heads / num_kv_heads;
  if (G != 1 && G != 2 && G != 4 && G != 8) return BI_GEMM_ERR_UNSUPPORTED;
  int dev = 0, sms = 0, per_sm = 0;
  if (const int rc = bifp4::check_device(&dev)) return rc;
  const biattn4::Kernel k = head_dim == 128 ? biattn4::kernel_of<128>(heads) : biattn4::kernel_of<64>(heads);
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k.fn, biattn4::kThreads, size_t(k.smem)) != cudaSuccess ||
      per_sm < 1) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  bi_attention4* h = new (std::nothrow) bi_attention4();
  if (!h) return BI_GEMM_ERR_OOM;
  h->Hq = int(num_q_heads);
  h->Hkv = int(num_kv_heads);
  h->D = int(head_dim);
  h->G = int(G);
  h->page_size = int(page_size);
  h->split = int(split);
  h->scale = scale;
  h->k_scale = k_scale;
  h->v_scale = v_scale;
  h->device = dev;
  h->max_ctas = per_sm * sms;
  h->heads = heads;
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

namespace {

struct Layout4 {
  int64_t splits, parts;   // of a token at most
  size_t part, total;      // bytes of the partial sums, and with the references and sums behind them
};
Layout4 layout4_of(const bi_attention4* h, int64_t T, int64_t max_pos) {
  Layout4 w{max_pos / h->split + 1, 0, 0, 0};
  w.parts = w.splits * (biattn4::kWarps / h->heads);
  if (w.parts > 1) {
    const size_t slots = size_t(std::min<int64_t>(T, biattn4::kTokens)) * h->Hkv * size_t(w.parts) * h->G;
    w.part = slots * h->D * sizeof(float);
    w.total = w.part + slots * 2 * sizeof(float);
  }
  return w;
}

}  // namespace

BI_GEMM_API int bi_attention4_workspace_size(bi_attention4_t h, int64_t T, int64_t max_pos, uint64_t* bytes) {
  if (!h || !bytes || T < 0 || max_pos < -1) return BI_GEMM_ERR_INVALID_ARG;
  *bytes = T == 0 || max_pos < 0 ? 0 : uint64_t(layout4_of(h, T, max_pos).total);
  return BI_GEMM_OK;
}

namespace {

// bi_attention4_run with the failure injection of the test controls (stall >= 0: that block loads nothing) and the
// limit of the waits.
int attention4_run(bi_attention4* h, const void* q, int64_t T, const int32_t* q_seq, const int32_t* q_pos,
                                  const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                                  int64_t num_pages, const int32_t* page_table, int64_t num_seqs, int64_t max_pages,
                                  int64_t max_pos, void* o, void* stream, int32_t stall, uint64_t timeout_ns) {
  if (!h || T < 0 || num_pages < 0 || num_seqs < 0 || max_pages < 0 || max_pos < -1) return BI_GEMM_ERR_INVALID_ARG;
  if (T == 0) return BI_GEMM_OK;
  if (T > (int64_t(1) << 24) || max_pos >= (int64_t(1) << 30)) return BI_GEMM_ERR_UNSUPPORTED;
  if (!q || !q_seq || !q_pos || !k_codes || !k_scales || !v_codes || !v_scales || !page_table || !o)
    return BI_GEMM_ERR_INVALID_ARG;
  auto bits = [](const void* a) { return reinterpret_cast<uintptr_t>(a); };
  if ((bits(q) | bits(o) | bits(k_codes) | bits(k_scales) | bits(v_codes) | bits(v_scales)) & 15u)
    return BI_GEMM_ERR_ALIGNMENT;
  if ((bits(q_seq) | bits(q_pos) | bits(page_table)) & 3u) return BI_GEMM_ERR_ALIGNMENT;
  const Layout4 w = layout4_of(h, T, std::max<int64_t>(max_pos, 0));
  const int64_t per_token = int64_t(h->Hkv) * w.parts;
  if (per_token * std::min<int64_t>(T, biattn4::kTokens) >= (int64_t(1) << 31)) return BI_GEMM_ERR_UNSUPPORTED;
  if (num_pages > int64_t(0xFFFFFFFE) / h->page_size / h->Hkv) return BI_GEMM_ERR_UNSUPPORTED;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  if (dev != h->device) return BI_GEMM_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (const int rc = h->ws.need(w.total, st)) return rc;
  biattn4::Params p;
  std::memset(&p, 0, sizeof(p));
  p.kc = static_cast<const uint8_t*>(k_codes);
  p.ks = static_cast<const uint8_t*>(k_scales);
  p.vc = static_cast<const uint8_t*>(v_codes);
  p.vs = static_cast<const uint8_t*>(v_scales);
  p.table = page_table;
  p.part = static_cast<float*>(h->ws.at);
  p.ml = reinterpret_cast<float*>(static_cast<uint8_t*>(h->ws.at) + w.part);
  p.status = h->d_status;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.B = num_seqs;
  p.Hq = h->Hq;
  p.Hkv = h->Hkv;
  p.G = h->G;
  p.page_size = h->page_size;
  p.split = h->split;
  p.parts = biattn4::kWarps / h->heads;
  p.max_parts = int32_t(w.parts);
  p.stall = stall;
  p.timeout_ns = timeout_ns;
  p.max_pos = int32_t(max_pos);
  int log2 = 0;
  while ((1 << log2) < h->page_size) ++log2;
  p.page_shift = 30 + log2;
  p.page_mul = uint32_t((uint64_t(1) << p.page_shift) / uint64_t(h->page_size) + 1);
  p.c = float(double(h->scale) * double(h->k_scale) * 1.4426950408889634);
  p.v_scale = h->v_scale;
  for (int64_t t0 = 0; t0 < T; t0 += biattn4::kTokens) {
    p.T = int32_t(std::min<int64_t>(biattn4::kTokens, T - t0));
    p.q = static_cast<const uint16_t*>(q) + t0 * h->Hq * h->D;
    p.o = static_cast<uint16_t*>(o) + t0 * h->Hq * h->D;
    p.q_seq = q_seq + t0;
    p.q_pos = q_pos + t0;
    const int blocks = h->Hkv / h->heads;
    const int64_t chains = std::min<int64_t>(int64_t(p.T) * w.splits, std::max(1, h->max_ctas / blocks));
    if (const int rc = bifp4::launch(h->kern.fn, unsigned(chains * blocks), biattn4::kThreads, size_t(h->kern.smem), st, &p))
      return rc;
    if (w.parts > 1)
      if (const int rc = bifp4::launch(biattn4::merge_of(h->D), unsigned(int64_t(p.T) * h->Hq), 32 * biattn4::kMergeWarps, 0,
                                       st, &p))
        return rc;
  }
  return BI_GEMM_OK;
}

}  // namespace

BI_GEMM_API int bi_attention4_run(bi_attention4_t h, const void* q, int64_t T, const int32_t* q_seq, const int32_t* q_pos,
                                  const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                                  int64_t num_pages, const int32_t* page_table, int64_t num_seqs, int64_t max_pages,
                                  int64_t max_pos, void* o, void* stream) {
  return attention4_run(h, q, T, q_seq, q_pos, k_codes, k_scales, v_codes, v_scales, num_pages, page_table, num_seqs,
                        max_pages, max_pos, o, stream, -1, biattn_tc::kTimeoutNs);
}

BI_GEMM_API int bi_attention4_expand(bi_attention4_t h, const void* k_codes, const void* k_scales, const void* v_codes,
                                     const void* v_scales, int64_t num_pages, const int32_t* pages, int64_t n, void* k_out,
                                     void* v_out, void* stream) {
  if (!h || num_pages < 0 || n < 0) return BI_GEMM_ERR_INVALID_ARG;
  if (n == 0) return BI_GEMM_OK;
  if (!k_codes || !k_scales || !v_codes || !v_scales || !pages || !k_out || !v_out) return BI_GEMM_ERR_INVALID_ARG;
  auto bits = [](const void* a) { return reinterpret_cast<uintptr_t>(a); };
  if ((bits(k_codes) | bits(k_scales) | bits(v_codes) | bits(v_scales) | bits(k_out) | bits(v_out)) & 15u)
    return BI_GEMM_ERR_ALIGNMENT;
  if (bits(pages) & 3u) return BI_GEMM_ERR_ALIGNMENT;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  if (dev != h->device) return BI_GEMM_ERR_INVALID_ARG;
  biattn4::ExpandParams p;
  std::memset(&p, 0, sizeof(p));
  p.kc = static_cast<const uint8_t*>(k_codes);
  p.ks = static_cast<const uint8_t*>(k_scales);
  p.vc = static_cast<const uint8_t*>(v_codes);
  p.vs = static_cast<const uint8_t*>(v_scales);
  p.pages = pages;
  p.ko = static_cast<uint16_t*>(k_out);
  p.vo = static_cast<uint16_t*>(v_out);
  p.status = h->d_status;
  p.num_pages = num_pages;
  p.per_page = int64_t(h->page_size) * h->Hkv * (h->D / 16);
  if (n > (int64_t(1) << 31) / p.per_page * 256) return BI_GEMM_ERR_UNSUPPORTED;
  p.blocks = n * p.per_page;
  p.k_scale = h->k_scale;
  p.v_scale = h->v_scale;
  if ((p.blocks + 255) / 256 >= (int64_t(1) << 31)) return BI_GEMM_ERR_UNSUPPORTED;
  return bifp4::launch(reinterpret_cast<const void*>(&biattn4::expand_kernel), unsigned((p.blocks + 255) / 256), 256, 0,
                       static_cast<cudaStream_t>(stream), &p);
}

BI_GEMM_API int bi_attention4_get_device_error(bi_attention4_t h, void* stream) {
  if (!h) return BI_GEMM_ERR_INVALID_ARG;
  return bifp4::read_status(h->d_status, static_cast<cudaStream_t>(stream), biattn_tc::kErrTimeout);
}

BI_GEMM_API int bi_attention4_get_config(bi_attention4_t h, bi_attention4_config* c) {
  if (!h || !c) return BI_GEMM_ERR_INVALID_ARG;
  c->num_q_heads = h->Hq;
  c->num_kv_heads = h->Hkv;
  c->head_dim = h->D;
  c->page_size = h->page_size;
  c->split_size = h->split;
  c->threads = biattn4::kThreads;
  c->max_ctas = h->max_ctas;
  c->tokens_per_launch = biattn4::kTokens;
  return BI_GEMM_OK;
}

BI_GEMM_API int bi_attention4_destroy(bi_attention4_t h) {
  if (!h) return BI_GEMM_OK;
  h->ws.release();
  if (h->d_status) cudaFree(h->d_status);
  delete h;
  return BI_GEMM_OK;
}
