// bi_attention4.cu — batch-invariant decode attention over a paged KV cache in 4 bits, and the expansion of its
// pages, for sm_103a.  Implements include/bi_attention4.h.
//
//   o_t = v_scale * sum_j w_j V_j / sum_j w_j,  w_j = 2^(c q_t . K_j - m),  c = scale k_scale log2(e)
//
// over the positions j of a token's request up to its own, K_j and V_j codes times block scales.
//
// A unit is (token, split, KV head); four warps run it.  Warp w takes the 32-position steps w, w + 4,
// ... of the split through a ring of its own (cp.async, no barrier with the other warps), keeps a running maximum
// reference, sum and the weighted values of its positions, and the four are merged in order at the unit's end.
//
// Per step, with g = lane / 4 and t = lane % 4 (mma.sync m16n8k16, f16 in, fp32 accumulate; the query heads of
// the KV head on the columns):
//   scores  S^T = K Q^T: 16 positions on the rows.  The order of the products' dimensions is free as long as both
//           operands agree, so lane t takes a quarter of a row, whole 16-byte chunks: eight codes become four f16
//           pairs by cvt, times their block's scale (exact: 2 + 4 significant bits).
//   weights P = 2^(s - m + 7) in fp32, rounded to f16 and transposed in registers (movmatrix).
//   values  O^T += V^T P^T.  A code pair that cvt makes is two dimensions at one position, and the MMA sums over the
//           pair.  G <= 4: a head has two columns, and a weight stands in one half of its pair and zero in the other, so
//           that one column gets the even dimensions and the other the odd ones (32 dimensions on the 16 rows, 8
//           positions deep).
//           G = 8: the codes of two positions are interleaved before cvt, a pair is one dimension at two positions (16
//           dimensions, 16 positions deep).  Lane g owns D / 8 consecutive dimensions either way.
//
// Tensor cores of the fifth generation would need codes and scales of the query too, of which eight bits would take
// four products, and a value's block scales lie along the dimensions where the MMA's lie along the sum.
//
// Bound (256 contexts of 1000 to 8192, 32/8 heads of 128, 265 us, 4.9 TB/s, 0.72 of the bytes' rate): the loads alone
// take nine tenths of it, a head's 64 bytes of every 512-byte row (the same bytes in rows of one KV head a tenth
// less), the arithmetic alone eight tenths at 270 instructions a sixteen of positions and head, the merge's launch 12
// us.  One token (700 positions: 7.9 us, 8.9 before its two splits merged in a cluster): the latencies of a launch, a
// lookup, a chain of steps.  Between them no unit is full: 133 ragged contexts at 16/2 heads of 64 (27.5 us) have
// ALUs at 37 % and DRAM at 26 % of their peaks with 23 % of the warps, 32 contexts of 1000 (16.6 us) 32 % and 27 %,
// 128 of 4096 at 64/8 heads (156 us) 42 % and 54 %.  Tried: a loading warp for eight computing ones, a warp a head
// (largest call 355 when this form took 391, but 96 registers, and one token's 700 positions 18.6 us instead of 9.3);
// three blocks an SM with rings of three steps (no change); splits of 256 positions (433 against 391, one token's
// 32768 21.4 against 18.5) and 1024 (379, 21.6).  For the blocks of four heads (285): one loading warp and rings that
// the heads share 421, four loading warps 333 (a stage waits for the slowest of four heads); pairs of such blocks
// with a cluster barrier a unit 325.  The last block to arrive merging a token's splits, instead of a second kernel:
// nothing for one token, 343 for the largest call (registers).  Splits joined in the block that runs them, the merge
// left with what chains cut: 1 % less.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
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

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kStep = 32;                 // positions of a step
constexpr int kRing = 2;                  // steps of a warp's ring
constexpr int kBlocksPerSm = 4;
constexpr int kTokens = 512;              // of a launch
constexpr int kHeads = 8;                 // columns of the MMA
constexpr int kGroup = 4;                 // KV heads of the larger blocks
constexpr int kDefaultSplit = 512;
constexpr int kMergeWarps = 8;
constexpr float kLift = 7.0f;             // weights are 2^7 at the reference, 2^15 at most
constexpr float kSlack = 8.0f;            // the reference moves when a score passes it by more
constexpr uint32_t kErrInput = 1u, kErrPage = 2u, kErrBound = 4u;

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
  float* part;        // [T, Hkv, max_splits, G, D] partial weighted sums
  float* ml;          // [T, Hkv, max_splits, G, 2] (reference, sum)
  uint32_t* status;
  int64_t max_pages, B;
  uint32_t num_pages;
  int32_t T, Hq, Hkv, G, page_size, split, max_splits, max_pos;
  int32_t cluster;    // blocks of a (token, KV head), a split each, that merge among themselves (0: runs of units)
  uint32_t page_mul;  // pos / page_size = 4 pos * page_mul >> (32 + page_shift) for pos < 2^30
  int32_t page_shift;
  float c;            // scale * k_scale * log2(e)
  float v_scale;
};

// HB: KV heads of a block, four warps each.
template <int D, int HB>
struct Cfg {
  static constexpr int THREADS = kThreads * HB;
  static constexpr int CODES = D / 2, SCALES = D / 16;           // bytes of a row
  // rows of values lie 16 bytes further apart than they are long, so that the rows 0, 2, 4, 6 that a load takes at
  // once are on different banks
  static constexpr int VROW = CODES + 16;
  static constexpr int OFF_V = kStep * CODES, OFF_KS = OFF_V + kStep * VROW, OFF_VS = OFF_KS + kStep * SCALES;
  static constexpr int STEP = OFF_VS + kStep * SCALES;
  static constexpr int RING = kRing * STEP;                      // of a warp
  static constexpr int OFF_ML = HB * kWarps * RING;
  static constexpr int OFF_CUM = OFF_ML + HB * kWarps * kHeads * 8;
  static constexpr int OFF_O = (OFF_CUM + (3 * kTokens + 1 + HB * kWarps) * 4 + 15) / 16 * 16;
  static_assert(STEP % 16 == 0 && OFF_ML % 16 == 0, "alignment");
  // The warps' parts meet in shared memory, eight heads in two halves of the dimensions: four blocks fit an SM.
  __host__ __device__ static constexpr int halves(int G) { return G == 8 ? 2 : 1; }
  __host__ __device__ static constexpr int row(int G) { return D / halves(G) + 4; }   // floats of a head
  static constexpr int smem(int G) { return OFF_O + HB * kWarps * G * row(G) * 4; }
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
// Both halves of a times the lower or upper half of b.
template <int kHalf>
__device__ __forceinline__ uint32_t mul_f16x2_by(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (kHalf == 0)
    asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 t;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 t, {l, l};\n\tmul.rn.f16x2 %0, %1, t;\n\t}"
        : "=r"(r) : "r"(a), "r"(b));
  else
    asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 t;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 t, {h, h};\n\tmul.rn.f16x2 %0, %1, t;\n\t}"
        : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t at) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
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

// kTwin: up to four heads, each on two of the MMA's columns.  kCluster: a block a split, the splits of a (token, KV
// head) in a cluster that merges them.
template <int D, bool kTwin, int HB, bool kCluster>
__global__ void __launch_bounds__(kThreads * HB, kBlocksPerSm / HB) attn_kernel(const Params p) {
  using C = Cfg<D, HB>;
  constexpr int HEADS = kTwin ? 1 : 2;                   // whose scores and sums a lane has
  constexpr int TILES = kTwin ? D / 32 : D / 16;         // of the weighted values
  extern __shared__ __align__(128) uint8_t smem[];
  int32_t* cum = reinterpret_cast<int32_t*>(smem + C::OFF_CUM);
  int32_t* seqs = cum + kTokens + 1;                     // the tokens' requests and positions
  int32_t* poss = seqs + kTokens;
  int32_t* sums = poss + kTokens;
  const int lane = int(threadIdx.x) & 31, g = lane >> 2, t4 = lane & 3;
  const int group = HB == 1 ? 0 : int(threadIdx.x) / kThreads;   // its KV head of the block's
  const int tid = int(threadIdx.x) - group * kThreads, warp = tid >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // (The next kernel is not asked for early: with its blocks waiting beside these, 133 ragged contexts at 16/2 heads
  // of 64 took 31 us instead of 27, 16 of 4096 at 32/8 of 128 26.8 instead of 26.0, and none less.)
  // first unit (of one KV head) of every token
  int32_t carry = 0;
  for (int base = 0; base < p.T; base += C::THREADS) {
    const int i = base + int(threadIdx.x);
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
    if (lane == 31) sums[group * kWarps + warp] = x;
    __syncthreads();
    int32_t before = carry;
#pragma unroll
    for (int w = 0; w < HB * kWarps; ++w) {
      const int32_t s = sums[w];
      if (w < group * kWarps + warp) before += s;
      carry += s;
    }
    if (i < p.T) cum[i] = before + x - n;
    __syncthreads();
  }
  if (threadIdx.x == 0) cum[p.T] = carry;
  __syncthreads();

  // Block (chain, kh) takes a run of consecutive (token, split) of its head, so that a token's query is prepared once
  // for its splits there; the blocks of a chain's heads read neighbouring rows at the same time.
  const uint32_t across = uint32_t(p.Hkv) / HB;          // blocks of a chain
  const int32_t chain = int32_t(blockIdx.x / across);
  const int32_t chains = int32_t(gridDim.x / across);
  // In clusters a block has one unit, or none.
  int32_t kh = int32_t(blockIdx.x % across) * HB + group, ct = 0, rank = 0, n_splits = 0;
  int32_t v_end = int32_t(int64_t(carry) * (chain + 1) / chains);
  if constexpr (kCluster) {
    const int32_t place = int32_t(blockIdx.x) / p.cluster;
    rank = int32_t(blockIdx.x) - place * p.cluster;
    ct = place / p.Hkv;
    kh = place - ct * p.Hkv;
    n_splits = cum[ct + 1] - cum[ct];
    v_end = cum[ct] + min(rank + 1, n_splits);
  }
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
    r.v = kCluster ? cum[ct] + min(rank, n_splits) : int32_t(int64_t(carry) * chain / chains);
    r.t = 0;
    if (r.v < v_end) locate(r);
  };
  auto advance = [&](Unit& r) {
    if (++r.v < v_end) locate(r);
  };

  // ---- this warp's loads, ahead of its products by kRing steps and across units
  const uint32_t ring = ptx::smem_u32(smem) + uint32_t(group * kWarps + warp) * C::RING;
  constexpr int CH = C::CODES / 16, ROWS = 32 / CH;      // 16-byte chunks of a row, rows an instruction
  const int row = lane / CH, ch = lane % CH;
  const uint8_t* kc = p.kc + ch * 16;
  const uint8_t* vc = p.vc + ch * 16;
  const uint32_t to_k = uint32_t(row * C::CODES + ch * 16), to_v = uint32_t(C::OFF_V + row * C::VROW + ch * 16);
  Unit L = {};                                           // unit of the next load
  int32_t lpos = 0;                                      // its position
  int32_t lpage = 0, lrow = 0;                           // this lane's page there, fetched ahead, and row of the page
  int lslot = 0;
  bool lmore = true;
  const int32_t* ltable = p.table;                       // its request's row of the page table
  auto fetch = [&]() {
    const uint32_t pos = uint32_t(min(lpos + lane, L.last)), pg = __umulhi(pos << 2, p.page_mul) >> p.page_shift;
    lrow = int32_t(pos - pg * uint32_t(p.page_size));
    lpage = __ldg(ltable + pg);
  };
  // Makes L the next unit (from itself on) in which this warp has a step.
  auto seek = [&]() {
    while (L.v < v_end) {
      lpos = L.first + warp * kStep;
      if (lpos <= L.last) {
        ltable = p.table + int64_t(seqs[L.t]) * p.max_pages;
        fetch();
        return;
      }
      advance(L);
    }
    lmore = false;
  };
  auto issue = [&]() {
    if (lmore) {
      const uint32_t dst = ring + uint32_t(lslot) * C::STEP;
      // a lane looks one position up; a row's place comes from its lane (fewer than 2^32 - 1 rows of a head: the host)
      const bool here = lpos + lane <= L.last, good = uint32_t(lpage) < p.num_pages;
      uint32_t at = (uint32_t(lpage) * uint32_t(p.page_size) + uint32_t(lrow)) * uint32_t(p.Hkv) + uint32_t(kh);
      if (__all_sync(0xFFFFFFFFu, here && good)) {
#pragma unroll
        for (int i = 0; i < kStep / ROWS; ++i) {
          const uint64_t off = uint64_t(__shfl_sync(0xFFFFFFFFu, at, i * ROWS + row)) * C::CODES;
          cp_async_16(dst + to_k + uint32_t(i * ROWS * C::CODES), kc + off);
          cp_async_16(dst + to_v + uint32_t(i * ROWS * C::VROW), vc + off);
        }
        cp_async<C::SCALES>(dst + C::OFF_KS + lane * C::SCALES, p.ks + uint64_t(at) * C::SCALES);
        cp_async<C::SCALES>(dst + C::OFF_VS + lane * C::SCALES, p.vs + uint64_t(at) * C::SCALES);
      } else {
        // the last step of a token, or a page that is not there: zeros in its place
        if (here && !good) atomicOr(p.status, kErrPage);
        if (!(here && good)) at = 0xFFFFFFFFu;
#pragma unroll 1
        for (int i = 0; i < kStep / ROWS; ++i) {
          const uint32_t a = __shfl_sync(0xFFFFFFFFu, at, i * ROWS + row), n = a != 0xFFFFFFFFu ? 16u : 0u;
          const uint64_t off = n ? uint64_t(a) * C::CODES : 0;
          ptx::cp_async_16(dst + to_k + uint32_t(i * ROWS * C::CODES), kc + off, n);
          ptx::cp_async_16(dst + to_v + uint32_t(i * ROWS * C::VROW), vc + off, n);
        }
        const uint32_t n = at != 0xFFFFFFFFu ? uint32_t(C::SCALES) : 0u;
        const uint64_t off = n ? uint64_t(at) * C::SCALES : 0;
        cp_async_zfill<C::SCALES>(dst + C::OFF_KS + lane * C::SCALES, p.ks + off, n);
        cp_async_zfill<C::SCALES>(dst + C::OFF_VS + lane * C::SCALES, p.vs + off, n);
      }
      if (++lslot == kRing) lslot = 0;
      lpos += kWarps * kStep;
      if (lpos <= L.last) {
        fetch();
      } else {
        advance(L);
        seek();
      }
    }
    ptx::cp_async_commit();
  };
  start(L);
  seek();
#pragma unroll 1
  for (int i = 0; i < kRing; ++i) issue();

  // ---- products
  auto meet = [&]() {                                    // the four warps of a head
    if constexpr (HB == 1)
      __syncthreads();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(kThreads) : "memory");
  };
  int slot = 0;
  float* so = reinterpret_cast<float*>(smem + C::OFF_O) + group * kWarps * p.G * C::row(p.G);
  float* sml = reinterpret_cast<float*>(smem + C::OFF_ML) + group * kWarps * kHeads * 2;
  int32_t token = -1;
  uint32_t qf[D / 8];
  float fac[HEADS];
  const int column = kTwin ? g >> 1 : g;                 // the head of this lane's column
  // (kTwin) the weights of two positions, one in either half, to the half that the column's dimensions are in
  const uint32_t even = g & 1 ? 0x1044u : 0x4410u, odd = g & 1 ? 0x3244u : 0x4432u;
  Unit U;
  for (start(U); U.v < v_end; advance(U)) {
    // the query in f16, relative to its head's largest element
    if (U.t != token) {
      token = U.t;
      const uint16_t* src = p.q + (int64_t(U.t) * p.Hq + kh * p.G + column) * D + t4 * (D / 4);
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 v = column < p.G ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
        qf[4 * i] = v.x, qf[4 * i + 1] = v.y, qf[4 * i + 2] = v.z, qf[4 * i + 3] = v.w;
      }
      most = bifp4::most_of(qf, D / 8);
      most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
      most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
      // times 2^11 / 2^exponent of the largest element (within fp32's range): sizes below 2^12
      const int e = min(max(int(most >> 7), 12), 254);
      const float up = __uint_as_float(uint32_t(265 - e) << 23), down = __uint_as_float(uint32_t(e - 11) << 23);
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        qf[i] = pack_f16x2(__uint_as_float(qf[i] << 16) * up, __uint_as_float(qf[i] & 0xFFFF0000u) * up);
      // the factors of the heads whose scores this lane has
      // (above zero, so that a hidden position's -inf stays one, and finite, so that a difference of zero stays one:
      // queries beyond 2^116 / c whose large elements meet keys of zero)
#pragma unroll
      for (int j = 0; j < HEADS; ++j)
        fac[j] = fminf(fmaxf(__fmul_rn(__shfl_sync(0xFFFFFFFFu, down, 8 * t4 + 4 * j), p.c), 1e-45f), FLT_MAX);
    }
    // (the reference m is a product's sum as it comes from the MMA; the difference to it is taken before the factor, so
    // that it is exact near the reference however large the scores are)
    float acc[TILES][4], m[HEADS], l[HEADS];
#pragma unroll
    for (int j = 0; j < HEADS; ++j) m[j] = -INFINITY, l[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < TILES; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    for (int32_t pos = U.first + warp * kStep; pos <= U.last; pos += kWarps * kStep) {
      ptx::cp_async_wait<kRing - 1>();
      __syncwarp();
      const uint8_t* src = smem + (group * kWarps + warp) * C::RING + slot * C::STEP;
      if (++slot == kRing) slot = 0;
      // scores: two sixteens of positions side by side, for two chains of products
      constexpr int W = D / 32;                           // words of codes a lane has of a row
      float s[2][4];
      uint32_t kw[4][W], ksc[4];                          // rows g, g + 8, g + 16, g + 24
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int at = 8 * r + g;
        if constexpr (D == 128) {
          const uint4 v = *reinterpret_cast<const uint4*>(src + at * C::CODES + t4 * 16);
          kw[r][0] = v.x, kw[r][1] = v.y, kw[r][2] = v.z, kw[r][3] = v.w;
          ksc[r] = bifp4::e4m3_pair(*reinterpret_cast<const uint16_t*>(src + C::OFF_KS + at * 8 + 2 * t4));
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(src + at * C::CODES + t4 * 8);
          kw[r][0] = v.x, kw[r][1] = v.y;
          ksc[r] = bifp4::e4m3_pair(src[C::OFF_KS + at * 4 + t4]);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[h][j] = 0.0f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t x[4], y[4];
          bifp4::values8(kw[2 * h][i], x);
          bifp4::values8(kw[2 * h + 1][i], y);
          // (D = 128: 32 dimensions a lane, two blocks)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (D == 64 || i < 2) {
              x[j] = mul_f16x2_by<0>(x[j], ksc[2 * h]), y[j] = mul_f16x2_by<0>(y[j], ksc[2 * h + 1]);
            } else {
              x[j] = mul_f16x2_by<1>(x[j], ksc[2 * h]), y[j] = mul_f16x2_by<1>(y[j], ksc[2 * h + 1]);
            }
          }
          mma(s[h], x[0], y[0], x[1], y[1], qf[4 * i], qf[4 * i + 1]);
          mma(s[h], x[2], y[2], x[3], y[3], qf[4 * i + 2], qf[4 * i + 3]);
        }
      }
      constexpr int VW = D / 64;                          // words of codes a lane has of a row of values
      uint32_t vw[kTwin ? 4 : 1][2][VW], vsc[kTwin ? 4 : 1];
      if constexpr (kTwin) {                              // (asked for before they are needed)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint8_t* a = src + C::OFF_V + (8 * q + 2 * t4 + r) * C::VROW + g * (C::CODES / 8);
            if constexpr (D == 128) {
              const uint2 v = *reinterpret_cast<const uint2*>(a);
              vw[q][r][0] = v.x, vw[q][r][1] = v.y;
            } else {
              vw[q][r][0] = *reinterpret_cast<const uint32_t*>(a);
            }
          }
          const uint8_t* a = src + C::OFF_VS + (8 * q + 2 * t4) * C::SCALES + (D == 128 ? g : g >> 1);
          vsc[q] = bifp4::e4m3_pair(uint32_t(a[0]) | uint32_t(a[C::SCALES]) << 8);
        }
      }
      if (pos + kStep - 1 > U.last) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (pos + 16 * h + 8 * (j >> 1) + g > U.last) s[h][j] = -INFINITY;
      }
      bool move = false;
      float top[HEADS];
#pragma unroll
      for (int j = 0; j < HEADS; ++j) {
        top[j] = fmaxf(fmaxf(s[0][j], s[0][j + 2]), fmaxf(s[1][j], s[1][j + 2]));
        move |= __fmul_rn(__fsub_rn(top[j], m[j]), fac[j]) > kSlack;
      }
      if (__any_sync(0xFFFFFFFFu, move)) {                // (a head's rule looks at that head alone)
        float f[HEADS];
#pragma unroll
        for (int j = 0; j < HEADS; ++j) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) top[j] = fmaxf(top[j], __shfl_xor_sync(0xFFFFFFFFu, top[j], o));
          const bool mv = __fmul_rn(__fsub_rn(top[j], m[j]), fac[j]) > kSlack;
          f[j] = mv ? ex2(__fmul_rn(__fsub_rn(m[j], top[j]), fac[j])) : 1.0f;
          if (mv) m[j] = top[j];
          l[j] *= f[j];
        }
#pragma unroll
        for (int i = 0; i < TILES; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] *= f[j & (HEADS - 1)];
      }
      if constexpr (kTwin) {
        // (columns 2 t4 and 2 t4 + 1 are one head's: s[h][j] and s[h][j + 1] are equal)
#pragma unroll
        for (int q = 0; q < 4; ++q) {                     // eight positions
          const float e = ex2(__fmaf_rn(__fsub_rn(s[q >> 1][2 * (q & 1)], m[0]), fac[0], kLift));
          l[0] += e;
          const uint32_t b = transposed(pack_f16x2(e, e));
          const uint32_t b0 = __byte_perm(b, 0u, even), b1 = __byte_perm(b, 0u, odd);
#pragma unroll
          for (int i = 0; i < VW; ++i) {
            uint32_t x[4], y[4];
            bifp4::values8(vw[q][0][i], x);
            bifp4::values8(vw[q][1][i], y);
#pragma unroll
            for (int j = 0; j < 2; ++j)
              mma(acc[2 * i + j], mul_f16x2_by<0>(x[2 * j], vsc[q]), mul_f16x2_by<0>(x[2 * j + 1], vsc[q]),
                  mul_f16x2_by<1>(y[2 * j], vsc[q]), mul_f16x2_by<1>(y[2 * j + 1], vsc[q]), b0, b1);
          }
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int k = j & (HEADS - 1);
            s[h][j] = ex2(__fmaf_rn(__fsub_rn(s[h][j], m[k]), fac[k], kLift));
          }
          l[0] += s[h][0] + s[h][2];
          l[HEADS - 1] += s[h][1] + s[h][3];
          const uint32_t b0 = transposed(pack_f16x2(s[h][0], s[h][1])), b1 = transposed(pack_f16x2(s[h][2], s[h][3]));
          constexpr int W = D / 64;                         // words of codes a lane has of a row
          uint32_t w[4][W], sc[2];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int at = 16 * h + 2 * t4 + (r & 1) + 8 * (r >> 1);
            const uint8_t* a = src + C::OFF_V + at * C::VROW + g * (C::CODES / 8);
            if constexpr (D == 128) {
              const uint2 v = *reinterpret_cast<const uint2*>(a);
              w[r][0] = v.x, w[r][1] = v.y;
            } else {
              w[r][0] = *reinterpret_cast<const uint32_t*>(a);
            }
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint8_t* a = src + C::OFF_VS + (16 * h + 2 * t4 + 8 * r) * C::SCALES + (D == 128 ? g : g >> 1);
            sc[r] = bifp4::e4m3_pair(uint32_t(a[0]) | uint32_t(a[C::SCALES]) << 8);
          }
#pragma unroll
          for (int i = 0; i < W; ++i) {
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
      __syncwarp();                                       // the slot may be refilled
      issue();
    }
    // ---- the four warps' parts, in order
    if constexpr (HB > 1) __syncthreads();               // (keeps the heads on neighbouring rows)
    const bool alone = U.split == 0 && U.last == poss[U.t];
    const int halves = C::halves(p.G), dims = D / halves, orow = C::row(p.G);
#pragma unroll
    for (int j = 0; j < HEADS; ++j) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[j] = __fadd_rn(l[j], __shfl_xor_sync(0xFFFFFFFFu, l[j], o));
      const int head = HEADS * t4 + j;
      if (g == 0 && head < p.G) {
        sml[(warp * kHeads + head) * 2] = __fmul_rn(m[j], fac[j]);
        sml[(warp * kHeads + head) * 2 + 1] = l[j];
      }
    }
    for (int half = 0; half < halves; ++half) {
      const int d0 = g * (D / 8) - half * dims;           // this lane's first dimension within the half
      if (d0 >= 0 && d0 < dims) {
#pragma unroll
        for (int j = 0; j < HEADS; ++j) {
          const int head = HEADS * t4 + j;
          if (head < p.G) {
            float* dst = so + (warp * p.G + head) * orow + d0;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
              if constexpr (kTwin)
                *reinterpret_cast<float4*>(dst + 4 * i) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
              else
                *reinterpret_cast<float4*>(dst + 4 * i) =
                    make_float4(acc[2 * i][j], acc[2 * i][j + 2], acc[2 * i + 1][j], acc[2 * i + 1][j + 2]);
            }
          }
        }
      }
      meet();
      for (int it = tid; it < p.G * (dims / 4); it += kThreads) {
        const int head = it / (dims / 4), d = (it - head * (dims / 4)) * 4;
        float M = -INFINITY, Ls = 0.0f;
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sml[(w * kHeads + head) * 2]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float mw = sml[(w * kHeads + head) * 2], lw = sml[(w * kHeads + head) * 2 + 1];
          // (a warp without a step has a sum of 0; one whose scores are all -inf or NaN has a NaN)
          const float f = mw == -INFINITY ? (lw == 0.0f ? 0.0f : NAN) : ex2(__fsub_rn(mw, M));
          const float4 v = *reinterpret_cast<const float4*>(so + (w * p.G + head) * orow + d);
          Ls = __fmaf_rn(lw, f, Ls);
          A.x = __fmaf_rn(v.x, f, A.x);
          A.y = __fmaf_rn(v.y, f, A.y);
          A.z = __fmaf_rn(v.z, f, A.z);
          A.w = __fmaf_rn(v.w, f, A.w);
        }
        const int at_d = half * dims + d;
        if (alone) {
          const float f = U.last < 0 ? 0.0f : __fdiv_rn(p.v_scale, Ls);
          const uint2 out = U.last < 0 ? make_uint2(0u, 0u)
                                       : make_uint2(ptx::pack_bf16x2(__fmul_rn(A.x, f), __fmul_rn(A.y, f)),
                                                    ptx::pack_bf16x2(__fmul_rn(A.z, f), __fmul_rn(A.w, f)));
          *reinterpret_cast<uint2*>(p.o + (int64_t(U.t) * p.Hq + kh * p.G + head) * D + at_d) = out;
        } else if (kCluster) {
          // (the rings are done with)
          float* keep = reinterpret_cast<float*>(smem);
          *reinterpret_cast<float4*>(keep + head * D + at_d) = A;
          if (at_d == 0) *reinterpret_cast<float2*>(keep + kHeads * D + 2 * head) = make_float2(M, Ls);
        } else {
          const int64_t at = ((int64_t(U.t) * p.Hkv + kh) * p.max_splits + U.split) * p.G + head;
          *reinterpret_cast<float4*>(p.part + at * D + at_d) = A;
          if (at_d == 0) *reinterpret_cast<float2*>(p.ml + at * 2) = make_float2(M, Ls);
        }
      }
      meet();
    }
  }
  ptx::cp_async_wait<0>();
  if constexpr (kCluster) {
    // The cluster's blocks have a split each: a warp a head sums them as merge_kernel would.
    __syncwarp();
    ptx::cluster_sync();
    for (int hd = rank * kWarps + warp; n_splits > 1 && hd < p.G; hd += p.cluster * kWarps) {
      constexpr int PER = D / 32;
      const uint32_t keep = ptx::smem_u32(smem);
      float mine = -INFINITY, sum = 0.0f;
      if (lane < n_splits) {
        const uint32_t at = ptx::mapa_shared(keep + uint32_t(kHeads * D + 2 * hd) * 4u, uint32_t(lane));
        mine = ld_cluster(at), sum = ld_cluster(at + 4u);
      }
      float M = mine, L = 0.0f, A[PER];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
#pragma unroll
      for (int j = 0; j < PER; ++j) A[j] = 0.0f;
      for (int s = 0; s < n_splits; ++s) {
        const uint32_t at = ptx::mapa_shared(keep + uint32_t(hd * D + lane * PER) * 4u, uint32_t(s));
        const float f = ex2(__fsub_rn(__shfl_sync(0xFFFFFFFFu, mine, s), M));
        L = __fmaf_rn(__shfl_sync(0xFFFFFFFFu, sum, s), f, L);
#pragma unroll
        for (int j = 0; j < PER; ++j) A[j] = __fmaf_rn(ld_cluster(at + 4u * j), f, A[j]);
      }
      uint16_t* o = p.o + (int64_t(ct) * p.Hq + kh * p.G + hd) * D;
      const float f = __fdiv_rn(p.v_scale, L);
#pragma unroll
      for (int j = 0; j < PER; j += 2)
        *reinterpret_cast<uint32_t*>(o + lane * PER + j) = ptx::pack_bf16x2(__fmul_rn(A[j], f), __fmul_rn(A[j + 1], f));
    }
    __syncwarp();
    ptx::cluster_sync();                                // nobody leaves while its splits are read
  }
}

// Up to kSolo splits of a token's query head are summed in ascending order by one warp (of a cluster's block, or here,
// eight heads a block: a block a head took 51 us for 8192 heads of 9 splits); more of them as eight consecutive
// groups of ceil(n / 8) by the warps of a block, ascending, the groups added in order.  n depends on the token's
// position alone.
constexpr int kSolo = 16;

// Splits s0 .. s1 - 1 of the head whose first is slot0, in order: the largest reference and, relative to it, the sum
// of the sums and this lane's dimensions.
template <int D>
__device__ __forceinline__ void sum_splits(const Params& p, int64_t slot0, int32_t s0, int32_t s1, int lane, float& M,
                                           float& L, float (&A)[D / 32]) {
  constexpr int PER = D / 32, BATCH = 8;
  const float2* mlp = reinterpret_cast<const float2*>(p.ml) + slot0;
  M = -INFINITY;
  for (int32_t s = s0 + lane; s < s1; s += 32) M = fmaxf(M, mlp[int64_t(s) * p.G].x);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  L = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) A[i] = 0.0f;
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
        const float f = ex2(__fsub_rn(ml[i].x, M));
        L = __fmaf_rn(ml[i].y, f, L);
#pragma unroll
        for (int j = 0; j < PER; ++j) A[j] = __fmaf_rn(v[i][j], f, A[j]);
      }
    }
  }
}

// Blocks of a token: one for eight heads where no token of the call can have more than kSolo splits.
__host__ __device__ constexpr uint32_t merge_blocks(int32_t Hq, int32_t max_splits) {
  return uint32_t(max_splits <= kSolo ? (Hq + kMergeWarps - 1) / kMergeWarps : Hq);
}

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_kernel(const Params p) {
  constexpr int PER = D / 32;                             // dimensions a lane
  __shared__ float sums[kMergeWarps][D];
  __shared__ float2 mls[kMergeWarps];
  const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t per = merge_blocks(p.Hq, p.max_splits);
  const int32_t t = int32_t(blockIdx.x / per);
  int32_t h = int32_t((blockIdx.x - uint32_t(t) * per) * (uint32_t(p.max_splits) <= kSolo ? kMergeWarps : 1));
  const int32_t n = splits_of(p, p.q_seq[t], p.q_pos[t], false);
  if (n <= 1) return;                                     // written by its unit, or refused
  const bool solo = n <= kSolo;
  if (solo) {
    if (h % kMergeWarps != 0) return;
    h += warp;
    if (h >= p.Hq) return;
  }
  const int32_t kh = h / p.G, hd = h - kh * p.G;
  const int64_t slot0 = (int64_t(t) * p.Hkv + kh) * p.max_splits * p.G + hd;
  const int32_t c = (n + kMergeWarps - 1) / kMergeWarps;
  const int32_t s0 = solo ? 0 : min(n, warp * c), s1 = solo ? n : min(n, s0 + c);
  float M, L, A[PER];
  sum_splits<D>(p, slot0, s0, s1, lane, M, L, A);
  uint16_t* o = p.o + (int64_t(t) * p.Hq + h) * D;
  if (solo) {
    const float f = __fdiv_rn(p.v_scale, L);
#pragma unroll
    for (int j = 0; j < PER; j += 2)
      *reinterpret_cast<uint32_t*>(o + lane * PER + j) = ptx::pack_bf16x2(__fmul_rn(A[j], f), __fmul_rn(A[j + 1], f));
    return;
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
      if (w * c < n) {                                    // (a group of no splits adds nothing)
        const float f = ex2(__fsub_rn(mls[w].x, top));
        Ls = __fmaf_rn(mls[w].y, f, Ls);
        a0 = __fmaf_rn(sums[w][2 * threadIdx.x], f, a0);
        a1 = __fmaf_rn(sums[w][2 * threadIdx.x + 1], f, a1);
      }
    }
    const float f = __fdiv_rn(p.v_scale, Ls);
    *reinterpret_cast<uint32_t*>(o + 2 * threadIdx.x) = ptx::pack_bf16x2(__fmul_rn(a0, f), __fmul_rn(a1, f));
  }
}

constexpr int kExpand = 4;                // pieces a thread expands

struct ExpandParams {
  const uint8_t* kc;
  const uint8_t* ks;
  const uint8_t* vc;
  const uint8_t* vs;
  const int32_t* pages;
  uint16_t* ko;
  uint16_t* vo;
  uint32_t* status;
  int64_t num_pages, pieces;              // pieces of eight elements in all
  int64_t per_page;                       // and of a page
  float k_scale, v_scale;
};

__global__ void __launch_bounds__(256) expand_kernel(const ExpandParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // eight elements a thread: half a block, so that a warp's stores are whole lines
  int64_t at[kExpand];
  uint32_t kc[kExpand], vc[kExpand], ks[kExpand], vs[kExpand];
  const int64_t first = int64_t(blockIdx.x) * (256 * kExpand) + threadIdx.x;
#pragma unroll
  for (int u = 0; u < kExpand; ++u) {
    const int64_t i = first + u * 256;
    at[u] = -1;
    if (i < p.pieces) {
      // (a page has no more pieces than the call)
      const int64_t n = p.pieces >> 32 ? i / p.per_page : int64_t(uint32_t(i) / uint32_t(p.per_page)), r = i - n * p.per_page;
      const int64_t page = p.pages[n];
      if (page >= 0 && page < p.num_pages) {
        at[u] = page * p.per_page + r;
        kc[u] = reinterpret_cast<const uint32_t*>(p.kc)[at[u]];
        vc[u] = reinterpret_cast<const uint32_t*>(p.vc)[at[u]];
        ks[u] = p.ks[at[u] >> 1];
        vs[u] = p.vs[at[u] >> 1];
      } else if (page != -1 && r == 0) {
        atomicOr(p.status, kErrPage);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kExpand; ++u) {
    if (at[u] < 0) continue;
    const int64_t i = first + u * 256;
    uint32_t out[4];
    bifp4::values_bf16(kc[u], bifp4::scale_value<true>(ks[u], p.k_scale), out);
    *reinterpret_cast<uint4*>(p.ko + i * 8) = make_uint4(out[0], out[1], out[2], out[3]);
    bifp4::values_bf16(vc[u], bifp4::scale_value<true>(vs[u], p.v_scale), out);
    *reinterpret_cast<uint4*>(p.vo + i * 8) = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

// With one KV head a block, in clusters or not (HB = 0, 1), or kGroup of them (heads of 128).
template <bool kTwin>
const void* attn_for(int D, int HB) {
  if (HB == 0)
    return D == 64 ? reinterpret_cast<const void*>(&attn_kernel<64, kTwin, 1, true>)
                   : reinterpret_cast<const void*>(&attn_kernel<128, kTwin, 1, true>);
  if (D == 64) return reinterpret_cast<const void*>(&attn_kernel<64, kTwin, 1, false>);
  return HB == 1 ? reinterpret_cast<const void*>(&attn_kernel<128, kTwin, 1, false>)
                 : reinterpret_cast<const void*>(&attn_kernel<128, kTwin, kGroup, false>);
}
inline const void* attn_of(int D, int G, int HB) { return G <= 4 ? attn_for<true>(D, HB) : attn_for<false>(D, HB); }
inline int smem_of(int D, int G, int HB) {
  if (D == 64) return Cfg<64, 1>::smem(G);
  return HB <= 1 ? Cfg<128, 1>::smem(G) : Cfg<128, kGroup>::smem(G);
}
inline const void* merge_of(int D) {
  return D == 128 ? reinterpret_cast<const void*>(&merge_kernel<128>) : reinterpret_cast<const void*>(&merge_kernel<64>);
}

}  // namespace biattn4

struct bi_attention4 {
  int Hq = 0, Hkv = 0, D = 0, G = 0, page_size = 0, split = 0;
  float scale = 0.0f, k_scale = 1.0f, v_scale = 1.0f;
  int device = 0, max_ctas = 0, smem = 0;
  int sms = 0, group_ctas = 0, group_smem = 0;   // of the blocks of kGroup heads (0: they are not for this shape)
  int cluster_ctas[2] = {0, 0};                  // resident blocks in clusters of two and of four
  uint32_t* d_status = nullptr;
  biattn_tc::Workspace ws;
};

namespace {

// The factor from a key's product with a query to the exponent of its weight.
double factor4(float scale, float k_scale) { return double(scale) * double(k_scale) * 1.4426950408889634; }

}  // namespace

BI_GEMM_API int bi_attention4_create(bi_attention4_t* out, int64_t num_q_heads, int64_t num_kv_heads, int64_t head_dim,
                                     int64_t page_size, float scale, float k_scale, float v_scale, int64_t split_size) {
  if (!out) return BI_GEMM_ERR_INVALID_ARG;
  *out = nullptr;
  auto fine = [](float s) { return s >= 0x1p-64f && s <= 0x1p64f; };
  if (!std::isfinite(scale) || scale <= 0.0f || !fine(k_scale) || !fine(v_scale) || factor4(scale, k_scale) > FLT_MAX)
    return BI_GEMM_ERR_INVALID_ARG;
  if (num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || page_size <= 0 || split_size < 0)
    return BI_GEMM_ERR_INVALID_ARG;
  const int64_t split = split_size ? split_size : biattn4::kDefaultSplit;
  if (num_q_heads % num_kv_heads != 0 || num_q_heads > 4096 || page_size > (1 << 20) || split % 128 != 0 || split > 4096 ||
      (head_dim != 64 && head_dim != 128))
    return BI_GEMM_ERR_UNSUPPORTED;
  const int64_t G = num_q_heads / num_kv_heads;
  if (G != 1 && G != 2 && G != 4 && G != 8) return BI_GEMM_ERR_UNSUPPORTED;
  int dev = 0, sms = 0;
  if (const int rc = bifp4::check_device(&dev)) return rc;
  // (the attribute is the kernel's, shared by every handle of the head size: the most any of them needs)
  auto ready = [&](int HB, int& smem, int& ctas) {
    const void* fn = biattn4::attn_of(int(head_dim), int(G), HB);
    smem = biattn4::smem_of(int(head_dim), int(G), HB);
    int per_sm = 0;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             biattn4::smem_of(int(head_dim), G <= 4 ? 4 : 8, HB)) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, biattn4::kThreads * std::max(HB, 1), smem) != cudaSuccess ||
        per_sm < 1)
      return false;
    ctas = per_sm * sms;
    return true;
  };
  // Blocks of four KV heads, for calls of many units (form4_of has their number): their warps read
  // neighbouring 64-byte pieces of long rows at about the same time.  us, 8 KV heads of 128 (a block a head / four):
  // 256 contexts of 4600 324 / 272, 64 of 4096 77 / 70, 128 of them at G = 8 167 / 156.  Rows of fewer or shorter
  // heads gain nothing: 4 of 128 51 / 53, 8 of 64 29 / 32.
  const bool grouped = head_dim == 128 && num_kv_heads >= 8 && num_kv_heads % biattn4::kGroup == 0;
  auto clusters = [&](int smem, int S, int& ctas) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(unsigned(S));
    cfg.blockDim = dim3(biattn4::kThreads);
    cfg.dynamicSmemBytes = size_t(smem);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(S);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, biattn4::attn_of(int(head_dim), int(G), 0), &cfg) != cudaSuccess) return false;
    ctas = n * S;
    return true;
  };
  int smem = 0, ctas = 0, group_smem = 0, group_ctas = 0, cluster_smem = 0, unused = 0, cluster_ctas[2] = {0, 0};
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || !ready(1, smem, ctas) ||
      !ready(0, cluster_smem, unused) || !clusters(cluster_smem, 2, cluster_ctas[0]) ||
      !clusters(cluster_smem, 4, cluster_ctas[1]) || (grouped && !ready(biattn4::kGroup, group_smem, group_ctas))) {
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
  h->max_ctas = ctas;
  h->smem = smem;
  h->sms = sms;
  h->group_ctas = group_ctas;
  h->group_smem = group_smem;
  h->cluster_ctas[0] = cluster_ctas[0];
  h->cluster_ctas[1] = cluster_ctas[1];
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

// How a launch of T tokens and `splits` splits at most runs.
struct Form4 {
  int HB;                  // KV heads of a block
  int32_t cluster;         // blocks of a cluster, whose splits merge there (0: none, the merge kernel does)
  int64_t blocks;
};
Form4 form4_of(const bi_attention4* h, int64_t T, int64_t splits) {
  const int64_t units = T * splits;
  // (us, a block a head / four: 32 x 1000, 512 heads' units, 16.3 / 16.6; 8 x 4096, 512 too, 17.8 / 17.0; 1 x 16384,
  // 256, 14.3 / 15.6; 4 x 4096, 256 too, 13.1 / 15.6; 1 x 700 7.9 / 14.4)
  const int HB = h->group_ctas && units * h->Hkv >= 3 * h->sms ? biattn4::kGroup : 1, across = h->Hkv / HB;
  // Clusters of two or four splits' blocks, where they run in one round: no second kernel.  us, without / with: 1 x
  // 700 8.9 / 7.9, 1 x 2000 9.3 / 8.1, 16 x 1000 14.5 / 11.8, 100 x 1000 at 8/1 heads 15.9 / 11.4; of eight: 1 x 4096
  // 9.3 / 9.0, but 4 x 4096 12.6 / 13.7.
  const int64_t S = splits <= 2 ? 2 : 4;
  if (HB == 1 && splits > 1 && splits <= 4 && T * h->Hkv * S <= h->cluster_ctas[S / 4])
    return {1, int32_t(S), T * h->Hkv * S};
  const int64_t chains = std::min<int64_t>(units, std::max(1, (HB == 1 ? h->max_ctas : h->group_ctas) / across));
  return {HB, 0, chains * across};
}

struct Layout4 {
  int64_t splits;
  size_t part, total;      // bytes of the partial sums, and with the references and sums behind them
};
Layout4 layout4_of(const bi_attention4* h, int64_t T, int64_t max_pos) {
  Layout4 w{max_pos / h->split + 1, 0, 0};
  // (a call's first launch is its largest: where that merges in clusters, all do)
  const int64_t first = std::min<int64_t>(T, biattn4::kTokens);
  if (w.splits > 1 && !form4_of(h, first, w.splits).cluster) {
    const size_t slots = size_t(first) * h->Hkv * size_t(w.splits) * h->G;
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

BI_GEMM_API int bi_attention4_run(bi_attention4_t h, const void* q, int64_t T, const int32_t* q_seq, const int32_t* q_pos,
                                  const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                                  int64_t num_pages, const int32_t* page_table, int64_t num_seqs, int64_t max_pages,
                                  int64_t max_pos, void* o, void* stream) {
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
  const int64_t per_token = int64_t(h->Hkv) * w.splits;
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
  p.num_pages = uint32_t(num_pages);      // (below 2^32 - 1, see above; a table's entry is below 2^31)
  p.max_pages = max_pages;
  p.B = num_seqs;
  p.Hq = h->Hq;
  p.Hkv = h->Hkv;
  p.G = h->G;
  p.page_size = h->page_size;
  p.split = h->split;
  p.max_splits = int32_t(w.splits);
  p.max_pos = int32_t(max_pos);
  int log2 = 0;
  while ((1 << log2) < h->page_size) ++log2;
  p.page_shift = log2;
  p.page_mul = uint32_t((uint64_t(1) << (30 + log2)) / uint64_t(h->page_size) + 1);
  p.c = float(factor4(h->scale, h->k_scale));
  p.v_scale = h->v_scale;
  for (int64_t t0 = 0; t0 < T; t0 += biattn4::kTokens) {
    p.T = int32_t(std::min<int64_t>(biattn4::kTokens, T - t0));
    p.q = static_cast<const uint16_t*>(q) + t0 * h->Hq * h->D;
    p.o = static_cast<uint16_t*>(o) + t0 * h->Hq * h->D;
    p.q_seq = q_seq + t0;
    p.q_pos = q_pos + t0;
    const Form4 f = form4_of(h, p.T, w.splits);
    p.cluster = f.cluster;
    if (const int rc = bifp4::launch(biattn4::attn_of(h->D, h->G, f.cluster ? 0 : f.HB), unsigned(f.blocks),
                                     biattn4::kThreads * f.HB, size_t(f.HB == 1 ? h->smem : h->group_smem), st, &p,
                                     unsigned(f.cluster)))
      return rc;
    if (w.splits > 1 && !f.cluster)
      if (const int rc = bifp4::launch(biattn4::merge_of(h->D),
                                       unsigned(p.T) * biattn4::merge_blocks(h->Hq, p.max_splits),
                                       32 * biattn4::kMergeWarps, 0, st, &p))
        return rc;
  }
  return BI_GEMM_OK;
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
  p.per_page = int64_t(h->page_size) * h->Hkv * (h->D / 8);
  constexpr int64_t kBlock = 256 * biattn4::kExpand;
  if (n > (((int64_t(1) << 31) - 1) * kBlock) / p.per_page) return BI_GEMM_ERR_UNSUPPORTED;
  p.pieces = n * p.per_page;
  p.k_scale = h->k_scale;
  p.v_scale = h->v_scale;
  const int64_t blocks = (p.pieces + kBlock - 1) / kBlock;
  if (blocks >= (int64_t(1) << 31)) return BI_GEMM_ERR_UNSUPPORTED;
  return bifp4::launch(reinterpret_cast<const void*>(&biattn4::expand_kernel), unsigned(blocks), 256, 0,
                       static_cast<cudaStream_t>(stream), &p);
}

BI_GEMM_API int bi_attention4_get_device_error(bi_attention4_t h, void* stream) {
  if (!h) return BI_GEMM_ERR_INVALID_ARG;
  return bifp4::read_status(h->d_status, static_cast<cudaStream_t>(stream), 0u);
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
  h->ws.release(h->device);
  if (h->d_status) cudaFree(h->d_status);
  delete h;
  return BI_GEMM_OK;
}
