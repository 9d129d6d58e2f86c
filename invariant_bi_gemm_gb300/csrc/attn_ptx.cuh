// attn_ptx.cuh — what the tcgen05 attention kernels share: PTX wrappers beyond ptx.cuh's, the
// bounded wait of their roles, and the loads of a 128-position block of a paged cache.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <mutex>
#include <vector>

#include "../../include/bi_gemm.h"
#include "ptx.cuh"

namespace biattn_tc {

namespace ptx = bigemm::ptx;

constexpr int kBlockPos = 128;                // positions of a key / value block
constexpr uint32_t kErrInput = 1u;            // lengths, positions or the page table's extent
constexpr uint32_t kErrPage = 2u;             // page outside [0, num_pages)
constexpr uint32_t kErrBound = 4u;            // a position above the host's max_pos
constexpr uint32_t kErrTimeout = 8u;          // a bounded wait expired
constexpr uint64_t kTimeoutNs = 2000000000ull;

// 3-D tiled bulk tensor load global -> shared (c0 innermost), completion counted in bytes on `bar`.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int32_t c0,
                                            int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// 3-D tiled bulk tensor store shared -> global, in this thread's bulk-async group.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, uint32_t src, int32_t c0, int32_t c1, int32_t c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(c0), "r"(c1), "r"(c2), "r"(src)
               : "memory");
}
// Wait until this thread's bulk groups have been written.
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// As tma_load_3d, five dimensions.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3, int32_t c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
      : "memory");
}

// D[tmem] (+)= A[tmem] x B[smem desc], bf16 inputs, fp32 accumulator.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Each thread of the warp writes 16 / 32 consecutive 32-bit columns of its own TMEM lane.
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void ld_shared_v4(uint32_t a, uint32_t (&w)[4]) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a) : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Three-input maximum (a NaN is passed over), and packed pairs of fp32 in one instruction.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Shared-memory matrix descriptor, 128-byte swizzle: start, leading / stride byte offsets, version 1.
__device__ __forceinline__ uint64_t sdesc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t((lbo >> 4) & 0x3FFFu) << 16) |
         (uint64_t((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}
// tcgen05 instruction descriptor (kind::f16): D = f32, A = B = bf16.
constexpr __host__ __device__ uint32_t idesc_bf16(int M, int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn_major ? 1u << 15 : 0u) | (b_mn_major ? 1u << 16 : 0u) |
         (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

// Named barrier `id` for 128 threads (four warps) with an OR over their predicates: every one of them
// gets the same answer.
__device__ __forceinline__ bool bar_or(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(uint32_t(x)), "r"(id)
      : "memory");
  return r != 0;
}

// An arrival that publishes nothing (what it announces is that reads are over): unlike
// ptx::mbar_arrive it does not order this thread's stores before it.
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// What every bounded wait of a block looks at.
struct Sync {
  volatile uint32_t* abort;   // shared: set once any role gives up
  uint32_t* status;           // global error word
  uint64_t timeout_ns;
};

// Bounded wait for a phase of a barrier: false (status and abort set) past the time limit, or soon
// after another role has aborted.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const Sync& s) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (*s.abort) return false;
    if (ptx::globaltimer() - t0 > s.timeout_ns) {
      atomicOr(s.status, kErrTimeout);
      *s.abort = 1u;
      return false;
    }
  }
  return true;
}

// The paged cache of a call and how a kernel loads a block of it.
struct Cache {
  const uint16_t* kc;
  const uint16_t* vc;
  const int32_t* table;       // [B, max_pages]
  int64_t num_pages, max_pages;
  int32_t Hkv, page_size;
};

// One 128-position block of one KV head goes to shared memory as 16 groups of 8 rows, a group as its
// D / 64 column halves of 8 rows of 128 bytes, 128-byte swizzled (16-byte chunk c of row r at chunk
// c ^ (r % 8)).  So a page of any multiple of 8 rows is one TMA box (64 x 8 x halves x groups of the
// cache seen as [Hkv][groups][halves][8][64]): a box costs its issue about 48 clocks, whatever it
// holds, and with a box per page and half, pages of 16 positions had bounded the prompt kernel.
template <int D>
struct BlockLayout {
  static constexpr uint32_t GROUP = D / 64 * 1024;            // bytes of 8 rows
  static constexpr uint32_t HALF = 1024;                      // between the halves of a group
  // 16-byte chunk c of row r
  __device__ static uint32_t chunk(int r, int c) {
    return uint32_t(r >> 3) * GROUP + uint32_t(c >> 3) * HALF + uint32_t((r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4));
  }
  // descriptors of the block at `a`: rows as the MMA's rows or columns, k step of 16 dimensions ...
  __device__ static uint64_t by_row(uint32_t a, int k) {
    return sdesc_sw128(a + uint32_t(k >> 2) * HALF + uint32_t(k & 3) * 32, 16, GROUP);
  }
  // ... or dimensions as rows or columns, k step of 16 positions
  __device__ static uint64_t by_dim(uint32_t a, int k) { return sdesc_sw128(a + uint32_t(k) * 2 * GROUP, HALF, GROUP); }
};

// TMA: lane l issues the box of the block's l-th page (of min(page_size, 128) rows).  block_box gives
// its first group in the cache, ahead of the wait for the ring: the page at or behind `last` and a page
// outside the cache (which sets *bad) load a box from past the cache's end, which TMA fills with zeros.
__device__ __forceinline__ int32_t block_box(const Cache& c, const int32_t* row, int32_t pos0, int32_t last, int lane,
                                             bool* bad) {
  const int32_t step = c.page_size < kBlockPos ? c.page_size : kBlockPos;
  const int32_t pos = pos0 + lane * step;
  const int32_t past = int32_t(c.num_pages * c.page_size / 8);
  if (lane * step >= kBlockPos || pos > last) return past;
  const int32_t page = __ldcg(row + pos / c.page_size);
  if (page < 0 || page >= c.num_pages) {
    *bad = true;
    return past;
  }
  return (page * c.page_size + pos % c.page_size) / 8;
}

template <int D>
__device__ __forceinline__ void load_block_tma(uint32_t dst, uint32_t bar, const CUtensorMap* m, const Cache& c,
                                               int32_t box, int32_t kh, int lane) {
  const int32_t step = c.page_size < kBlockPos ? c.page_size : kBlockPos;
  if (lane == 0) ptx::mbar_arrive_expect_tx(bar, uint32_t(kBlockPos * D * 2));
  __syncwarp();
  if (lane * step < kBlockPos)
    tma_load_5d(dst + uint32_t(lane * (step / 8)) * BlockLayout<D>::GROUP, m, bar, 0, 0, 0, box, kh);
}

// Any page size: lane l owns rows l, l + 32, l + 64, l + 96 of the block; off[k] = the row's element
// offset in the caches (without the KV head), -1 for a row of no page.
__device__ __forceinline__ void block_rows(const Cache& c, const int32_t* row, int32_t pos0, int32_t last, int D,
                                           int lane, int64_t (&off)[4], bool* bad) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int32_t pos = pos0 + lane + 32 * k;
    off[k] = -1;
    if (pos <= last) {
      const int64_t page = __ldcg(row + pos / c.page_size);
      if (page >= 0 && page < c.num_pages)
        off[k] = (page * c.page_size + pos % c.page_size) * c.Hkv * D;
      else
        *bad = true;
    }
  }
}

// Eight lanes copy 128 bytes of a row, so an instruction takes four rows and a row's offset is fetched
// from its lane once for both of its halves.
template <int D>
__device__ __forceinline__ void load_block_rows(uint32_t dst, const uint16_t* base, const int64_t (&off)[4],
                                                int32_t kh, int lane) {
  const int sub = lane >> 3, ch = lane & 7;
  const uint16_t* src0 = base + int64_t(kh) * D + ch * 8;
  const uint32_t even = BlockLayout<D>::chunk(sub, ch), odd = BlockLayout<D>::chunk(sub + 4, ch);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t o = __shfl_sync(0xFFFFFFFFu, off[k], 4 * i + sub);
      const uint32_t to = dst + uint32_t(4 * k + (i >> 1)) * BlockLayout<D>::GROUP + ((i & 1) ? odd : even);
      const uint16_t* src = o >= 0 ? src0 + o : base;
      const uint32_t bytes = o >= 0 ? 16u : 0u;
#pragma unroll
      for (int h = 0; h < D / 64; ++h) ptx::cp_async_16(to + uint32_t(h) * BlockLayout<D>::HALF, src + h * 64, bytes);
    }
  }
}

// Page sizes whose blocks are whole TMA boxes: powers of two from 8 (one 1024-byte swizzle atom) up.
inline bool tma_page_size(int64_t ps) { return ps >= 8 && (ps & (ps - 1)) == 0; }

// A handle's device scratch, grown in stream order.  A block that a captured call uses lives until the
// handle does, since the graph may still be replayed; any other is freed behind the calls that used it.
struct Workspace {
  // growth doubles up to this step, so that a bound that climbs with every call does not move the
  // scratch at each, and no handle holds more than this beyond what a call has asked for
  static constexpr size_t kStep = size_t(64) << 20;
  void* at = nullptr;
  size_t bytes = 0;
  bool captured = false;        // a captured call uses `at`
  std::vector<void*> earlier;

  // A call being captured cannot allocate for good: it uses what earlier calls left.
  int need(size_t n, cudaStream_t st) {
    if (n == 0) return BI_GEMM_OK;
    cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &capturing) != cudaSuccess) {
      cudaGetLastError();
      return BI_GEMM_ERR_CUDA;
    }
    if (n <= bytes) {
      captured |= capturing != cudaStreamCaptureStatusNone;
      return BI_GEMM_OK;
    }
    if (capturing != cudaStreamCaptureStatusNone) return BI_GEMM_ERR_SCRATCH_LIMIT;
    try {
      if (captured) earlier.reserve(earlier.size() + 1);
    } catch (...) {
      return BI_GEMM_ERR_OOM;
    }
    const size_t step = bytes + (bytes < kStep ? bytes : kStep);
    size_t size = n > step ? n : step;
    void* p = allocate(size, st);
    if (!p && size > n) p = allocate(size = n, st);
    if (!p && at && !captured) {          // the block that it replaces may be the room it needs
      cudaFreeAsync(at, st);
      at = nullptr;
      bytes = 0;
      p = allocate(size, st);
    }
    if (!p) return BI_GEMM_ERR_OOM;
    if (captured) earlier.push_back(at);
    else if (at) cudaFreeAsync(at, st);
    at = p;
    bytes = size;
    captured = false;
    return BI_GEMM_OK;
  }
  void release() {
    if (at) cudaFree(at);
    for (void* p : earlier) cudaFree(p);
    at = nullptr;
    bytes = 0;
    captured = false;
    earlier.clear();
  }
  static void* allocate(size_t n, cudaStream_t st) {
    void* p = nullptr;
    if (cudaMallocAsync(&p, n, st) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    return p;
  }
};

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

inline bool encode_bf16(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                        const cuuint32_t* box) {
  auto fn = encode_fn();
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cuuint32_t(rank), const_cast<void*>(base), dims, strides, box,
                  ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query rows [T, H, D]: boxes of 64 dims x `heads` x `tokens`, zero fill outside.
inline bool encode_queries(CUtensorMap* m, const void* q, int64_t T, int H, int D, int heads, int tokens) {
  const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(H), cuuint64_t(T)};
  const cuuint64_t strides[2] = {cuuint64_t(D) * 2, cuuint64_t(H) * D * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(heads), cuuint32_t(tokens)};
  return encode_bf16(m, q, 3, dims, strides, box);
}

// A cache of `rows` = pages x page_size rows for load_block_tma.
inline bool encode_pages(CUtensorMap* m, const void* cache, int64_t rows, int Hkv, int D, int page_size) {
  const cuuint64_t pitch = cuuint64_t(Hkv) * D * 2;
  const cuuint64_t dims[5] = {64, 8, cuuint64_t(D / 64), cuuint64_t(rows / 8), cuuint64_t(Hkv)};
  const cuuint64_t strides[4] = {pitch, 128, 8 * pitch, cuuint64_t(D) * 2};
  const cuuint32_t box[5] = {64, 8, cuuint32_t(D / 64), cuuint32_t((page_size < kBlockPos ? page_size : kBlockPos) / 8), 1};
  return encode_bf16(m, cache, 5, dims, strides, box);
}

}  // namespace biattn_tc
