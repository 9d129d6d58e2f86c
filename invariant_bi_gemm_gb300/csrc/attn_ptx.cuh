// attn_ptx.cuh — what the tcgen05 attention kernels share: PTX wrappers beyond ptx.cuh's, the
// bounded wait of their roles, and the loads of a 128-position block of a paged cache.
#pragma once
#include <cstdint>
#include <cuda.h>

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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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

// One 128-position block of one KV head goes to shared memory as D / 64 column halves of 128 rows
// of 128 bytes, 128-byte swizzled (16-byte chunk c of row r at chunk c ^ (r % 8)), whoever writes it:
// `pg` holds lane l's page of the block (pages of min(page_size, 128) rows; -1: zeros), from
// block_page.  TMA: lane l issues its page's boxes; a page outside the cache loads a box from past
// the cache's end, which TMA fills with zeros.
__device__ __forceinline__ int32_t block_page(const Cache& c, const int32_t* row, int32_t pos0, int32_t last, int lane,
                                              bool* bad) {
  const int32_t step = c.page_size < kBlockPos ? c.page_size : kBlockPos;
  const int32_t pos = pos0 + lane * step;
  if (lane * step >= kBlockPos || pos > last) return -1;
  const int32_t page = row[pos / c.page_size];
  if (page < 0 || page >= c.num_pages) {
    *bad = true;
    return -1;
  }
  return page;
}

template <int D>
__device__ __forceinline__ void load_block_tma(uint32_t dst, uint32_t bar, const CUtensorMap* m, const Cache& c,
                                               int32_t page, int32_t pos0, int32_t kh, int lane) {
  const int32_t step = c.page_size < kBlockPos ? c.page_size : kBlockPos;
  if (lane == 0) ptx::mbar_arrive_expect_tx(bar, uint32_t(kBlockPos * D * 2));
  __syncwarp();
  if (lane * step < kBlockPos) {
    const int32_t row = page >= 0 ? page * c.page_size + (pos0 + lane * step) % c.page_size
                                  : int32_t(c.num_pages * c.page_size);
#pragma unroll
    for (int hh = 0; hh < D / 64; ++hh)
      tma_load_3d(dst + uint32_t(hh * kBlockPos * 128 + lane * step * 128), m, bar, hh * 64, kh, row);
  }
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
      const int64_t page = row[pos / c.page_size];
      if (page >= 0 && page < c.num_pages)
        off[k] = (page * c.page_size + pos % c.page_size) * c.Hkv * D;
      else
        *bad = true;
    }
  }
}

template <int D>
__device__ __forceinline__ void load_block_rows(uint32_t dst, const uint16_t* base, const int64_t (&off)[4],
                                                int32_t kh, int lane) {
  constexpr int CH = D / 8, RPI = 32 / CH;      // chunks per row, rows per step of the warp
  const int ch = lane % CH, sub = lane / CH;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
#pragma unroll 4
    for (int i = 0; i < 32 / RPI; ++i) {
      const int rl = i * RPI + sub;
      const int64_t o = __shfl_sync(0xFFFFFFFFu, off[k], rl);
      const int r = 32 * k + rl;
      ptx::cp_async_16(dst + uint32_t((ch >> 3) * kBlockPos * 128 + r * 128 + (((ch & 7) ^ (r & 7)) << 4)),
                       o >= 0 ? base + o + int64_t(kh) * D + ch * 8 : base, o >= 0 ? 16u : 0u);
    }
  }
}

// Page sizes whose blocks are whole TMA boxes: powers of two from 8 (one 1024-byte swizzle atom) up.
inline bool tma_page_size(int64_t ps) { return ps >= 8 && (ps & (ps - 1)) == 0; }

}  // namespace biattn_tc
