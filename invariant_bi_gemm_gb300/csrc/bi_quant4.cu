// bi_quant4.cu — rows of bf16 to E2M1 codes with block scales, and back, for sm_103a.  Implements the
// quantisation of include/bi_fp4.h.
//
// Bound: HBM bandwidth (2 bytes an element read, 0.53 or 0.56 written) and, close behind, the ALUs, which are busy for
// 60 % of the time: 14336 x 4096 take 25 us with mxfp4 (5.9 TB/s), 30 with nvfp4 (whose scales want a division each,
// and whose elements another), and 24 back (6.1 TB/s).  Two pieces a thread: one 27.5 and 34, four 26 and 40.  A
// thread has sixteen consecutive elements: a block of BI_NVFP4, half a block of BI_MXFP4 (the two halves meet in one
// shuffle).  K is a multiple of 128, so the lanes that share a block, or the four scales that lie side by side in a
// tile and leave as one 32-bit store, are always of one row, and threads run over the matrix without regard to where
// rows end.
#include <cuda_runtime.h>

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

namespace biq4 {

using namespace bifp4;

constexpr int kThreads = 256;
constexpr int kUnroll = 2;                // pieces of sixteen elements a thread loads at once

struct Params {
  const uint16_t* x;
  uint8_t* codes;
  uint8_t* scales;
  uint16_t* y;
  int64_t pieces;                        // of sixteen elements, in all
  int64_t stride;                        // of x, in elements
  int32_t per_row;                       // pieces of a row: 8 .. 2^20
  uint32_t row_mul;                      // i / per_row = i * row_mul >> row_shift for i < 2^21
  int32_t row_shift;
  float g, six_g, inv_six_g;
};

// Byte offset of the 32-bit word that holds the scales c .. c + 3 (c % 4 == 0) of row r.
__device__ __forceinline__ int64_t scale_word(int64_t r, int c, int per_tile_row) {
  return ((r >> 7) * per_tile_row + (c >> 2)) * 512 + int64_t((r & 31) * 16 + ((r >> 5) & 3) * 4);
}

// Where a block's pieces lie: its first one's row by one division, the others' by a multiplication.
struct Place {
  int64_t row0;
  uint32_t rest;
  __device__ __forceinline__ Place(const Params& p, int64_t first) {
    row0 = p.pieces >> 32 ? first / p.per_row : int64_t(uint32_t(first) / uint32_t(p.per_row));
    rest = uint32_t(first - row0 * p.per_row);
  }
  __device__ __forceinline__ void operator()(const Params& p, uint32_t off, int64_t& row, int& piece) const {
    const uint32_t i = rest + off, r = uint32_t(uint64_t(i) * p.row_mul >> p.row_shift);
    row = row0 + r;
    piece = int(i - r * uint32_t(p.per_row));
  }
};

template <bool kNv>
__global__ void __launch_bounds__(kThreads) quant_kernel(const Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t first = int64_t(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
  const Place place(p, int64_t(blockIdx.x) * (kThreads * kUnroll));
  uint32_t w[kUnroll][8];
  int64_t row[kUnroll];
  int piece[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = first + u * kThreads;
    place(p, threadIdx.x + u * kThreads, row[u], piece[u]);
    if (i < p.pieces) {
      const uint4* src = reinterpret_cast<const uint4*>(p.x + row[u] * p.stride + piece[u] * 16);
      const uint4 a = src[0], b = src[1];
      w[u][0] = a.x, w[u][1] = a.y, w[u][2] = a.z, w[u][3] = a.w;
      w[u][4] = b.x, w[u][5] = b.y, w[u][6] = b.z, w[u][7] = b.w;
    }
  }
  const int lane = int(threadIdx.x) & 31;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    // the pieces that are there end at a multiple of eight lanes: whole groups leave
    if (first + u * kThreads >= p.pieces) return;
    const uint32_t mask = 0xFFu << (lane & 24);
    uint32_t most = most_of(w[u], 8);
    if (!kNv) most = max(most, __shfl_xor_sync(mask, most, 1));
    const Scale s = kNv ? nvfp4_scale(most, p.g, p.six_g, p.inv_six_g) : mxfp4_scale(most);
    const uint2 codes = make_uint2(quantise8<kNv>(w[u], s), quantise8<kNv>(w[u] + 4, s));
    *reinterpret_cast<uint2*>(p.codes + (row[u] * p.per_row + piece[u]) * 8) = codes;
    // four scales to one lane
    if constexpr (kNv) {
      uint32_t word = s.byte << (8 * (lane & 3));
      word |= __shfl_xor_sync(mask, word, 1);
      word |= __shfl_xor_sync(mask, word, 2);
      if ((lane & 3) == 0)
        *reinterpret_cast<uint32_t*>(p.scales + scale_word(row[u], piece[u], p.per_row >> 2)) = word;
    } else {
      uint32_t word = s.byte << (8 * ((lane >> 1) & 3));
      word |= __shfl_xor_sync(mask, word, 2);
      word |= __shfl_xor_sync(mask, word, 4);
      if ((lane & 7) == 0)
        *reinterpret_cast<uint32_t*>(p.scales + scale_word(row[u], piece[u] >> 1, p.per_row >> 3)) = word;
    }
  }
}

// Eight elements a thread, so that a warp's stores are whole lines (sixteen: 30 us for 14336 x 4096, in halves of
// lines).
template <bool kNv>
__global__ void __launch_bounds__(kThreads) expand_kernel(const Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t first = int64_t(blockIdx.x) * (kThreads * 2 * kUnroll) + threadIdx.x, halves = 2 * p.pieces;
  const Place place(p, int64_t(blockIdx.x) * (kThreads * kUnroll));
  uint32_t codes[2 * kUnroll], byte[2 * kUnroll];
#pragma unroll
  for (int u = 0; u < 2 * kUnroll; ++u) {
    const int64_t i = first + u * kThreads;
    if (i < halves) {
      int64_t row;
      int piece;
      place(p, (threadIdx.x + u * kThreads) >> 1, row, piece);
      const int c = kNv ? piece : piece >> 1;
      codes[u] = reinterpret_cast<const uint32_t*>(p.codes)[i];
      byte[u] = p.scales[scale_word(row, c, kNv ? p.per_row >> 2 : p.per_row >> 3) + (c & 3)];
    }
  }
#pragma unroll
  for (int u = 0; u < 2 * kUnroll; ++u) {
    const int64_t i = first + u * kThreads;
    if (i >= halves) return;
    uint32_t out[4];
    values_bf16(codes[u], scale_value<kNv>(byte[u], p.g), out);
    *reinterpret_cast<uint4*>(p.y + i * 8) = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

}  // namespace biq4

struct bi_quant4 {
  int64_t K = 0;
  int nv = 0, device = 0;
  float g = 1.0f;
};

BI_GEMM_API int bi_quant4_create(bi_quant4_t* out, int64_t K, int32_t format, float tensor_scale) {
  if (!out) return BI_GEMM_ERR_INVALID_ARG;
  *out = nullptr;
  if (K <= 0 || (format != BI_MXFP4 && format != BI_NVFP4)) return BI_GEMM_ERR_INVALID_ARG;
  if (!(tensor_scale >= 0x1p-64f && tensor_scale <= 0x1p64f) || (format == BI_MXFP4 && tensor_scale != 1.0f))
    return BI_GEMM_ERR_INVALID_ARG;
  if (K % 128 != 0 || K > (1 << 24)) return BI_GEMM_ERR_UNSUPPORTED;
  int dev = 0;
  if (const int rc = bifp4::check_device(&dev)) return rc;
  bi_quant4* h = new (std::nothrow) bi_quant4();
  if (!h) return BI_GEMM_ERR_OOM;
  h->K = K;
  h->nv = format == BI_NVFP4;
  h->device = dev;
  h->g = tensor_scale;
  *out = h;
  return BI_GEMM_OK;
}

BI_GEMM_API int bi_quant4_scale_bytes(bi_quant4_t h, int64_t M, uint64_t* bytes) {
  if (!h || !bytes || M < 0) return BI_GEMM_ERR_INVALID_ARG;
  *bytes = uint64_t((M + 127) / 128) * uint64_t(h->K / (h->nv ? 64 : 128)) * 512;
  return BI_GEMM_OK;
}

namespace {

int quant4_launch(bi_quant4* h, const void* fn, biq4::Params& p, int64_t M, void* stream) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  if (dev != h->device) return BI_GEMM_ERR_INVALID_ARG;
  p.per_row = int32_t(h->K / 16);
  p.pieces = M * p.per_row;
  p.g = h->g;
  p.six_g = 6.0f * h->g;
  p.inv_six_g = 1.0f / p.six_g;
  int log2 = 0;
  while ((1 << log2) < p.per_row) ++log2;
  p.row_shift = 21 + log2;
  p.row_mul = uint32_t((uint64_t(1) << p.row_shift) / uint64_t(p.per_row) + 1);
  const int64_t per_block = biq4::kThreads * biq4::kUnroll, blocks = (p.pieces + per_block - 1) / per_block;
  static_assert(biq4::kThreads * biq4::kUnroll < (1 << 20), "Place: offsets below 2^21");
  if (blocks >= (int64_t(1) << 31)) return BI_GEMM_ERR_UNSUPPORTED;
  return bifp4::launch(fn, unsigned(blocks), biq4::kThreads, 0, static_cast<cudaStream_t>(stream), &p);
}

}  // namespace

BI_GEMM_API int bi_quant4_run(bi_quant4_t h, const void* x, int64_t M, int64_t x_stride, void* codes, void* scales,
                              void* stream) {
  if (!h || M < 0) return BI_GEMM_ERR_INVALID_ARG;
  if (M == 0) return BI_GEMM_OK;
  if (!x || !codes || !scales) return BI_GEMM_ERR_INVALID_ARG;
  if (x_stride % 8 != 0 || x_stride < h->K || M > (int64_t(1) << 31)) return BI_GEMM_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(codes) | reinterpret_cast<uintptr_t>(scales)) & 15u)
    return BI_GEMM_ERR_ALIGNMENT;
  biq4::Params p;
  std::memset(&p, 0, sizeof(p));
  p.x = static_cast<const uint16_t*>(x);
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = static_cast<uint8_t*>(scales);
  p.stride = x_stride;
  return quant4_launch(h, h->nv ? reinterpret_cast<const void*>(&biq4::quant_kernel<true>)
                                : reinterpret_cast<const void*>(&biq4::quant_kernel<false>), p, M, stream);
}

BI_GEMM_API int bi_quant4_expand(bi_quant4_t h, const void* codes, const void* scales, int64_t M, void* y,
                                 void* stream) {
  if (!h || M < 0) return BI_GEMM_ERR_INVALID_ARG;
  if (M == 0) return BI_GEMM_OK;
  if (!y || !codes || !scales) return BI_GEMM_ERR_INVALID_ARG;
  if (M > (int64_t(1) << 31)) return BI_GEMM_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(codes) | reinterpret_cast<uintptr_t>(scales)) & 15u)
    return BI_GEMM_ERR_ALIGNMENT;
  biq4::Params p;
  std::memset(&p, 0, sizeof(p));
  p.codes = static_cast<uint8_t*>(const_cast<void*>(codes));
  p.scales = static_cast<uint8_t*>(const_cast<void*>(scales));
  p.y = static_cast<uint16_t*>(y);
  return quant4_launch(h, h->nv ? reinterpret_cast<const void*>(&biq4::expand_kernel<true>)
                                : reinterpret_cast<const void*>(&biq4::expand_kernel<false>), p, M, stream);
}

BI_GEMM_API int bi_quant4_get_config(bi_quant4_t h, bi_quant4_config* c) {
  if (!h || !c) return BI_GEMM_ERR_INVALID_ARG;
  c->K = int32_t(h->K);
  c->format = h->nv ? BI_NVFP4 : BI_MXFP4;
  c->block = h->nv ? 16 : 32;
  c->threads = biq4::kThreads;
  return BI_GEMM_OK;
}

BI_GEMM_API int bi_quant4_destroy(bi_quant4_t h) {
  delete h;
  return BI_GEMM_OK;
}
