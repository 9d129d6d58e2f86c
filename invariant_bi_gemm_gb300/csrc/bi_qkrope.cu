// bi_qkrope.cu — per-head RMSNorm of queries and keys, rotation by position and append of keys and
// values to the paged cache, in one pass over the fused projection's output, for sm_103a.
// Implements include/bi_qkrope.h.
//
// Bound: HBM bandwidth (every element read once, written once, about eight operations each); one
// launch's latency for a few tokens.  A head of D elements belongs to D / 8 lanes, one 16-byte
// load, one store and eight fp32 values each, so the norm's sum is a butterfly inside the warp and
// a rotation partner D / 2 away is one shuffle.  A token has a power of two of such lane groups,
// each with up to kHeads heads at a time in registers: their loads are issued before the token's
// position is known, and its cosines, sines and the norm weights are read once for all of them.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>

#include "../../include/bi_qkrope.h"

#ifndef BI_GEMM_API
#define BI_GEMM_API extern "C" __attribute__((visibility("default")))
#endif

namespace biqkr {

constexpr int kThreads = 256;
constexpr int kHeads = 4;                // heads a lane group holds at a time
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
  float D, eps;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void widen(const uint4& v, float (&x)[8]) {
  x[0] = bf16_lo(v.x), x[1] = bf16_hi(v.x), x[2] = bf16_lo(v.y), x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z), x[5] = bf16_hi(v.z), x[6] = bf16_lo(v.w), x[7] = bf16_hi(v.w);
}

template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 4) qkrope_kernel(const Params p) {
  constexpr int LANES = D / 8;
  // Programmatic dependent launch: the block may start while the previous kernel finishes and
  // waits for it (and its memory) before its first global access.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = int(threadIdx.x);
  const int l = tid & (LANES - 1);                      // lane of the head: dimensions 8 l .. 8 l + 7
  const int groups = 1 << p.groups_log2;
  const int g = (tid / LANES) & (groups - 1);           // lane group of the token
  const int per_block = (kThreads / LANES) >> p.groups_log2;
  const int64_t t = int64_t(blockIdx.x) * per_block + ((tid / LANES) >> p.groups_log2);
  const bool live = t < p.T;                            // (whole lane groups: the shuffles stay inside them)
  const int H = p.Hq + 2 * p.Hkv;

  const uint16_t* row = p.qkv + (live ? t : 0) * p.stride + l * 8;
  uint4 raw[kHeads];
  auto load = [&](int h0) {
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const int h = h0 + k * groups;
      raw[k] = live && h < H ? *reinterpret_cast<const uint4*>(row + int64_t(h) * D) : make_uint4(0, 0, 0, 0);
    }
  };
  load(g);

  int32_t b = -1, pos = -1;
  if (live) {
    b = p.q_seq[t];
    pos = p.q_pos[t];
  }
  bool ok = live && b >= 0 && b < p.B && pos >= 0 && pos < p.num_positions &&
            int64_t(pos / p.page_size) < p.max_pages;
  if (live && !ok) atomicOr(p.status, kErrInput);
  int64_t slot = 0;
  float co[8], si[8];
  // the rotation of this lane's dimensions: cosines and (signed) sines per element
  const int half = p.rot >> 1;
  const bool turned = 8 * l < p.rot;
#pragma unroll
  for (int e = 0; e < 8; ++e) co[e] = 1.0f, si[e] = 0.0f;
  if (ok) {
    const int64_t page = p.table[int64_t(b) * p.max_pages + pos / p.page_size];
    if (page < 0 || page >= p.num_pages) {
      ok = false;
      atomicOr(p.status, kErrPage);
    }
    slot = page * p.page_size + pos % p.page_size;
    if (turned) {
      const float* c = p.cs + int64_t(pos) * p.rot;
      if constexpr (kInterleaved) {
        const float4 cv = *reinterpret_cast<const float4*>(c + 4 * l);
        const float4 sv = *reinterpret_cast<const float4*>(c + half + 4 * l);
        const float cc[4] = {cv.x, cv.y, cv.z, cv.w}, ss[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) co[e] = cc[e >> 1], si[e] = (e & 1) ? ss[e >> 1] : -ss[e >> 1];
      } else {
        const bool first = 8 * l < half;
        const int i = 8 * l - (first ? 0 : half);
#pragma unroll
        for (int e4 = 0; e4 < 8; e4 += 4) {
          const float4 cv = *reinterpret_cast<const float4*>(c + i + e4);
          const float4 sv = *reinterpret_cast<const float4*>(c + half + i + e4);
          co[e4] = cv.x, co[e4 + 1] = cv.y, co[e4 + 2] = cv.z, co[e4 + 3] = cv.w;
          si[e4] = first ? -sv.x : sv.x, si[e4 + 1] = first ? -sv.y : sv.y;
          si[e4 + 2] = first ? -sv.z : sv.z, si[e4 + 3] = first ? -sv.w : sv.w;
        }
      }
    }
  }
  // lane (of the warp) that holds the rotation partners of this lane's elements: half = 8 k, so
  // they sit k lanes away in the same head
  const int warp_lane = tid & 31;
  const int partner = kInterleaved || !turned ? warp_lane : warp_lane + (8 * l < half ? half / 8 : -(half / 8));

  for (int h0 = g;; h0 += kHeads * groups) {
    // The loop is uniform over a lane group, not over a warp: a shuffle names its group's lanes.
    const uint32_t mask = LANES == 16 ? 0xFFFFu << (warp_lane & 16) : 0xFFu << (warp_lane & 24);
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const int h = h0 + k * groups;
      if (h >= H) break;
      if (h >= p.Hq + p.Hkv) {
        if (ok)
          *reinterpret_cast<uint4*>(p.vc + (slot * p.Hkv + (h - p.Hq - p.Hkv)) * D + l * 8) = raw[k];
        continue;
      }
      const bool key = h >= p.Hq;
      float x[8];
      widen(raw[k], x);
      if (p.gq) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s = __fmaf_rn(x[e], x[e], s);
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) s = __fadd_rn(s, __shfl_xor_sync(mask, s, o));
        const float r = __frsqrt_rn(__fadd_rn(__fdiv_rn(s, p.D), p.eps));
        float w[8];
        widen(*reinterpret_cast<const uint4*>((key ? p.gk : p.gq) + l * 8), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(__fmul_rn(x[e], r), w[e]);
      }
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float other = kInterleaved ? x[e ^ 1] : __shfl_sync(mask, x[e], partner);
        y[e] = turned ? __fmaf_rn(x[e], co[e], __fmul_rn(other, si[e])) : x[e];
      }
      if (ok) {
        uint16_t* dst = key ? p.kc + (slot * p.Hkv + (h - p.Hq)) * D : p.q_out + (t * p.Hq + h) * D;
        *reinterpret_cast<uint4*>(dst + l * 8) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                            pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
      }
    }
    if (h0 + kHeads * groups >= H) break;
    load(h0 + kHeads * groups);
  }
}

using Kernel = void (*)(const Params);
inline Kernel kernel_of(int D, bool interleaved) {
  if (D == 128) return interleaved ? qkrope_kernel<128, true> : qkrope_kernel<128, false>;
  return interleaved ? qkrope_kernel<64, true> : qkrope_kernel<64, false>;
}

}  // namespace biqkr

struct bi_qkrope {
  int Hq = 0, Hkv = 0, D = 0, page_size = 0, rot = 0, interleaved = 0;
  float eps = 0.0f;
  int device = 0, groups_log2 = 0, per_block = 0;
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

BI_GEMM_API int bi_qkrope_run(bi_qkrope_t h, const void* qkv, int64_t T, int64_t qkv_stride, const void* gq,
                              const void* gk, const float* cos_sin, int64_t num_positions, const int32_t* q_seq,
                              const int32_t* q_pos, void* k_cache, void* v_cache, int64_t num_pages,
                              const int32_t* page_table, int64_t num_seqs, int64_t max_pages, void* q_out,
                              void* stream) {
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
  p.D = float(h->D);
  p.eps = h->eps;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(unsigned((T + h->per_block - 1) / h->per_block));
  cfg.blockDim = dim3(biqkr::kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, biqkr::kernel_of(h->D, h->interleaved != 0), p) != cudaSuccess) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  return BI_GEMM_OK;
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
  return BI_GEMM_ERR_INVALID_ARG;
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
  return BI_GEMM_OK;
}

BI_GEMM_API int bi_qkrope_destroy(bi_qkrope_t h) {
  if (!h) return BI_GEMM_OK;
  if (h->d_status) cudaFree(h->d_status);
  delete h;
  return BI_GEMM_OK;
}
