// bi_qkrope.cu — per-head RMSNorm of queries and keys, rotation by position and append of keys and
// values to the paged cache, in one pass over the fused projection's output, for sm_103a.
// Implements include/bi_qkrope.h.
//
// Bound: HBM bandwidth (every element read once, written once) beside the instructions, about eight
// operations an element; one launch's latency for a few tokens.  A head of D elements belongs to D / 8
// lanes, eight elements each: two runs of four that are rotation partners (dimensions 4 j and
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
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t widen(uint32_t w) { return pair(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t narrow(uint64_t v) {
  float lo, hi;
  unpair(v, lo, hi);
  return pack_bf16x2(lo, hi);
}

template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 4) qkrope_kernel(const Params p) {
  constexpr int LANES = D / 8;
  // Programmatic dependent launch: the block may start while the previous kernel finishes and
  // waits for it (and its memory) before its first global access.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = int(threadIdx.x);
  const int l = tid & (LANES - 1);                      // lane of the head
  const int groups = 1 << p.groups_log2;
  const int g = (tid / LANES) & (groups - 1);           // lane group of the token
  const int per_block = (kThreads / LANES) >> p.groups_log2;
  const int64_t t = int64_t(blockIdx.x) * per_block + ((tid / LANES) >> p.groups_log2);
  const bool live = t < p.T;                            // (whole lane groups: the shuffles stay inside them)
  const int H = p.Hq + 2 * p.Hkv;
  // this lane's two runs of four dimensions, and whether they are rotated
  const int half = p.rot >> 1, eighth = p.rot >> 3;
  const bool turned = l < eighth;
  const int da = kInterleaved || !turned ? 8 * l : 4 * l, db = kInterleaved || !turned ? da + 4 : da + half;

  const uint16_t* row = p.qkv + (live ? t : 0) * p.stride;
  uint2 ra[kHeads], rb[kHeads];
  auto load = [&](int h0) {
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const int h = h0 + k * groups;
      ra[k] = rb[k] = make_uint2(0, 0);
      if (live && h < H) {
        ra[k] = *reinterpret_cast<const uint2*>(row + h * D + da);
        rb[k] = *reinterpret_cast<const uint2*>(row + h * D + db);
      }
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
  // cosines and sines of the lane's pairs: of the four pairs (a, b) of its runs, or, interleaved, of each
  // two neighbours, both alike and the sine with either sign
  uint64_t co[kInterleaved ? 4 : 2], si[kInterleaved ? 4 : 2];
#pragma unroll
  for (int e = 0; e < (kInterleaved ? 4 : 2); ++e) co[e] = si[e] = 0;
  if (ok) {
    const int64_t page = p.table[int64_t(b) * p.max_pages + pos / p.page_size];
    if (page < 0 || page >= p.num_pages) {
      ok = false;
      atomicOr(p.status, kErrPage);
    }
    slot = page * p.page_size + pos % p.page_size;
    if (turned) {
      const float* c = p.cs + int64_t(pos) * p.rot + 4 * l;
      const float4 cv = *reinterpret_cast<const float4*>(c);
      const float4 sv = *reinterpret_cast<const float4*>(c + half);
      if constexpr (kInterleaved) {
        co[0] = pair(cv.x, cv.x), co[1] = pair(cv.y, cv.y), co[2] = pair(cv.z, cv.z), co[3] = pair(cv.w, cv.w);
        si[0] = pair(-sv.x, sv.x), si[1] = pair(-sv.y, sv.y), si[2] = pair(-sv.z, sv.z), si[3] = pair(-sv.w, sv.w);
      } else {
        co[0] = pair(cv.x, cv.y), co[1] = pair(cv.z, cv.w);
        si[0] = pair(sv.x, sv.y), si[1] = pair(sv.z, sv.w);
      }
    }
  }
  uint2 wqa = make_uint2(0, 0), wqb = wqa, wka = wqa, wkb = wqa;
  if (p.gq) {
    wqa = *reinterpret_cast<const uint2*>(p.gq + da), wqb = *reinterpret_cast<const uint2*>(p.gq + db);
    wka = *reinterpret_cast<const uint2*>(p.gk + da), wkb = *reinterpret_cast<const uint2*>(p.gk + db);
  }
  // The loop is uniform over a lane group, not over a warp: a shuffle names its group's lanes.
  const uint32_t mask = LANES == 16 ? 0xFFFFu << (tid & 16) : 0xFFu << (tid & 24);

  for (int h0 = g;; h0 += kHeads * groups) {
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const int h = h0 + k * groups;
      if (h >= H) break;
      if (h >= p.Hq + p.Hkv) {                          // values: as they are
        if (ok) {
          uint16_t* dst = p.vc + (slot * p.Hkv + (h - p.Hq - p.Hkv)) * D;
          *reinterpret_cast<uint2*>(dst + da) = ra[k];
          *reinterpret_cast<uint2*>(dst + db) = rb[k];
        }
        continue;
      }
      const bool key = h >= p.Hq;
      uint64_t x[4] = {widen(ra[k].x), widen(ra[k].y), widen(rb[k].x), widen(rb[k].y)};
      if (p.gq) {
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
            const uint64_t a = x[e], c = x[e + 2];
            float lo, hi;
            unpair(mul2(c, si[e]), lo, hi);
            x[e] = fma2(a, co[e], pair(-lo, -hi));
            x[e + 2] = fma2(c, co[e], mul2(a, si[e]));
          }
        }
      }
      if (ok) {
        uint16_t* dst = key ? p.kc + (slot * p.Hkv + (h - p.Hq)) * D : p.q_out + (t * p.Hq + h) * D;
        *reinterpret_cast<uint2*>(dst + da) = make_uint2(narrow(x[0]), narrow(x[1]));
        *reinterpret_cast<uint2*>(dst + db) = make_uint2(narrow(x[2]), narrow(x[3]));
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
