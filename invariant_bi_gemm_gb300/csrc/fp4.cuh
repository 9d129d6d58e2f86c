// fp4.cuh — E2M1 codes and their block scales on the device: what quantisation, the append to a cache in 4
// bits and its readers share.  include/bi_fp4.h defines the format.
#pragma once
#include <cstdint>
#include <cstring>
#include <cuda_runtime.h>

#include "../../include/bi_gemm.h"

namespace bifp4 {

// Four pairs of fp32 values -> eight codes, element 0 in the lowest four bits (nearest, ties to even, at
// most 6 in size).
__device__ __forceinline__ uint32_t codes8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Eight codes -> four f16 pairs (exact), pair i the elements 2 i and 2 i + 1.
__device__ __forceinline__ void values8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Two E4M3 bytes (bits 0-7 and 8-15) -> an f16 pair (exact).
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t bytes) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(bytes));
  return r;
}
__device__ __forceinline__ float f16_lo(uint32_t h) {
  float f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}" : "=f"(f) : "r"(h));
  return f;
}
__device__ __forceinline__ float f16_hi(uint32_t h) {
  float f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, b;\n\t}" : "=f"(f) : "r"(h));
  return f;
}

// E4M3 byte of a value >= 0: nearest, ties to even, at most 448.
__device__ __forceinline__ uint32_t e4m3_of(float v) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %2, %1;\n\tcvt.u32.u16 %0, t;\n\t}"
      : "=r"(r)
      : "f"(v), "f"(0.0f));
  return r & 0xFFu;
}

constexpr uint32_t kNanE4M3 = 0x7Fu, kNanE8M0 = 0xFFu;

// What a block's largest size (as bf16 bits, non-finite ones above 0x7F7F) makes of it: the scale's byte,
// and the unit and factor with which `in_units` gives an element's place on the codes' grid.
struct Scale {
  uint32_t byte;
  float unit, inv;
  bool zero;          // every code is 0
  bool wide;          // above the largest scale: a quotient may be far above the codes'
};
// q = x / d for a d whose reciprocal r is known to an ulp: the product with r, corrected by its remainder, which is
// exact (Markstein's correction of a quotient).  With a rounded reciprocal it is the rounded quotient; with one an
// ulp off it still lies on the rounded quotient's side of every tie between codes, but for one divisor's mantissa
// (2^24 - 1, whose rcp.approx is the reciprocal that does not miss: the tests have the proof and that divisor).
__device__ __forceinline__ float divided(float x, float d, float r) {
  const float q = __fmul_rn(x, r);
  return __fmaf_rn(__fmaf_rn(-q, d, x), r, q);
}
// (inv_six_g: the rounded reciprocal of six_g)
__device__ __forceinline__ Scale nvfp4_scale(uint32_t amax_bits, float g, float six_g, float inv_six_g) {
  Scale s;
  const float amax = __uint_as_float(amax_bits << 16);
  s.wide = !(__fmul_rn(amax, inv_six_g) <= 448.0f);
  s.byte = s.wide ? 0x7Eu : e4m3_of(divided(amax, six_g, inv_six_g));
  s.unit = __fmul_rn(f16_lo(e4m3_pair(s.byte)), g);
  s.zero = s.byte == 0u;
  if (amax_bits >= 0x7F80u) s.byte = kNanE4M3, s.zero = true;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.inv) : "f"(s.unit));
  return s;
}
__device__ __forceinline__ Scale mxfp4_scale(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 7;                // (an exponent of a value below 2^-126 is no more than -127)
  Scale s;
  s.byte = e > 2u ? e - 2u : 0u;
  s.zero = amax_bits >= 0x7F80u;
  s.unit = 1.0f;
  s.wide = false;
  s.inv = s.zero ? 0.0f : __uint_as_float((254u - s.byte) << 23);
  if (s.zero) s.byte = kNanE8M0;
  return s;
}
// The places of two bf16 values (a word) on the codes' grid: x / unit.
template <bool kNv>
__device__ __forceinline__ void in_units(uint32_t w, const Scale& s, float& lo, float& hi) {
  const uint32_t a = w << 16, b = w & 0xFFFF0000u;
  if constexpr (!kNv) {
    lo = __fmul_rn(__uint_as_float(a), s.inv), hi = __fmul_rn(__uint_as_float(b), s.inv);
  } else {
    // `divided`, both at a time; a zero keeps its sign
    uint64_t x, r, d, q, e;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "r"(a), "r"(b));
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(s.inv));
    asm("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(-s.unit));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(x), "l"(r));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(e) : "l"(q), "l"(d), "l"(x));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(e), "l"(r), "l"(q));
    uint32_t y, z;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(y), "=r"(z) : "l"(q));
    lo = __uint_as_float(y | (a & 0x80000000u)), hi = __uint_as_float(z | (b & 0x80000000u));
  }
}

// Largest size, as bits, among the bf16 pairs of w (a NaN is above every number).
__device__ __forceinline__ uint32_t most_of(const uint32_t* w, int n) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < n; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
  return max(m & 0xFFFFu, m >> 16);
}

// Eight bf16 values (four words) -> their codes.  A wide block's quotients are out of the range that `divided`
// corrects: its values are clamped first (nvfp4, 14336 x 4096: 30.1 us, with a division in its place 32.4).
template <bool kNv>
__device__ __forceinline__ uint32_t quantise8(const uint32_t* w, const Scale& s) {
  if (s.zero && kNv) {
    // zeros keep their sign; a block that is not finite has codes of 0
    uint32_t r = 0;
    if (s.byte != kNanE4M3) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        r |= ((w[i] >> 15 & 1u) << (8 * i + 3)) | ((w[i] >> 31) << (8 * i + 7));
    }
    return r;
  }
  if (s.zero) return 0u;
  uint32_t x[4] = {w[0], w[1], w[2], w[3]};
  if (kNv && s.wide) {
    // sizes from 8 units on become 8 units, a 6 all the same
    const uint32_t most = __float_as_uint(__fmul_rn(8.0f, s.unit)) >> 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (x[i] & 0x80008000u) | __vminu2(x[i] & 0x7FFF7FFFu, most | most << 16);
  }
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) in_units<kNv>(x[i], s, v[2 * i], v[2 * i + 1]);
  return codes8(v);
}

// A scale's byte -> its value (NaN for the NaN byte).  (2^-127 is a denormal of fp32.)
template <bool kNv>
__device__ __forceinline__ float scale_value(uint32_t byte, float g) {
  if constexpr (kNv) return __fmul_rn(f16_lo(e4m3_pair(byte)), g);
  return byte == kNanE8M0 ? __uint_as_float(0x7FC00000u)
                          : __uint_as_float(byte ? byte << 23 : 1u << 22);
}
// Eight codes times their scale, as bf16 pairs (in fp32 and then bf16).
__device__ __forceinline__ void values_bf16(uint32_t codes, float scale, uint32_t* out) {
  uint32_t h[4];
  values8(codes, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = __fmul_rn(f16_lo(h[i]), scale), hi = __fmul_rn(f16_hi(h[i]), scale);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out[i]) : "f"(hi), "f"(lo));
  }
}

// ------------------------------------------------------------------ host

// The current device, which has to be an sm_103 one.
inline int check_device(int* dev) {
  int major = 0, minor = 0;
  if (cudaGetDevice(dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *dev) != cudaSuccess) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  return major == 10 && minor == 3 ? BI_GEMM_OK : BI_GEMM_ERR_UNSUPPORTED;
}

// A kernel of one parameter block, as a programmatic dependent of its predecessor.
inline int launch(const void* fn, unsigned blocks, unsigned threads, size_t smem, cudaStream_t st, void* params,
                  unsigned cluster = 0) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  void* args[1] = {params};
  if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  return BI_GEMM_OK;
}

// What a handle's status word says since it was last read; cleared.
inline int read_status(uint32_t* status, cudaStream_t st, uint32_t timeout_bit) {
  uint32_t s = 0;
  if (cudaMemcpyAsync(&s, status, sizeof(s), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  if (s == 0) return BI_GEMM_OK;
  if (cudaMemsetAsync(status, 0, sizeof(uint32_t), st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess) {
    cudaGetLastError();
    return BI_GEMM_ERR_CUDA;
  }
  return (s & timeout_bit) ? BI_GEMM_ERR_TIMEOUT : BI_GEMM_ERR_INVALID_ARG;
}

}  // namespace bifp4
