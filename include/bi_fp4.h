/*
 * bi_fp4.h — C ABI of the operators on matrices in 4 bits (in libbi_gemm.so), sm_103a: quantisation of rows,
 * the values that they stand for, and the batch-invariant product.
 *
 * Format.  A row of K elements is K E2M1 codes (OCP: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign in bit 3), two a
 * byte, element 2 i in the low half, and one scale per block of consecutive elements:
 *
 *   BI_MXFP4   32 elements, E8M0: value = code * 2^(byte - 127)          (255 is NaN)
 *   BI_NVFP4   16 elements, E4M3: value = code * scale * g               g: a constant of the tensor
 *
 * codes [rows, K / 2] uint8, row-major.  Scales lie in tiles of 128 rows x 4 blocks of 512 bytes, the layout
 * in which the tensor cores take them: row r's scale of block c is byte
 *   (r % 32) * 16 + (r / 32 % 4) * 4 + c % 4   of tile   (r / 128) * (C / 4) + c / 4,   C = K / block,
 * ceil(rows / 128) * C / 4 tiles in all; the bytes of rows that are not there are never used.
 *
 * Quantisation (fp32, each operation rounded once):
 *   BI_MXFP4   e = floor(log2 max|x|) - 2, at least -127; byte = e + 127; code = RN(x / 2^e)
 *   BI_NVFP4   scale = RN_e4m3(min(max|x| / (6 g), 448)); code = RN(x / (scale g)), 0 where the scale is 0
 * with RN to the nearest E2M1 value, ties to even, at most 6 in size, zeros keeping their sign.  A block with
 * an infinity or a NaN gets a NaN scale and codes of 0, so that it reads as NaN.  g is given, not derived
 * from the data: a row's bits would else depend on the rows around it.
 *
 * Product:  y[i, j] = alpha sum_k x[i, k] w[j, k]   with the values above (g left out: alpha carries the
 * tensor scales), x [M, K] and w [N, K] both row-major along K; products exact, fp32 accumulation on the
 * tensor cores (tcgen05 mxf4, 64 elements of K an instruction, ascending), alpha and one rounding at the
 * end.  Batch invariance: an element's sequence of instructions is a function of K alone; row i depends on
 * x[i] and w only, bit for bit, for every M.
 *
 * Conventions (as in bi_gemm.h, whose BI_GEMM_* return codes these functions use): data are DEVICE pointers
 * owned by the caller, 16-byte aligned (else BI_GEMM_ERR_ALIGNMENT); outputs must not overlap inputs;
 * `stream` is a cudaStream_t passed as void* (NULL = legacy default stream); nothing is allocated by a run,
 * which may be captured into a graph; a handle belongs to the device that was current when it was made
 * (else BI_GEMM_ERR_INVALID_ARG) and is not thread-safe.
 */
#ifndef BI_FP4_H
#define BI_FP4_H

#include <stdint.h>

#include "bi_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { BI_MXFP4 = 0, BI_NVFP4 = 1 } bi_fp4_format;

/* ---------------------------------------------------------------- quantisation */

typedef struct bi_quant4* bi_quant4_t;

typedef struct {
  int32_t K, format, block;   /* block: elements per scale */
  int32_t threads;
} bi_quant4_config;

/* Create a handle for rows of K elements.  Requirements: K a multiple of 128, 128 .. 2^24; an sm_103 device
 * (else BI_GEMM_ERR_UNSUPPORTED).  tensor_scale: g, in [2^-64, 2^64]; 1 for BI_MXFP4 (else
 * BI_GEMM_ERR_INVALID_ARG).  Checks on the arguments come before any CUDA call.  *out is NULL on failure. */
int bi_quant4_create(bi_quant4_t* out, int64_t K, int32_t format, float tensor_scale);

/* Bytes of the scales of M rows. */
int bi_quant4_scale_bytes(bi_quant4_t h, int64_t M, uint64_t* bytes);

/* codes [M, K / 2] and scales of x bf16 [M, K], rows x_stride elements apart (a multiple of 8, at least K;
 * else BI_GEMM_ERR_UNSUPPORTED).  Asynchronous, one kernel; M = 0 queues nothing. */
int bi_quant4_run(bi_quant4_t h, const void* x, int64_t M, int64_t x_stride, void* codes, void* scales,
                  void* stream);

/* y bf16 [M, K]: the values of codes and scales times the handle's tensor scale: scale g, then code times that, in fp32
 * (exact where g is a power of two), then to bf16. */
int bi_quant4_expand(bi_quant4_t h, const void* codes, const void* scales, int64_t M, void* y, void* stream);

int bi_quant4_get_config(bi_quant4_t h, bi_quant4_config* c);
int bi_quant4_destroy(bi_quant4_t h);

/* ---------------------------------------------------------------- product */

typedef struct bi_gemm4* bi_gemm4_t;

typedef struct {
  int32_t K, N, format, out_f32;
  int32_t tile_rows, tile_cols;  /* of y per CTA pair, and                                    */
  int32_t stages, max_groups;    /* the pipeline's depth and the pairs at most                 */
  int32_t few_rows;              /* up to this M, and for larger ones whose tiles are no more
                                    than the SMs, a form of smaller tiles runs: the same bits  */
  int32_t smem_bytes;
} bi_gemm4_config;

/* Create a handle for w [N, K].  Requirements: K a multiple of 128, 128 .. 2^24; N a multiple of 8, 8 ..
 * 2^24; an sm_103 device (else BI_GEMM_ERR_UNSUPPORTED); out_f32 0 (y bf16) or 1 (y fp32). */
int bi_gemm4_create(bi_gemm4_t* out, int64_t K, int64_t N, int32_t format, int32_t out_f32);

/* y [M, N] for codes x, w and their scales sx, sw in tiles.  alpha finite (else BI_GEMM_ERR_INVALID_ARG).
 * Asynchronous, one kernel; M = 0 queues nothing.  The waits inside the kernel are bounded (2 s): past the
 * limit it stops, y is undefined and bi_gemm4_get_device_error reports BI_GEMM_ERR_TIMEOUT. */
int bi_gemm4_run(bi_gemm4_t h, const void* x, const void* sx, int64_t M, const void* w, const void* sw,
                 float alpha, void* y, void* stream);

/* Synchronise `stream`; BI_GEMM_ERR_TIMEOUT if a bounded wait expired since the last call (the status is
 * then cleared); BI_GEMM_ERR_CUDA if synchronisation failed; else BI_GEMM_OK. */
int bi_gemm4_get_device_error(bi_gemm4_t h, void* stream);

int bi_gemm4_get_config(bi_gemm4_t h, bi_gemm4_config* c);
int bi_gemm4_destroy(bi_gemm4_t h);

#ifdef __cplusplus
}
#endif
#endif
