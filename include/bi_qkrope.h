/*
 * bi_qkrope.h — C ABI of the step between the fused projection and attention (in libbi_gemm.so),
 * sm_103a: per-head RMSNorm of queries and keys, rotation by position, append to the paged cache.
 *
 * For each token t — request b = q_seq[t] at position p = q_pos[t] — the row qkv[t] holds Hq query
 * heads, then Hkv key heads, then Hkv value heads of D elements.  For every query and key head x
 * with norm weight g (gq or gk), in fp32:
 *
 *     r = 1 / sqrt( (sum_j x_j^2) / D + eps ),   y_j = (x_j r) g_j        (y = x without weights)
 *     (y_a, y_b) <- (y_a cos_i - y_b sin_i,  y_b cos_i + y_a sin_i)       i = 0 .. rot_dim / 2 - 1
 *
 * with (a, b) = (i, i + rot_dim / 2), or (2 i, 2 i + 1) for an interleaved handle; cos_i =
 * cos_sin[p, i], sin_i = cos_sin[p, rot_dim / 2 + i]; dimensions from rot_dim on are not rotated.
 * One rounding to bf16 at the end.  Query heads go to q_out[t]; key heads and, unchanged, value
 * heads to the cache slot of (b, p), k_cache[page_table[b][p / page_size], p % page_size, kh, :]
 * and v_cache alike: the layout that bi_attention.h and bi_prompt.h read.
 *
 * Batch invariance: a head's squares are summed by D / 8 lanes, each its eight elements (fixed by
 * rot_dim and the pairing) in two chains of fma, combined by a fixed xor butterfly; nothing else of
 * the call enters, so q_out[t] and the slot's contents are a function of qkv[t], the weights and p.
 *
 * Conventions (as in bi_gemm.h, whose BI_GEMM_* return codes these functions use):
 *   - qkv bf16 [T, (Hq + 2 Hkv) D] with rows qkv_stride elements apart; gq, gk bf16 [D] (both, or
 *     both NULL: no norm); cos_sin fp32 [num_positions, rot_dim]; q_out bf16 [T, Hq, D]; k_cache,
 *     v_cache bf16 [num_pages, page_size, Hkv, D]; page_table int32 [num_seqs, max_pages] (entry
 *     -1 = no page); q_seq, q_pos int32 [T].  All DEVICE pointers owned by the caller; the bf16
 *     and fp32 arrays 16-byte aligned, the int32 ones 4-byte (else BI_GEMM_ERR_ALIGNMENT).
 *     Outputs must not overlap inputs.
 *   - Inputs the host cannot see (a q_seq outside [0, num_seqs), a q_pos that is negative, not
 *     below num_positions or past max_pages pages, a page outside [0, num_pages)) are caught by
 *     the kernel: the token's q_out row and slot are left as they were and
 *     bi_qkrope_get_device_error reports BI_GEMM_ERR_INVALID_ARG.
 *   - The (request, position) pairs of a call name different slots.  Two tokens of one call on the
 *     same slot leave it with 8-byte pieces of either.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).  A handle keeps
 *     no workspace, only its status word; it is not thread-safe.
 */
#ifndef BI_QKROPE_H
#define BI_QKROPE_H

#include <stdint.h>

#include "bi_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct bi_qkrope* bi_qkrope_t;

typedef struct {
  int32_t num_q_heads, num_kv_heads, head_dim, page_size;
  int32_t rot_dim;            /* rotated dimensions of a head                              */
  int32_t interleaved;        /* 1: pairs (2 i, 2 i + 1); 0: pairs (i, i + rot_dim / 2)      */
  int32_t threads;            /* threads per block of the form for few tokens                */
  int32_t tokens_per_block;
  int32_t ring_tokens;        /* the form for many tokens: tokens on their way per block (0:
                                 rows too long for it), and its resident blocks              */
  int32_t ring_ctas;
  int32_t ring_from;          /* the T from which it runs (bi_qkrope_run4's may be lower)     */
} bi_qkrope_config;

/* Create a handle.  Requirements: head_dim 64 or 128; rot_dim a multiple of 16, 16..head_dim;
 * at most 4096 heads in all; page_size 1..2^20; an sm_103 device (else BI_GEMM_ERR_UNSUPPORTED).
 * Non-positive sizes, eps not finite or negative, interleaved not 0 or 1:
 * BI_GEMM_ERR_INVALID_ARG.  Checks on the arguments come before any CUDA call.  *out is NULL on
 * failure. */
int bi_qkrope_create(bi_qkrope_t* out, int64_t num_q_heads, int64_t num_kv_heads, int64_t head_dim,
                     int64_t page_size, int64_t rot_dim, int32_t interleaved, float eps);

/* One call for T tokens (T = 0 queues nothing).  qkv_stride: elements between rows, a multiple of
 * 8 and at least (Hq + 2 Hkv) D (else BI_GEMM_ERR_UNSUPPORTED).  Asynchronous, one kernel;
 * allocates nothing; safe inside CUDA graph capture. */
int bi_qkrope_run(bi_qkrope_t h, const void* qkv, int64_t T, int64_t qkv_stride, const void* gq, const void* gk,
                  const float* cos_sin, int64_t num_positions, const int32_t* q_seq, const int32_t* q_pos,
                  void* k_cache, void* v_cache, int64_t num_pages, const int32_t* page_table, int64_t num_seqs,
                  int64_t max_pages, void* q_out, void* stream);

/* bi_qkrope_run into a cache in 4 bits, the layout that bi_attention4.h reads (q_out is bi_qkrope_run's):
 * a key head, rounded to bf16 as above, and a value head are quantised in the BI_NVFP4 format of bi_fp4.h with the
 * tensor scales k_scale and v_scale (in [2^-64, 2^64], else BI_GEMM_ERR_INVALID_ARG) and go to the slot's rows of
 * k_codes, v_codes [num_pages, page_size, Hkv, D / 2] and k_scales, v_scales [num_pages, page_size, Hkv, D / 16]
 * (uint8, 16-byte aligned).  So the cache holds the quantised rows of the one that bi_qkrope_run would fill, bit
 * for bit.  Two tokens of one call on the same slot leave it with pieces of either.
 * A token with q_pos[t] = -1, whatever its q_seq, is an empty place of a padded batch, as bi_attention4_run has it:
 * nothing is appended, its q_out row stays as it was, and no error is reported (bi_qkrope_run reports one). */
int bi_qkrope_run4(bi_qkrope_t h, const void* qkv, int64_t T, int64_t qkv_stride, const void* gq, const void* gk,
                   const float* cos_sin, int64_t num_positions, const int32_t* q_seq, const int32_t* q_pos,
                   void* k_codes, void* k_scales, void* v_codes, void* v_scales, float k_scale, float v_scale,
                   int64_t num_pages, const int32_t* page_table, int64_t num_seqs, int64_t max_pages, void* q_out,
                   void* stream);

/* Synchronise `stream`; BI_GEMM_ERR_TIMEOUT if a bounded wait (2 s) expired, else
 * BI_GEMM_ERR_INVALID_ARG if a kernel caught a bad input, since the last call (the status is then
 * cleared); BI_GEMM_ERR_CUDA if synchronisation failed; else BI_GEMM_OK. */
int bi_qkrope_get_device_error(bi_qkrope_t h, void* stream);

int bi_qkrope_get_config(bi_qkrope_t h, bi_qkrope_config* c);

/* Release the handle (NULL is a no-op). */
int bi_qkrope_destroy(bi_qkrope_t h);

#ifdef __cplusplus
}
#endif
#endif
