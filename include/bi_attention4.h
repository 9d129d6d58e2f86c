/*
 * bi_attention4.h — C ABI of the batch-invariant decode attention over a paged KV cache in 4 bits (in
 * libbi_gemm.so), sm_103a, and of the expansion of such a cache's pages to bf16.
 *
 * For each query token t — request b = q_seq[t] at position p = q_pos[t] — and each query head h (KV head
 * h / G, G = num_q_heads / num_kv_heads):
 *
 *     o[t, h, :] = sum_{j <= p} softmax_j(scale * q[t, h, :] . K_b[j, h/G, :]) V_b[j, h/G, :]
 *
 * as in bi_attention.h, with K and V held in the BI_NVFP4 format of bi_fp4.h along head_dim: E2M1 codes, two
 * a byte, and an E4M3 scale per 16 elements beside each row,
 *
 *     k_codes, v_codes   uint8 [num_pages, page_size, num_kv_heads, head_dim / 2]
 *     k_scales, v_scales uint8 [num_pages, page_size, num_kv_heads, head_dim / 16]
 *     K_b[j, kh, i] = k_scale * scale_i/16 * code_i of page_table[b][j / page_size], row j % page_size (V alike)
 *
 * which bi_qkrope_run4 fills; k_scale and v_scale are constants of the handle.  4.5 bits an element: 3.6 times
 * the positions of a bf16 cache in the same memory.
 *
 * A token with q_pos[t] = -1 sees no position: its output is zeros (an empty place of a padded batch).
 *
 * Batch invariance: the keys 0..p are cut at multiples of split_size, a split is four interleaved sequences of
 * 32 positions in ascending order, merged in order, and the n splits are merged in ascending order, above 16 of them
 * as eight consecutive groups of ceil(n / 8) and then group by group: all of it a function of p.  o[t] is a function
 * of q[t], p and K_b, V_b[0..p], bit for bit, whatever else the call holds.  Arithmetic: codes times scales exactly in f16;
 * queries in f16 relative to their head's largest element (a bf16 element at least 2^-25 of it is exact, any
 * other within 2^-36 of it); scores on the tensor cores in fp32; weights exp2 of the score less a running
 * reference of the maximum (moved when passed by more than 8), summed in fp32, rounded to f16 (11 bits) for
 * the product with the values, fp32 accumulation; fp32 merges and division; one bf16 rounding at the end.
 *
 * Conventions (as in bi_gemm.h, whose BI_GEMM_* return codes these functions use):
 *   - q, o bf16 [T, num_q_heads, head_dim]; page_table int32 [num_seqs, max_pages] (entry -1 = no page); q_seq,
 *     q_pos int32 [T].  All DEVICE pointers owned by the caller; the int32 arrays 4-byte aligned, the others
 *     16-byte (else BI_GEMM_ERR_ALIGNMENT).  o must not overlap the inputs.
 *   - Inputs the host cannot see (a q_seq outside [0, num_seqs) unless q_pos is -1, a q_pos below -1 or above
 *     max_pos, a position whose entry lies past max_pages or names no page in [0, num_pages)) are caught by
 *     the kernels: the token's output is then undefined and bi_attention4_get_device_error reports
 *     BI_GEMM_ERR_INVALID_ARG.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).  A handle is not thread-safe
 *     and must not be used on two streams at once; captured calls of one handle share its workspace, so their
 *     graphs must not run at the same time.
 */
#ifndef BI_ATTENTION4_H
#define BI_ATTENTION4_H

#include <stdint.h>

#include "bi_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct bi_attention4* bi_attention4_t;

typedef struct {
  int32_t num_q_heads, num_kv_heads, head_dim, page_size;
  int32_t split_size;       /* positions per split (fixed for the handle)                      */
  int32_t threads;          /* threads per block                                               */
  int32_t max_ctas;         /* resident blocks of one KV head                                  */
  int32_t tokens_per_launch; /* calls of more tokens are served as several                      */
} bi_attention4_config;

/* Create a handle.  Requirements (else BI_GEMM_ERR_UNSUPPORTED): head_dim 64 or 128; num_q_heads /
 * num_kv_heads in {1, 2, 4, 8}; num_q_heads <= 4096; page_size 1 .. 2^20; split_size (0 = 512) a multiple of
 * 128 up to 4096; an sm_103 device.  scale finite and > 0, k_scale and v_scale in [2^-64, 2^64], scale k_scale log2(e)
 * below 2^128 (else BI_GEMM_ERR_INVALID_ARG).  Checks on the arguments come before any CUDA call.  *out is NULL on
 * failure. */
int bi_attention4_create(bi_attention4_t* out, int64_t num_q_heads, int64_t num_kv_heads, int64_t head_dim,
                         int64_t page_size, float scale, float k_scale, float v_scale, int64_t split_size);

/* o = attention(q) for T query tokens.  max_pos: an upper bound (on the host) of every q_pos; it sizes the
 * workspace and changes no result.  T = 0 queues nothing.  The run grows the handle's workspace in stream
 * order when it needs more than before (BI_GEMM_ERR_OOM if that fails; BI_GEMM_ERR_SCRATCH_LIMIT in a call
 * being captured into a graph that needs more than an earlier call left; a graph stays valid when later
 * calls grow it), then queues the attention and, where max_pos leaves more than one split and the
 * splits' blocks do not merge among themselves, the merge (of each 512 tokens).  num_pages x page_size x num_kv_heads
 * below 2^32 - 1, max_pos below 2^30 (else BI_GEMM_ERR_UNSUPPORTED).  Asynchronous; only the blocks of a cluster, which
 * run together, wait for one another. */
int bi_attention4_run(bi_attention4_t h, const void* q, int64_t T, const int32_t* q_seq, const int32_t* q_pos,
                      const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                      int64_t num_pages, const int32_t* page_table, int64_t num_seqs, int64_t max_pages,
                      int64_t max_pos, void* o, void* stream);

/* Workspace bytes a run with T tokens and the bound max_pos needs (0: none, where the bound leaves one split or the
 * splits' blocks merge among themselves). */
int bi_attention4_workspace_size(bi_attention4_t h, int64_t T, int64_t max_pos, uint64_t* bytes);

/* k_out, v_out bf16 [n, page_size, num_kv_heads, head_dim]: the values of pages[i] (int32 [n], 4-byte aligned),
 * i = 0 .. n - 1, rounded as bi_quant4_expand rounds them, for operators that read a bf16 cache (bi_prompt_run over a
 * cached context: page i of the result is page i of its table).  An entry of -1 leaves page i as it was; any other
 * outside [0, num_pages) does too and is reported by bi_attention4_get_device_error.  One kernel; allocates nothing. */
int bi_attention4_expand(bi_attention4_t h, const void* k_codes, const void* k_scales, const void* v_codes,
                         const void* v_scales, int64_t num_pages, const int32_t* pages, int64_t n, void* k_out,
                         void* v_out, void* stream);

/* Synchronise `stream`; BI_GEMM_ERR_INVALID_ARG if a kernel caught a bad input since the last call (the
 * status is then cleared); BI_GEMM_ERR_CUDA if synchronisation failed; else BI_GEMM_OK. */
int bi_attention4_get_device_error(bi_attention4_t h, void* stream);

int bi_attention4_get_config(bi_attention4_t h, bi_attention4_config* c);

/* Release the handle and, behind everything that its device has queued, its workspace (NULL is a no-op).  Not to
 * be called while a stream is being captured. */
int bi_attention4_destroy(bi_attention4_t h);

#ifdef __cplusplus
}
#endif
#endif
