/*
 * bi_prompt.h — C ABI of the batch-invariant prompt attention (in libbi_gemm.so), sm_103a: causal
 * attention of whole prompts, or of chunks of them behind a cached context, packed one after the
 * other, over the paged KV cache that bi_attention.h reads.
 *
 * Sequence b (0 <= b < num_seqs) has the n_b = q_start[b + 1] - q_start[b] query tokens q[q_start[b]
 * ...], the positions q_pos0[b], q_pos0[b] + 1, ... of request b.  For its token at position p and
 * query head h (KV head h / G, G = num_q_heads / num_kv_heads):
 *
 *     o[t, h, :] = sum_{j <= p} softmax_j(scale * q[t, h, :] . K_b[j, h/G, :]) V_b[j, h/G, :]
 *
 * K_b[j, kh, :] = k_cache[page_table[b][j / page_size], j % page_size, kh, :] (V alike).  The cache
 * holds positions 0 .. q_pos0[b] + n_b - 1 of every request before the call, its own tokens
 * included (bi_qkrope_run writes them): a whole prompt has q_pos0[b] = 0, a chunk the number of
 * positions cached before it.
 *
 * Batch invariance: tiles of queries and blocks of 128 keys are cut at fixed positions of the
 * request, whatever part of it a call holds; a row's blocks are taken in ascending order with its
 * own running maximum and sum.  So o[t] is a function of q[t], p and K_b, V_b[0..p] only, bit for
 * bit: it depends neither on the other sequences, nor on the chunk that the token came in, nor on
 * where pages sit or how large they are.  Arithmetic: scores on the tensor cores (bf16 products,
 * fp32 accumulation); weights exp2 of the score minus a running reference in fp32, rounded to bf16
 * for the product with the values (fp32 accumulation) and summed in fp32 unrounded; one division
 * and one bf16 rounding at the end.  The bits are this operator's own: bi_attention_run, which
 * serves single tokens, keeps 16 bits of every weight and sums in another order.
 *
 * Values that are not finite count where they are seen and nowhere else: a key or value at a
 * position behind p (or in an unused slot of a page) never reaches o[t].  An infinite value that is
 * seen under a weight that has underflowed to zero leaves an infinity or a NaN: which of the two is,
 * like every other bit, a function of q[t], p and K_b, V_b[0..p] alone.
 *
 * Conventions (as in bi_gemm.h, whose BI_GEMM_* return codes these functions use):
 *   - q [T, num_q_heads, head_dim] and o likewise, bf16 row-major; k_cache, v_cache
 *     [num_pages, page_size, num_kv_heads, head_dim] bf16; page_table int32 [num_seqs,
 *     max_pages] (entry -1 = no page); q_start int32 [num_seqs + 1], ascending; q_pos0 int32
 *     [num_seqs].  All DEVICE pointers owned by the caller; the bf16 arrays 16-byte aligned, the
 *     int32 ones 4-byte (else BI_GEMM_ERR_ALIGNMENT).  o must not overlap the inputs.
 *   - Rows of o before q_start[0] and from q_start[num_seqs] on are left as they were.
 *   - Inputs the host cannot see (a q_start that descends or leaves [0, T], a negative q_pos0, a
 *     last position above max_pos or past max_pages pages, a page outside [0, num_pages)) are
 *     caught by the kernels: the sequence's output is then undefined (it is not computed, or a bad
 *     page's rows count as zeros; of a q_start that descends nothing is computed) and
 *     bi_prompt_get_device_error reports BI_GEMM_ERR_INVALID_ARG.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).  A handle is
 *     not thread-safe and must not be used on two streams at once; captured calls of one handle
 *     share its workspace, so their graphs must not run at the same time.
 */
#ifndef BI_PROMPT_H
#define BI_PROMPT_H

#include <stdint.h>

#include "bi_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct bi_prompt* bi_prompt_t;

typedef struct {
  int32_t num_q_heads, num_kv_heads, head_dim, page_size;
  int32_t tile_positions;   /* positions of a work unit (two tiles of 128 query rows)        */
  int32_t block_positions;  /* keys per block                                              */
  int32_t stages;           /* depth of the key / value ring                                */
  int32_t threads;          /* threads per block of the attention kernel                    */
  int32_t max_ctas;         /* persistent grid bound (one block per SM)                     */
  int32_t tma_pages;        /* 1: pages are loaded as TMA boxes; 0: row by row (cp.async)    */
} bi_prompt_config;

/* Create a handle.  Requirements (else BI_GEMM_ERR_UNSUPPORTED): head_dim 64 or 128;
 * num_q_heads / num_kv_heads = G in {1, 2, 4, 8}; page_size 1..2^20; an sm_103 device.  scale must
 * be finite and > 0 (else BI_GEMM_ERR_INVALID_ARG; 1 / sqrt(head_dim) is the usual value).  Checks
 * on the arguments come before any CUDA call.  *out is NULL on failure. */
int bi_prompt_create(bi_prompt_t* out, int64_t num_q_heads, int64_t num_kv_heads, int64_t head_dim,
                     int64_t page_size, float scale);

/* o = attention(q) for the T packed query tokens of num_seqs sequences.  max_pos: an upper bound
 * (on the host) of every position; it changes no result.  T = 0 or num_seqs = 0 queues nothing.
 * The run grows the handle's workspace (stream-ordered cudaMallocAsync) when T or num_seqs outgrow
 * it (BI_GEMM_ERR_OOM if that fails; BI_GEMM_ERR_SCRATCH_LIMIT in a call being captured into a graph,
 * which uses what an earlier call of its size left; a graph stays valid when later calls grow the
 * workspace), then queues two kernels: a plan of the units (longest first) and the attention.  A call
 * that can have no more units than the GPU has SMs needs neither plan nor workspace.  Asynchronous.
 * The kernel's waits are bounded (2 s): past the limit the block stops, its output is undefined and
 * bi_prompt_get_device_error reports BI_GEMM_ERR_TIMEOUT. */
int bi_prompt_run(bi_prompt_t h, const void* q, int64_t T, const int32_t* q_start, const int32_t* q_pos0,
                  int64_t num_seqs, const void* k_cache, const void* v_cache, int64_t num_pages,
                  const int32_t* page_table, int64_t max_pages, int64_t max_pos, void* o, void* stream);

/* Workspace bytes a run with T tokens in num_seqs sequences needs (0 for few).  The handle holds up to
 * twice what a run has needed, at most 64 MiB more, and the smaller ones that captured calls use. */
int bi_prompt_workspace_size(bi_prompt_t h, int64_t T, int64_t num_seqs, uint64_t* bytes);

/* Synchronise `stream`; BI_GEMM_ERR_TIMEOUT if a bounded wait expired, else
 * BI_GEMM_ERR_INVALID_ARG if a kernel caught a bad input, since the last call (the status is then
 * cleared); BI_GEMM_ERR_CUDA if synchronisation failed; else BI_GEMM_OK. */
int bi_prompt_get_device_error(bi_prompt_t h, void* stream);

int bi_prompt_get_config(bi_prompt_t h, bi_prompt_config* c);

/* Release the handle and, behind everything that its device has queued, its workspace (NULL is a no-op).  Not to
 * be called while a stream is being captured. */
int bi_prompt_destroy(bi_prompt_t h);

#ifdef __cplusplus
}
#endif
#endif
