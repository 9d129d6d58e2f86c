/*
 * bi_paged_controls.h — TEST-ONLY entry points of libbi_gemm_controls.so for the operators around the
 * paged cache: this library's own copies (a handle made here is used only here) and failure
 * injection.  Each *_stall is the product's run (same arguments and codes) with block 0 of the
 * kernel (of the prompts' kernel, whose blocks take their units as they come: every block with a
 * unit of sequence 0) never issuing its loads and the waits limited to timeout_ns (> 0): the block's waits
 * expire, it stops, and *_get_device_error then reads BI_GEMM_ERR_TIMEOUT; outputs are undefined
 * and the handle stays usable.  No GPU fault is raised.
 */
#ifndef BI_PAGED_CONTROLS_H
#define BI_PAGED_CONTROLS_H

#include <stdint.h>

#include "../../include/bi_attention.h"
#include "../../include/bi_prompt.h"
#include "../../include/bi_qkrope.h"

#ifdef __cplusplus
extern "C" {
#endif

int bi_ctl_prompt_create(bi_prompt_t* out, int64_t num_q_heads, int64_t num_kv_heads, int64_t head_dim,
                         int64_t page_size, float scale);
int bi_ctl_prompt_run(bi_prompt_t h, const void* q, int64_t T, const int32_t* q_start, const int32_t* q_pos0,
                      int64_t num_seqs, const void* k_cache, const void* v_cache, int64_t num_pages,
                      const int32_t* page_table, int64_t max_pages, int64_t max_pos, void* o, void* stream);
int bi_ctl_prompt_stall(bi_prompt_t h, const void* q, int64_t T, const int32_t* q_start, const int32_t* q_pos0,
                        int64_t num_seqs, const void* k_cache, const void* v_cache, int64_t num_pages,
                        const int32_t* page_table, int64_t max_pages, int64_t max_pos, void* o,
                        uint64_t timeout_ns, void* stream);
int bi_ctl_prompt_get_device_error(bi_prompt_t h, void* stream);
int bi_ctl_prompt_destroy(bi_prompt_t h);

/* On a handle of bi_ctl_attention_create; the groups' kernel stalls. */
int bi_ctl_attention_shared_stall(bi_attention_t h, const void* q, int64_t T, const int32_t* q_seq,
                                  const int32_t* q_pos, const void* k_cache, const void* v_cache, int64_t num_pages,
                                  const int32_t* page_table, int64_t num_seqs, int64_t max_pages, int64_t max_pos,
                                  const int32_t* group_start, const int32_t* group_len, int64_t num_groups, void* o,
                                  uint64_t timeout_ns, void* stream);

int bi_ctl_qkrope_create(bi_qkrope_t* out, int64_t num_q_heads, int64_t num_kv_heads, int64_t head_dim,
                         int64_t page_size, int64_t rot_dim, int32_t interleaved, float eps);
/* The form for many tokens stalls (T at least the configuration's ring_from). */
int bi_ctl_qkrope_stall(bi_qkrope_t h, const void* qkv, int64_t T, int64_t qkv_stride, const void* gq,
                        const void* gk, const float* cos_sin, int64_t num_positions, const int32_t* q_seq,
                        const int32_t* q_pos, void* k_cache, void* v_cache, int64_t num_pages,
                        const int32_t* page_table, int64_t num_seqs, int64_t max_pages, void* q_out,
                        uint64_t timeout_ns, void* stream);
int bi_ctl_qkrope_get_device_error(bi_qkrope_t h, void* stream);
int bi_ctl_qkrope_destroy(bi_qkrope_t h);

#ifdef __cplusplus
}
#endif
#endif
