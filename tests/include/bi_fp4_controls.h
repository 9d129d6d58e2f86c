/*
 * bi_fp4_controls.h — TEST-ONLY entry points of libbi_gemm_controls.so for the operators in 4 bits: this library's own
 * copies (a handle made here is used only here) and failure injection.  Each *_stall is the product's run (same
 * arguments and codes) with no operand loaded (the product; the append: by block 0 of its form for many tokens) and the
 * waits limited to timeout_ns (> 0): they expire, the kernel stops, and *_get_device_error then reads
 * BI_GEMM_ERR_TIMEOUT; outputs are undefined and the handle stays usable.  No GPU fault is raised.
 */
#ifndef BI_FP4_CONTROLS_H
#define BI_FP4_CONTROLS_H

#include <stdint.h>

#include "../../include/bi_fp4.h"
#include "../../include/bi_qkrope.h"

#ifdef __cplusplus
extern "C" {
#endif

int bi_ctl_gemm4_create(bi_gemm4_t* out, int64_t K, int64_t N, int32_t format, int32_t out_f32);
int bi_ctl_gemm4_run(bi_gemm4_t h, const void* x, const void* sx, int64_t M, const void* w, const void* sw, float alpha,
                     void* y, void* stream);
int bi_ctl_gemm4_stall(bi_gemm4_t h, const void* x, const void* sx, int64_t M, const void* w, const void* sw, float alpha,
                       void* y, uint64_t timeout_ns, void* stream);
/* What a product of M rows runs as on a device of `sms` SMs, without touching one: rows of w a CTA in the form of smaller
 * tiles, and its CTAs an SM, stages and slots a stage; 0 in the form of CTA pairs. */
int bi_ctl_gemm4_form(int64_t K, int64_t N, int32_t format, int32_t out_f32, int32_t sms, int64_t M, int32_t* per_sm,
                      int32_t* stages, int32_t* slots);
int bi_ctl_gemm4_get_device_error(bi_gemm4_t h, void* stream);
int bi_ctl_gemm4_destroy(bi_gemm4_t h);

/* On a handle of bi_ctl_qkrope_create (T at least the configuration's ring_from). */
int bi_ctl_qkrope_stall4(bi_qkrope_t h, const void* qkv, int64_t T, int64_t qkv_stride, const void* gq, const void* gk,
                         const float* cos_sin, int64_t num_positions, const int32_t* q_seq, const int32_t* q_pos,
                         void* k_codes, void* k_scales, void* v_codes, void* v_scales, float k_scale, float v_scale,
                         int64_t num_pages, const int32_t* page_table, int64_t num_seqs, int64_t max_pages, void* q_out,
                         uint64_t timeout_ns, void* stream);

#ifdef __cplusplus
}
#endif
#endif
