/*
 * Entry points of libparallax.so for this package's own binding (marshal.cpp):
 * forms of the calls in parallax.h that its users do not need.
 */
#ifndef PARALLAX_INTERNAL_H
#define PARALLAX_INTERNAL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/*
 * parallax_norm_rope_append; the rows of q_out (clear_rest bit 0) and r_out (bit 1)
 * that have no token (padding, idle rows) become zeros, for outputs that the binding
 * has just allocated.
 */
int parallax_internal_norm_rope_append(
    const void* q, const void* r, const void* k, const void* v, const void* q_weight,
    const void* r_weight, const void* k_weight, const float* cos_sin, const int32_t* positions,
    const int32_t* cu_seqlens_q, const int32_t* cache_seqlens, const int32_t* block_table,
    void* q_out, void* r_out, void* k_pages, void* v_pages, int B, int total_tokens, int Hq,
    int Hkv, int D, int rotary_dim, int interleaved, int max_positions, float eps,
    long long q_stride, long long r_stride, long long k_stride, long long v_stride, int num_pages,
    int page_size, int max_pages_per_seq, int dtype, void* stream, void* workspace,
    size_t workspace_bytes,
    int clear_rest);

#ifdef __cplusplus
}
#endif

#endif /* PARALLAX_INTERNAL_H */
