/*
 * parallax_testing.h - testing hook of libparallax.so.
 *
 * Not part of the API, and with no counterpart in the pages: these hooks
 * exist so that tests can watch the kernels' bounded waits give up on a GPU
 * without hanging or faulting it.
 */
#ifndef PARALLAX_TESTING_H
#define PARALLAX_TESTING_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/*
 * parallax_decode (same arguments and checks) with two changes: every wait
 * inside the split-KV kernel is bounded by timeout_ms (1 .. 10000) instead of
 * the default 2 s, and the producer never fills the first pipeline stage of
 * each CTA, so the consumers' wait on it must run out. The kernels then set
 * PARALLAX_DEVICE_STATUS_TIMEOUT in the workspace status word and return; the
 * output is invalid; the CUDA context stays usable. Returns
 * PARALLAX_ERR_BAD_SHAPE for a timeout outside the range.
 */
int parallax_testing_decode_stalled(const void* q, const void* r, const void* k_cache,
                                    const void* v_cache, const int32_t* cache_seqlens,
                                    void* out, int B, int Hq, int Hkv, int D, float scale,
                                    void* stream, int Lmax, int num_splits, void* workspace,
                                    size_t workspace_bytes, int timeout_ms);

/*
 * parallax_prefill (same arguments and checks) with the same two changes for
 * the tcgen05 forward: every wait bounded by timeout_ms (1 .. 10000), and the
 * TMA producer never loads the first K tile of each CTA, so the UMMA issuer's
 * wait on it runs out. Each CTA then records PARALLAX_DEVICE_STATUS_TIMEOUT,
 * waits (bounded) for its own copies in flight, frees its tensor memory and
 * returns; the output is invalid; the CUDA context stays usable.
 */
int parallax_testing_prefill_stalled(const void* q, const void* r, const void* k, const void* v,
                                     void* out, int B, int Hq, int Hkv, int L, int D,
                                     float scale, int causal, void* stream, int out_dtype,
                                     void* workspace, size_t workspace_bytes, int timeout_ms);

/*
 * parallax_prefill_paged (cu_seqlens_q required) with the same two changes: every
 * wait bounded by timeout_ms (1 .. 10000), the first K tile of each CTA never
 * loaded.
 */
int parallax_testing_prefill_paged_stalled(
    const void* q, const void* r, const void* k_pages, const void* v_pages,
    const int32_t* block_table, const int32_t* cu_seqlens_q, const int32_t* cache_seqlens,
    void* out, int B, int total_tokens, int Hq, int Hkv, int D, float scale, int causal,
    void* stream, int num_pages, int page_size, int max_pages_per_seq, int probe, void* workspace,
    size_t workspace_bytes, int timeout_ms);

/*
 * Changes the next call that this host thread makes of parallax_qk_norm_rope, its
 * backward pass or parallax_norm_rope_append (one that is refused may use it up):
 * every wait is bounded by timeout_ms (1 .. 10000), and the first rows of each kind of
 * head are never loaded, so that the wait of the warp that has them runs out. It records
 * PARALLAX_DEVICE_STATUS_TIMEOUT, waits (bounded) for its own copies in flight and leaves
 * its rows unwritten; the other warps finish theirs. Returns PARALLAX_ERR_BAD_SHAPE for a
 * timeout outside the range.
 */
int parallax_testing_norm_rope_stall_next(int timeout_ms);

/*
 * The work partition of parallax_prefill_paged, walked on the host by the kernel's own
 * arithmetic (csrc/chunk_partition.cuh). Host pointers: cu_seqlens_q [B + 1] or NULL,
 * cache_seqlens [B]. For each of `ctas` CTAs, merges gets 5 ints (token, ntok, kv head,
 * first range, whether that is a first piece) and pieces 8 per piece (CTA, sequence, kv
 * head, row tile, first tile, last tile + 1, complete, first). Returns the number of
 * pieces, or PARALLAX_ERR_BAD_SHAPE for more than max_pieces.
 */
int parallax_testing_chunk_walk(const int32_t* cu_seqlens_q, const int32_t* cache_seqlens, int B,
                                int total_tokens, int Lmax, int Hkv, int tokens_per_tile,
                                int causal, int ctas, int32_t* pieces, int max_pieces,
                                int32_t* merges);

/* n / d (0 <= n, 1 <= d) as the norm and rotation kernels compute it. */
int parallax_testing_divide(int n, int d);

#ifdef __cplusplus
}
#endif

#endif /* PARALLAX_TESTING_H */
