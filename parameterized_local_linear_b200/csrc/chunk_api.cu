// C ABI of the chunk attention over a paged cache (include/parallax.h):
// argument checks, tensor maps and launches of the kernels in kernel_chunk.cuh.
#include <algorithm>
#include <atomic>
#include <cstdlib>

#include "parallax.h"
#include "parallax_testing.h"

#include "common.cuh"
#include "host.cuh"
#include "kernel_chunk.cuh"

using namespace plx;

namespace {

constexpr unsigned long long kChunkTimeoutNs = 2000000000ull;  // 2 s per wait

// [total][Hq][D] bf16 viewed as {64 dims, G heads of a group, tokens, D/64
// halves, Hkv groups}: a box of G heads x tpt tokens lands as one swizzled
// [tpt * G rows][128 bytes] block, rows ordered (token, head).
int encode_rows_by_group(CUtensorMap* map, const void* base, int D, int total, int G, int Hkv,
                         int tpt) {
  auto enc = tensor_map_encoder();
  if (!enc) return PARALLAX_ERR_CUDA;
  cuuint64_t dims[5] = {64, (cuuint64_t)G, (cuuint64_t)total, (cuuint64_t)(D / 64),
                        (cuuint64_t)Hkv};
  cuuint64_t strides[4] = {(cuuint64_t)D * 2, (cuuint64_t)G * Hkv * D * 2, 128,
                           (cuuint64_t)G * D * 2};
  cuuint32_t box[5] = {64, (cuuint32_t)G, (cuuint32_t)tpt, 1, 1};
  cuuint32_t elem[5] = {1, 1, 1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims,
                   strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PARALLAX_OK : PARALLAX_ERR_CUDA;
}

// The status header, what to merge per CTA, and two partial records per CTA.
size_t chunk_records_offset(int ctas) { return kWorkspaceHeaderBytes + ctas * sizeof(ChunkMerge); }
size_t chunk_workspace(int ctas, int D) {
  return chunk_records_offset(ctas) + (size_t)2 * ctas * chunk_rec_floats(D) * sizeof(float);
}

template <int D, bool PROBE>
int launch_chunk(const void* q, const void* r, const void* k, const void* v, const ChunkParams& p,
                 int ctas, cudaStream_t stream) {
  static std::atomic<int> done[256];
  auto kernel = parallax_chunk_kernel<D, PROBE>;
  int st = set_smem_once(kernel, ChGeom<D>::kSmem, done);
  if (st != PARALLAX_OK) return st;
  CUtensorMap tq, tr, tk, tv;
  const ChunkSpace& sp = p.sp;
  if ((st = encode_rows_by_group(&tq, q, D, sp.total, p.G, sp.Hkv, sp.tpt)) != PARALLAX_OK)
    return st;
  tr = tq;
  if (PROBE &&
      (st = encode_rows_by_group(&tr, r, D, sp.total, p.G, sp.Hkv, sp.tpt)) != PARALLAX_OK)
    return st;
  // the pool [pages][page_size][Hkv][D] is a (kv_len, H, D) cache of pages
  if ((st = encode_cache_map(&tk, k, D, p.page_size, sp.Hkv, p.num_pages, PARALLAX_KV_BSHD)) !=
          PARALLAX_OK ||
      (st = encode_cache_map(&tv, v, D, p.page_size, sp.Hkv, p.num_pages, PARALLAX_KV_BSHD)) !=
          PARALLAX_OK)
    return st;
  st = launch_pdl(kernel, dim3((unsigned)ctas), kChThreads, ChGeom<D>::kSmem, stream, tq, tr, tk,
                  tv, p);
  if (st != PARALLAX_OK) return st;
  return launch_pdl(parallax_chunk_merge_kernel<D, PROBE>,
                    dim3((unsigned)ctas, (unsigned)(D / 4 / kChunkMergeCols)), kChunkRows, 0,
                    stream, p);
}

int run_chunk(const void* q, const void* r, const void* k_pages, const void* v_pages,
              const int32_t* block_table, const int32_t* cu_seqlens_q,
              const int32_t* cache_seqlens, void* out, int B, int total_tokens, int Hq, int Hkv,
              int D, float scale, int causal, void* stream, int num_pages, int page_size,
              int max_pages_per_seq, int probe, void* workspace, size_t workspace_bytes,
              unsigned long long timeout_ns, int debug_skip_first_k) {
  if (!q || (probe && !r) || !k_pages || !v_pages || !block_table || !cache_seqlens || !out ||
      !workspace)
    return PARALLAX_ERR_NULL_POINTER;
  if (B < 1 || total_tokens < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq > 65535 ||
      Hq / Hkv > kChunkRows || num_pages < 1 || max_pages_per_seq < 1 || page_size < kChunkKeys ||
      page_size % kChunkKeys != 0 || (long long)page_size * max_pages_per_seq > 0x7fffffffLL ||
      (cu_seqlens_q == nullptr && total_tokens != B))
    return PARALLAX_ERR_BAD_SHAPE;
  if (!(scale > 0.f) || !(scale < 3.0e38f)) return PARALLAX_ERR_BAD_SHAPE;  // positive, finite
  if (D != 64 && D != 128) return PARALLAX_ERR_UNSUPPORTED_HEAD_DIM;
  if (!aligned16(q) || (probe && !aligned16(r)) || !aligned16(k_pages) || !aligned16(v_pages) ||
      !aligned16(out) || !aligned16(workspace) || (reinterpret_cast<uintptr_t>(block_table) & 3u) ||
      (reinterpret_cast<uintptr_t>(cu_seqlens_q) & 3u) ||
      (reinterpret_cast<uintptr_t>(cache_seqlens) & 3u))
    return PARALLAX_ERR_MISALIGNED;
  // One token per sequence: the decode over the same cache where its TMA kernel takes
  // the group. Measured, 32 sequences of 4096 keys, 8 kv heads of 128, decode against
  // chunk kernel: groups of 1 to 4 with the probe 88 to 90 us and 130 us, without it (to
  // 8) 87 to 92 and 104; one sequence 7 to 9 us and 21 to 26. Larger groups, which the
  // decode has only its generic kernel for: 4700 us against 134 (1 sequence: 105, 26).
  if (cu_seqlens_q == nullptr && decode_on_tma(PARALLAX_DTYPE_BF16, probe, Hq / Hkv))
    return parallax_decode_paged(q, r, k_pages, v_pages, block_table, cache_seqlens, out, B, Hq,
                                 Hkv, D, scale, stream, num_pages, page_size, max_pages_per_seq,
                                 probe, PARALLAX_DTYPE_BF16, PARALLAX_DTYPE_BF16, 0, workspace,
                                 workspace_bytes);
  int sm = 0;
  const int st = current_sm_count(&sm);
  if (st != PARALLAX_OK) return st;
  if (workspace_bytes < chunk_workspace(sm, D)) return PARALLAX_ERR_WORKSPACE_TOO_SMALL;
  ChunkParams p{};
  p.G = Hq / Hkv;
  p.sp = ChunkSpace{cu_seqlens_q, cache_seqlens,       B, total_tokens, page_size * max_pages_per_seq,
                    Hkv,          kChunkRows / p.G, causal != 0 && cu_seqlens_q != nullptr};
  p.out = static_cast<__nv_bfloat16*>(out);
  p.status = static_cast<unsigned int*>(workspace);
  p.merges = reinterpret_cast<ChunkMerge*>(static_cast<char*>(workspace) + kWorkspaceHeaderBytes);
  p.records = reinterpret_cast<float*>(static_cast<char*>(workspace) + chunk_records_offset(sm));
  p.table = block_table;
  p.Hq = Hq;
  p.page_size = page_size;
  p.num_pages = num_pages;
  p.max_pages = max_pages_per_seq;
  p.scale_log2 = (float)((double)scale * 1.4426950408889634);
  p.timeout_ns = timeout_ns;
  p.debug_skip_first_k = debug_skip_first_k;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (D == 128)
    return probe ? launch_chunk<128, true>(q, r, k_pages, v_pages, p, sm, s)
                 : launch_chunk<128, false>(q, r, k_pages, v_pages, p, sm, s);
  return probe ? launch_chunk<64, true>(q, r, k_pages, v_pages, p, sm, s)
               : launch_chunk<64, false>(q, r, k_pages, v_pages, p, sm, s);
}

}  // namespace

extern "C" size_t parallax_prefill_paged_workspace_bytes(int B, int total_tokens, int Hq, int Hkv,
                                                         int D) {
  if (B < 1 || total_tokens < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > kChunkRows ||
      (D != 64 && D != 128))
    return 0;
  int sm = 0;
  if (current_sm_count(&sm) != PARALLAX_OK) return 0;
  // the decode that a call with one token per sequence runs, at its most
  // partitions (one per 64 keys of the longest cache, at most one per SM)
  const size_t decode = parallax_decode_workspace_bytes(B, Hq, Hkv, D, 64 * sm, 0);
  return std::max(chunk_workspace(sm, D), decode);
}

extern "C" int parallax_prefill_paged(const void* q, const void* r, const void* k_pages,
                                      const void* v_pages, const int32_t* block_table,
                                      const int32_t* cu_seqlens_q, const int32_t* cache_seqlens,
                                      void* out, int B, int total_tokens, int Hq, int Hkv, int D,
                                      float scale, int causal, void* stream, int num_pages,
                                      int page_size, int max_pages_per_seq, int probe,
                                      void* workspace, size_t workspace_bytes) {
  return run_chunk(q, r, k_pages, v_pages, block_table, cu_seqlens_q, cache_seqlens, out, B,
                   total_tokens, Hq, Hkv, D, scale, causal, stream, num_pages, page_size,
                   max_pages_per_seq, probe, workspace, workspace_bytes, kChunkTimeoutNs, 0);
}

extern "C" int parallax_testing_prefill_paged_stalled(
    const void* q, const void* r, const void* k_pages, const void* v_pages,
    const int32_t* block_table, const int32_t* cu_seqlens_q, const int32_t* cache_seqlens,
    void* out, int B, int total_tokens, int Hq, int Hkv, int D, float scale, int causal,
    void* stream, int num_pages, int page_size, int max_pages_per_seq, int probe, void* workspace,
    size_t workspace_bytes, int timeout_ms) {
  if (timeout_ms < 1 || timeout_ms > 10000 || cu_seqlens_q == nullptr)
    return PARALLAX_ERR_BAD_SHAPE;
  return run_chunk(q, r, k_pages, v_pages, block_table, cu_seqlens_q, cache_seqlens, out, B,
                   total_tokens, Hq, Hkv, D, scale, causal, stream, num_pages, page_size,
                   max_pages_per_seq, probe, workspace, workspace_bytes,
                   (unsigned long long)timeout_ms * 1000000ull, 1);
}

extern "C" int parallax_testing_chunk_walk(const int32_t* cu_seqlens_q,
                                           const int32_t* cache_seqlens, int B, int total_tokens,
                                           int Lmax, int Hkv, int tokens_per_tile, int causal,
                                           int ctas, int32_t* pieces, int max_pieces,
                                           int32_t* merges) {
  const ChunkSpace sp{cu_seqlens_q, cache_seqlens,   B,          total_tokens, Lmax,
                      Hkv,          tokens_per_tile, causal != 0};
  const auto cost = [&](const ChunkSeq& s) { return chunk_cost(sp, s, chunk_row_tiles(sp, s)); };
  long long total = 0;
  for (int b = 0; b < B; ++b) total += cost(chunk_seq(sp, b)) * Hkv;
  int count = 0;
  for (int c = 0; c < ctas; ++c) {
    ChunkRange r{};
    chunk_bounds(r, total, c, ctas);
    if (r.lo < r.hi) {  // the item at r.lo, in chunk_locate's steps without its searches
      long long rem = r.lo;
      r.s = chunk_seq(sp, 0);
      while (rem >= cost(r.s) * Hkv) {
        rem -= cost(r.s) * Hkv;
        r.s = chunk_seq(sp, ++r.b);
      }
      r.g = (int)div_pos(rem, cost(r.s));
      rem -= cost(r.s) * r.g;
      while (r.rt + 1 < chunk_row_tiles(sp, r.s) && chunk_cost(sp, r.s, r.rt + 1) <= rem) ++r.rt;
      r.off = (int)(rem - chunk_cost(sp, r.s, r.rt));
    }
    const ChunkMerge mg = chunk_merge_note(sp, r);
    const int note[5] = {mg.token, mg.ntok, mg.g, mg.c0, mg.c0_first};
    std::copy(note, note + 5, merges + (size_t)c * 5);
    ChunkCursor cur(r);
    ChunkPiece pc;
    while (cur.next(sp, pc)) {
      if (count == max_pieces) return PARALLAX_ERR_BAD_SHAPE;
      const int row[8] = {c, pc.b, pc.g, pc.rt, pc.t0, pc.t1, pc.complete, pc.first};
      std::copy(row, row + 8, pieces + (size_t)count++ * 8);
    }
  }
  return count;
}
