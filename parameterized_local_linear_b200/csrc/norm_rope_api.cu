// C ABI of the norm + rotation entry points (include/parallax.h): argument
// checks and launches of the kernels in kernel_norm_rope.cuh.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "parallax.h"
#include "parallax_testing.h"

#include "common.cuh"
#include "host.cuh"
#include "internal.h"
#include "kernel_norm_rope.cuh"

using namespace plx;

namespace {

size_t elem_size(int dtype) { return dtype == PARALLAX_DTYPE_BF16 ? 2 : 4; }

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Rows `stride` elements apart that hold H heads of D elements, 16-byte words.
bool stride_ok(long long stride, int H, int D, int dtype) {
  return stride >= (long long)H * D && stride % (long long)(16 / elem_size(dtype)) == 0;
}

// The checks the three entry points share. heads[i] is 0 for an absent kind.
int check_common(int tokens, int Hq, int Hkv, int D, int rot, int max_pos, float eps, int dtype,
                 const float* cs, const int32_t* pos, void* ws, size_t ws_bytes, size_t need) {
  if (!cs || !ws) return PARALLAX_ERR_NULL_POINTER;
  if (tokens < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq > 65535 || max_pos < 1 ||
      (long long)tokens * Hq > 0x7fffffffLL)  // (such a tensor does not fit the GPU)
    return PARALLAX_ERR_BAD_SHAPE;
  if (!(eps > 0.f) || !(eps < 3.0e38f)) return PARALLAX_ERR_BAD_SHAPE;
  if (D != 64 && D != 128) return PARALLAX_ERR_UNSUPPORTED_HEAD_DIM;
  if (rot < 16 || rot > D || rot % 16 != 0) return PARALLAX_ERR_BAD_SHAPE;
  if (dtype != PARALLAX_DTYPE_BF16 && dtype != PARALLAX_DTYPE_F32)
    return PARALLAX_ERR_UNSUPPORTED_DTYPE;
  if (!aligned16(cs) || !aligned4(pos) || !aligned16(ws)) return PARALLAX_ERR_MISALIGNED;
  if (ws_bytes < need) return PARALLAX_ERR_WORKSPACE_TOO_SMALL;
  return PARALLAX_OK;
}

// One kind's input: rows, stride and weight.
int check_rows(const void* x, long long stride, const void* w, int H, int D, int dtype) {
  if (!x) return PARALLAX_ERR_NULL_POINTER;
  if (!stride_ok(stride, H, D, dtype)) return PARALLAX_ERR_BAD_SHAPE;
  if (!aligned16(x) || !aligned16(w)) return PARALLAX_ERR_MISALIGNED;
  return PARALLAX_OK;
}

// Blocks of a grid that fits the GPU at once (`most`, a few per SM): each kind
// as many as its units fill, or where that is more than `most`, its share of
// the work (one block over would run alone at the end: 445 blocks on 444 places
// took 100 us where 441 took 73). Many tokens: a unit fills a ring stage
// (`stage_rows`), so that a token's angles serve all its heads; few (less than
// two steps of 32 / (D/16) rows per warp): single steps, so that more warps
// share them. A unit's own part (its copies, angles and place) takes as long as
// `unit_cost` steps.
void deal_blocks(NormRopeParams& p, int kinds, int most, int D, int stage_rows, double unit_cost) {
  const int groups = 32 / (D / 16);
  long long steps[4] = {}, all_steps = 0, fill[4] = {}, filled = 0;
  double work[4] = {}, all_work = 0;
  for (int i = 0; i < kinds; ++i) {
    steps[i] = (p.H[i] + groups - 1) / groups;
    all_steps += p.tokens * steps[i];
  }
  p.seq_div = NrDivisor::of(std::max(1, p.seq_len));
  p.unit_rows = all_steps >= 2LL * most * kNrWarps ? stage_rows : groups;
  for (int i = 0; i < kinds; ++i) {
    const long long units = (p.H[i] + p.unit_rows - 1) / p.unit_rows;
    p.unit_div[i] = NrDivisor::of(std::max(1, (int)units));
    filled += fill[i] = (p.tokens * units + kNrWarps - 1) / kNrWarps;
    all_work += work[i] = steps[i] + unit_cost * units;
  }
  p.first_block[0] = 0;
  for (int i = 0; i < kinds; ++i) {
    // kinds that would get no block take one; `most` leaves room for them
    const long long share = std::max(1LL, (long long)((most - kinds) * work[i] / all_work));
    p.first_block[i + 1] =
        p.first_block[i] + (int)(filled <= most ? fill[i] : std::min(share, fill[i]));
  }
}

constexpr int kNrForwardBlocksPerSm = 2;
constexpr double kNrForwardUnitCost = 1.5;  // (the backward's steps are longer: 0)
constexpr int kNrBackwardBlocksPerSm = 2;
constexpr int kNrDoneWord = 8;  // of the workspace header: counters that are 0 between calls

template <typename T, int D, bool INTER, bool APPEND>
int launch_forward(NormRopeParams& p, cudaStream_t s) {
  static std::atomic<int> done[256];
  auto kernel = parallax_norm_rope_kernel<T, D, INTER, APPEND>;
  constexpr int kSmem = NrForwardRing::kSmem;
  int sm = 0;
  int st = current_sm_count(&sm);
  if (st != PARALLAX_OK || (st = set_smem_once(kernel, kSmem, done)) != PARALLAX_OK) return st;
  constexpr int kKinds = APPEND ? 4 : 3;
  deal_blocks(p, kKinds, kNrForwardBlocksPerSm * sm, D,
              NrForwardRing::kBytes / (D * (int)sizeof(T)), kNrForwardUnitCost);
  return launch_pdl(kernel, dim3((unsigned)p.first_block[kKinds]), kNrThreads, kSmem, s, p);
}

template <bool APPEND, typename T>
int dispatch_forward_t(NormRopeParams& p, int D, bool inter, cudaStream_t s) {
  if (D == 128) return inter ? launch_forward<T, 128, true, APPEND>(p, s)
                             : launch_forward<T, 128, false, APPEND>(p, s);
  return inter ? launch_forward<T, 64, true, APPEND>(p, s)
               : launch_forward<T, 64, false, APPEND>(p, s);
}

template <bool APPEND>
int dispatch_forward(NormRopeParams& p, int D, int inter, int dtype, cudaStream_t s) {
  return dtype == PARALLAX_DTYPE_BF16
             ? dispatch_forward_t<APPEND, __nv_bfloat16>(p, D, inter != 0, s)
             : dispatch_forward_t<APPEND, float>(p, D, inter != 0, s);
}

size_t backward_workspace(int sm, int D) {  // a partial per block: at most one more per kind
  return kWorkspaceHeaderBytes + (size_t)(kNrBackwardBlocksPerSm * sm + 3) * D * sizeof(float);
}

template <typename T, int D, bool INTER>
int launch_backward(const NormRopeParams& p, cudaStream_t s) {
  static std::atomic<int> done[256];
  auto kernel = parallax_norm_rope_backward_kernel<T, D, INTER>;
  constexpr int kSmem = NrBackwardRing::kSmem;
  int st = set_smem_once(kernel, kSmem, done);
  if (st != PARALLAX_OK) return st;
  return launch_pdl(kernel, dim3((unsigned)p.first_block[3]), kNrThreads, kSmem, s, p);
}

template <typename T>
int dispatch_backward(const NormRopeParams& p, int D, bool inter, cudaStream_t s) {
  if (D == 128)
    return inter ? launch_backward<T, 128, true>(p, s) : launch_backward<T, 128, false>(p, s);
  return inter ? launch_backward<T, 64, true>(p, s) : launch_backward<T, 64, false>(p, s);
}

constexpr unsigned long long kNrTimeoutNs = 2000000000ull;  // 2 s per wait
thread_local unsigned long long stalled_timeout_ns = 0;  // of the next call, if not 0

NormRopeParams base_params(int tokens, int Hq, int Hkv, int rot, int max_pos, float eps,
                           const float* cs, const int32_t* pos, bool probe, void* ws) {
  NormRopeParams p{};
  p.H[0] = Hq;
  p.H[1] = probe ? Hq : 0;
  p.H[2] = Hkv;
  p.cs = cs;
  p.pos = pos;
  p.tokens = tokens;
  p.rot = rot;
  p.max_pos = max_pos;
  p.eps = eps;
  p.status = static_cast<unsigned int*>(ws);
  p.timeout_ns = stalled_timeout_ns ? stalled_timeout_ns : kNrTimeoutNs;
  p.debug_skip_unit = stalled_timeout_ns ? 0 : -1;
  stalled_timeout_ns = 0;
  return p;
}

}  // namespace

extern "C" int parallax_rope_table(float* cos_sin, int max_positions, int rotary_dim, double base,
                                   void* stream) {
  if (!cos_sin) return PARALLAX_ERR_NULL_POINTER;
  if (max_positions < 1 || rotary_dim < 16 || rotary_dim > 128 || rotary_dim % 16 != 0 ||
      !(base > 0.0) || !std::isfinite(base))
    return PARALLAX_ERR_BAD_SHAPE;
  if (!aligned16(cos_sin)) return PARALLAX_ERR_MISALIGNED;
  const long long n = (long long)max_positions * (rotary_dim / 2);
  const long long blocks = (n + kNrThreads - 1) / kNrThreads;
  if (blocks > 0x7fffffffLL) return PARALLAX_ERR_BAD_SHAPE;
  parallax_rope_table_kernel<<<(unsigned)blocks, kNrThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      cos_sin, max_positions, rotary_dim, base);
  return cudaGetLastError() == cudaSuccess ? PARALLAX_OK : PARALLAX_ERR_CUDA;
}

extern "C" int parallax_qk_norm_rope(const void* q, const void* r, const void* k,
                                     const void* q_weight, const void* r_weight,
                                     const void* k_weight, const float* cos_sin,
                                     const int32_t* positions, void* q_out, void* r_out,
                                     void* k_out, int tokens, int Hq, int Hkv, int D,
                                     int rotary_dim, int interleaved, int max_positions, float eps,
                                     long long q_stride, long long r_stride, long long k_stride,
                                     int seq_len, int dtype, void* stream, void* workspace,
                                     size_t workspace_bytes) {
  int st = check_common(tokens, Hq, Hkv, D, rotary_dim, max_positions, eps, dtype, cos_sin,
                        positions, workspace, workspace_bytes, kWorkspaceHeaderBytes);
  if (st != PARALLAX_OK) return st;
  if (seq_len < 0 || (seq_len > 0 && tokens % seq_len != 0)) return PARALLAX_ERR_BAD_SHAPE;
  const bool probe = r != nullptr;
  if (!q_out || !k_out || (probe && !r_out)) return PARALLAX_ERR_NULL_POINTER;
  if ((st = check_rows(q, q_stride, q_weight, Hq, D, dtype)) != PARALLAX_OK) return st;
  if (probe && (st = check_rows(r, r_stride, r_weight, Hq, D, dtype)) != PARALLAX_OK) return st;
  if ((st = check_rows(k, k_stride, k_weight, Hkv, D, dtype)) != PARALLAX_OK) return st;
  if (!aligned16(q_out) || !aligned16(k_out) || (probe && !aligned16(r_out)))
    return PARALLAX_ERR_MISALIGNED;
  NormRopeParams p = base_params(tokens, Hq, Hkv, rotary_dim, max_positions, eps, cos_sin,
                                 positions, probe, workspace);
  p.seq_len = seq_len;
  p.x[0] = q, p.x[1] = r, p.x[2] = k;
  p.w[0] = q_weight, p.w[1] = r_weight, p.w[2] = k_weight;
  p.y[0] = q_out, p.y[1] = r_out, p.y[2] = k_out;
  p.xs[0] = q_stride, p.xs[1] = r_stride, p.xs[2] = k_stride;
  return dispatch_forward<false>(p, D, interleaved, dtype, static_cast<cudaStream_t>(stream));
}

extern "C" size_t parallax_qk_norm_rope_backward_workspace_bytes(int tokens, int Hq, int Hkv,
                                                                 int D) {
  if (tokens < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || (D != 64 && D != 128)) return 0;
  int sm = 0;
  if (current_sm_count(&sm) != PARALLAX_OK) return 0;
  return backward_workspace(sm, D);
}

extern "C" int parallax_qk_norm_rope_backward(
    const void* dq_out, const void* dr_out, const void* dk_out, const void* q, const void* r,
    const void* k, const void* q_weight, const void* r_weight, const void* k_weight,
    const float* cos_sin, const int32_t* positions, void* dq, void* dr, void* dk,
    float* dq_weight, float* dr_weight, float* dk_weight, int tokens, int Hq, int Hkv, int D,
    int rotary_dim, int interleaved, int max_positions, float eps, long long q_stride,
    long long r_stride, long long k_stride, long long dq_stride, long long dr_stride,
    long long dk_stride, int seq_len, int dtype, void* stream, void* workspace,
    size_t workspace_bytes) {
  int st = check_common(tokens, Hq, Hkv, D, rotary_dim, max_positions, eps, dtype, cos_sin,
                        positions, workspace, workspace_bytes, kWorkspaceHeaderBytes);
  if (st != PARALLAX_OK) return st;
  if (seq_len < 0 || (seq_len > 0 && tokens % seq_len != 0)) return PARALLAX_ERR_BAD_SHAPE;
  const bool probe = r != nullptr;
  const void* const x[3] = {q, r, k};
  const void* const w[3] = {q_weight, r_weight, k_weight};
  const void* const dy[3] = {dq_out, dr_out, dk_out};
  void* const dx[3] = {dq, dr, dk};
  float* const dw[3] = {dq_weight, dr_weight, dk_weight};
  const long long xs[3] = {q_stride, r_stride, k_stride}, dxs[3] = {dq_stride, dr_stride, dk_stride};
  NormRopeParams p = base_params(tokens, Hq, Hkv, rotary_dim, max_positions, eps, cos_sin,
                                 positions, probe, workspace);
  p.seq_len = seq_len;
  for (int i = 0; i < 3; ++i) {
    if (p.H[i] == 0) continue;
    if ((st = check_rows(x[i], xs[i], w[i], p.H[i], D, dtype)) != PARALLAX_OK) return st;
    if (!dy[i] || !dx[i] || (w[i] && !dw[i])) return PARALLAX_ERR_NULL_POINTER;
    if (!stride_ok(dxs[i], p.H[i], D, dtype)) return PARALLAX_ERR_BAD_SHAPE;
    if (!aligned16(dy[i]) || !aligned16(dx[i]) || !aligned4(dw[i])) return PARALLAX_ERR_MISALIGNED;
    p.x[i] = x[i];
    p.w[i] = w[i];
    p.xs[i] = xs[i];
    p.dy[i] = dy[i];
    p.dx[i] = dx[i];
    p.dxs[i] = dxs[i];
    p.dw[i] = dw[i];
  }
  int sm = 0;
  if ((st = current_sm_count(&sm)) != PARALLAX_OK) return st;
  if (workspace_bytes < backward_workspace(sm, D)) return PARALLAX_ERR_WORKSPACE_TOO_SMALL;
  deal_blocks(p, 3, kNrBackwardBlocksPerSm * sm, D,
              NrBackwardRing::kBytes / (D * (int)elem_size(dtype)), 0.0);
  p.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + kWorkspaceHeaderBytes);
  p.done = p.status + kNrDoneWord;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == PARALLAX_DTYPE_BF16 ? dispatch_backward<__nv_bfloat16>(p, D, interleaved != 0, s)
                                      : dispatch_backward<float>(p, D, interleaved != 0, s);
}

extern "C" int parallax_internal_norm_rope_append(
    const void* q, const void* r, const void* k, const void* v, const void* q_weight,
    const void* r_weight, const void* k_weight, const float* cos_sin, const int32_t* positions,
    const int32_t* cu_seqlens_q, const int32_t* cache_seqlens, const int32_t* block_table,
    void* q_out, void* r_out, void* k_pages, void* v_pages, int B, int total_tokens, int Hq,
    int Hkv, int D, int rotary_dim, int interleaved, int max_positions, float eps,
    long long q_stride, long long r_stride, long long k_stride, long long v_stride, int num_pages,
    int page_size, int max_pages_per_seq, int dtype, void* stream, void* workspace,
    size_t workspace_bytes, int clear_rest) {
  int st = check_common(total_tokens, Hq, Hkv, D, rotary_dim, max_positions, eps, dtype, cos_sin,
                        positions, workspace, workspace_bytes, kWorkspaceHeaderBytes);
  if (st != PARALLAX_OK) return st;
  const bool probe = r != nullptr;
  if (!q_out || (probe && !r_out) || !k_pages || !v_pages || !cache_seqlens || !block_table)
    return PARALLAX_ERR_NULL_POINTER;
  if (B < 1 || (cu_seqlens_q == nullptr && total_tokens != B) || num_pages < 1 ||
      page_size < 1 || max_pages_per_seq < 1 ||
      (long long)page_size * max_pages_per_seq > 0x7fffffffLL)
    return PARALLAX_ERR_BAD_SHAPE;
  if ((st = check_rows(q, q_stride, q_weight, Hq, D, dtype)) != PARALLAX_OK) return st;
  if (probe && (st = check_rows(r, r_stride, r_weight, Hq, D, dtype)) != PARALLAX_OK) return st;
  if ((st = check_rows(k, k_stride, k_weight, Hkv, D, dtype)) != PARALLAX_OK) return st;
  if ((st = check_rows(v, v_stride, nullptr, Hkv, D, dtype)) != PARALLAX_OK) return st;
  if (!aligned16(q_out) || (probe && !aligned16(r_out)) || !aligned16(k_pages) ||
      !aligned16(v_pages) || !aligned4(cu_seqlens_q) || !aligned4(cache_seqlens) ||
      !aligned4(block_table))
    return PARALLAX_ERR_MISALIGNED;
  NormRopeParams p = base_params(total_tokens, Hq, Hkv, rotary_dim, max_positions, eps, cos_sin,
                                 positions, probe, workspace);
  p.H[3] = Hkv;
  p.x[0] = q, p.x[1] = r, p.x[2] = k, p.x[3] = v;
  p.w[0] = q_weight, p.w[1] = r_weight, p.w[2] = k_weight;
  p.y[0] = q_out, p.y[1] = r_out, p.y[2] = k_pages, p.y[3] = v_pages;
  p.xs[0] = q_stride, p.xs[1] = r_stride, p.xs[2] = k_stride, p.xs[3] = v_stride;
  p.cu = cu_seqlens_q;
  p.lens = cache_seqlens;
  p.table = block_table;
  p.B = B;
  p.page_size = page_size;
  p.page_div = NrDivisor::of(page_size);
  p.num_pages = num_pages;
  p.max_pages = max_pages_per_seq;
  p.clear_rest = clear_rest & 3;
  return dispatch_forward<true>(p, D, interleaved, dtype, static_cast<cudaStream_t>(stream));
}

extern "C" int parallax_norm_rope_append(
    const void* q, const void* r, const void* k, const void* v, const void* q_weight,
    const void* r_weight, const void* k_weight, const float* cos_sin, const int32_t* positions,
    const int32_t* cu_seqlens_q, const int32_t* cache_seqlens, const int32_t* block_table,
    void* q_out, void* r_out, void* k_pages, void* v_pages, int B, int total_tokens, int Hq,
    int Hkv, int D, int rotary_dim, int interleaved, int max_positions, float eps,
    long long q_stride, long long r_stride, long long k_stride, long long v_stride, int num_pages,
    int page_size, int max_pages_per_seq, int dtype, void* stream, void* workspace,
    size_t workspace_bytes) {
  return parallax_internal_norm_rope_append(
      q, r, k, v, q_weight, r_weight, k_weight, cos_sin, positions, cu_seqlens_q, cache_seqlens,
      block_table, q_out, r_out, k_pages, v_pages, B, total_tokens, Hq, Hkv, D, rotary_dim,
      interleaved, max_positions, eps, q_stride, r_stride, k_stride, v_stride, num_pages,
      page_size, max_pages_per_seq, dtype, stream, workspace, workspace_bytes, 0);
}

extern "C" int parallax_testing_norm_rope_stall_next(int timeout_ms) {
  if (timeout_ms < 1 || timeout_ms > 10000) return PARALLAX_ERR_BAD_SHAPE;
  stalled_timeout_ns = (unsigned long long)timeout_ms * 1000000ull;
  return PARALLAX_OK;
}

extern "C" int parallax_testing_divide(int n, int d) { return NrDivisor::of(d).quotient(n); }
