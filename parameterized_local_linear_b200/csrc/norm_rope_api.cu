// C ABI of the norm + rotation entry points (include/parallax.h): argument
// checks and launches of the kernels in kernel_norm_rope.cuh.
#include <algorithm>
#include <cmath>

#include "parallax.h"

#include "common.cuh"
#include "host.cuh"
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
  if (tokens < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq > 65535 || max_pos < 1)
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

template <typename T, int D, int U, bool APPEND>
int launch_forward(const NormRopeParams& p, cudaStream_t s) {
  constexpr int kRows = U * 32 / (D / 16);
  const int heads = p.H[0] + p.H[1] + p.H[2] + (APPEND ? p.H[3] : 0);
  const long long units = (long long)p.tokens * ((heads + kRows - 1) / kRows);
  const long long blocks = (units + kNrThreads / 32 - 1) / (kNrThreads / 32);
  if (blocks > 0x7fffffffLL) return PARALLAX_ERR_BAD_SHAPE;
  return launch_pdl(parallax_norm_rope_kernel<T, D, U, APPEND>, dim3((unsigned)blocks), kNrThreads,
                    0, s, p);
}

template <typename T, int D, bool APPEND>
int launch_forward_u(const NormRopeParams& p, cudaStream_t s) {
  int sm = 0;
  const int st = current_sm_count(&sm);
  if (st != PARALLAX_OK) return st;
  const int heads = p.H[0] + p.H[1] + p.H[2] + (APPEND ? p.H[3] : 0);
  constexpr int kRows4 = 4 * 32 / (D / 16);
  const long long units = (long long)p.tokens * ((heads + kRows4 - 1) / kRows4);
  return units >= 8LL * sm ? launch_forward<T, D, 4, APPEND>(p, s)
                           : launch_forward<T, D, 1, APPEND>(p, s);
}

template <bool APPEND>
int dispatch_forward(const NormRopeParams& p, int D, int dtype, cudaStream_t s) {
  if (dtype == PARALLAX_DTYPE_BF16)
    return D == 128 ? launch_forward_u<__nv_bfloat16, 128, APPEND>(p, s)
                    : launch_forward_u<__nv_bfloat16, 64, APPEND>(p, s);
  return D == 128 ? launch_forward_u<float, 128, APPEND>(p, s)
                  : launch_forward_u<float, 64, APPEND>(p, s);
}

// Blocks of the backward kernel: two per SM, dealt to the kinds by their rows,
// each kind's at most one per 8 tokens.
constexpr int kNrBackwardBlocksPerSm = 2;

size_t backward_workspace(int sm, int D) {
  return kWorkspaceHeaderBytes + (size_t)(kNrBackwardBlocksPerSm * sm + 3) * D * sizeof(float);
}

template <typename T, int D>
int launch_backward(const NormRopeParams& p, cudaStream_t s) {
  constexpr int kU = sizeof(T) == 2 ? 2 : 1;  // fp32 rows: 2 at a time spill
  int st = launch_pdl(parallax_norm_rope_backward_kernel<T, D, kU>, dim3((unsigned)p.first_block[3]),
                      kNrThreads, 0, s, p);
  if (st != PARALLAX_OK) return st;
  if (!p.w[0] && !p.w[1] && !p.w[2]) return PARALLAX_OK;
  return launch_pdl(parallax_norm_rope_dw_kernel<D>, dim3(3), 1024, 0, s, p);
}

NormRopeParams base_params(int tokens, int Hq, int Hkv, int rot, int interleaved, int max_pos,
                           float eps, const float* cs, const int32_t* pos, bool probe, void* ws) {
  NormRopeParams p{};
  p.H[0] = Hq;
  p.H[1] = probe ? Hq : 0;
  p.H[2] = Hkv;
  p.cs = cs;
  p.pos = pos;
  p.tokens = tokens;
  p.rot = rot;
  p.interleaved = interleaved != 0;
  p.max_pos = max_pos;
  p.eps = eps;
  p.status = static_cast<unsigned int*>(ws);
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
  NormRopeParams p = base_params(tokens, Hq, Hkv, rotary_dim, interleaved, max_positions, eps,
                                 cos_sin, positions, probe, workspace);
  p.seq_len = seq_len;
  p.x[0] = q, p.x[1] = r, p.x[2] = k;
  p.w[0] = q_weight, p.w[1] = r_weight, p.w[2] = k_weight;
  p.y[0] = q_out, p.y[1] = r_out, p.y[2] = k_out;
  p.xs[0] = q_stride, p.xs[1] = r_stride, p.xs[2] = k_stride;
  return dispatch_forward<false>(p, D, dtype, static_cast<cudaStream_t>(stream));
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
  NormRopeParams p = base_params(tokens, Hq, Hkv, rotary_dim, interleaved, max_positions, eps,
                                 cos_sin, positions, probe, workspace);
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
  const long long rows = (long long)p.H[0] + p.H[1] + p.H[2];
  for (int i = 0; i < 3; ++i) {
    const long long share = ((long long)kNrBackwardBlocksPerSm * sm * p.H[i] + rows / 2) / rows;
    const long long most = ((long long)tokens + kNrThreads / 32 - 1) / (kNrThreads / 32);
    p.first_block[i + 1] =
        p.first_block[i] + (p.H[i] == 0 ? 0 : (int)std::max(1LL, std::min(share, most)));
  }
  p.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + kWorkspaceHeaderBytes);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == PARALLAX_DTYPE_BF16)
    return D == 128 ? launch_backward<__nv_bfloat16, 128>(p, s)
                    : launch_backward<__nv_bfloat16, 64>(p, s);
  return D == 128 ? launch_backward<float, 128>(p, s) : launch_backward<float, 64>(p, s);
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
  NormRopeParams p = base_params(total_tokens, Hq, Hkv, rotary_dim, interleaved, max_positions, eps,
                                 cos_sin, positions, probe, workspace);
  p.H[3] = Hkv;
  p.x[0] = q, p.x[1] = r, p.x[2] = k, p.x[3] = v;
  p.w[0] = q_weight, p.w[1] = r_weight, p.w[2] = k_weight;
  p.y[0] = q_out, p.y[1] = r_out;
  p.xs[0] = q_stride, p.xs[1] = r_stride, p.xs[2] = k_stride, p.xs[3] = v_stride;
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.cu = cu_seqlens_q;
  p.lens = cache_seqlens;
  p.table = block_table;
  p.B = B;
  p.page_size = page_size;
  p.num_pages = num_pages;
  p.max_pages = max_pages_per_seq;
  return dispatch_forward<true>(p, D, dtype, static_cast<cudaStream_t>(stream));
}
