// Per-head RMS norm and rotary position rotation of the query, probe and key
// heads in one pass (forward, backward, and forward with the cache append).
//
// For a head row x of D values with weight w, at a token whose position's
// table row holds cos_p, sin_p for the pairs p of its first `rot` dimensions:
//   xh = x / sqrt(mean(x^2) + eps),  n = xh w          (no weight: n = x)
//   y_a = n_a cos_p - n_b sin_p,  y_b = n_a sin_p + n_b cos_p
// for pair p = (a, b): (p, p + rot/2), or (2p, 2p + 1) interleaved; the other
// dimensions pass through. Backward, from dy:
//   dz_a = dy_a cos_p + dy_b sin_p,  dz_b = dy_b cos_p - dy_a sin_p,
//   dn = dz w,  dx = (dn - xh mean(dn xh)) / sqrt(mean(x^2) + eps),
//   dw = sum over tokens and heads of dz xh              (no weight: dx = dz)
// All arithmetic is fp32 with one rounding to the output type.
//
// Bound: HBM. A row is read once and written once; the table row of a token
// (4 rot bytes) is read once per warp and kept in registers over the heads.
// D/16 lanes share a row, 16 values each: two 16-byte chunks for bf16 whose
// dimensions pair up under the rotation (chunks c and c + rot/16), so the
// rotation needs no exchange and the norm log2(D/16) shuffles.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace plx {

constexpr int kNrThreads = 256;
constexpr unsigned int kNrStatusClamped = 2u;   // PARALLAX_DEVICE_STATUS_SEQLEN_CLAMPED
constexpr unsigned int kNrStatusPosition = 4u;  // PARALLAX_DEVICE_STATUS_POSITION_CLAMPED

struct NormRopeParams {
  // kinds: 0 query, 1 probe, 2 key, 3 value (append only, copied)
  const void* x[4];       // [tokens] rows xs[i] elements apart, heads D apart
  const void* w[3];       // [D], or nullptr: no norm
  void* y[3];             // outputs (append: y[2] is unused)
  long long xs[4];
  int H[4];               // heads of each kind; 0 leaves it out
  const float* cs;        // [max_pos][rot]: cosines, then sines
  const int32_t* pos;     // [tokens], or nullptr
  int tokens, rot, interleaved, seq_len, max_pos;
  float eps;
  unsigned int* status;
  // append
  void *k_pages, *v_pages;
  const int32_t *cu, *lens, *table;
  int B, page_size, num_pages, max_pages;
  // backward: dy in the layout of y, dx rows dxs[i] elements apart
  const void* dy[3];
  void* dx[3];
  long long dxs[3];
  float* partial;         // [blocks][D] sums of dz xh
  float* dw[3];
  int first_block[4];     // blocks of kind i: first_block[i] .. first_block[i + 1]
};

// The two 8-value chunks a lane holds of a D-value row, and which of them the
// rotation touches. Halves: chunks (i, i + rot/16) rotate as pairs for
// i < rot/16, the other lanes hold the chunks that pass through. Interleaved:
// chunks (i, i + D/16), each with its pairs inside.
template <int D>
struct NrLane {
  int a, b;          // chunk indices
  bool rot_a, rot_b;
  __device__ NrLane(int i, int rot, int interleaved) {
    if (interleaved) {
      a = i;
      b = i + D / 16;
      rot_a = a < rot / 8;
      rot_b = b < rot / 8;
    } else {
      const int rc = rot / 16;
      a = i < rc ? i : 2 * i;
      b = i < rc ? i + rc : 2 * i + 1;
      rot_a = rot_b = i < rc;
    }
  }
};

template <typename T>
struct NrChunk;  // 8 values as loaded
template <>
struct NrChunk<__nv_bfloat16> {
  uint4 u;
  __device__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ void get(float* f) const {
    const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo_to_float(v[i]);
      f[2 * i + 1] = bf16_hi_to_float(v[i]);
    }
  }
  __device__ void set(const float* f) {
    u = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7]));
  }
  __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = u; }
};
template <>
struct NrChunk<float> {
  float4 lo, hi;
  __device__ void load(const float* p) {
    lo = reinterpret_cast<const float4*>(p)[0];
    hi = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ void get(float* f) const {
    f[0] = lo.x, f[1] = lo.y, f[2] = lo.z, f[3] = lo.w;
    f[4] = hi.x, f[5] = hi.y, f[6] = hi.z, f[7] = hi.w;
  }
  __device__ void set(const float* f) {
    lo = make_float4(f[0], f[1], f[2], f[3]);
    hi = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = lo;
    reinterpret_cast<float4*>(p)[1] = hi;
  }
};

// The cosines and sines a lane applies (8 pairs) of one table row.
template <int D>
__device__ __forceinline__ void nr_load_angles(const float* row, const NrLane<D>& ln, int rot,
                                               int interleaved, float (&c)[8], float (&s)[8]) {
  const float* const sn = row + rot / 2;
  const auto four = [](const float* p, float* f) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
  };
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] = 1.f;
    s[i] = 0.f;
  }
  if (interleaved) {
    if (ln.rot_a) {
      four(row + 4 * ln.a, c);
      four(sn + 4 * ln.a, s);
    }
    if (ln.rot_b) {
      four(row + 4 * ln.b, c + 4);
      four(sn + 4 * ln.b, s + 4);
    }
  } else if (ln.rot_a) {
    four(row + 8 * ln.a, c);
    four(row + 8 * ln.a + 4, c + 4);
    four(sn + 8 * ln.a, s);
    four(sn + 8 * ln.a + 4, s + 4);
  }
}

// Rotates v (chunk a in v[0..8), chunk b in v[8..16)) forwards (SIGN = 1) or
// back (-1). Values outside the rotated dimensions are not touched, so an
// infinity or a NaN there stays where it is.
template <int D, int SIGN>
__device__ __forceinline__ void nr_rotate(float (&v)[16], const NrLane<D>& ln, int interleaved,
                                          const float (&c)[8], const float (&s)[8]) {
  const auto turn = [](float& x, float& y, float co, float si) {
    const float x0 = x, y0 = y, sg = SIGN > 0 ? si : -si;
    x = x0 * co - y0 * sg;
    y = x0 * sg + y0 * co;
  };
  if (interleaved) {
    if (ln.rot_a) {
#pragma unroll
      for (int i = 0; i < 4; ++i) turn(v[2 * i], v[2 * i + 1], c[i], s[i]);
    }
    if (ln.rot_b) {
#pragma unroll
      for (int i = 0; i < 4; ++i) turn(v[8 + 2 * i], v[9 + 2 * i], c[4 + i], s[4 + i]);
    }
  } else if (ln.rot_a) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(v[i], v[8 + i], c[i], s[i]);
  }
}

// Sum over the D/16 lanes of a row.
template <int D>
__device__ __forceinline__ float nr_row_sum(float x) {
#pragma unroll
  for (int o = D / 32; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int D>
__device__ __forceinline__ float nr_rstd(const float (&v)[16], float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) ss = fmaf(v[i], v[i], ss);
  return 1.f / sqrtf(nr_row_sum<D>(ss) * (1.f / D) + eps);
}

// Element offset of (token t, head h) in an output: [tokens][H][D], or with
// seq_len L > 0 [tokens / L][H][L][D].
__device__ __forceinline__ size_t nr_out_offset(int t, int h, int H, int L, int D) {
  if (L > 0) return (((size_t)(t / L) * H + h) * L + t % L) * D;
  return ((size_t)t * H + h) * D;
}

// The table row of token t's position (clamped into the table and flagged).
__device__ __forceinline__ const float* nr_table_row(const NormRopeParams& p, long long pos) {
  if (pos < 0 || pos >= p.max_pos) {
    atomicOr(p.status, kNrStatusPosition);
    pos = pos < 0 ? 0 : p.max_pos - 1;
  }
  return p.cs + (size_t)pos * p.rot;
}

// The sequence of packed row t: the largest b with cu[b] <= t < cu[b + 1], or
// -1 outside every sequence. Warp-cooperative (one 32-way step per 32 x),
// bounded for any contents of cu.
__device__ __forceinline__ int nr_find_sequence(const int32_t* cu, int B, int t) {
  const int lane = threadIdx.x & 31;
  if (t < __ldg(cu) || t >= __ldg(cu + B)) return -1;
  int lo = 0, hi = B;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + (lane + 1) * step;
    const bool below = i < hi && __ldg(cu + i) <= t;
    const int n = __ffs(~__ballot_sync(0xffffffffu, below) | 0x80000000u) - 1;
    lo += n * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// Forward. One warp per (token, block of U x 32 / (D/16) head rows); lane
// group g of the warp takes rows g, g + groups, ... The U loads of a lane are
// issued before any is used. U = 1 spreads a few tokens over more warps;
// U = 4 keeps enough bytes in flight for many.
template <typename T, int D, int U, bool APPEND>
__global__ void __launch_bounds__(kNrThreads) parallax_norm_rope_kernel(const NormRopeParams p) {
  constexpr int kLanes = D / 16, kGroups = 32 / kLanes, kRows = U * kGroups;
  pdl_wait_primary();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, li = lane % kLanes, grp = lane / kLanes;
  const int heads = p.H[0] + p.H[1] + p.H[2] + (APPEND ? p.H[3] : 0);
  const int per_token = (heads + kRows - 1) / kRows;
  const long long unit =
      (long long)blockIdx.x * (kNrThreads / 32) + (int)(threadIdx.x >> 5);
  if (unit >= (long long)p.tokens * per_token) return;
  const int t = (int)(unit / per_token), blk = (int)(unit - (long long)t * per_token);
  long long pos = t;
  size_t slot_row = 0;  // append: the token's row of the page pools
  bool in_cache = false;
  if (APPEND) {
    int b = t;
    long long at;
    if (p.cu != nullptr) {
      b = nr_find_sequence(p.cu, p.B, t);
      if (b < 0) return;  // a padding row: left as it is
      at = (long long)__ldg(p.lens + b) - __ldg(p.cu + b + 1) + t;
    } else {
      at = (long long)__ldg(p.lens + b) - 1;
    }
    pos = at;
    in_cache = at >= 0 && at < (long long)p.max_pages * p.page_size;
    if (in_cache) {
      const int page = __ldg(p.table + (size_t)b * p.max_pages + (int)at / p.page_size);
      in_cache = page >= 0 && page < p.num_pages;
      slot_row = (size_t)(in_cache ? page : 0) * p.page_size + (int)at % p.page_size;
    }
    if (!in_cache && lane == 0) atomicOr(p.status, kNrStatusClamped);
  } else if (p.seq_len > 0) {
    pos = t % p.seq_len;
  }
  if (p.pos != nullptr) pos = __ldg(p.pos + t);
  const NrLane<D> ln(li, p.rot, p.interleaved);
  float c[8], s[8];
  nr_load_angles<D>(nr_table_row(p, pos), ln, p.rot, p.interleaved, c, s);

  NrChunk<T> xa[U], xb[U];
  int kind[U], head[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    int h = blk * kRows + u * kGroups + grp;
    int k = 0;
    while (k < 4 && h >= p.H[k]) h -= p.H[k++];
    if (k >= (APPEND ? 4 : 3)) k = -1;
    kind[u] = k;
    head[u] = h;
    if (k >= 0) {
      const T* const row = static_cast<const T*>(p.x[k]) + (size_t)t * p.xs[k] + (size_t)h * D;
      xa[u].load(row + 8 * ln.a);
      xb[u].load(row + 8 * ln.b);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int k = kind[u];
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
    if (k >= 0) {
      xa[u].get(v);
      xb[u].get(v + 8);
    }
    const float rstd = nr_rstd<D>(v, p.eps);  // every lane takes part in the shuffles
    if (k < 0) continue;
    T* out;
    if (APPEND && k >= 2) {
      if (!in_cache) continue;
      out = static_cast<T*>(k == 2 ? p.k_pages : p.v_pages) +
            (slot_row * p.H[k] + (size_t)head[u]) * D;
    } else {
      out = static_cast<T*>(p.y[k]) + nr_out_offset(t, head[u], p.H[k], APPEND ? 0 : p.seq_len, D);
    }
    if (k < 3) {
      if (p.w[k] != nullptr) {
        NrChunk<T> wa, wb;
        float w[16];
        wa.load(static_cast<const T*>(p.w[k]) + 8 * ln.a);
        wb.load(static_cast<const T*>(p.w[k]) + 8 * ln.b);
        wa.get(w);
        wb.get(w + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = v[i] * rstd * w[i];
      }
      nr_rotate<D, 1>(v, ln, p.interleaved, c, s);
      xa[u].set(v);
      xb[u].set(v + 8);
    }
    xa[u].store(out + 8 * ln.a);
    xb[u].store(out + 8 * ln.b);
  }
}

// Backward. The blocks of a kind walk its tokens, one token per warp and
// step, all its heads (U row blocks at a time); dw stays in 16 registers per
// lane and is summed over the block's rows in shared memory at the end, one
// [D] partial per block in a fixed order.
template <typename T, int D, int U>
__global__ void __launch_bounds__(kNrThreads, 2)
    parallax_norm_rope_backward_kernel(const NormRopeParams p) {
  constexpr int kLanes = D / 16, kGroups = 32 / kLanes, kWarps = kNrThreads / 32;
  __shared__ float red[kWarps][D];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, li = lane % kLanes,
            grp = lane / kLanes;
  int k = 0;
  while (k < 2 && (int)blockIdx.x >= p.first_block[k + 1]) ++k;
  const int blk = (int)blockIdx.x - p.first_block[k], nblk = p.first_block[k + 1] - p.first_block[k];
  const int H = p.H[k];
  const T* const x = static_cast<const T*>(p.x[k]);
  const T* const dy = static_cast<const T*>(p.dy[k]);
  T* const dx = static_cast<T*>(p.dx[k]);
  const bool norm = p.w[k] != nullptr;
  const NrLane<D> ln(li, p.rot, p.interleaved);
  float w[16], dw[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    w[i] = 1.f;
    dw[i] = 0.f;
  }
  if (norm) {
    NrChunk<T> wa, wb;
    wa.load(static_cast<const T*>(p.w[k]) + 8 * ln.a);
    wb.load(static_cast<const T*>(p.w[k]) + 8 * ln.b);
    wa.get(w);
    wb.get(w + 8);
  }
  for (long long tt = (long long)blk * kWarps + warp; tt < p.tokens;
       tt += (long long)nblk * kWarps) {
    const int t = (int)tt;
    const long long pos = p.pos != nullptr ? __ldg(p.pos + t) : (p.seq_len > 0 ? t % p.seq_len : t);
    float c[8], s[8];
    nr_load_angles<D>(nr_table_row(p, pos), ln, p.rot, p.interleaved, c, s);
    for (int h0 = 0; h0 < H; h0 += U * kGroups) {
      NrChunk<T> xa[U], xb[U], ga[U], gb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * kGroups + grp;
        if (h < H) {
          const T* const g = dy + nr_out_offset(t, h, H, p.seq_len, D);
          ga[u].load(g + 8 * ln.a);
          gb[u].load(g + 8 * ln.b);
          if (norm) {
            const T* const row = x + (size_t)t * p.xs[k] + (size_t)h * D;
            xa[u].load(row + 8 * ln.a);
            xb[u].load(row + 8 * ln.b);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * kGroups + grp;
        float v[16], g[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = g[i] = 0.f;
        if (h < H) {
          ga[u].get(g);
          gb[u].get(g + 8);
          if (norm) {
            xa[u].get(v);
            xb[u].get(v + 8);
          }
        }
        nr_rotate<D, -1>(g, ln, p.interleaved, c, s);
        if (norm) {
          const float rstd = nr_rstd<D>(v, p.eps);
          float dot = 0.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            v[i] *= rstd;                    // xh
            dw[i] = fmaf(g[i], v[i], dw[i]);  // dz xh
            g[i] *= w[i];                    // dn
            dot = fmaf(g[i], v[i], dot);
          }
          dot = nr_row_sum<D>(dot) * (1.f / D);
#pragma unroll
          for (int i = 0; i < 16; ++i) g[i] = rstd * (g[i] - v[i] * dot);
        }
        if (h < H) {
          T* const out = dx + (size_t)t * p.dxs[k] + (size_t)h * D;
          ga[u].set(g);
          gb[u].set(g + 8);
          ga[u].store(out + 8 * ln.a);
          gb[u].store(out + 8 * ln.b);
        }
      }
    }
  }
  if (!norm) return;  // the whole block: one kind
#pragma unroll
  for (int i = 0; i < 16; ++i) {
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1) dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], o);
  }
  if (grp == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      red[warp][8 * ln.a + i] = dw[i];
      red[warp][8 * ln.b + i] = dw[8 + i];
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kNrThreads) {
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) sum += red[v][d];
    p.partial[(size_t)blockIdx.x * D + d] = sum;
  }
}

// dw of each kind from its blocks' partials, in block order per thread.
template <int D>
__global__ void __launch_bounds__(1024) parallax_norm_rope_dw_kernel(const NormRopeParams p) {
  constexpr int kParts = 1024 / D;
  __shared__ float red[kParts][D];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int k = blockIdx.x, d = threadIdx.x % D, part = threadIdx.x / D;
  if (p.H[k] == 0 || p.w[k] == nullptr) return;
  float sum = 0.f;
  for (int b = p.first_block[k] + part; b < p.first_block[k + 1]; b += kParts)
    sum += __ldcg(p.partial + (size_t)b * D + d);
  red[part][d] = sum;
  __syncthreads();
  if (part == 0) {
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < kParts; ++i) all += red[i][d];
    p.dw[k][d] = all;
  }
}

// cos_sin[t][p], cos_sin[t][rot/2 + p] = cos, sin of t base^(-2p/rot), the
// angle in fp64: at position 10^6 an fp32 angle is off by up to 0.03.
__global__ void __launch_bounds__(kNrThreads)
    parallax_rope_table_kernel(float* cs, int max_pos, int rot, double base) {
  const long long i = (long long)blockIdx.x * kNrThreads + threadIdx.x;
  const int half = rot / 2;
  if (i >= (long long)max_pos * half) return;
  const int t = (int)(i / half), q = (int)(i % half);
  double sn, co;
  sincos((double)t * pow(base, -2.0 * q / rot), &sn, &co);
  cs[(size_t)t * rot + q] = (float)co;
  cs[(size_t)t * rot + half + q] = (float)sn;
}

}  // namespace plx
