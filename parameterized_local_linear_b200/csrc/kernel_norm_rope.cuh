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
// Bound: HBM for many tokens (a row is read once and written once, the table
// row of a token, 4 rot bytes, once per warp), launch latency for few. Measured,
// bf16, 16384 tokens of 16 + 16 + 8 heads of 128: forward 58.5 us, 5.8 TB/s,
// backward 94.4 us, 5.4 TB/s (a plain copy: 6.55); the append of 1 token 2.6 us,
// of 128 tokens 3.6, of 2674 tokens in 12 chunks 17.9 (3.7 TB/s).
//  - D/16 lanes share a row, 16 values each: two chunks of 8 whose dimensions
//    pair up under the rotation (chunks c and c + rot/16), so the rotation
//    needs no exchange and the norm log2(D/16) shuffles. A warp holds
//    32 / (D/16) heads of one token per step.
//  - A block works on one kind of head (query, probe, key, value), so its
//    weight stays in registers, multiplied into the token's cosines and sines:
//    a value costs two packed multiply-adds and a scaling.
//  - A warp's rows come through a ring of its own in shared memory, a token's
//    heads by one bulk copy, the next ones in flight while it works: as loads to
//    registers the forward took 102 us, with too few bytes in flight.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace plx {

constexpr int kNrThreads = 256;
constexpr int kNrWarps = kNrThreads / 32;
constexpr unsigned int kNrStatusClamped = 2u;   // PARALLAX_DEVICE_STATUS_SEQLEN_CLAMPED
constexpr unsigned int kNrStatusPosition = 4u;  // PARALLAX_DEVICE_STATUS_POSITION_CLAMPED

// n / d for 0 <= n < 2^31 without a division instruction sequence (Granlund
// and Montgomery, "Division by invariant integers using multiplication"): with
// 2^s >= d > 2^(s-1) and m = floor(2^32 (2^s - d) / d) + 1, the quotient is
// (mulhi(m, n) + n) >> s. Units of work are placed by two divisions each.
struct NrDivisor {
  uint32_t d, m, s;
  __host__ static NrDivisor of(int d) {
    NrDivisor r{(uint32_t)d, 0, 0};
    while ((1ull << r.s) < (unsigned long long)d) ++r.s;
    r.m = (uint32_t)((((1ull << r.s) - d) << 32) / d + 1);
    return r;
  }
  __host__ __device__ int quotient(int n) const {
#ifdef __CUDA_ARCH__
    const uint32_t hi = __umulhi(m, (uint32_t)n);
#else
    const uint32_t hi = (uint32_t)((uint64_t)m * (uint32_t)n >> 32);
#endif
    return (int)((hi + (uint32_t)n) >> s);
  }
};

struct NormRopeParams {
  // kinds: 0 query, 1 probe, 2 key, 3 value (append only, copied)
  const void* x[4];       // [tokens] rows xs[i] elements apart, heads D apart
  const void* w[4];       // [D], or nullptr: no norm
  void* y[4];             // outputs; append: y[2], y[3] are the pools
  long long xs[4];
  int H[4];               // heads of each kind; 0 leaves it out
  const float* cs;        // [max_pos][rot]: cosines, then sines
  const int32_t* pos;     // [tokens], or nullptr
  int tokens, rot, seq_len, max_pos;
  NrDivisor seq_div, unit_div[4];  // by seq_len; by a token's units of each kind
  float eps;
  unsigned int* status;
  int first_block[5];     // blocks of kind i: first_block[i] .. first_block[i + 1]
  int unit_rows;          // heads of a token that a warp takes at a time
  // append
  const int32_t *cu, *lens, *table;
  int B, page_size, num_pages, max_pages;
  NrDivisor page_div;     // by page_size
  int clear_rest;         // zeros to the query (bit 0), probe (bit 1) rows without a token
  // backward: dy in the layout of y, dx rows dxs[i] elements apart
  const void* dy[3];
  void* dx[3];
  long long dxs[3];
  float* partial;         // [blocks][D] sums of dz xh
  unsigned int* done;     // [3] blocks of each kind whose partials are written
  float* dw[3];
  unsigned long long timeout_ns;  // of each wait
  int debug_skip_unit;            // testing hook: a unit of each kind whose rows are never loaded
};

// The two 8-value chunks a lane holds of a D-value row, and which of them the
// rotation touches. Halves: chunks (i, i + rot/16) rotate as pairs for
// i < rot/16, the other lanes hold the chunks that pass through. Interleaved:
// chunks (i, i + D/16), each with its pairs inside.
template <int D, bool INTER>
struct NrLane {
  int a, b;  // chunk indices
  bool rot_a, rot_b;
  __device__ NrLane(int i, int rot) {
    if (INTER) {
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

// 8 values as packed pairs, from or to memory.
__device__ __forceinline__ void nr_get(const __nv_bfloat16* p, f32x2 (&f)[4]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2_pack(bf16_lo_to_float(v[i]), bf16_hi_to_float(v[i]));
}
__device__ __forceinline__ void nr_get(const float* p, f32x2 (&f)[4]) {
  const float4 u = reinterpret_cast<const float4*>(p)[0], v = reinterpret_cast<const float4*>(p)[1];
  f[0] = f2_pack(u.x, u.y), f[1] = f2_pack(u.z, u.w);
  f[2] = f2_pack(v.x, v.y), f[3] = f2_pack(v.z, v.w);
}
__device__ __forceinline__ void nr_put(__nv_bfloat16* p, const f32x2 (&f)[4]) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_unpack(f[i], lo, hi);
    v[i] = pack_bf16x2(lo, hi);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void nr_put(float* p, const f32x2 (&f)[4]) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f2_unpack(f[i], v[2 * i], v[2 * i + 1]);
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// The rotation's factors of one lane: y_a = x_a ca + z_a sa, y_b = x_b cb +
// z_b sb, where z is the other member of each pair (halves: the other chunk;
// interleaved: the pair swapped). BACK rotates the other way.
struct NrAngles {
  f32x2 ca[4], sa[4], cb[4], sb[4];
};

template <int D, bool INTER, bool BACK>
__device__ __forceinline__ NrAngles nr_angles(const float* row, const NrLane<D, INTER>& ln,
                                              int rot) {
  NrAngles g;
  const float* const sn = row + rot / 2;
  if (INTER) {
    const auto chunk = [&](int c, bool on, f32x2(&co)[4], f32x2(&si)[4]) {
      float4 x = make_float4(1.f, 1.f, 1.f, 1.f), y = make_float4(0.f, 0.f, 0.f, 0.f);
      if (on) {
        x = *reinterpret_cast<const float4*>(row + 4 * c);
        y = *reinterpret_cast<const float4*>(sn + 4 * c);
      }
      const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        co[i] = f2_pack(xs[i], xs[i]);
        si[i] = BACK ? f2_pack(ys[i], -ys[i]) : f2_pack(-ys[i], ys[i]);
      }
    };
    chunk(ln.a, ln.rot_a, g.ca, g.sa);
    chunk(ln.b, ln.rot_b, g.cb, g.sb);
  } else {
    const f32x2 minus = f2_pack(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      g.ca[i] = f2_pack(1.f, 1.f);
      g.sa[i] = 0;
    }
    if (ln.rot_a) {
      nr_get(row + 8 * ln.a, g.ca);
      nr_get(sn + 8 * ln.a, g.sa);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      g.cb[i] = g.ca[i];
      g.sb[i] = BACK ? f2_mul(g.sa[i], minus) : g.sa[i];
      if (!BACK) g.sa[i] = f2_mul(g.sa[i], minus);
    }
  }
  return g;
}

// Chunks that the rotation does not touch only take their factor: an infinity
// or a NaN stays in its place.
template <int D, bool INTER>
__device__ __forceinline__ void nr_rotate(f32x2 (&a)[4], f32x2 (&b)[4],
                                          const NrLane<D, INTER>& ln, const NrAngles& g) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 x = a[i], y = b[i];
    const f32x2 za = INTER ? f2_swap(x) : y, zb = INTER ? f2_swap(y) : x;
    a[i] = f2_mul(x, g.ca[i]);
    b[i] = f2_mul(y, g.cb[i]);
    if (ln.rot_a) a[i] = f2_fma(za, g.sa[i], a[i]);
    if (ln.rot_b) b[i] = f2_fma(zb, g.sb[i], b[i]);
  }
}

// Sum over the D/16 lanes of a row.
template <int D>
__device__ __forceinline__ float nr_row_sum(float x) {
#pragma unroll
  for (int o = D / 32; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// sum of a.x + b.y over a lane's 16 values
__device__ __forceinline__ float nr_dot(const f32x2 (&a)[4], const f32x2 (&x)[4],
                                        const f32x2 (&b)[4], const f32x2 (&y)[4]) {
  f32x2 s = f2_mul(a[0], x[0]), u = f2_mul(b[0], y[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    s = f2_fma(a[i], x[i], s);
    u = f2_fma(b[i], y[i], u);
  }
  float s0, s1, u0, u1;
  f2_unpack(s, s0, s1);
  f2_unpack(u, u0, u1);
  return (s0 + s1) + (u0 + u1);
}

// 1 / sqrt(mean(x^2) + eps) of a row
template <int D>
__device__ __forceinline__ float nr_rstd(const f32x2 (&a)[4], const f32x2 (&b)[4], float eps) {
  return rsqrtf(nr_row_sum<D>(nr_dot(a, a, b, b)) * (1.f / D) + eps);
}

// The table row of a position (clamped into the table and flagged).
__device__ __forceinline__ const float* nr_table_row(const NormRopeParams& p, long long pos) {
  if (pos < 0 || pos >= p.max_pos) {
    atomicOr(p.status, kNrStatusPosition);
    pos = pos < 0 ? 0 : p.max_pos - 1;
  }
  return p.cs + (size_t)pos * p.rot;
}

// The sequences of an append's packed rows. Up to 32 of them are kept by the
// warp, one per lane; more are searched in memory.
struct NrBatch {
  int end, len, begin;  // cu[lane + 1], lens[lane], cu[0]
  __device__ NrBatch(const int32_t* cu, const int32_t* lens, int B) : end(0x7fffffff), len(0), begin(0) {
    const int lane = threadIdx.x & 31;
    if (cu != nullptr && B <= 32) {
      begin = __ldg(cu);
      if (lane < B) {
        end = __ldg(cu + lane + 1);
        len = __ldg(lens + lane);
      }
    }
  }
  // The key index that row t becomes and (slot) its sequence; slot -1 and key -1
  // outside every sequence. A key below 0 or past the table is not stored; the
  // caller sees it by the page it then lacks.
  __device__ long long key(const int32_t* cu, const int32_t* lens, int B, int t, int& b) const {
    if (cu == nullptr) {
      const int n = __ldg(lens + t);
      b = n == 0 ? -1 : t;  // a length of 0: an idle row
      return (long long)n - 1;
    }
    int last, n;
    if (B <= 32) {
      // the largest b with cu[b] <= t < cu[b + 1]: as many ends in a row are <= t
      const unsigned past = __ballot_sync(0xffffffffu, end <= t);
      b = past == 0xffffffffu ? 32 : __ffs(~past) - 1;
      if (t < begin || b >= B) {
        b = -1;
        return -1;
      }
      last = __shfl_sync(0xffffffffu, end, b);
      n = __shfl_sync(0xffffffffu, len, b);
    } else {
      b = search(cu, B, t);
      if (b < 0) return -1;
      last = __ldg(cu + b + 1);
      n = __ldg(lens + b);
    }
    return (long long)n - last + t;
  }
  // The largest b with cu[b] <= t < cu[b + 1], or -1. Warp-cooperative (one
  // 32-way step per 32 x), bounded for any contents of cu.
  static __device__ int search(const int32_t* cu, int B, int t) {
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
};

// A unit of work is up to `rows` heads of one kind and token. A warp's units
// are `stride` apart.
struct NrUnits {
  int unit, stride, count, rows;
  NrDivisor per_token;
  __device__ NrUnits(int first, int stride_, int tokens, const NrDivisor& per, int rows_)
      : unit(first), stride(stride_), rows(rows_), per_token(per) {
    count = tokens * (int)per.d;  // below 2^31: the entry points check tokens x heads
  }
  __device__ bool valid() const { return unit < count; }
  __device__ void place(int& t, int& h0) const {
    t = per_token.quotient(unit);
    h0 = (unit - t * (int)per_token.d) * rows;
  }
  __device__ void next() { unit = count - unit > stride ? unit + stride : count; }
};

// The ring of one warp: kStages stages of PARTS x BYTES of head rows, a table
// row (up to 512 bytes) and a note, filled by bulk copies that an mbarrier per
// stage counts.
template <int PARTS, int BYTES, int STAGES>
struct NrRing {
  static constexpr int kStages = STAGES, kBytes = BYTES;
  static constexpr int kStageBytes = PARTS * BYTES + 512 + 16;
  static constexpr int kWarpBytes = STAGES * (kStageBytes + 16);
  static constexpr int kSmem = kNrWarps * kWarpBytes;
  uint8_t* base;  // this warp's
  __device__ uint8_t* rows(int st, int part) const {
    return base + st * kStageBytes + part * BYTES;
  }
  __device__ float* table(int st) const {
    return reinterpret_cast<float*>(base + st * kStageBytes + PARTS * BYTES);
  }
  __device__ long long* note(int st) const {
    return reinterpret_cast<long long*>(base + st * kStageBytes + PARTS * BYTES + 512);
  }
  __device__ uint32_t bar(int st) const { return smem_u32(base + STAGES * kStageBytes + st * 16); }
  __device__ void init() const {  // one lane
    for (int st = 0; st < STAGES; ++st) mbar_init(bar(st), 1);
    mbar_fence_init();
  }
  // Waits for the copies of a unit. Where they do not land, reports it, gives those
  // of the units after it as long (the ones started: up to STAGES - 1) and fails.
  __device__ bool wait(int st, uint32_t parity, NrUnits at, const NormRopeParams& p) const {
    const bool got = mbar_wait_bounded(bar(st), parity, p.timeout_ns, nullptr);
    if (__all_sync(0xffffffffu, got)) return true;  // (the warp goes on or gives up as one)
    atomicOr(p.status, 1u /* PARALLAX_DEVICE_STATUS_TIMEOUT */);
    for (int i = 1; i < STAGES; ++i) {
      at.next();
      if (!at.valid()) break;
      if (++st == STAGES) {
        st = 0;
        parity ^= 1;
      }
      mbar_wait_bounded(bar(st), parity, p.timeout_ns, nullptr);
    }
    return false;
  }
};

// 4 KB of rows per stage: 16 heads of 128 bf16 dimensions. Two blocks per SM
// (16 warps with 12 KB each in flight; two stages measure the same as three).
using NrForwardRing = NrRing<1, 4096, 3>;
// 2 KB of dy and as much of x. Two blocks per SM.
using NrBackwardRing = NrRing<2, 2048, 3>;

template <typename T, int D, bool INTER, bool APPEND>
__global__ void __launch_bounds__(kNrThreads, 2)
    parallax_norm_rope_kernel(const NormRopeParams p) {
  using Ring = NrForwardRing;
  constexpr int kLanes = D / 16, kGroups = 32 / kLanes, kSt = Ring::kStages;
  constexpr int kRowBytes = D * (int)sizeof(T);
  constexpr int kKinds = APPEND ? 4 : 3;
  extern __shared__ __align__(16) uint8_t ring_bytes[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, li = lane % kLanes,
            grp = lane / kLanes;
  const Ring ring{ring_bytes + warp * Ring::kWarpBytes};
  if (lane == 0) ring.init();
  __syncwarp();
  int k = 0;
  while (k < kKinds - 1 && (int)blockIdx.x >= p.first_block[k + 1]) ++k;
  const int blk = (int)blockIdx.x - p.first_block[k],
            nblk = p.first_block[k + 1] - p.first_block[k];
  const int H = p.H[k];
  const T* const x = static_cast<const T*>(p.x[k]);
  T* const y = static_cast<T*>(p.y[k]);
  const T* const wt = static_cast<const T*>(p.w[k]);
  const long long xs = p.xs[k];
  const NrLane<D, INTER> ln(li, p.rot);
  pdl_wait_primary();
  pdl_launch_dependents();
  NrUnits at(blk * kNrWarps + warp, nblk * kNrWarps, p.tokens, p.unit_div[k], p.unit_rows),
      load_at = at;
  const NrBatch batch(APPEND ? p.cu : nullptr, APPEND ? p.lens : nullptr, p.B);
  // A unit's place: its position, and (append) the page that takes its key. The
  // append's chain of loads (length, page id) is looked up one unit ahead, so
  // that none is waited for when the copies start (2674 tokens 20.5 -> 17.9 us);
  // the plain forward's one position is not: with it ahead, 16384 tokens take 64
  // us instead of 58.5.
  struct Place {
    int pos, page, slot;  // slot -1: a padding row; page and slot of kinds 2, 3
  };
  const auto look_up = [&](const NrUnits& u) {
    Place f{0, -1, -1};
    if (!u.valid()) return f;
    int t, h0;
    u.place(t, h0);
    long long key = t;
    f.slot = 0;
    if (APPEND) {
      key = batch.key(p.cu, p.lens, p.B, t, f.slot);
      if (k >= 2 && key >= 0 && key < (long long)p.max_pages * p.page_size) {
        const int i = p.page_div.quotient((int)key);
        f.page = __ldg(p.table + (size_t)f.slot * p.max_pages + i);
        f.slot = (int)key - i * p.page_size;
      }
    } else if (p.seq_len > 0) {
      key = t - p.seq_div.quotient(t) * p.seq_len;
    }
    f.pos = (int)max(-1LL, min(key, 0x7fffffffLL));  // (outside the table: clamped below)
    if (p.pos != nullptr && k < 3 && f.slot >= 0) f.pos = __ldg(p.pos + t);
    return f;
  };
  Place ahead{};  // APPEND
  if (APPEND) ahead = look_up(load_at);
  // Starts the copies of the next unit. Its note: the first row (in units of D
  // elements) of its token's heads in the output, or -1 where it has none; ~row of
  // a query or probe row without a token that is to be cleared.
  const auto load = [&](int st) {
    if (!load_at.valid()) return;
    int t, h0;
    load_at.place(t, h0);
    const Place f = APPEND ? ahead : look_up(load_at);
    load_at.next();
    const uint32_t bytes = (uint32_t)(min(load_at.rows, H - h0) * kRowBytes);
    if (lane == 0) {
      mbar_arrive_expect_tx(ring.bar(st), bytes + (k < 3 ? p.rot * 4 : 0));
      bulk_load(smem_u32(ring.rows(st, 0)), x + (size_t)t * xs + (size_t)h0 * D, bytes,
                ring.bar(st));
      long long note = (long long)t * H;
      if (APPEND && f.slot < 0) {
        note = p.clear_rest >> k & 1 ? ~note : -1;
      } else if (APPEND && k >= 2) {  // the key's place in the pools
        const bool held = f.page >= 0 && f.page < p.num_pages;
        note = held ? ((long long)f.page * p.page_size + f.slot) * H : -1;
        if (!held) atomicOr(p.status, kNrStatusClamped);
      } else if (!APPEND && p.seq_len > 0) {
        const int row = p.seq_div.quotient(t);
        note = (long long)row * H * p.seq_len + (t - row * p.seq_len);
      }
      if (k < 3)
        bulk_load(smem_u32(ring.table(st)), f.slot < 0 ? p.cs : nr_table_row(p, f.pos), p.rot * 4,
                  ring.bar(st));
      *ring.note(st) = note;
    }
    if (APPEND) ahead = look_up(load_at);
  };
#pragma unroll 1
  for (int st = 0; st < kSt; ++st) {
    if (load_at.unit != p.debug_skip_unit) {
      load(st);
    } else {
      load_at.next();
      if (APPEND) ahead = look_up(load_at);
    }
  }
  __syncwarp();  // the notes (later ones: the barrier that frees each stage)

  f32x2 wa[4], wb[4];
  const bool norm = wt != nullptr;
  if (norm) {
    nr_get(wt + 8 * ln.a, wa);
    nr_get(wt + 8 * ln.b, wb);
  }
  // heads of an output row are D apart, or with seq_len > 0 seq_len * D
  const size_t head_step = (!APPEND && p.seq_len > 0 ? (size_t)p.seq_len : 1) * D;
  int st = 0;
  uint32_t parity = 0;
  for (; at.valid(); at.next()) {
    int t, h0;
    at.place(t, h0);
    if (!ring.wait(st, parity, at, p)) break;
    const long long out_row = *ring.note(st);
    const int n = min(at.rows, H - h0);
    if (out_row >= 0) {
      NrAngles ang;
      if (k < 3) {
        ang = nr_angles<D, INTER, false>(ring.table(st), ln, p.rot);
        if (norm) {
          // the weight belongs to the source of each term: n_a cos, n_b sin, ...
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ang.ca[i] = f2_mul(ang.ca[i], wa[i]);
            ang.cb[i] = f2_mul(ang.cb[i], wb[i]);
            ang.sa[i] = f2_mul(ang.sa[i], INTER ? f2_swap(wa[i]) : wb[i]);
            ang.sb[i] = f2_mul(ang.sb[i], INTER ? f2_swap(wb[i]) : wa[i]);
          }
        }
      }
      T* out = y + (size_t)out_row * D + (size_t)(h0 + grp) * head_step;
      const T* row = reinterpret_cast<const T*>(ring.rows(st, 0)) + grp * D;
#pragma unroll 2
      for (int h = grp; h < n + grp; h += kGroups) {  // the warp's groups together
        f32x2 a[4], b[4];
        nr_get(row + 8 * ln.a, a);  // past the unit's rows: stale, not stored
        nr_get(row + 8 * ln.b, b);
        if (k < 3) {
          const float rstd = norm ? nr_rstd<D>(a, b, p.eps) : 1.f;
          nr_rotate<D, INTER>(a, b, ln, ang);
          if (norm) {
            const f32x2 rr = f2_pack(rstd, rstd);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              a[i] = f2_mul(a[i], rr);
              b[i] = f2_mul(b[i], rr);
            }
          }
        }
        if (h < n) {
          nr_put(out + 8 * ln.a, a);
          nr_put(out + 8 * ln.b, b);
        }
        out += kGroups * head_step;
        row += kGroups * D;
      }
    } else if (APPEND && (p.clear_rest >> k & 1)) {
      const f32x2 zero[4] = {0, 0, 0, 0};
      for (int h = grp; h < n; h += kGroups) {
        T* const out = y + ((size_t)~out_row + h0 + h) * D;
        nr_put(out + 8 * ln.a, zero);
        nr_put(out + 8 * ln.b, zero);
      }
    }
    __syncwarp();  // the warp is done with this stage
    load(st);
    if (++st == kSt) {
      st = 0;
      parity ^= 1;
    }
  }
}

// Backward: dw stays in 16 registers per lane and is summed over the block's
// rows in shared memory at the end, one [D] partial per block in a fixed order,
// and over the blocks by the last of them. (In a kernel of its own that sum took
// 2 us more of a 777-token call.)
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kNrThreads, 2)
    parallax_norm_rope_backward_kernel(const NormRopeParams p) {
  using Ring = NrBackwardRing;
  constexpr int kLanes = D / 16, kGroups = 32 / kLanes, kSt = Ring::kStages;
  constexpr int kRowBytes = D * (int)sizeof(T);
  extern __shared__ __align__(16) uint8_t ring_bytes[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, li = lane % kLanes,
            grp = lane / kLanes;
  const Ring ring{ring_bytes + warp * Ring::kWarpBytes};
  if (lane == 0) ring.init();
  __syncwarp();
  int k = 0;
  while (k < 2 && (int)blockIdx.x >= p.first_block[k + 1]) ++k;
  const int blk = (int)blockIdx.x - p.first_block[k],
            nblk = p.first_block[k + 1] - p.first_block[k];
  const int H = p.H[k];
  const T* const x = static_cast<const T*>(p.x[k]);
  const T* const dy = static_cast<const T*>(p.dy[k]);
  T* const dx = static_cast<T*>(p.dx[k]);
  const T* const wt = static_cast<const T*>(p.w[k]);
  const long long xs = p.xs[k], dxs = p.dxs[k];
  const bool norm = wt != nullptr;
  const NrLane<D, INTER> ln(li, p.rot);
  pdl_wait_primary();
  pdl_launch_dependents();
  NrUnits at(blk * kNrWarps + warp, nblk * kNrWarps, p.tokens, p.unit_div[k], p.unit_rows),
      load_at = at;
  const auto position = [&](const NrUnits& u) {  // looked up one unit ahead, 1% faster
    int t, h0;
    u.place(t, h0);
    if (p.pos != nullptr) return u.valid() ? __ldg(p.pos + t) : 0;
    return p.seq_len > 0 ? t - p.seq_div.quotient(t) * p.seq_len : t;
  };
  int ahead = position(load_at);
  const auto load = [&](int st) {
    if (!load_at.valid()) return;
    int t, h0;
    load_at.place(t, h0);
    load_at.next();
    const int pos = ahead;
    const int n = min(load_at.rows, H - h0);
    const uint32_t bytes = (uint32_t)(n * kRowBytes);
    long long dy_row = (long long)t * H + h0;
    if (p.seq_len > 0) {
      const int row = p.seq_div.quotient(t), i = t - row * p.seq_len;
      dy_row = ((long long)row * H + h0) * p.seq_len + i;
    }
    if (lane == 0) {
      mbar_arrive_expect_tx(ring.bar(st), (norm ? 2 : 1) * bytes + p.rot * 4);
      if (norm)
        bulk_load(smem_u32(ring.rows(st, 1)), x + (size_t)t * xs + (size_t)h0 * D, bytes,
                  ring.bar(st));
      if (p.seq_len == 0)
        bulk_load(smem_u32(ring.rows(st, 0)), dy + (size_t)dy_row * D, bytes, ring.bar(st));
      bulk_load(smem_u32(ring.table(st)), nr_table_row(p, pos), p.rot * 4, ring.bar(st));
    }
    if (p.seq_len > 0) {  // a head's rows are seq_len apart: one copy per head
      __syncwarp();       // after the expected bytes are set
      if (lane < n)
        bulk_load(smem_u32(ring.rows(st, 0)) + lane * kRowBytes,
                  dy + (size_t)(dy_row + (long long)lane * p.seq_len) * D, kRowBytes, ring.bar(st));
    }
    ahead = position(load_at);
  };
#pragma unroll 1
  for (int st = 0; st < kSt; ++st) {
    if (load_at.unit != p.debug_skip_unit) {
      load(st);
    } else {
      load_at.next();
      ahead = position(load_at);
    }
  }

  f32x2 wa[4], wb[4], da[4] = {0, 0, 0, 0}, db[4] = {0, 0, 0, 0};
  if (norm) {
    nr_get(wt + 8 * ln.a, wa);
    nr_get(wt + 8 * ln.b, wb);
  }
  int st = 0;
  uint32_t parity = 0;
  for (; at.valid(); at.next()) {
    int t, h0;
    at.place(t, h0);
    if (!ring.wait(st, parity, at, p)) break;
    const int n = min(at.rows, H - h0);
    const NrAngles ang = nr_angles<D, INTER, true>(ring.table(st), ln, p.rot);
    T* out = dx + (size_t)t * dxs + (size_t)(h0 + grp) * D;
    const T* gr = reinterpret_cast<const T*>(ring.rows(st, 0)) + grp * D;
    const T* xr = reinterpret_cast<const T*>(ring.rows(st, 1)) + grp * D;
#pragma unroll 2
    for (int h = grp; h < n + grp; h += kGroups) {  // the warp's groups together
      f32x2 ga[4], gb[4], a[4], b[4];
      const bool live = h < n;
      nr_get(gr + 8 * ln.a, ga);  // past the unit's rows: stale, not stored or summed
      nr_get(gr + 8 * ln.b, gb);
      nr_rotate<D, INTER>(ga, gb, ln, ang);  // dz
      if (norm) {
        nr_get(xr + 8 * ln.a, a);
        nr_get(xr + 8 * ln.b, b);
        const float rstd = nr_rstd<D>(a, b, p.eps);
        const f32x2 rr = f2_pack(rstd, rstd);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = f2_mul(a[i], rr);  // xh
          b[i] = f2_mul(b[i], rr);
          if (live) {
            da[i] = f2_fma(ga[i], a[i], da[i]);  // dz xh
            db[i] = f2_fma(gb[i], b[i], db[i]);
          }
          ga[i] = f2_mul(ga[i], wa[i]);  // dn
          gb[i] = f2_mul(gb[i], wb[i]);
        }
        // rstd (dn - xh mean(dn xh))
        const float m = nr_row_sum<D>(nr_dot(ga, a, gb, b)) * (-1.f / D);
        const f32x2 mm = f2_pack(m, m);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ga[i] = f2_mul(f2_fma(a[i], mm, ga[i]), rr);
          gb[i] = f2_mul(f2_fma(b[i], mm, gb[i]), rr);
        }
      }
      if (live) {
        nr_put(out + 8 * ln.a, ga);
        nr_put(out + 8 * ln.b, gb);
      }
      out += kGroups * D;
      gr += kGroups * D;
      xr += kGroups * D;
    }
    __syncwarp();  // the warp is done with this stage
    load(st);
    if (++st == kSt) {
      st = 0;
      parity ^= 1;
    }
  }
  if (!norm) return;  // the whole block: one kind
  __syncthreads();  // no copy is in flight; the rings' space now holds the warps' sums
  float(*const red)[D] = reinterpret_cast<float(*)[D]>(ring_bytes);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[4];
    f2_unpack(da[i], v[0], v[1]);
    f2_unpack(db[i], v[2], v[3]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int o = kLanes; o < 32; o <<= 1) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
      if (grp == 0) red[warp][8 * (j < 2 ? ln.a : ln.b) + 2 * i + (j & 1)] = v[j];
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kNrThreads) {
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < kNrWarps; ++v) sum += red[v][d];
    __stcg(p.partial + (size_t)blockIdx.x * D + d, sum);
  }
  // The kind's last block sums the partials, each thread and then the threads of
  // a column in a fixed order. The counter wraps to 0 for the next call.
  __shared__ bool last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicInc(p.done + k, nblk - 1) == (unsigned)nblk - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  constexpr int kCols = D / 4, kParts = kNrThreads / kCols;
  float4(*const sums)[kCols] = reinterpret_cast<float4(*)[kCols]>(ring_bytes);
  const int c = threadIdx.x % kCols, part = threadIdx.x / kCols;
  const float4* from = reinterpret_cast<const float4*>(p.partial) + (size_t)p.first_block[k] * kCols + c;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int b = part; b < nblk; b += kParts) {
    const float4 v = __ldcg(from + (size_t)b * kCols);
    s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
  }
  sums[part][c] = s;
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kNrThreads) {
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < kParts; ++i) all += reinterpret_cast<const float*>(sums[i])[d];
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
