// How the chunk attention over a paged cache is dealt to its CTAs; shared by
// the attention kernel and its merge kernel.
//
// A row tile is `tpt` consecutive new tokens of one sequence with all G query
// heads of one kv head (tpt = 128 / G, so at most 128 rows); an item is a row
// tile and a kv head. It walks the 64-key tiles its last row can see, at least
// one (a masked one, if it sees no key: its rows are then written as zeros).
// The items are laid end to end, ordered by (sequence, kv head, row tile), each
// kChunkItemCost + tiles long: the fixed part stands for the tiles' worth of
// time that loading Q and R and writing the result take (2 and 5 instead of 3:
// within 1% on large batches; 5 costs three short sequences 6%). P CTAs cut the line
// into equal ranges, so whatever the lengths, every CTA gets the same work and
// the last key of a long row tile does not leave one CTA running alone. The
// part of an item inside a range is a piece; a piece that does not hold all of
// its item's tiles writes a partial record to slot 2c (a piece at the start of
// range c) or 2c + 1 (one at its end), and the CTA in whose range the item ends
// merges them.
#pragma once

#include <cstdint>

#include "partition.cuh"

// The arithmetic also compiles for the host, where tests walk it.
#define PLX_HD __host__ __device__ __forceinline__

namespace plx {

PLX_HD int chunk_load(const int32_t* p) {
#ifdef __CUDA_ARCH__
  return __ldg(p);
#else
  return *p;
#endif
}

constexpr int kChunkRows = 128;
constexpr int kChunkKeys = 64;
constexpr int kChunkItemCost = 3;

struct ChunkSpace {
  const int32_t* cu;    // [B + 1] first new token of each sequence, or NULL: one each
  const int32_t* lens;  // [B] cached keys, the new tokens' included
  int B, total, Lmax, Hkv, tpt, causal;
};

struct ChunkSeq {
  int s0, q, n;  // first packed row, new tokens, cached keys
};

PLX_HD int chunk_clamp(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }
PLX_HD int chunk_min(int a, int b) { return a < b ? a : b; }
PLX_HD int chunk_max(int a, int b) { return a > b ? a : b; }

PLX_HD ChunkSeq chunk_seq(const ChunkSpace& sp, int b) {
  ChunkSeq s;
  s.s0 = sp.cu ? chunk_clamp(chunk_load(sp.cu + b), 0, sp.total) : b;
  s.q = sp.cu ? chunk_clamp(chunk_load(sp.cu + b + 1), s.s0, sp.total) - s.s0 : 1;
  s.n = clamp_len(chunk_load(sp.lens + b), sp.Lmax);
  return s;
}

PLX_HD int chunk_row_tiles(const ChunkSpace& sp, const ChunkSeq& s) {
  return (s.q + sp.tpt - 1) / sp.tpt;
}

// A sequence whose bounds or length chunk_seq clamped, or with more new tokens
// than keys.
__device__ __forceinline__ bool chunk_seq_clamped(const ChunkSpace& sp, int b) {
  const int a = sp.cu ? __ldg(sp.cu + b) : b, e = sp.cu ? __ldg(sp.cu + b + 1) : b + 1;
  const int n = __ldg(sp.lens + b);
  return a < 0 || e < a || e > sp.total || n < 0 || n > sp.Lmax || (sp.causal && n < e - a);
}

// The tiles that hold the keys the last row of row tile rt sees.
PLX_HD int chunk_tiles(const ChunkSpace& sp, const ChunkSeq& s, int rt) {
  const int kend = sp.causal ? s.n - s.q + chunk_min(s.q, (rt + 1) * sp.tpt) : s.n;
  return chunk_max(1, (kend + kChunkKeys - 1) / kChunkKeys);
}

// sum of ceil((a + i T) / 64) over i = 1 .. m, for a >= 0: with i = 64 u + v, the
// terms of a whole period of 64 rise by T from one period to the next. T a divisor
// or multiple of 64 (any power of two) has a shorter one.
PLX_HD long long chunk_ceil_sum(int a, int T, int m) {
  const int period = T >= 64 ? (T % 64 == 0 ? 1 : 64) : (64 % T == 0 ? 64 / T : 64);
  const int rise = period * T / 64;  // of a term, one period later
  const int u = m / period, v = m - u * period;
  long long sum = 0;
  for (int i = 1; i <= chunk_min(m, period); ++i) {
    const long long first = (a + (long long)i * T + 63) / 64;
    const long long terms = u + (i <= v ? 1 : 0);
    sum += terms * first + rise * (terms * (terms - 1) / 2);
  }
  return sum;
}

// The length of the first m items of one kv head of a sequence. A loop where
// some rows see no key (more new tokens than keys).
PLX_HD long long chunk_cost(const ChunkSpace& sp, const ChunkSeq& s, int m) {
  if (!sp.causal) return m * (long long)(chunk_tiles(sp, s, 0) + kChunkItemCost);
  long long c = (long long)m * kChunkItemCost;
  if (s.n < s.q) {
    for (int rt = 0; rt < m; ++rt) c += chunk_tiles(sp, s, rt);
    return c;
  }
  const int whole = m > 0 && m == chunk_row_tiles(sp, s) ? m - 1 : m;  // the last may be cut short
  c += chunk_ceil_sum(s.n - s.q, sp.tpt, whole);
  if (whole < m) c += chunk_tiles(sp, s, whole);
  return c;
}

struct ChunkRange {
  long long per, lo, hi;  // this CTA's range [lo, hi) of the line
  int b, g, rt;           // the item at lo (valid if lo < hi)
  int off;                // lo's offset in it
  ChunkSeq s;
  int clamped;
};

// Range c of P of a line of length total.
PLX_HD void chunk_bounds(ChunkRange& r, long long total, int c, int P) {
  // at least one tile past the fixed part, so that no range is all overhead (with
  // three, fewer records but longer ranges: three short sequences 18.3 -> 19.1 us)
  const long long per = div_pos(total + P - 1, P);
  r.per = per > kChunkItemCost ? per : kChunkItemCost + 1;
  r.lo = c * r.per < total ? c * r.per : total;
  r.hi = r.lo + r.per < total ? r.lo + r.per : total;
}

// What the merge kernel does for one CTA: the item that ends in its range after
// tiles in earlier ones. Written by the attention kernel, so that the merge
// need not find the item again.
struct alignas(16) ChunkMerge {
  int token, ntok;      // first packed row and tokens of the row tile; ntok 0: nothing
  int g;                // kv head
  int c0, c0_first;     // the range of its first tile, and whether that is a first piece
  int pad[3];
};

PLX_HD ChunkMerge chunk_merge_note(const ChunkSpace& sp, const ChunkRange& r) {
  ChunkMerge mg{};
  const int len = r.lo < r.hi ? chunk_tiles(sp, r.s, r.rt) + kChunkItemCost : 0;
  // some of the item's tiles come before this range, and its last one in it
  if (len > 0 && r.off > kChunkItemCost && len - r.off <= r.hi - r.lo) {
    const long long start = r.lo - r.off;
    mg.token = r.s.s0 + r.rt * sp.tpt;
    mg.ntok = chunk_min(sp.tpt, r.s.q - r.rt * sp.tpt);
    mg.g = r.g;
    mg.c0 = (int)div_pos(start + kChunkItemCost, r.per);
    mg.c0_first = (long long)mg.c0 * r.per >= start;
  }
  return mg;
}

// Warp-cooperative, no barrier: each lane sums a contiguous chunk of the
// sequences, a scan gives the prefix, the lane whose chunk holds lo finds the
// sequence, and the lanes together its row tile.
__device__ inline ChunkRange chunk_locate(const ChunkSpace& sp, int c, int P) {
  const int lane = threadIdx.x & 31;
  const int chunk = (sp.B + 31) / 32;
  const int b0 = min(sp.B, lane * chunk), b1 = min(sp.B, b0 + chunk);
  long long local = 0;
  int clamped = 0;
  for (int b = b0; b < b1; ++b) {
    const ChunkSeq s = chunk_seq(sp, b);
    clamped |= chunk_seq_clamped(sp, b);
    local += chunk_cost(sp, s, chunk_row_tiles(sp, s)) * sp.Hkv;
  }
  long long incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  ChunkRange r{};
  r.clamped = __any_sync(0xffffffffu, clamped);
  const long long total = __shfl_sync(0xffffffffu, incl, 31);
  chunk_bounds(r, total, c, P);
  long long pos = incl - local;
  int fb = -1;
  if (r.lo < r.hi && r.lo >= pos && r.lo < incl) {
    fb = b0;
    if (b1 - b0 > 1) {
      for (; fb < b1; ++fb) {
        const ChunkSeq s = chunk_seq(sp, fb);
        const long long w = chunk_cost(sp, s, chunk_row_tiles(sp, s)) * sp.Hkv;
        if (r.lo < pos + w) break;
        pos += w;
      }
    }
  }
  const unsigned owner = __ballot_sync(0xffffffffu, fb >= 0);
  if (owner) {
    const int src = __ffs(owner) - 1;
    r.b = __shfl_sync(0xffffffffu, fb, src);
    r.s = chunk_seq(sp, r.b);
    long long rem = r.lo - __shfl_sync(0xffffffffu, pos, src);
    const long long w = chunk_cost(sp, r.s, chunk_row_tiles(sp, r.s));
    r.g = (int)div_pos(rem, w);
    rem -= w * r.g;
    // the largest rt with chunk_cost(rt) <= rem, in steps of 32 candidates
    int lo = 0, hi = chunk_row_tiles(sp, r.s);
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, i = lo + (lane + 1) * step;
      const bool below = i < hi && chunk_cost(sp, r.s, i) <= rem;
      const int k = __ffs(~__ballot_sync(0xffffffffu, below) | 0x80000000u) - 1;
      lo += k * step;
      hi = min(hi, lo + step);
    }
    r.rt = lo;
    r.off = (int)(rem - chunk_cost(sp, r.s, lo));
  }
  return r;
}

struct ChunkPiece {
  int b, g, rt;
  int t0, t1;     // its tiles
  bool complete;  // all of the item's tiles
  bool first;     // at the start of the CTA's range
  ChunkSeq s;
};

// Walks the pieces of one range; every role of a CTA walks the same list.
struct ChunkCursor {
  long long pos, lo, hi;
  int b, g, rt, off;
  ChunkSeq s;

  __host__ __device__ explicit ChunkCursor(const ChunkRange& r)
      : pos(r.lo), lo(r.lo), hi(r.hi), b(r.b), g(r.g), rt(r.rt), off(r.off), s(r.s) {}

  __host__ __device__ bool next(const ChunkSpace& sp, ChunkPiece& pc) {
    while (pos < hi) {
      const int nt = chunk_tiles(sp, s, rt), len = nt + kChunkItemCost;
      const int take = hi - pos < len - off ? (int)(hi - pos) : len - off;
      pc.b = b;
      pc.g = g;
      pc.rt = rt;
      pc.s = s;
      pc.t0 = chunk_max(0, off - kChunkItemCost);
      pc.t1 = chunk_max(0, off + take - kChunkItemCost);
      pc.complete = pc.t0 == 0 && pc.t1 == nt;
      pc.first = pos == lo;
      pos += take;
      off += take;
      if (off == len) {
        off = 0;
        if (++rt >= chunk_row_tiles(sp, s)) {
          rt = 0;
          if (++g == sp.Hkv) {
            g = 0;
            do {
              if (pos >= hi || ++b >= sp.B) {
                hi = pos;  // past the last item
                break;
              }
              s = chunk_seq(sp, b);
            } while (s.q == 0);
          }
        }
      }
      if (pc.t1 > pc.t0) return true;
    }
    return false;
  }
};

// A partial record: m, l, b of the 128 rows, then A and C as [D / 4][128 rows]
// float4, so that a warp's rows are contiguous when written and when merged.
__host__ __device__ constexpr int chunk_rec_floats(int D) { return kChunkRows * (4 + 2 * D); }

}  // namespace plx
