// Attention of a chunk of new tokens over a paged cache, on the tcgen05 tensor
// cores: a persistent kernel over equal ranges of all sequences' work.
//
// New token j of a sequence with q new tokens and n cached keys (the new ones
// included) sees keys 0 .. n - q + j (causal) or all n; its output is that of
// the decode over them:
//   t_i = scale q.k_i, s_i = r.k_i, e_i = 2^(t_i log2e - m),
//   l = sum e, b = sum e s, A = sum e v, C = sum e s v,
//   o = A/l + C/l - (b/l)(A/l)   (without the probe: o = A/l).
// As in the prefill kernel, S = Q K^T and T = R K^T and the value products are
// UMMAs with fp32 accumulators in TMEM. What differs:
//  - the rows of a tile are the G query heads of one kv head for 128 / G
//    consecutive tokens, so every K and V tile is loaded once for the group;
//  - K and V tiles come from the page pool: a 64-key tile lies in one page, its
//    page id is read 32 tiles at a time by the producer warp;
//  - the work is cut into equal ranges (chunk_partition.cuh), so a long context
//    with few rows spreads over all SMs and ragged batches stay balanced. Each
//    CTA runs its pieces back to back, the next piece's Q, R, K and V loading
//    while the last tile of the one before is worked on; cut items go through
//    partial records and the merge kernel;
//  - V is turned from bf16 into fp16 in shared memory by two warps of its own.
//
// The weights. The value of key i is weighted by e_i (1 + s_i - b/l), so a
// weight's rounding error is multiplied by the probe score, which reaches tens:
// one bf16 term (8 bits) is not enough. e and e s enter as one fp16 term each
// (11 bits), half the value products of a bf16 hi + lo pair, and l and b are
// summed from exactly the rounded values, so the weights stay consistent.
//  - e 2^11: the stale row maximum is kept until it is exceeded by 2^4, so the
//    values reach 2^15 and stay normal fp16 numbers down to e = 2^-25.
//  - e s 2^sigma: 2^sigma is a power of two per row, set by the row's largest |s|
//    so far (to |s| 2^sigma in [2^8, 2^9), growing to below 2^11) and lowered with
//    O_C and b when that grows further, as O_A and l are when the maximum does. It
//    is never raised within a piece: e s is normal in fp16 down to 2^-22 of the
//    largest |s|, and within 2^-33 of it below.
//  - V: a block of 16 keys whose values are all 0 or of magnitude [2^-25, 2^8)
//    becomes fp16, times 2^8, which is exact for every one of them (8 significant
//    bits; fp16's last step is 2^-24). Any other block (far values, tiny ones,
//    infinities) stays bf16, and its keys' weights are rounded to 17 bits and
//    enter, times 2^8 too, as exact bf16 hi + lo pairs. A UMMA takes 16 keys, so
//    each takes the form of its block. (Looking only at a block's largest value
//    takes 119 us instead of 120.5 for 4 drafted tokens, 79 instead of 83.5 for 512
//    rows, 178 instead of 183 for a mixed batch, but loses the bits of a dimension
//    that is small in every key. Of the ways to look at both: one vote over a warp's
//    two blocks; a vote for each costs the drafts 129 us, blocks one after the other
//    144, the exponent's bits moved instead of converted 122.)
//
// What bounds it. A 128 x 64 tile of D = 128 is 8.4 MFLOP of useful work and, at
// the rates measured for these UMMAs one by one (S, T: 50 cycles per 16 dims, fed
// from shared memory; value products: 65 per 16 keys), 1320 cycles of tensor
// pipe. Observed 2000: the issuer's loop (its 24 UMMAs and two waits), a softmax
// warp's chain (TMEM load, mask, maximum, 2^x, conversion, TMEM store, barrier:
// 2600 cycles, two warps per scheduler) and the V conversion (two warps) are each
// near that. More softmax or converting warps leave too few registers (alternate
// tiles to two sets of eight warps: 15% slower). Measured, 16 query on 8 kv heads
// of 128, in a graph at full clock, and in a loop of calls, where the power limit
// holds the clock at 1.5 to 1.8 GHz: 2048 rows over 32768 keys 1080 and 1265 us
// (0.99 and 0.84 PFLOP/s), 512 rows over 8192 keys 83 and 91 us, 4 drafted tokens
// of 32 sequences of 4096 keys 121 (4.4 TB/s) and 144 to 154 us. Softmax form: 900,
// 65 and 115 us in a loop. D = 64: 865 and 71 us.
//
// Slots past a sequence's length may hold anything (NaN too): their scores are
// masked before use, and the converting warps zero their V rows, which weight 0
// would not remove.
//
// Warps 0-7 softmax (16 rows each, four threads for rows ra and ra + 8), 8
// producer, 9 UMMA issuer, 10-11 V. TMEM columns as in the prefill kernel: S
// [0,64) T [64,128) P [128,256), two buffers of fp16 weights (e, then e s, 32
// columns each) or one of hi + lo pairs, O_A [256,256+D) O_C [256+D,256+2D).
// Every wait is bounded.
#pragma once

#include "chunk_partition.cuh"
#include "common.cuh"
#include "kernel_prefill.cuh"
#include "ptx.cuh"

namespace plx {

// Three warps per scheduler, 168 registers a thread (four converting warps
// instead of two left 128, and the softmax spilled)
constexpr int kChThreads = 384;
constexpr int kChConvertWarps = 2;
// fp16 values carry 2^kChValueShift, and so O_A and O_C
constexpr int kChValueShift = 8;
constexpr float kChValueScale = 1 << kChValueShift;

struct ChunkParams {
  ChunkSpace sp;
  __nv_bfloat16* out;      // [total][Hq][D]
  ChunkMerge* merges;      // one per CTA
  float* records;          // 2 * gridDim.x partial records
  unsigned int* status;
  const int32_t* table;    // [B][max_pages]
  int Hq, G, page_size, num_pages, max_pages;
  float scale_log2;        // > 0
  unsigned long long timeout_ns;
  int debug_skip_first_k;  // testing hook: the producer never loads the first K tile
};

template <int D>
struct ChGeom {
  static constexpr int kStages = 4;  // depth of the K ring and of the V ring
  static constexpr int kH = D / 64;
  static constexpr int kQBytes = kH * kChunkRows * 128;   // Q (or R) tile
  static constexpr int kKVBytes = kH * kChunkKeys * 128;  // K (or V) tile
  static constexpr int kOffQ = 0, kOffR = kQBytes, kOffK = 2 * kQBytes;
  static constexpr int kOffV = kOffK + kStages * kKVBytes;
  static constexpr int kOffRed = kOffV + kStages * kKVBytes;  // l, b, 2^-sigma, m of each row
  static constexpr int kOffBar = kOffRed + 2 * 4 * kChunkRows * 4;  // two pieces' worth
  static constexpr int kSmem = kOffBar + 512 + 1024;  // barriers, flags, alignment
  static constexpr uint32_t kColOA = 256, kColOC = 256 + D;
};

// 2^x of two packed values, one fused multiply-add for both arguments.
__device__ __forceinline__ void ch_exp2(f32x2 s, f32x2 c, f32x2 neg_m, float& e0, float& e1) {
  float a, b;
  f2_unpack(f2_fma(s, c, neg_m), a, b);
  e0 = ex2_approx(a);
  e1 = ex2_approx(b);
}

template <int D, bool PROBE>
__global__ void __launch_bounds__(kChThreads, 1)
    parallax_chunk_kernel(const __grid_constant__ CUtensorMap tmQ,
                          const __grid_constant__ CUtensorMap tmR,
                          const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const ChunkParams p) {
  using Geo = ChGeom<D>;
  constexpr int kSt = Geo::kStages;
  constexpr uint32_t kIdescS = umma_idesc_bf16(kChunkRows, kChunkKeys, false);
  constexpr uint32_t kIdescPV = umma_idesc_bf16(kChunkRows, D, true);
  constexpr uint32_t kIdescPV16 = umma_idesc_f16(kChunkRows, D, true);
  const float kNegInf = __int_as_float(0xff800000u);

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  const uint32_t sQ = base + Geo::kOffQ, sR = base + Geo::kOffR;
  const uint32_t sK = base + Geo::kOffK, sV = base + Geo::kOffV;
  const uint32_t bar = base + Geo::kOffBar;
  // One per ring stage: K, V loaded; V converted; S and T written (which frees K);
  // the value products done (which frees V). p_full: one per P buffer, since a
  // warp may finish tile j + 1 before another finishes tile j.
  const uint32_t k_full = bar, v_full = k_full + 8 * kSt, v_ready = v_full + 8 * kSt,
                 s_full = v_ready + 8 * kSt, o_done = s_full + 8 * kSt;
  const uint32_t s_free = o_done + 8 * kSt, p_full = s_free + 8, q_full = s_free + 24,
                 bar_drain = s_free + 32, red_full = s_free + 40;
  constexpr int kOffMisc = Geo::kOffBar + 5 * 8 * kSt + 48;
  // per stage, one word per 16 keys, written by the warp that converted them:
  // bit 0 the block is fp16, bit 1 the tile's page is in the pool
  int4* const v_info = reinterpret_cast<int4*>(gbase + kOffMisc);
  volatile int* const tile_ok = reinterpret_cast<volatile int*>(gbase + kOffMisc + 16 * kSt);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gbase + kOffMisc + 20 * kSt);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(gbase + kOffMisc + 20 * kSt + 4);
  float* const red = reinterpret_cast<float*>(gbase + Geo::kOffRed);
  ChunkRange* const range_slot = reinterpret_cast<ChunkRange*>(gbase + kOffMisc + 20 * kSt + 16);
  static_assert(kOffMisc % 16 == 0 &&
                    5 * 8 * kSt + 48 + 20 * kSt + 16 + sizeof(ChunkRange) <= 512,
                "misc area");

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be warp-uniform
  if (tid == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < kSt; ++s) {
      mbar_init(k_full + 8 * s, 1);
      mbar_init(v_full + 8 * s, 1);
      mbar_init(v_ready + 8 * s, kChConvertWarps);
      mbar_init(s_full + 8 * s, 1);
      mbar_init(o_done + 8 * s, 1);
    }
    mbar_init(s_free, kPfSoftmaxWarps);
    mbar_init(p_full, kPfSoftmaxWarps);
    mbar_init(p_full + 8, kPfSoftmaxWarps);
    mbar_init(bar_drain, 1);
    mbar_init(red_full, kPfSoftmaxWarps);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 9) tmem_alloc(smem_u32(tmem_slot), kPfTmemCols);
  if (tid == 8 * 32) {
    prefetch_tensormap(&tmQ);
    if (PROBE) prefetch_tensormap(&tmR);
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  pdl_wait_primary();  // nothing above reads global memory
  pdl_launch_dependents();

  // one warp finds this CTA's range, the roles take it from shared memory
  if (warp == 8) {
    const ChunkRange range = chunk_locate(p.sp, (int)blockIdx.x, (int)gridDim.x);
    if (lane == 0) {
      *range_slot = range;
      if (blockIdx.x == 0 && range.clamped)
        atomicOr(p.status, 2u /* PARALLAX_DEVICE_STATUS_SEQLEN_CLAMPED */);
      p.merges[blockIdx.x] = chunk_merge_note(p.sp, range);
    }
  }
  __syncthreads();
  const ChunkRange range = *range_slot;
  ChunkCursor cur(range);
  ChunkPiece pc;
  // Every role walks the same pieces and counts tiles over all of them: tile
  // jt uses ring stage jt % kSt in its (jt / kSt)-th round.
  const auto round_parity = [](int jt) { return (uint32_t)(jt / kSt) & 1u; };
  const auto wait_round = [&](uint32_t bars, int jt) {
    return mbar_wait_bounded(bars + 8 * (jt % kSt), round_parity(jt), p.timeout_ns, abort_flag);
  };

  if (warp == 8) {
    // ------------------------------------------------- producer of K and V --
    bool ok = true, skipped_k0 = false;
    int last = -1;  // the last tile whose K and V loads both started
    int jt = 0;
    while (ok && cur.next(p.sp, pc)) {
      const int32_t* const row = p.table + (size_t)pc.b * p.max_pages;
      int ids = 0;
      for (int j = pc.t0; j < pc.t1; ++j, ++jt) {
        const int k0 = j * kChunkKeys, w = (j - pc.t0) & 31;
        if (w == 0) {  // the page ids of the next 32 tiles, one per lane
          // (none past the piece's tiles, whose key index need not fit an int)
          const int kl = j + lane < pc.t1 ? (j + lane) * kChunkKeys : pc.s.n;
          ids = kl < pc.s.n ? __ldg(row + kl / p.page_size) : -1;
          // a page id outside the pool: its keys are left out
          if (kl < pc.s.n && (ids < 0 || ids >= p.num_pages)) atomicOr(p.status, 2u);
        }
        int page = __shfl_sync(0xffffffffu, ids, w);
        const bool in_pool = page >= 0 && page < p.num_pages;
        if (!in_pool) page = p.num_pages;  // out of range for the TMA too: reads zeros
        const int st = jt % kSt;
        const uint32_t ph = round_parity(jt);
        ok = jt < kSt || wait_round(s_full, jt - kSt);  // the stage's last K is read
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          if (jt == 0 && p.debug_skip_first_k) {
            skipped_k0 = true;  // the UMMA issuer's wait on this tile must run out
          } else {
            mbar_arrive_expect_tx(k_full + 8 * st, Geo::kKVBytes);
            tma_load_5d_plain(sK + st * Geo::kKVBytes, &tmK, 0, k0 % p.page_size, 0, pc.g, page,
                              k_full + 8 * st);
          }
        }
        __syncwarp();
        ok = jt < kSt || wait_round(o_done, jt - kSt);
        if (!__all_sync(0xffffffffu, ok)) {
          if (!(jt == 0 && skipped_k0))
            mbar_wait_bounded(k_full + 8 * st, ph, p.timeout_ns, nullptr);  // K in flight
          ok = false;
          break;
        }
        if (lane == 0) {
          tile_ok[st] = in_pool;
          mbar_arrive_expect_tx(v_full + 8 * st, Geo::kKVBytes);
          tma_load_5d_plain(sV + st * Geo::kKVBytes, &tmV, 0, k0 % p.page_size, 0, pc.g, page,
                            v_full + 8 * st);
        }
        last = jt;
      }
    }
    if (lane == 0) {
      if (!ok) {
        *abort_flag = 1;
        atomicOr(p.status, 1u /* PARALLAX_DEVICE_STATUS_TIMEOUT */);
      }
      // Wait (bounded) until every copy this CTA started has landed: the
      // latest load into each buffer is the last one started there.
      for (int j = max(0, last - kSt + 1); j <= last; ++j) {
        const int s = j % kSt;
        if (!(j == 0 && skipped_k0))
          mbar_wait_bounded(k_full + 8 * s, round_parity(j), p.timeout_ns, nullptr);
        mbar_wait_bounded(v_full + 8 * s, round_parity(j), p.timeout_ns, nullptr);
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------- UMMA issuer --
    // The whole warp runs this, one lane issues.
    const uint32_t lead = elect_lane();
    bool ok = true;
    const auto wait_scores = [&](int jt) {  // S, T are free and tile jt's K is here
      const bool got =
          (jt == 0 || mbar_poll_bounded(s_free, (jt - 1) & 1, p.timeout_ns, abort_flag)) &&
          mbar_poll_bounded(k_full + 8 * (jt % kSt), round_parity(jt), p.timeout_ns, abort_flag);
      tc_fence_after_sync();
      return __all_sync(0xffffffffu, got) != 0;
    };
    const uint64_t dQ = umma_smem_desc(sQ, 16, 1024), dR = umma_smem_desc(sR, 16, 1024),
                   dK = umma_smem_desc(sK, 16, 1024),
                   dV = umma_smem_desc(sV, kChunkKeys * 128, 1024);  // + bytes / 16
    // O_A += P V, O_C += (P o T) V for tile jv. fp16: bit kk set where keys
    // 16 kk .. +15 are; acc0 0: the first product clears O
    const auto values = [&](int jv, uint32_t fp16, uint32_t acc0) {
      const uint64_t v = dV + (uint32_t)((jv % kSt) * (Geo::kKVBytes / 16));
      if (fp16 == 15u) {
        const uint32_t tp = tmem + kPfColP + 64 * (jv & 1);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t acc = kk > 0 ? 1u : acc0;
          umma_ts_lead(tmem + Geo::kColOA, tp + 8 * kk, v + kk * 128, kIdescPV16, acc, lead);
          if (PROBE)
            umma_ts_lead(tmem + Geo::kColOC, tp + 32 + 8 * kk, v + kk * 128, kIdescPV16, acc, lead);
        }
      } else {
#pragma unroll 1
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t tp = tmem + kPfColP + 8 * kk, acc = kk > 0 ? 1u : acc0;
          const bool one = (fp16 >> kk & 1u) != 0;
          const uint32_t id = one ? kIdescPV16 : kIdescPV;
          umma_ts_lead(tmem + Geo::kColOA, tp, v + kk * 128, id, acc, lead);
          if (PROBE) umma_ts_lead(tmem + Geo::kColOC, tp + 32, v + kk * 128, id, acc, lead);
          if (!one) {
            umma_ts_lead(tmem + Geo::kColOA, tp + 64, v + kk * 128, id, 1u, lead);
            if (PROBE) umma_ts_lead(tmem + Geo::kColOC, tp + 96, v + kk * 128, id, 1u, lead);
          }
        }
      }
    };
    int np = 0;  // pieces whose Q and R loads started
    const auto load_queries = [&](const ChunkPiece& x) {
      if (lead) {
        const int tok = x.s.s0 + x.rt * p.sp.tpt;
        mbar_arrive_expect_tx(q_full, (PROBE ? 2 : 1) * Geo::kH * (uint32_t)(p.sp.tpt * p.G) * 128u);
        for (int h = 0; h < Geo::kH; ++h) {
          tma_load_5d_plain(sQ + h * kChunkRows * 128, &tmQ, 0, 0, tok, h, x.g, q_full);
          if (PROBE) tma_load_5d_plain(sR + h * kChunkRows * 128, &tmR, 0, 0, tok, h, x.g, q_full);
        }
      }
      __syncwarp();
      ++np;
    };
    // Per tile: its scores, then the value products of the tile before. The next
    // piece's Q and R load as soon as the last scores are done.
    int jt = 0;
    bool more = cur.next(p.sp, pc);
    if (more) load_queries(pc);
    while (ok && more) {
      ChunkPiece nx;
      more = cur.next(p.sp, nx);
      const bool got = mbar_wait_bounded(q_full, (np - 1) & 1, p.timeout_ns, abort_flag);
      if (!(ok = __all_sync(0xffffffffu, got) != 0)) break;
      for (int j = pc.t0; j <= pc.t1; ++j) {
        if (j < pc.t1) {  // S = Q K^T, T = R K^T
          if (!(ok = wait_scores(jt))) break;
          const uint64_t k = dK + (uint32_t)((jt % kSt) * (Geo::kKVBytes / 16));
#pragma unroll
          for (int x = 0; x < (PROBE ? 2 : 1); ++x) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t ko = (kk >> 2) * (kChunkKeys * 128) + (kk & 3) * 32;
              const uint32_t qo = (kk >> 2) * (kChunkRows * 128) + (kk & 3) * 32;
              umma_ss_lead(tmem + (x == 0 ? kPfColS : kPfColT), (x == 0 ? dQ : dR) + qo / 16,
                           k + ko / 16, kIdescS, kk > 0, lead);
            }
          }
          umma_commit_lead(s_full + 8 * (jt % kSt), lead);
          ++jt;
        } else if (more) {
          const bool done = wait_round(s_full, jt - 1);
          if (!(ok = __all_sync(0xffffffffu, done) != 0)) break;
          load_queries(nx);
        }
        if (j > pc.t0) {  // tile jv: P is written (and V was ready for that)
          const int jv = j < pc.t1 ? jt - 2 : jt - 1;
          const bool full = mbar_poll_bounded(p_full + 8 * (jv & 1), (uint32_t)(jv >> 1) & 1u,
                                              p.timeout_ns, abort_flag);
          if (!(ok = __all_sync(0xffffffffu, full) != 0)) break;
          tc_fence_after_sync();
          const int4 vi = v_info[jv % kSt];
          const uint32_t fp16 = __shfl_sync(
              0xffffffffu, (vi.x & 1) | (vi.y & 1) << 1 | (vi.z & 1) << 2 | (vi.w & 1) << 3, 0);
          values(jv, fp16, j > pc.t0 + 1 ? 1u : 0u);
          umma_commit_lead(o_done + 8 * (jv % kSt), lead);
        }
      }
      pc = nx;
    }
    if (!ok && lead) {
      *abort_flag = 1;
      atomicOr(p.status, 1u);
    }
    // the last Q and R loads have landed, and every UMMA issued above is done
    if (np > 0) mbar_wait_bounded(q_full, (np - 1) & 1, p.timeout_ns, nullptr);
    umma_commit_lead(bar_drain, lead);
    mbar_wait_bounded(bar_drain, 0, p.timeout_ns, nullptr);
  } else if (warp >= 10) {
    // ------------------------------- V: bf16 to fp16, rows past the end to 0 --
    constexpr int kWords = Geo::kH * 16 * 8 / 32;  // 16-byte words per lane
    // bf16 bits of 2^8 and 2^-25, and what multiplies a pair of values below 2^8 by 2^8
    // (a 0 becomes 2^-119, which is 0 in fp16)
    constexpr uint32_t kBelow = (127 + 16 - kChValueShift) << 7,
                       kFrom = (127 - 17 - kChValueShift) << 7, kPair = 0x00010001u,
                       kTimes = kPair * (kChValueShift << 7);
    const auto turn = [](uint32_t v) {
      v += kTimes;
      return pack_f16x2(bf16_lo_to_float(v), bf16_hi_to_float(v));
    };
    // Per half: max(far, 2 (|v| - kFrom)) of unsigned 16 bits, so that values below kFrom
    // wrap to far ones. (v + v drops the signs; the low half's goes into the last bit of
    // the high half, where it changes no comparison with an even bound.)
    const auto range_max = [](uint32_t far, uint32_t v) {
      return __viaddmax_u16x2(v + v, kPair * (0x10000u - 2 * kFrom), far);
    };
    bool ok = true;
    int jt = 0;
    while (ok && cur.next(p.sp, pc)) {
      for (int j = pc.t0; j < pc.t1; ++j, ++jt) {
        const int st = jt % kSt;
        ok = mbar_wait_bounded(v_full + 8 * st, round_parity(jt), p.timeout_ns, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        // both of this warp's blocks of 16 keys at once: warp - 10 and the next but one
        constexpr int kBlocks = kChunkKeys / 16 / kChConvertWarps;
        uint4* const tile = reinterpret_cast<uint4*>(gbase + Geo::kOffV + st * Geo::kKVBytes) + lane;
        const int left = pc.s.n - j * kChunkKeys;  // rows of the tile below the length
        // word i of block y: row (i % 4) * 4 + lane / 8 (8 words in each half)
        const auto word = [&](int y, int i) -> uint4& {
          const int w = warp - 10 + kChConvertWarps * y;
          return tile[(i / 4) * kChunkKeys * 8 + w * 16 * 8 + (i % 4) * 32];
        };
        uint4 x[kBlocks][kWords];
#pragma unroll
        for (int y = 0; y < kBlocks; ++y)
#pragma unroll
          for (int i = 0; i < kWords; ++i) x[y][i] = word(y, i);
        if (left < kChunkKeys) {
#pragma unroll
          for (int y = 0; y < kBlocks; ++y)
#pragma unroll
            for (int i = 0; i < kWords; ++i)
              if ((warp - 10 + kChConvertWarps * y) * 16 + (i % 4) * 4 + lane / 8 >= left)
                x[y][i] = make_uint4(0, 0, 0, 0);
        }
        uint32_t far[4] = {0, 0, 0, 0};  // independent chains
#pragma unroll
        for (int y = 0; y < kBlocks; ++y)
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
            far[0] = range_max(far[0], x[y][i].x);
            far[1] = range_max(far[1], x[y][i].y);
            far[2] = range_max(far[2], x[y][i].z);
            far[3] = range_max(far[3], x[y][i].w);
          }
        constexpr uint32_t kMost = kPair * (2 * (kBelow - kFrom) - 1);
        const uint32_t f = __vmaxu2(__vmaxu2(far[0], far[1]), __vmaxu2(far[2], far[3]));
        bool f16[kBlocks];
        if (__all_sync(0xffffffffu, __vmaxu2(f, kMost) == kMost)) {
#pragma unroll
          for (int y = 0; y < kBlocks; ++y) {
            f16[y] = true;
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
              uint4& v = x[y][i];
              v = make_uint4(turn(v.x), turn(v.y), turn(v.z), turn(v.w));
            }
          }
        } else {  // some are zeros or out of fp16's range: block by block
#pragma unroll
          for (int y = 0; y < kBlocks; ++y) {
            uint32_t most = 0;
            const auto take = [&](uint32_t w) {  // (a 0 counts as the smallest in range)
              const uint32_t m = w & 0x7fff7fffu;
              most = __vmaxu2(most, __vsub2(m, kPair * kFrom) & ~__vcmpeq2(m, 0));
            };
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
              take(x[y][i].x);
              take(x[y][i].y);
              take(x[y][i].z);
              take(x[y][i].w);
            }
            f16[y] = __all_sync(0xffffffffu, max(most & 0xffffu, most >> 16) < kBelow - kFrom);
            if (f16[y]) {
#pragma unroll
              for (int i = 0; i < kWords; ++i) {
                uint4& v = x[y][i];
                v = make_uint4(turn(v.x), turn(v.y), turn(v.z), turn(v.w));
              }
            }
          }
        }
#pragma unroll
        for (int y = 0; y < kBlocks; ++y) {
#pragma unroll
          for (int i = 0; i < kWords; ++i) word(y, i) = x[y][i];
          if (lane == 0)
            reinterpret_cast<int*>(v_info + st)[warp - 10 + kChConvertWarps * y] =
                (f16[y] ? 1 : 0) | (tile_ok[st] ? 2 : 0);
        }
        fence_proxy_async_smem();  // the UMMAs read these rows through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(v_ready + 8 * st);
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      atomicOr(p.status, 1u);
    }
  } else {
    // ------------------------------------------------------------ softmax --
    // Warp w has 16 rows of its quarter of the TMEM lanes: four threads share
    // rows ra and ra + 8 (tmem_ld16x64), each with 16 of the 64 keys.
    const int quarter = warp & 3, half = warp >> 2;
    const int ra = quarter * 32 + half * 16 + (lane >> 2), col = 2 * (lane & 3);
    const uint32_t t16 = tmem + ((uint32_t)(quarter * 32 + half * 16) << 16);
    const float c = p.scale_log2;
    const int tok_a = ra / p.G, tok_b = (ra + 8) / p.G;
    // the epilogue's row: one per thread and half of the columns
    const int r = quarter * 32 + lane, r_tok = r / p.G, r_head = r - r_tok * p.G;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    struct Row {
      float m, l, b;                // running max, sums over this thread's keys
      float s_scale, s_unscale;     // 2^sigma, 2^-sigma; the first tile sets them
    };
    bool ok = true;
    int jt = 0, np = 0;
    bool wide = false;     // the tile before filled both P buffers
    bool more = cur.next(p.sp, pc);
    while (ok && more) {
      ChunkPiece nx;
      more = cur.next(p.sp, nx);
      const int j0 = pc.rt * p.sp.tpt;
      const int ntok = min(p.sp.tpt, pc.s.q - j0);  // tokens of this row tile
      // keys below lim are seen by a row, keys below kall by every row
      const int seen0 = p.sp.causal ? pc.s.n - pc.s.q + j0 + 1 : pc.s.n;  // the first token's
      const auto row_limit = [&](int tok) {
        if (tok >= ntok) return 0;
        return p.sp.causal ? min(pc.s.n, seen0 + tok) : pc.s.n;
      };
      const int lim_a = row_limit(tok_a), lim_b = row_limit(tok_b), kall = min(pc.s.n, seen0);
      Row A{kNegInf, 0.f, 0.f, 0.f, 0.f}, B = A;
      // A warp whose rows are all past the tile's tokens only keeps the barriers'
      // pace: the products of its rows are not used, whatever P holds there. With
      // few rows the others then have the schedulers for themselves.
      if ((quarter * 32 + half * 16) / p.G >= ntok) {
        for (int j = pc.t0; j < pc.t1; ++j, ++jt) {
          ok = wait_round(s_full, jt);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            mbar_arrive(s_free);
            mbar_arrive(p_full + 8 * (jt & 1));
          }
        }
      } else {
        for (int j = pc.t0; j < pc.t1; ++j, ++jt) {
          const int st = jt % kSt;
          // the tile's V is ready, and its flags with it, before its scores are
          ok = mbar_wait_bounded(v_ready + 8 * st, round_parity(jt), p.timeout_ns, abort_flag);
          const int4 vi = v_info[st];
          const bool in_pool = (vi.x & 2) != 0;
          const bool f16 = (vi.x & vi.y & vi.z & vi.w & 1) != 0;
          ok = ok && wait_round(s_full, jt);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          float sv[32], tv[32];
          tmem_ld16x64(t16 + kPfColS, sv);
          if constexpr (PROBE) tmem_ld16x64(t16 + kPfColT, tv);
          tmem_wait_ld();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free);
          // mask
          const int k0 = j * kChunkKeys;
          if (!(in_pool && k0 + kChunkKeys <= kall)) {
            const int la = in_pool ? lim_a - k0 - col : 0, lb = in_pool ? lim_b - k0 - col : 0;
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              const bool own = 8 * (x >> 2) + (x & 1) < ((x & 2) ? lb : la);
              sv[x] = own ? sv[x] : kNegInf;
              if constexpr (PROBE) tv[x] = own ? tv[x] : 0.f;
            }
          }
          // Lazy rescale: keep the stale max unless this tile exceeds it by 2^4,
          // and 2^sigma unless |s| 2^sigma reaches 2^11.
          const auto within = [&](const Row& w, float mx, float sx) {
            return mx * c <= w.m + 4.f && (!PROBE || (sx * w.s_scale < 2048.f && w.s_scale > 0.f));
          };
          float alpha[2] = {1.f, 1.f}, alpha_c[2] = {1.f, 1.f};  // factors of l, A and of b, C
          const auto update = [&](float ma, float mb, float sa, float sb) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              Row& w = y ? B : A;
              float mx = (y ? mb : ma) * c, sx = y ? sb : sa;  // (the scale is positive)
#pragma unroll
              for (int o = 1; o < 4; o <<= 1) {
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                sx = fmaxf(sx, __shfl_xor_sync(0xffffffffu, sx, o));
              }
              float alpha_s = 1.f;
              if (mx > w.m + 4.f) {
                alpha[y] = w.m == kNegInf ? 0.f : ex2_approx(w.m - mx);
                w.m = mx;
              }
              if (PROBE && !(sx * w.s_scale < 2048.f && w.s_scale > 0.f)) {
                // sx 2^sigma in [2^8, 2^9): room to grow before the next change
                const int ex = max((int)((__float_as_uint(sx) >> 23) & 0xffu) - 127, -100);
                const float ns = __int_as_float((135 - ex) << 23);
                alpha_s = ns * w.s_unscale;
                w.s_scale = ns;
                w.s_unscale = __int_as_float((119 + ex) << 23);
              }
              alpha_c[y] = alpha[y] * alpha_s;
              w.l *= alpha[y];
              w.b *= alpha_c[y];
            }
          };
          const f32x2 c2 = f2_pack(c, c);
          f32x2 lt[2], bt[2];  // per row: the sums of the even and the odd keys
          f32x2 nm[2], ss[2];
          const auto factors = [&]() {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const Row& w = y ? B : A;
              const float neg_m = (w.m == kNegInf ? 0.f : -w.m) + 11.f;  // no key yet: e = 0
              nm[y] = f2_pack(neg_m, neg_m);
              const float sc = w.s_scale * (1.f / 2048.f);  // of e 2^11
              ss[y] = f2_pack(sc, sc);
              lt[y] = bt[y] = 0;
            }
          };
          // fp16 weights of the 32 values
          uint32_t ph[16], th[PROBE ? 16 : 1];
          const auto weights = [&]() {
#pragma unroll
            for (int u = 0; u < 16; ++u) {  // pair u / 2 of row u % 2
              const int y = u & 1;
              float e0, e1;
              ch_exp2(f2_pack(sv[2 * u], sv[2 * u + 1]), c2, nm[y], e0, e1);
              ph[u] = pack_f16x2(e0, e1);
              const f32x2 a = f2_pack(f16_lo_to_float(ph[u]), f16_hi_to_float(ph[u]));
              lt[y] = f2_add(lt[y], a);
              if constexpr (PROBE) {  // e s from the rounded e: the weights P applies
                float x0, x1;
                f2_unpack(f2_mul(f2_mul(a, ss[y]), f2_pack(tv[2 * u], tv[2 * u + 1])), x0, x1);
                th[u] = pack_f16x2(x0, x1);
                bt[y] = f2_add(bt[y], f2_pack(f16_lo_to_float(th[u]), f16_hi_to_float(th[u])));
              }
            }
          };
          float ma = sv[0], mb = sv[2], sa = 0.f, sb = 0.f;  // the largest t and |s| of both rows
#pragma unroll
          for (int x = 0; x < 32; x += 4) {
            ma = max3(ma, sv[x], sv[x + 1]);
            mb = max3(mb, sv[x + 2], sv[x + 3]);
            if constexpr (PROBE) {
              sa = max3_abs(sa, tv[x], tv[x + 1]);
              sb = max3_abs(sb, tv[x + 2], tv[x + 3]);
            }
          }
          const bool grow =
              __any_sync(0xffffffffu, !(within(A, ma, sa) && within(B, mb, sb)) && in_pool);
          if (grow) update(ma, mb, sa, sb);  // (the row's four threads need a common value)
          factors();
          if (f16) weights();
          // Tiles of fp16 blocks alternate between two P buffers, and this one's is
          // free: the value products of tile jt - 2 were issued before the scores
          // of jt, whose commit (s_full) covers them. A tile with hi + lo weights
          // fills both buffers, and O may need a rescale: for either, the products
          // of the tile before must be done.
          const auto prev_done_and_rescale = [&]() -> bool {
            const bool wait = j > pc.t0 && (grow || wide || !f16);
            wide = !f16;
            if (!wait) return true;
            const bool got = wait_round(o_done, jt - 1);
            if (!__all_sync(0xffffffffu, got)) return false;
            tc_fence_after_sync();
            if (grow) {
#pragma unroll 1
              for (int c0 = 0; c0 < (PROBE ? 2 * D : D); c0 += 64) {
                const float fa = c0 < D ? alpha[0] : alpha_c[0], fb = c0 < D ? alpha[1] : alpha_c[1];
                float o[32];
                tmem_ld16x64(t16 + Geo::kColOA + c0, o);  // O_C follows O_A
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 32; ++x) o[x] *= (x & 2) ? fb : fa;
                tmem_st16x64(t16 + Geo::kColOA + c0, o);
              }
            }
            return true;
          };
          if (f16) {
            if (!prev_done_and_rescale()) {
              ok = false;
              break;
            }
            tmem_st16x32u(t16 + kPfColP + 64 * (jt & 1), ph);
            if constexpr (PROBE) tmem_st16x32u(t16 + kPfColP + 64 * (jt & 1) + 32, th);
          } else {
            if (!prev_done_and_rescale()) {
              ok = false;
              break;
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {  // 16 keys: fp16, or bf16 hi + lo
              const bool g16 = ((g == 0 ? vi.x : g == 1 ? vi.y : g == 2 ? vi.z : vi.w) & 1) != 0;
              uint32_t hi[4], lo[4], thi[4], tlo[4];
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const int y = u & 1, x = 8 * g + 2 * u;
                float e0, e1, t0 = 0.f, t1 = 0.f;
                ch_exp2(f2_pack(sv[x], sv[x + 1]), c2, nm[y], e0, e1);
                if constexpr (PROBE) f2_unpack(f2_mul(ss[y], f2_pack(tv[x], tv[x + 1])), t0, t1);
                lo[u] = tlo[u] = 0;
                if (g16) {
                  hi[u] = pack_f16x2(e0, e1);
                  e0 = f16_lo_to_float(hi[u]);
                  e1 = f16_hi_to_float(hi[u]);
                  thi[u] = pack_f16x2(e0 * t0, e1 * t1);
                  t0 = f16_lo_to_float(thi[u]);
                  t1 = f16_hi_to_float(thi[u]);
                } else {
                  e0 = round17(e0);
                  e1 = round17(e1);
                  split_hi_lo(e0 * kChValueScale, e1 * kChValueScale, hi[u], lo[u]);
                  t0 = round17(e0 * t0);
                  t1 = round17(e1 * t1);
                  split_hi_lo(t0 * kChValueScale, t1 * kChValueScale, thi[u], tlo[u]);
                }
                lt[y] = f2_add(lt[y], f2_pack(e0, e1));
                bt[y] = f2_add(bt[y], f2_pack(t0, t1));
              }
              tmem_st16x8u(t16 + kPfColP + 8 * g, hi);
              tmem_st16x8u(t16 + kPfColP + 64 + 8 * g, lo);
              if constexpr (PROBE) {
                tmem_st16x8u(t16 + kPfColP + 32 + 8 * g, thi);
                tmem_st16x8u(t16 + kPfColP + 96 + 8 * g, tlo);
              }
            }
          }
          tmem_wait_st();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full + 8 * (jt & 1));
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            Row& w = y ? B : A;
            float x0, x1;
            f2_unpack(lt[y], x0, x1);
            w.l += x0 + x1;
            if constexpr (PROBE) {
              f2_unpack(bt[y], x0, x1);
              w.b += x0 + x1;
            }
          }
        }
      }
      if (!ok) break;
      // The rows' sums over their four threads, and what else the epilogue's
      // threads need, through shared memory (two buffers: a warp that writes
      // the next piece's may run ahead of this one's readers)
      float* const rd = red + (np & 1) * 4 * kChunkRows;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        Row& w = y ? B : A;
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          w.l += __shfl_xor_sync(0xffffffffu, w.l, o);
          w.b += __shfl_xor_sync(0xffffffffu, w.b, o);
        }
        if ((lane & 3) == 0) {
          rd[ra + 8 * y] = w.l;
          rd[kChunkRows + ra + 8 * y] = w.b;
          rd[2 * kChunkRows + ra + 8 * y] = w.s_unscale;
          rd[3 * kChunkRows + ra + 8 * y] = w.m;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(red_full);
      ok = mbar_wait_bounded(red_full, np & 1, p.timeout_ns, abort_flag) &&
           wait_round(o_done, jt - 1);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      ++np;
      tc_fence_after_sync();
      const bool live = r_tok < ntok;
      const float lsum = rd[r], cs = rd[2 * kChunkRows + r] * 2048.f;
      // l and A carry 2^11; C and b, which carry 2^sigma, are brought to it. The
      // values' 2^8 leaves A and C here.
      const float bfull = PROBE ? rd[kChunkRows + r] * cs : 0.f;
      constexpr float kUnscale = 1.f / kChValueScale;
      const float c_unscale = cs * kUnscale;
      const float inv = lsum > 0.f ? 1.f / lsum : 0.f, bl = bfull * inv;
      const size_t orow =
          ((size_t)(pc.s.s0 + j0 + r_tok) * p.Hq + (size_t)pc.g * p.G + r_head) * D;
      float* const rec =
          p.records + (size_t)piece_slot((int)blockIdx.x, pc.first) * chunk_rec_floats(D);
      if (!pc.complete && live && half == 0) {
        rec[r] = rd[3 * kChunkRows + r];
        rec[kChunkRows + r] = lsum;
        rec[2 * kChunkRows + r] = bfull;
      }
#pragma unroll 1
      for (int c0 = half * (D / 2); c0 < (half + 1) * (D / 2); c0 += 32) {
        float a[32], cc[32];
        tmem_ld32(tmem + lane_base + Geo::kColOA + c0, a);
        if constexpr (PROBE) tmem_ld32(tmem + lane_base + Geo::kColOC + c0, cc);
        tmem_wait_ld();
        if (live && pc.complete) {
#pragma unroll
          for (int x = 0; x < 32; x += 8) {
            uint32_t w[4];
#pragma unroll
            for (int y = 0; y < 8; y += 2) {
              float o2[2];
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const float vbar = a[x + y + z] * kUnscale * inv;
                o2[z] = PROBE ? vbar + (cc[x + y + z] * c_unscale * inv - bl * vbar) : vbar;
              }
              w[y / 2] = pack_bf16x2(o2[0], o2[1]);
            }
            *reinterpret_cast<uint4*>(p.out + orow + c0 + x) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else if (live) {
          float4* const ra = reinterpret_cast<float4*>(rec + 4 * kChunkRows);
#pragma unroll
          for (int x = 0; x < 32; x += 4) {
            const int col = (c0 + x) / 4;
            ra[col * kChunkRows + r] = make_float4(a[x] * kUnscale, a[x + 1] * kUnscale,
                                                   a[x + 2] * kUnscale, a[x + 3] * kUnscale);
            if constexpr (PROBE)
              ra[(D / 4 + col) * kChunkRows + r] =
                  make_float4(cc[x] * c_unscale, cc[x + 1] * c_unscale, cc[x + 2] * c_unscale,
                              cc[x + 3] * c_unscale);
          }
        }
        __syncwarp();
      }
      tc_fence_before_sync();  // O is read: the next piece's products follow p_full
      pc = nx;
    }
    if (!ok) {
      *abort_flag = 1;
      if (lane == 0) atomicOr(p.status, 1u);
    }
  }
  // teardown: every role is done with TMEM (UMMAs drained, loads waited)
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 9) tmem_dealloc(tmem, kPfTmemCols);
}

// Combines the partial records of every cut item: block (c, y) merges slice y of
// the columns (kChunkMergeCols float4 columns of A and of C) of the item that
// ends in range c, one row per thread, the records in order:
//   M = max_j m_j, w_j = 2^(m_j - M), sums of w_j (l_j, b_j, A_j, C_j).
// Latency: 3 to 4 us behind the attention kernel. 16 (D = 128) slices per item
// rather than one block, so that a few items use many SMs.
constexpr int kChunkMergeCols = 2;

template <int D, bool PROBE>
__global__ void __launch_bounds__(kChunkRows) parallax_chunk_merge_kernel(const ChunkParams p) {
  const float kNegInf = __int_as_float(0xff800000u);
  const int c = (int)blockIdx.x, r = threadIdx.x, r_tok = r / p.G, r_head = r - r_tok * p.G;
  pdl_wait_primary();
  pdl_launch_dependents();
  const int4* const mp = reinterpret_cast<const int4*>(p.merges + c);
  const int4 m0 = __ldcg(mp), m1 = __ldcg(mp + 1);
  const int token = m0.x, ntok = m0.y, g = m0.z, c0 = m0.w;
  const bool c0_first = m1.x != 0;
  if (r_tok >= ntok) return;
  const auto record = [&](int j) {
    return p.records + (size_t)piece_slot(j, j > c0 || c0_first) * chunk_rec_floats(D);
  };
  float M = kNegInf;
  for (int j = c0; j <= c; ++j) M = fmaxf(M, __ldcg(record(j) + r));
  float l = 0.f, b = 0.f;
  float4 A[kChunkMergeCols], C[kChunkMergeCols];
#pragma unroll
  for (int i = 0; i < kChunkMergeCols; ++i) A[i] = C[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int col0 = (int)blockIdx.y * kChunkMergeCols;
#pragma unroll 2
  for (int j = c0; j <= c; ++j) {
    const float* const rec = record(j);
    const float mj = __ldcg(rec + r);
    const float w = mj == kNegInf ? 0.f : ex2_approx(mj - M);
    l += w * __ldcg(rec + kChunkRows + r);
    if (PROBE) b += w * __ldcg(rec + 2 * kChunkRows + r);
    const float4* const ra = reinterpret_cast<const float4*>(rec + 4 * kChunkRows);
#pragma unroll
    for (int i = 0; i < kChunkMergeCols; ++i) {
      const float4 a = ld_cg_f4(ra + (col0 + i) * kChunkRows + r);
      A[i].x += w * a.x, A[i].y += w * a.y, A[i].z += w * a.z, A[i].w += w * a.w;
      if (PROBE) {
        const float4 x = ld_cg_f4(ra + (D / 4 + col0 + i) * kChunkRows + r);
        C[i].x += w * x.x, C[i].y += w * x.y, C[i].z += w * x.z, C[i].w += w * x.w;
      }
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f, bl = b * inv;
  __nv_bfloat16* const out =
      p.out + ((size_t)(token + r_tok) * p.Hq + (size_t)g * p.G + r_head) * D;
  const auto fin = [&](float a, float x) {
    const float vbar = a * inv;
    return PROBE ? vbar + (x * inv - bl * vbar) : vbar;
  };
#pragma unroll
  for (int i = 0; i < kChunkMergeCols; ++i) {
    uint2 w;
    w.x = pack_bf16x2(fin(A[i].x, C[i].x), fin(A[i].y, C[i].y));
    w.y = pack_bf16x2(fin(A[i].z, C[i].z), fin(A[i].w, C[i].w));
    *reinterpret_cast<uint2*>(out + 4 * (col0 + i)) = w;
  }
}

}  // namespace plx
