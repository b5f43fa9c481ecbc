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
//  - e s 2^sigma: sigma is a power of two per row, set by the row's largest |s|
//    so far (|s| 2^sigma below 2^11) and lowered with O_C and b when it grows,
//    as O_A and l are when the maximum does.
//  - V: a block of 16 keys whose largest |v| is 0 or in [2^-8, 2^16) becomes
//    fp16: exact down to 2^-17, within 2^-25 below. Any other block (far
//    values, tiny ones, infinities) stays bf16, and its keys' weights are
//    rounded to 17 bits and enter as exact bf16 hi + lo pairs. A UMMA takes 16
//    keys, so each takes the form of its block.
//
// Slots past a sequence's length may hold anything (NaN too): their scores are
// masked before use, and the converting warps zero their V rows, which weight 0
// would not remove.
//
// Warps 0-7 softmax (two threads per row), 8 producer, 9 UMMA issuer, 10-11 V.
// TMEM columns as in the prefill kernel: S [0,64) T [64,128) P [128,256) O_A
// [256,256+D) O_C [256+D,256+2D). Every wait is bounded.
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

struct ChunkParams {
  ChunkSpace sp;
  __nv_bfloat16* out;      // [total][Hq][D]
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
  static constexpr int kOffRed = kOffV + kStages * kKVBytes;  // l, b of both key halves
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
  const uint32_t q_full = bar, q_empty = bar + 8, k_full = bar + 16, k_empty = k_full + 8 * kSt,
                 v_full = k_empty + 8 * kSt, v_ready = v_full + 8 * kSt,
                 v_empty = v_ready + 8 * kSt;
  const uint32_t s_full = v_empty + 8 * kSt, s_free = s_full + 8, p_full = s_full + 16,
                 o_done = s_full + 24, bar_drain = s_full + 32, red_full = s_full + 40;
  constexpr int kOffMisc = Geo::kOffBar + 16 + 5 * 8 * kSt + 48;
  // per stage, one word per 16 keys, written by the warp that converted them:
  // bit 0 the block is fp16, bit 1 the tile's page is in the pool
  int4* const v_info = reinterpret_cast<int4*>(gbase + kOffMisc);
  volatile int* const tile_ok = reinterpret_cast<volatile int*>(gbase + kOffMisc + 16 * kSt);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gbase + kOffMisc + 20 * kSt);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(gbase + kOffMisc + 20 * kSt + 4);
  float* const red = reinterpret_cast<float*>(gbase + Geo::kOffRed);
  static_assert(kOffMisc % 16 == 0 && 16 + 5 * 8 * kSt + 48 + 20 * kSt + 8 <= 512, "misc area");

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be warp-uniform
  if (tid == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < kSt; ++s) {
      mbar_init(k_full + 8 * s, 1);
      mbar_init(k_empty + 8 * s, 1);
      mbar_init(v_full + 8 * s, 1);
      mbar_init(v_ready + 8 * s, kChConvertWarps);
      mbar_init(v_empty + 8 * s, 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_free, kPfSoftmaxWarps);
    mbar_init(p_full, kPfSoftmaxWarps);
    mbar_init(o_done, 1);
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

  const ChunkRange range = chunk_locate(p.sp, (int)blockIdx.x, (int)gridDim.x);
  if (blockIdx.x == 0 && tid == 0 && range.clamped)
    atomicOr(p.status, 2u /* PARALLAX_DEVICE_STATUS_SEQLEN_CLAMPED */);
  ChunkCursor cur(range);
  ChunkPiece pc;
  // Every role walks the same pieces and counts tiles over all of them: tile
  // jt uses ring stage jt % kSt in its (jt / kSt)-th round.
  const auto round_parity = [](int jt) { return (uint32_t)(jt / kSt) & 1u; };

  if (warp == 8) {
    // ------------------------------------------------------------ producer --
    bool ok = true, skipped_k0 = false;
    int np = 0, last = -1;  // pieces started, last tile whose K and V loads both started
    int jt = 0;
    while (ok && cur.next(p.sp, pc)) {
      if (np > 0) ok = mbar_wait_bounded(q_empty, (np - 1) & 1, p.timeout_ns, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        const int tok = pc.s.s0 + pc.rt * p.sp.tpt;
        const uint32_t rows = (uint32_t)(p.sp.tpt * p.G);
        mbar_arrive_expect_tx(q_full, (PROBE ? 2 : 1) * Geo::kH * rows * 128u);
        for (int h = 0; h < Geo::kH; ++h) {
          tma_load_5d_plain(sQ + h * kChunkRows * 128, &tmQ, 0, 0, tok, h, pc.g, q_full);
          if (PROBE) tma_load_5d_plain(sR + h * kChunkRows * 128, &tmR, 0, 0, tok, h, pc.g, q_full);
        }
      }
      ++np;
      const int32_t* const row = p.table + (size_t)pc.b * p.max_pages;
      int ids = 0;
      for (int j = pc.t0; j < pc.t1; ++j, ++jt) {
        const int k0 = j * kChunkKeys, w = (j - pc.t0) & 31;
        if (w == 0) {  // the page ids of the next 32 tiles, one per lane
          const int kl = (j + lane) * kChunkKeys;
          ids = kl < pc.s.n ? __ldg(row + kl / p.page_size) : -1;
          // a page id outside the pool: its keys are left out
          if (j + lane < pc.t1 && kl < pc.s.n && (ids < 0 || ids >= p.num_pages))
            atomicOr(p.status, 2u);
        }
        int page = __shfl_sync(0xffffffffu, ids, w);
        const bool in_pool = page >= 0 && page < p.num_pages;
        if (!in_pool) page = p.num_pages;  // out of range for the TMA too: reads zeros
        const int st = jt % kSt;
        const uint32_t ph = round_parity(jt);
        ok = mbar_wait_bounded(k_empty + 8 * st, ph ^ 1, p.timeout_ns, abort_flag);
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
        ok = mbar_wait_bounded(v_empty + 8 * st, ph ^ 1, p.timeout_ns, abort_flag);
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
      if (np > 0) mbar_wait_bounded(q_full, (np - 1) & 1, p.timeout_ns, nullptr);
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
          (jt == 0 || mbar_wait_bounded(s_free, (jt - 1) & 1, p.timeout_ns, abort_flag)) &&
          mbar_wait_bounded(k_full + 8 * (jt % kSt), round_parity(jt), p.timeout_ns, abort_flag);
      tc_fence_after_sync();
      return __all_sync(0xffffffffu, got) != 0;
    };
    const uint64_t dQ = umma_smem_desc(sQ, 16, 1024), dR = umma_smem_desc(sR, 16, 1024),
                   dK = umma_smem_desc(sK, 16, 1024),
                   dV = umma_smem_desc(sV, kChunkKeys * 128, 1024);  // + bytes / 16
    const auto scores = [&](int jt) {  // S = Q K^T, T = R K^T
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
      umma_commit_lead(s_full, lead);  // also frees the K stage: softmax warp 0 passes it on
    };
    uint32_t fp16 = 0;  // bit kk: keys 16 kk .. +15 of the tile are fp16
    const auto wait_values = [&](int j) {  // P is written (and V was ready for that)
      const bool got = mbar_wait_bounded(p_full, j & 1, p.timeout_ns, abort_flag);
      tc_fence_after_sync();
      const int4 vi = v_info[j % kSt];
      fp16 = (vi.x & 1) | (vi.y & 1) << 1 | (vi.z & 1) << 2 | (vi.w & 1) << 3;
      fp16 = __shfl_sync(0xffffffffu, fp16, 0);
      return __all_sync(0xffffffffu, got) != 0;
    };
    // O_A += P V, O_C += (P o T) V for keys 16 k0 .. 16 k1 - 1 of tile j
    const auto values = [&](int j, int k0, int k1, uint32_t acc0) {
      const uint64_t v = dV + (uint32_t)((j % kSt) * (Geo::kKVBytes / 16));
      if (fp16 == 15u) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (kk < k0 || kk >= k1) continue;
          const uint32_t tp = tmem + kPfColP + 64 * (kk >> 1) + 8 * (kk & 1);
          umma_ts_lead(tmem + Geo::kColOA, tp, v + kk * 128, kIdescPV16, kk > 0 ? 1u : acc0, lead);
          if (PROBE)
            umma_ts_lead(tmem + Geo::kColOC, tp + 32, v + kk * 128, kIdescPV16,
                         kk > 0 ? 1u : acc0, lead);
        }
      } else {
#pragma unroll 1
        for (int kk = k0; kk < k1; ++kk) {
          const uint32_t tp = tmem + kPfColP + 64 * (kk >> 1) + 8 * (kk & 1);
          const uint32_t acc = kk > 0 ? 1u : acc0;
          const bool one = (fp16 >> kk & 1u) != 0;
          const uint32_t id = one ? kIdescPV16 : kIdescPV;
          umma_ts_lead(tmem + Geo::kColOA, tp, v + kk * 128, id, acc, lead);
          if (PROBE) umma_ts_lead(tmem + Geo::kColOC, tp + 32, v + kk * 128, id, acc, lead);
          if (!one) {
            umma_ts_lead(tmem + Geo::kColOA, tp + 16, v + kk * 128, id, 1u, lead);
            if (PROBE) umma_ts_lead(tmem + Geo::kColOC, tp + 48, v + kk * 128, id, 1u, lead);
          }
        }
      }
    };
    // Per tile: its scores, then the value products of the tile before. The
    // waits for the next tile's scores fall between those products, so that
    // the tensor pipe has work queued while they are checked.
    int jt = 0, np = 0;
    uint32_t acc0 = 0;  // 0: tile jt - 1 was the first of its piece and clears O
    while (ok && cur.next(p.sp, pc)) {
      bool waited = false;
      for (int j = pc.t0; j < pc.t1; ++j, ++jt) {
        const bool start = j == pc.t0;
        if (start) {
          if (jt > 0) {
            // the last tile of the piece before, ahead of the wait for the new Q and R
            if (!(ok = wait_values(jt - 1))) break;
            values(jt - 1, 0, 4, acc0);
            umma_commit_lead(o_done, lead);
          }
          const bool got = mbar_wait_bounded(q_full, np++ & 1, p.timeout_ns, abort_flag);
          if (!(ok = __all_sync(0xffffffffu, got) != 0)) break;
        }
        if (!waited && !(ok = wait_scores(jt))) break;
        scores(jt);
        waited = false;
        if (!start) {
          if (!(ok = wait_values(jt - 1))) break;
          values(jt - 1, 0, 3, acc0);
          if (j + 1 < pc.t1 && !(ok = waited = wait_scores(jt + 1))) break;
          values(jt - 1, 3, 4, acc0);
          umma_commit_lead(o_done, lead);  // also frees the V stage: softmax warp 0 passes it on
        }
        acc0 = start ? 0u : 1u;
      }
    }
    if (ok && jt > 0 && (ok = wait_values(jt - 1))) {
      values(jt - 1, 0, 4, acc0);
      umma_commit_lead(o_done, lead);
    }
    if (!ok && lead) {
      *abort_flag = 1;
      atomicOr(p.status, 1u);
    }
    umma_commit_lead(bar_drain, lead);  // every UMMA issued above is done once this arrives
    mbar_wait_bounded(bar_drain, 0, p.timeout_ns, nullptr);
  } else if (warp >= 10) {
    // ------------------------------- V: bf16 to fp16, rows past the end to 0 --
    constexpr int kWords = Geo::kH * 16 * 8 / 32;  // 16-byte words per lane
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
#pragma unroll 1
        for (int w = warp - 10; w < kChunkKeys / 16; w += kChConvertWarps) {  // keys 16 w .. +15
          const int held = pc.s.n - j * kChunkKeys - 16 * w;  // this block's rows below the length
          uint4* const blk =
              reinterpret_cast<uint4*>(gbase + Geo::kOffV + st * Geo::kKVBytes) + w * 16 * 8 + lane;
          uint4 x[kWords];
          uint32_t mx = 0;
#pragma unroll
          for (int i = 0; i < kWords; ++i) {  // a row is 8 words in each 64-dimension half
            const int half = i / 4, off = (i % 4) * 32;
            x[i] = blk[half * kChunkKeys * 8 + off];
            if ((off + lane) / 8 >= held) x[i] = make_uint4(0, 0, 0, 0);
            const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int y = 0; y < 4; ++y) mx = __vmaxu2(mx, u[y] & 0x7fff7fffu);
          }
          mx = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
          // bf16 bits: 2^16 is 0x4780, 2^-8 is 0x3b80
          const bool f16 = mx == 0 || (mx >= 0x3b80u && mx < 0x4780u);
          if (f16 || held < 16) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
              const int half = i / 4, off = (i % 4) * 32;
              if (f16) {
                x[i].x = pack_f16x2(bf16_lo_to_float(x[i].x), bf16_hi_to_float(x[i].x));
                x[i].y = pack_f16x2(bf16_lo_to_float(x[i].y), bf16_hi_to_float(x[i].y));
                x[i].z = pack_f16x2(bf16_lo_to_float(x[i].z), bf16_hi_to_float(x[i].z));
                x[i].w = pack_f16x2(bf16_lo_to_float(x[i].w), bf16_hi_to_float(x[i].w));
              }
              blk[half * kChunkKeys * 8 + off] = x[i];
            }
            fence_proxy_async_smem();  // the UMMAs read these rows through the async proxy
          }
          if (lane == 0)
            reinterpret_cast<int*>(v_info + st)[w] = (f16 ? 1 : 0) | (tile_ok[st] ? 2 : 0);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(v_ready + 8 * st);
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      atomicOr(p.status, 1u);
    }
  } else {
    // ------------------------------------- softmax: two threads per row --
    const int quarter = warp & 3, half = warp >> 2;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_base + kPfColS, tT = tmem + lane_base + kPfColT;
    const uint32_t tP = tmem + lane_base + kPfColP + 64 * half;  // this half's 64 columns
    const float c = p.scale_log2;
    const int r_tok = r / p.G, r_head = r - r_tok * p.G;
    bool ok = true;
    int jt = 0, np = 0;
    while (ok && cur.next(p.sp, pc)) {
      const int j0 = pc.rt * p.sp.tpt;
      const int ntok = min(p.sp.tpt, pc.s.q - j0);  // tokens of this row tile
      const bool live = r_tok < ntok;
      // keys below klim are seen by this row, keys below kall by every row
      const int seen0 = p.sp.causal ? pc.s.n - pc.s.q + j0 + 1 : pc.s.n;  // the first token's
      const int klim = live ? (p.sp.causal ? min(pc.s.n, seen0 + r_tok) : pc.s.n) : 0;
      const int kall = min(pc.s.n, seen0);
      float m_used = kNegInf, l = 0.f, bsum = 0.f;
      // 2^sigma and 2^-sigma; the first tile that is worked on sets them
      float s_scale = 0.f, s_unscale = 0.f;
      for (int j = pc.t0; j < pc.t1; ++j, ++jt) {
        const int st = jt % kSt;
        ok = mbar_wait_bounded(s_full, jt & 1, p.timeout_ns, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        // S_j, T_j complete: the score UMMAs have read K_j (and Q, R at a piece's end)
        if (warp == 0 && lane == 0) {
          mbar_arrive(k_empty + 8 * st);
          if (j == pc.t1 - 1) mbar_arrive(q_empty);
        }
        // The other half's scores are only needed for the row's largest t and |s|
        float sv[32], tv[32];
        tmem_ld32(tS + 32 * (half ^ 1), sv);
        if constexpr (PROBE) tmem_ld32(tT + 32 * (half ^ 1), tv);
        ok = mbar_wait_bounded(v_ready + 8 * st, round_parity(jt), p.timeout_ns, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          tmem_wait_ld();
          break;
        }
        const int4 vi = v_info[st];
        const bool in_pool = (vi.x & 2) != 0;
        const bool f16 = (vi.x & vi.y & vi.z & vi.w & 1) != 0;
        const int k0 = j * kChunkKeys;
        const bool whole = in_pool && k0 + kChunkKeys <= kall;  // nothing to mask
        const int lim = in_pool ? klim : 0;
        float mx = kNegInf, my = kNegInf, sx = 0.f, sy = 0.f;
        const auto reduce = [&](int kfirst, bool keep) {
          if (whole) {
#pragma unroll
            for (int x = 0; x < 32; x += 4) {  // two chains
              mx = max3(mx, sv[x], sv[x + 1]);
              my = max3(my, sv[x + 2], sv[x + 3]);
              if constexpr (PROBE) {
                sx = max3_abs(sx, tv[x], tv[x + 1]);
                sy = max3_abs(sy, tv[x + 2], tv[x + 3]);
              }
            }
          } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              const bool own = kfirst + x < lim;
              const float sm = own ? sv[x] : kNegInf;
              mx = fmaxf(mx, sm);
              if (keep) sv[x] = sm;
              if constexpr (PROBE) {
                const float tm = own ? tv[x] : 0.f;
                sx = fmaxf(sx, fabsf(tm));
                if (keep) tv[x] = tm;
              }
            }
          }
        };
        tmem_wait_ld();
        reduce(k0 + 32 * (half ^ 1), false);
        tmem_ld32(tS + 32 * half, sv);
        if constexpr (PROBE) tmem_ld32(tT + 32 * half, tv);
        tmem_wait_ld();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free);
        reduce(k0 + 32 * half, true);
        sx = fmaxf(sx, sy);
        mx = fmaxf(mx, my) * c;  // the scale is positive: this is the max of the scaled scores
        // lazy rescale: keep the stale max unless this tile exceeds it by 2^4,
        // and 2^sigma unless |s| 2^sigma reaches 2^11
        float alpha = 1.f, alpha_s = 1.f;
        const bool grow_m = mx > m_used + 4.f;
        const bool grow_s = PROBE && !(sx * s_scale < 2048.f && s_scale > 0.f);
        if (grow_m) {
          alpha = m_used == kNegInf ? 0.f : ex2_approx(m_used - mx);
          m_used = mx;
        }
        if (grow_s) {
          // sx 2^sigma in [2^8, 2^9): room to grow before the next change
          const int ex = max((int)((__float_as_uint(sx) >> 23) & 0xffu) - 127, -100);
          const float ns = __int_as_float((135 - ex) << 23);
          alpha_s = ns * s_unscale;
          s_scale = ns;
          s_unscale = __int_as_float((119 + ex) << 23);
        }
        const bool grow = grow_m || grow_s;
        const float alpha_c = alpha * alpha_s;
        const float neg_m = (m_used == kNegInf ? 0.f : -m_used) + 11.f;  // no key yet: e = 0
        const f32x2 c2 = f2_pack(c, c), nm2 = f2_pack(neg_m, neg_m);
        const float ss = s_scale * (1.f / 2048.f);  // of e 2^11
        const f32x2 ss2 = f2_pack(ss, ss);
        f32x2 lt = 0, bt = 0;  // (+0, +0)
        // P is single-buffered and O may need a rescale: the value products of
        // the tile before must be done
        const auto prev_done_and_rescale = [&]() -> bool {
          if (j == pc.t0) return true;
          const bool got = mbar_wait_bounded(o_done, (jt - 1) & 1, p.timeout_ns, abort_flag);
          if (!__all_sync(0xffffffffu, got)) return false;
          tc_fence_after_sync();
          if (warp == 0 && lane == 0) mbar_arrive(v_empty + 8 * ((jt - 1) % kSt));
          if (__any_sync(0xffffffffu, grow) && (PROBE || half == 0)) {  // warp-uniform
            const uint32_t tO = tmem + lane_base + (half ? Geo::kColOC : Geo::kColOA);
            const float f = half ? alpha_c : alpha;  // 1 on the rows that keep theirs
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              float o[32];
              tmem_ld32(tO + c0, o);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] *= f;
              tmem_st32(tO + c0, o);
            }
          }
          return true;
        };
        if (f16) {
          uint32_t ph[16], th[PROBE ? 16 : 1];
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            float e0, e1;
            ch_exp2(f2_pack(sv[2 * u], sv[2 * u + 1]), c2, nm2, e0, e1);
            ph[u] = pack_f16x2(e0, e1);
            const f32x2 a = f2_pack(f16_lo_to_float(ph[u]), f16_hi_to_float(ph[u]));
            lt = f2_add(lt, a);
            if constexpr (PROBE) {  // e s from the rounded e: the weights P applies
              float x0, x1;
              f2_unpack(f2_mul(f2_mul(a, ss2), f2_pack(tv[2 * u], tv[2 * u + 1])), x0, x1);
              th[u] = pack_f16x2(x0, x1);
              bt = f2_add(bt, f2_pack(f16_lo_to_float(th[u]), f16_hi_to_float(th[u])));
            }
          }
          if (!prev_done_and_rescale()) {
            ok = false;
            break;
          }
          tmem_st16u(tP, ph);
          if constexpr (PROBE) tmem_st16u(tP + 32, th);
        } else {
          if (!prev_done_and_rescale()) {
            ok = false;
            break;
          }
#pragma unroll
          for (int g = 0; g < 2; ++g) {  // 16 keys: fp16, or bf16 hi + lo
            const bool g16 = ((half ? (g ? vi.w : vi.z) : (g ? vi.y : vi.x)) & 1) != 0;
            uint32_t hi[8], lo[8], thi[8], tlo[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              float e0, e1, t0 = 0.f, t1 = 0.f;
              const int x = 16 * g + 2 * u;
              ch_exp2(f2_pack(sv[x], sv[x + 1]), c2, nm2, e0, e1);
              if constexpr (PROBE) {
                t0 = tv[x] * ss;
                t1 = tv[x + 1] * ss;
              }
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
                split_hi_lo(e0, e1, hi[u], lo[u]);
                t0 = round17(e0 * t0);
                t1 = round17(e1 * t1);
                split_hi_lo(t0, t1, thi[u], tlo[u]);
              }
              lt = f2_add(lt, f2_pack(e0, e1));
              bt = f2_add(bt, f2_pack(t0, t1));
            }
            tmem_st8u(tP + 8 * g, hi);
            tmem_st8u(tP + 16 + 8 * g, lo);
            if constexpr (PROBE) {
              tmem_st8u(tP + 32 + 8 * g, thi);
              tmem_st8u(tP + 48 + 8 * g, tlo);
            }
          }
        }
        float x0, x1;  // the sums of the even and of the odd keys
        f2_unpack(lt, x0, x1);
        l = l * alpha + (x0 + x1);
        if constexpr (PROBE) {
          f2_unpack(bt, x0, x1);
          bsum = bsum * alpha_c + (x0 + x1);
        }
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
      }
      if (!ok) break;
      // l and b of the two key halves meet in shared memory (two buffers: a
      // warp that writes the next piece's may run ahead of this one's readers)
      float* const rd = red + (np & 1) * 4 * kChunkRows;
      rd[half * kChunkRows + r] = l;
      if constexpr (PROBE) rd[(2 + half) * kChunkRows + r] = bsum;
      __syncwarp();
      if (lane == 0) mbar_arrive(red_full);
      ok = mbar_wait_bounded(red_full, np & 1, p.timeout_ns, abort_flag) &&
           mbar_wait_bounded(o_done, (jt - 1) & 1, p.timeout_ns, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      ++np;
      const float lsum = rd[r] + rd[kChunkRows + r];
      const float bfull =
          PROBE ? (rd[2 * kChunkRows + r] + rd[3 * kChunkRows + r]) * s_unscale * 2048.f : 0.f;
      tc_fence_after_sync();
      if (warp == 0 && lane == 0) mbar_arrive(v_empty + 8 * ((jt - 1) % kSt));
      // l and A carry 2^11; C and b, which carry 2^sigma, are brought to it
      const float inv = lsum > 0.f ? 1.f / lsum : 0.f, bl = bfull * inv;
      const float cs = s_unscale * 2048.f;
      const size_t orow =
          ((size_t)(pc.s.s0 + j0 + r_tok) * p.Hq + (size_t)pc.g * p.G + r_head) * D;
      float* const rec =
          p.records + (size_t)piece_slot((int)blockIdx.x, pc.first) * chunk_rec_floats(D);
      if (!pc.complete && live && half == 0) {
        rec[r] = m_used;
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
                const float vbar = a[x + y + z] * inv;
                o2[z] = PROBE ? vbar + (cc[x + y + z] * cs * inv - bl * vbar) : vbar;
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
            ra[col * kChunkRows + r] = make_float4(a[x], a[x + 1], a[x + 2], a[x + 3]);
            if constexpr (PROBE)
              ra[(D / 4 + col) * kChunkRows + r] =
                  make_float4(cc[x] * cs, cc[x + 1] * cs, cc[x + 2] * cs, cc[x + 3] * cs);
          }
        }
        __syncwarp();
      }
      tc_fence_before_sync();  // O is read: the next piece's products follow p_full
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

// Combines the partial records of every cut item: block (c, y) owns the item
// that ends in range c after tiles in an earlier one, and merges slice y of
// its columns (kChunkMergeCols float4 columns of A and of C), one row per
// thread, the records in order:
//   M = max_j m_j, w_j = 2^(m_j - M), sums of w_j (l_j, b_j, A_j, C_j).
constexpr int kChunkMergeCols = 2;

template <int D, bool PROBE>
__global__ void __launch_bounds__(kChunkRows) parallax_chunk_merge_kernel(const ChunkParams p) {
  const float kNegInf = __int_as_float(0xff800000u);
  pdl_wait_primary();
  pdl_launch_dependents();
  const int c = (int)blockIdx.x, P = (int)gridDim.x;
  const ChunkRange rg = chunk_locate(p.sp, c, P);
  if (rg.lo >= rg.hi || rg.off <= kChunkItemCost) return;  // no tile of it before this range
  const int len = chunk_tiles(p.sp, rg.s, rg.rt) + kChunkItemCost;
  if (len - rg.off > rg.hi - rg.lo) return;  // it ends in a later range
  const long long start = rg.lo - rg.off;
  // the range that holds the item's first tile
  const int c0 = (int)div_pos(start + kChunkItemCost, rg.per);
  const bool c0_first = (long long)c0 * rg.per >= start;
  const int j0 = rg.rt * p.sp.tpt, ntok = min(p.sp.tpt, rg.s.q - j0);
  const int r = threadIdx.x, r_tok = r / p.G, r_head = r - r_tok * p.G;
  if (r_tok >= ntok) return;
  const auto record = [&](int j) {
    return p.records +
           (size_t)piece_slot(j, j > c0 || c0_first) * chunk_rec_floats(D);
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
      p.out + ((size_t)(rg.s.s0 + j0 + r_tok) * p.Hq + (size_t)rg.g * p.G + r_head) * D;
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
