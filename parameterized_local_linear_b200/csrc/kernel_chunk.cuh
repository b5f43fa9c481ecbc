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
// UMMAs with fp32 accumulators in TMEM; e and e s are rounded to 17 significant
// bits and enter as exact bf16 hi + lo pairs (each weight is multiplied by the
// probe scores, which reach tens, so one bf16 term is not enough), and l and b
// are summed from exactly the values the products apply.
//
// What differs from the prefill kernel:
//  - the rows of a tile are the G query heads of one kv head for 128 / G
//    consecutive tokens, so every K and V tile is loaded once for the group;
//  - K and V tiles come from the page pool: a 64-key tile lies in one page, its
//    page id is read 32 tiles at a time by the producer warp;
//  - the work is cut into equal ranges (chunk_partition.cuh), so a long context
//    with few rows spreads over all SMs and ragged batches stay balanced. Each
//    CTA runs its pieces back to back, the next piece's Q, R, K and V loading
//    while the last tile of the one before is worked on; cut items go through
//    partial records and the merge kernel;
//  - slots past a sequence's length may hold anything (NaN too): their scores
//    are masked before use and their V rows zeroed in shared memory before the
//    value products read them.
// Warps 0-7 softmax (two threads per row), 8 producer, 9 UMMA issuer. TMEM
// columns as in the prefill kernel: S [0,64) T [64,128) P [128,256) O_A
// [256,256+D) O_C [256+D,256+2D). Every wait is bounded.
#pragma once

#include "chunk_partition.cuh"
#include "common.cuh"
#include "kernel_prefill.cuh"
#include "ptx.cuh"

namespace plx {

constexpr int kChThreads = 320;

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
  static constexpr int kSmem = kOffBar + 512 + 1024;  // barriers, slots, alignment
  static constexpr uint32_t kColOA = 256, kColOC = 256 + D;
};

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
  const float kNegInf = __int_as_float(0xff800000u);

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  const uint32_t sQ = base + Geo::kOffQ, sR = base + Geo::kOffR;
  const uint32_t sK = base + Geo::kOffK, sV = base + Geo::kOffV;
  const uint32_t bar = base + Geo::kOffBar;
  const uint32_t q_full = bar, q_empty = bar + 8, k_full = bar + 16, k_empty = k_full + 8 * kSt,
                 v_full = k_empty + 8 * kSt, v_empty = v_full + 8 * kSt;
  const uint32_t s_full = v_empty + 8 * kSt, s_free = s_full + 8, p_full = s_full + 16,
                 o_done = s_full + 24, bar_drain = s_full + 32, red_full = s_full + 40;
  constexpr int kOffMisc = Geo::kOffBar + 16 + 4 * 8 * kSt + 48;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gbase + kOffMisc);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(gbase + kOffMisc + 4);
  // per stage: the tile's page id was in the pool
  volatile int* const tile_ok = reinterpret_cast<volatile int*>(gbase + kOffMisc + 8);
  float* const red = reinterpret_cast<float*>(gbase + Geo::kOffRed);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < kSt; ++s) {
      mbar_init(k_full + 8 * s, 1);
      mbar_init(k_empty + 8 * s, kPfSoftmaxWarps);
      mbar_init(v_full + 8 * s, 1);
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

  if (warp == 8) {
    // ------------------------------------------------------------ producer --
    bool ok = true, skipped_k0 = false;
    int np = 0, last = -1;  // pieces started, last tile whose K and V loads both started
    int jt = 0;             // tiles so far, over all pieces
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
        const uint32_t ph = (uint32_t)(jt / kSt) & 1u;
        ok = mbar_wait_bounded(k_empty + 8 * st, ph ^ 1, p.timeout_ns, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          tile_ok[st] = in_pool;
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
        const uint32_t par = (uint32_t)(j / kSt) & 1u;
        if (!(j == 0 && skipped_k0)) mbar_wait_bounded(k_full + 8 * s, par, p.timeout_ns, nullptr);
        mbar_wait_bounded(v_full + 8 * s, par, p.timeout_ns, nullptr);
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------- UMMA issuer --
    if (lane == 0) {
      bool ok = true;
      // O_A += P V, O_C += (P o T) V for tile j, the first of its piece or not
      const auto value_products = [&](int j, bool piece_start) -> bool {
        const int st = j % kSt;
        if (!mbar_wait_bounded(p_full, j & 1, p.timeout_ns, abort_flag) ||
            !mbar_wait_bounded(v_full + 8 * st, (uint32_t)(j / kSt) & 1u, p.timeout_ns, abort_flag))
          return false;
        tc_fence_after_sync();
        const uint32_t sVs = sV + st * Geo::kKVBytes;
#pragma unroll
        for (int pm = 0; pm < (PROBE ? 4 : 2); ++pm) {  // P_hi, P_lo -> O_A; PT_hi, PT_lo -> O_C
          const uint32_t dO = tmem + (pm < 2 ? Geo::kColOA : Geo::kColOC);
#pragma unroll
          for (int kk = 0; kk < kChunkKeys / 16; ++kk) {
            const bool acc = !(piece_start && (pm & 1) == 0 && kk == 0);
            umma_ts(dO, tmem + kPfColP + 64 * (kk >> 1) + 16 * pm + 8 * (kk & 1),
                    umma_smem_desc(sVs + kk * 16 * 128, kChunkKeys * 128, 1024), kIdescPV, acc);
          }
        }
        umma_commit(o_done);  // also frees the V stage: softmax warp 0 passes it on
        return true;
      };
      int jt = 0, np = 0;
      bool prev_start = false;  // tile jt - 1 was the first of its piece
      while (ok && cur.next(p.sp, pc)) {
        for (int j = pc.t0; j < pc.t1 && ok; ++j, ++jt) {
          const bool start = j == pc.t0;
          if (start) {
            // the last tile of the piece before, ahead of the wait for the new Q and R
            if (jt > 0 && !value_products(jt - 1, prev_start)) ok = false;
            if (ok && !mbar_wait_bounded(q_full, np & 1, p.timeout_ns, abort_flag)) ok = false;
            ++np;
          }
          const int st = jt % kSt;
          if (!ok ||
              (jt > 0 && !mbar_wait_bounded(s_free, (jt - 1) & 1, p.timeout_ns, abort_flag)) ||
              !mbar_wait_bounded(k_full + 8 * st, (uint32_t)(jt / kSt) & 1u, p.timeout_ns,
                                 abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t sKs = sK + st * Geo::kKVBytes;
#pragma unroll
          for (int x = 0; x < (PROBE ? 2 : 1); ++x) {  // S = Q K^T, T = R K^T
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t ko = (kk >> 2) * (kChunkKeys * 128) + (kk & 3) * 32;
              const uint32_t qo = (kk >> 2) * (kChunkRows * 128) + (kk & 3) * 32;
              umma_bf16(tmem + (x == 0 ? kPfColS : kPfColT),
                        umma_smem_desc((x == 0 ? sQ : sR) + qo, 16, 1024),
                        umma_smem_desc(sKs + ko, 16, 1024), kIdescS, kk > 0);
            }
          }
          umma_commit(s_full);  // also frees the K stage: softmax warp 0 passes it on
          if (!start && !value_products(jt - 1, prev_start)) ok = false;
          prev_start = start;
        }
      }
      if (ok && jt > 0 && !value_products(jt - 1, prev_start)) ok = false;
      if (!ok) {
        *abort_flag = 1;
        atomicOr(p.status, 1u);
      }
      umma_commit(bar_drain);  // every UMMA issued above is done once this arrives
      mbar_wait_bounded(bar_drain, 0, p.timeout_ns, nullptr);
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
      for (int j = pc.t0; j < pc.t1; ++j, ++jt) {
        const int st = jt % kSt;
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(s_full, jt & 1, p.timeout_ns, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        float sv[32], so[32], tv[32];
        tmem_ld32(tS + 32 * half, sv);
        tmem_ld32(tS + 32 * (half ^ 1), so);
        if constexpr (PROBE) tmem_ld32(tT + 32 * half, tv);
        tmem_wait_ld();
        tc_fence_before_sync();
        // this tile's K load completed before its UMMAs; the wait makes the
        // producer's tile_ok write visible here
        const bool full_ok = mbar_wait_bounded(k_full + 8 * st, (uint32_t)(jt / kSt) & 1u,
                                               p.timeout_ns, abort_flag);
        const bool in_pool = full_ok && tile_ok[st] != 0;
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(s_free);
          mbar_arrive(k_empty + 8 * st);  // K is read, and so is this warp's tile_ok
          if (warp == 0 && j == pc.t1 - 1) mbar_arrive(q_empty);  // the last read of Q and R
        }
        // mask, and the row max over all 64 keys
        const int k0 = j * kChunkKeys, kown = k0 + 32 * half, kother = k0 + 32 * (half ^ 1);
        float mx = kNegInf;
        if (in_pool && k0 + kChunkKeys <= kall) {
#pragma unroll
          for (int x = 0; x < 32; ++x) mx = fmaxf(mx, fmaxf(sv[x], so[x]));
        } else {
          const int lim = in_pool ? klim : 0;
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            const bool own = kown + x < lim;
            sv[x] = own ? sv[x] : kNegInf;
            if constexpr (PROBE) tv[x] = own ? tv[x] : 0.f;
            mx = fmaxf(mx, fmaxf(sv[x], kother + x < lim ? so[x] : kNegInf));
          }
        }
        mx *= c;  // the scale is positive: this is the max of the scaled scores
        // lazy rescale: keep the stale max unless this tile exceeds it by 2^8
        float alpha = 1.f;
        const bool grow = mx > m_used + 8.f;
        if (grow) {
          alpha = m_used == kNegInf ? 0.f : ex2_approx(m_used - mx);
          m_used = mx;
        }
        const float neg_m = m_used == kNegInf ? 0.f : -m_used;  // no key yet: every e is 0
        // the weights of this thread's 32 keys, before the wait for the
        // products of the tile before, so that they overlap them
        uint32_t pp[32], pt[PROBE ? 32 : 1];
        float lt = 0.f, bt = 0.f;
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          const float e0 = ex2_approx(fmaf(sv[2 * u], c, neg_m));
          const float e1 = ex2_approx(fmaf(sv[2 * u + 1], c, neg_m));
          lt += split_hi_lo(e0, e1, pp[u], pp[16 + u]);
          if constexpr (PROBE)  // e*s from the rounded e: the weights P applies
            bt += split_hi_lo(round17(e0) * tv[2 * u], round17(e1) * tv[2 * u + 1], pt[u],
                              pt[16 + u]);
        }
        if (j > pc.t0) {
          // P is single-buffered and O may need a rescale: the value products
          // of the tile before must be done
          if (!__all_sync(0xffffffffu,
                          mbar_wait_bounded(o_done, (jt - 1) & 1, p.timeout_ns, abort_flag))) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          if (warp == 0 && lane == 0) mbar_arrive(v_empty + 8 * ((jt - 1) % kSt));
          if (__any_sync(0xffffffffu, grow)) {  // warp-uniform: alpha is 1 on the other rows
            if (PROBE || half == 0) {
              const uint32_t tO = tmem + lane_base + (half ? Geo::kColOC : Geo::kColOA);
#pragma unroll 1
              for (int c0 = 0; c0 < D; c0 += 32) {
                float o[32];
                tmem_ld32(tO + c0, o);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 32; ++x) o[x] *= alpha;
                tmem_st32(tO + c0, o);
              }
            }
          }
        }
        tmem_st32u(tP, pp);
        if constexpr (PROBE) tmem_st32u(tP + 32, pt);
        if (k0 + kChunkKeys > pc.s.n) {
          // slots past the length may hold NaN: zero their V rows, which weight
          // 0 does not remove. Rows are 128 bytes in each 64-dimension half.
          ok = __all_sync(0xffffffffu,
                          mbar_wait_bounded(v_full + 8 * st, (uint32_t)(jt / kSt) & 1u,
                                            p.timeout_ns, abort_flag));
          if (!ok) break;
          const int from = max(0, pc.s.n - k0);
          for (int x = from * 8 + tid; x < kChunkKeys * 8; x += kPfSoftmaxWarps * 32)
#pragma unroll
            for (int h = 0; h < Geo::kH; ++h)
              st_shared_v4(sV + st * Geo::kKVBytes + h * (kChunkKeys * 128) + x * 16, 0, 0, 0, 0);
          fence_proxy_async_smem();  // the UMMAs read these rows through the async proxy
        }
        l = l * alpha + lt;
        if constexpr (PROBE) bsum = bsum * alpha + bt;
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
      const float bfull = PROBE ? rd[2 * kChunkRows + r] + rd[3 * kChunkRows + r] : 0.f;
      tc_fence_after_sync();
      if (warp == 0 && lane == 0) mbar_arrive(v_empty + 8 * ((jt - 1) % kSt));
      const float inv = lsum > 0.f ? 1.f / lsum : 0.f, bl = bfull * inv;
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
                o2[z] = PROBE ? vbar + (cc[x + y + z] * inv - bl * vbar) : vbar;
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
                  make_float4(cc[x], cc[x + 1], cc[x + 2], cc[x + 3]);
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
