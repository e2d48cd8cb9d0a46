// dQ of the cross attention's backward, query-major: for query row n with the len_b keys of its
// batch entry
//   P_nm = exp(scale q_n.k_m - LSE_n),  dS_nm = P_nm (dO_n.v_m - D_n),  dQ_n = scale sum_m dS_nm k_m.
//
// Per 128 keys the tensor cores form S = Q K^T and dP = dO V^T again, the elementwise warps dS, and
// dQ += dS K accumulates in TMEM: 1536 clocks of products, 1024 of exponentials (all on the MUFU
// unit: with a quarter of them on the FMA pipe the whole backward took 656 in place of 650 us for the
// pair of lengths below, and a score of -inf got a small weight where 0 is meant).  A window holds
// thousands of keys, a prompt one to four steps' worth, so what counts here is that nothing drains
// between units:
//   * three regions of TMEM columns rotate: S of step G + 1 goes where dS of step G - 1 was, dP of
//     step G + 1 where S of step G was, so both are ready when the elementwise warps end step G
//     (with Q and dO as TMEM operands there was room for one of each, and dP waited for dS);
//   * a unit's dQ is read out in the next unit's first step, after its dS is written and before it is
//     handed over (that step's product overwrites dQ), and leaves through shared memory and TMA
//     stores;
//   * the row statistics of a unit are loaded during the unit before;
//   * K and V of short key sequences stay in shared memory for all consecutive units of their kv
//     head; a CTA's (pair's) units are a contiguous range of equal cost, as in the forward, whose
//     units these are.
// More than 128 rows per head run on CTA pairs, as in the forward (kPair): every product is one M
// = 256 tcgen05.mma.cta_group::2 over 256 rows.  A CTA holds half of every operand, and K twice:
// its half of a step's keys for the scores and its half of the channels for the dQ product, each
// with a ring of its own and released by its own product.  (24 heads x 35840 rows over 512 and 203
// keys, whole backward: 650 us, and 695 with this pass on single CTAs.)
//
// What bounds it: 289 us there, 3200 clocks per step.  Latency: the tensor pipe is active 40% of the
// time, L2 at 18% of its rate; the MMA warp goes through seven waits of 200 clocks a step,
// which follow one another, a unit's start and its dQ take 3000 to 3500 clocks of the elementwise
// warps, and of the stalls of a warp a fifth are for instructions (long unrolled code, run once a
// step).  Ring depth counts: two entries in place of three cost 40%.  Measured and not kept: rings of two entries with two Q tiles (430 us); one wait per step for all loads, behind
// a warp that collects them (336); dQ stored from registers, four V entries in its place (350).
//
// Persistent and warp-specialised, 384 threads:
//   warp 8      TMA producer of K
//   warp 10     TMA producer of V and of Q and dO
//   warp 11     takes each K chunk of the dQ product as it lands, zeroes the rows past the last key
//               that the product will read (against dS = 0, but 0 * NaN is NaN) and hands it over
//   warp 9      MMA issuer (pair: the even CTA's), per step G: S(G + 1); dP(G + 1) once the
//               elementwise warps hold S(G) in registers; dQ += dS(G) K(G) once dS(G) is written
//   warps 0-7   elementwise, two threads per row: thread h takes keys [64h, 64h + 64) of a step
// TMEM (512 columns): three regions of 128 [0, 384), dQ [384, 512).
#pragma once

#include <stdint.h>

#include "dsa_bwd_dq.cuh"
#include "dsa_cross_fwd.cuh"
#include "sm100.cuh"

namespace dsa {

struct CrossDqParams : CrossShape {
  const float* lse;    // [B, heads, Lq]
  const float* delta;
  __nv_bfloat16* dq;   // through strides (batch, head, row)
  int64_t dq_s[3];
  float* dq_part;      // n_split > 1: [n_split, B * heads * Lq, 128]
  uint32_t q_bytes;    // bytes a unit's Q (or dO) boxes load
  int qb, qk, qg, db, dk, dg, kb, kh, vb, vh;  // 1, or 0 for a broadcast (stride 0) dimension of q, dO, k, v
  float scale, scale_log2;
};

namespace crossdq {
constexpr int kThreads = bdq::kThreads;
constexpr int kKWarp = 8, kMmaWarp = 9, kVWarp = 10, kHandWarp = 11;
constexpr uint32_t kTile = 128 * 128 * 2, kHalf = kTile / 2;
// Shared memory: 224 KB of tiles and the barriers.  Q and dO (32 KB each); single: K 3 and V 2
// chunks of 32 KB; pair: K 3 entries of 64 keys (scores) and 3 of 64 channels (dQ product), V 2 of
// 64 keys, 16 KB each, and 32 KB through which dQ leaves.
template <bool kPair>
struct Mem {
  static constexpr int kK = 3, kV = 2;  // chunks
  static constexpr uint32_t kEntry = kPair ? kHalf : kTile;
  static constexpr uint32_t kOffQ = 0, kOffDO = kTile, kOffK = 2 * kTile, kOffV = kOffK + kK * kEntry;
  static constexpr uint32_t kOffK2 = kPair ? kOffV + kV * kEntry : kOffK;  // K of the dQ product
  static constexpr uint32_t kOffOut = kPair ? kOffK2 + kK * kEntry : kOffQ;
  static_assert((kPair ? kOffOut + kTile : kOffV + kV * kEntry) == 7 * kTile, "both forms use 224 KB");
};
constexpr uint32_t kOffBar = 7 * kTile;
constexpr uint32_t kSmemUsed = kOffBar + 320;
constexpr uint32_t kSmemBytes = 227 * 1024;
static_assert(kSmemUsed <= kSmemBytes, "shared memory layout too large");

// Regions of 128 TMEM columns rotate: S of step G at region(G), dP (then dS) at the one after it.
__device__ __forceinline__ int next_region(int r) { return r == 0 ? 2 : r - 1; }  // S of the next step
__device__ __forceinline__ uint32_t col_s(int r) { return 128 * r; }
__device__ __forceinline__ uint32_t col_dp(int r) { return 128 * (r == 2 ? 0 : r + 1); }

// D = A B^T over 128 channels: A (Q or dO, K-major) and B (a K-major tile of the step's 128 keys;
// pair: 64 of them in either CTA) from shared memory.
template <bool kPair>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc) {
  mma_ss_128<kPair, kHalf, kPair ? kHalf / 2 : kHalf>(d_tmem, a_desc, b_desc,
                                                      kPair ? idesc_bf16_f32(256, 128, 0, 0) : bdq::kIdescS, 0);
}

// dQ (+)= dS K over 16 keys (dS of keys [16kk, 16kk + 16) at the columns of its region t_ds that
// their thread wrote).
template <bool kPair>
__device__ __forceinline__ void issue_dq(uint32_t tmem, uint32_t t_ds, int kk, uint64_t k_desc, bool accumulate) {
  const uint32_t ds = t_ds + 64 * (kk >> 2) + 8 * (kk & 3);
  if constexpr (kPair)
    mma_ts_pair_warp(tmem + bdq::kColDQ, ds, fwd::desc_add(k_desc, kk * 2048), idesc_bf16_f32(256, 128, 0, 1), accumulate);
  else
    mma_ts_warp(tmem + bdq::kColDQ, ds, fwd::desc_add(k_desc, kk * 2048), bdq::kIdescDQ, accumulate);
}
}  // namespace crossdq

// kPair: launched as clusters of two; tmK and tmV have boxes of 64 keys, tmK2 of 128.  Single: all of
// 128, tmK2 is not used.
template <bool kPair>
__global__ void __launch_bounds__(crossdq::kThreads, 1)
    cross_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDO,
                    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmK2,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDQ,
                    CrossDqParams p) {
  using namespace crossdq;
  using crossf::arrive;
  using crossf::commit;
  using crossf::lead_bar;
  using crossf::wait_lead;
  using M = Mem<kPair>;
  using Cur = crossf::Cursor<kPair ? 256 : 128>;
  constexpr int kK = M::kK, kV = M::kV, kCtas = kPair ? 2 : 1;
  using bdq::kColDQ;
  using fwd::desc_add;
  using fwd::warp_wait;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
  if (pad + kSmemUsed > kSmemBytes) {  // uniform over the CTA: nothing has started yet
    if (threadIdx.x == 0) device_report(DSA_DEV_BOUNDS, 6);
    return;
  }
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw + pad;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* q_full = bars;               // Q of a unit has landed
  uint64_t* q_empty = bars + 1;
  uint64_t* do_full = bars + 2;          // dO
  uint64_t* do_empty = bars + 3;
  uint64_t* k_land = bars + 4;           // [kK] K of the dQ product has landed in this CTA
  uint64_t* k2_full = k_land + kK;       // [kK] handed over (by each CTA)
  uint64_t* k2_empty = k2_full + kK;     // [kK]
  uint64_t* k_full = k2_empty + kK;      // [kK] pair: K of the scores
  uint64_t* k_empty = k_full + kK;       // [kK]
  uint64_t* v_full = k_empty + kK;       // [kV]
  uint64_t* v_empty = v_full + kV;       // [kV]
  uint64_t* s_full = v_empty + kV;       // [2] S of a step (by its parity) ready
  uint64_t* s_read = s_full + 2;         // [2] loaded (8 per CTA)
  uint64_t* dp_full = s_full + 4;        // [2] dP of a step ready
  uint64_t* ds_full = s_full + 6;        // [2] dS written (8 per CTA); a unit's first: also the previous dQ read
  uint64_t* dq_done = s_full + 8;        // every dQ product of a unit done
  uint64_t* drain = s_full + 9;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_full + 10);
  volatile int* abort = reinterpret_cast<volatile int*>(s_full + 10) + 1;
  int* range = reinterpret_cast<int*>(s_full + 11);  // [2]
  static_assert(4 + 5 * kK + 2 * kV + 12 <= 320 / 8, "barriers must fit their 320 bytes");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = kPair ? static_cast<int>(cluster_ctarank()) : 0;
  const bool lead = rank == 0;
  if (tid == 0) {
    tma_prefetch_map(&tmQ);
    tma_prefetch_map(&tmDO);
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(do_full, 1);
    mbar_init(do_empty, 1);
    for (int s = 0; s < kK; ++s) {
      mbar_init(k_land + s, 1);
      mbar_init(k2_full + s, kCtas);
      mbar_init(k2_empty + s, 1);
      mbar_init(k_full + s, 1);
      mbar_init(k_empty + s, 1);
    }
    for (int s = 0; s < kV; ++s) {
      mbar_init(v_full + s, 1);
      mbar_init(v_empty + s, 1);
    }
    for (int e = 0; e < 2; ++e) {
      mbar_init(s_full + e, 1);
      mbar_init(s_read + e, 8 * kCtas);
      mbar_init(dp_full + e, 1);
      mbar_init(ds_full + e, 8 * kCtas);
    }
    mbar_init(dq_done, 1);
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    int b, e;
    crossf::unit_range(p, blockIdx.x / kCtas, gridDim.x / kCtas, b, e);
    if (lane == 0) {
      range[0] = b;
      range[1] = e;
    }
  }
  if (warp == kMmaWarp) {
    if constexpr (kPair) {
      tmem_alloc_pair(tmem_slot, bdq::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, bdq::kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();  // both CTAs' barriers are ready before either arrives on the other's
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int begin = range[0], end = range[1];

  if (warp >= 8) {
    setmaxnreg_dec<bdq::kRegsAux>();
    if (warp == kKWarp) {
      // ------------------------------------------------------------------ TMA producer of K
      if (lane == 0) {
        Cur c, d;  // the scores' K of the next step, the dQ product's K of this one
        c.start(p, begin, end);
        c.settle(p);
        d = c;
        int ld = 0, ld2 = 0;
        bool ok = true;
        // this CTA's half of the keys of c's step for the scores (pair)
        auto load_scores = [&]() {
          if (!c.reuse(kK)) {
            const int st = ld % kK;
            ok = mbar_wait(k_empty + st, ((ld / kK) & 1) ^ 1, abort, 170);
            if (!ok) return;
            ++ld;
            if (lead) mbar_arrive_expect_tx(k_full + st, 2 * M::kEntry);
            const uint32_t bar = lead_bar<kPair>(k_full + st);
            uint8_t* dst = smem + M::kOffK + st * M::kEntry;
            const int row = 128 * (c.c0 + c.t) + 64 * rank;
            tma_load_4d_pair(dst, &tmK, bar, 0, row, c.x.kvh * p.kh, c.x.b * p.kb);
            tma_load_4d_pair(dst + kHalf / 2, &tmK, bar, 64, row, c.x.kvh * p.kh, c.x.b * p.kb);
          }
          c.next_chunk(p);
        };
        if (kPair && c.valid()) load_scores();
        while (ok && d.valid()) {
          if (kPair && c.valid()) load_scores();
          if (ok && !d.reuse(kK)) {
            const int st = ld2 % kK;
            ok = mbar_wait(k2_empty + st, ((ld2 / kK) & 1) ^ 1, abort, 171);
            if (!ok) break;
            ++ld2;
            uint8_t* dst = smem + M::kOffK2 + st * M::kEntry;
            mbar_arrive_expect_tx(k_land + st, M::kEntry);
            const CUtensorMap* map = kPair ? &tmK2 : &tmK;
            tma_load_4d(dst, map, k_land + st, 64 * rank, 128 * (d.c0 + d.t), d.x.kvh * p.kh, d.x.b * p.kb);
            if constexpr (!kPair)
              tma_load_4d(dst + kHalf, map, k_land + st, 64, 128 * (d.c0 + d.t), d.x.kvh * p.kh, d.x.b * p.kb);
          }
          d.next_chunk(p);
        }
      }
    } else if (warp == kHandWarp) {
      // ------------------------------------------------------------------ K hand-over (whole warp)
      Cur c;
      c.start(p, begin, end);
      int ld = 0;
      bool ok = true;
      for (c.settle(p); ok && c.valid(); c.next_unit(p)) {
        if (c.reuse(kK)) continue;
        for (int j = 0; j < c.n; ++j, ++ld) {
          const int st = ld % kK;
          ok = warp_wait(k_land + st, (ld / kK) & 1, abort, 172);
          if (!ok) break;
          const int keys = c.keys(j);
          if (keys & 15) {
            const int pad_rows = 16 - (keys & 15);
            const uint32_t k0 = sbase + M::kOffK2 + st * M::kEntry + (lane & 7) * 16 + (kPair ? 0u : (lane >> 3 & 1) * kHalf);
            for (int rr = lane >> (kPair ? 3 : 4); rr < pad_rows; rr += kPair ? 4 : 2)
              st_shared_v4(k0 + (keys + rr) * 128, 0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) {
            if constexpr (kPair)
              mbar_arrive_release_cluster(lead_bar<kPair>(k2_full + st));
            else
              mbar_arrive(k2_full + st);
          }
        }
      }
    } else if (warp == kVWarp) {
      // ------------------------------------------------------------------ TMA producer of V, Q and dO
      if (lane == 0) {
        Cur c;
        c.start(p, begin, end);
        int ld = 0, un = 0;
        bool ok = true;
        for (c.settle(p); ok && c.valid(); c.next_unit(p), ++un) {
          const int row = c.x.row + 128 * rank;
          auto load = [&](uint64_t* full, uint64_t* empty, uint32_t off, const CUtensorMap* map, int g, int kvh, int b,
                          int site) -> bool {
            if (!mbar_wait(empty, (un & 1) ^ 1, abort, site)) return false;
            if (lead) mbar_arrive_expect_tx(full, kCtas * p.q_bytes);
            if constexpr (kPair) {
              const uint32_t bar = lead_bar<kPair>(full);
              tma_load_5d_pair(smem + off, map, bar, 0, row, g, kvh, b);
              tma_load_5d_pair(smem + off + kHalf, map, bar, 64, row, g, kvh, b);
            } else {
              tma_load_5d(smem + off, map, full, 0, row, g, kvh, b);
              tma_load_5d(smem + off + kHalf, map, full, 64, row, g, kvh, b);
            }
            return true;
          };
          ok = load(q_full, q_empty, M::kOffQ, &tmQ, c.x.g * p.qg, c.x.kvh * p.qk, c.x.b * p.qb, 173) &&
               load(do_full, do_empty, M::kOffDO, &tmDO, c.x.g * p.dg, c.x.kvh * p.dk, c.x.b * p.db, 174);
          if (!ok) break;
          if (c.reuse(kV)) continue;
          for (int j = 0; j < c.n; ++j, ++ld) {
            const int st = ld % kV;
            ok = mbar_wait(v_empty + st, ((ld / kV) & 1) ^ 1, abort, 175);
            if (!ok) break;
            uint8_t* dst = smem + M::kOffV + st * M::kEntry;
            const int at = 128 * (c.c0 + j) + (kPair ? 64 * rank : 0);
            if (lead) mbar_arrive_expect_tx(v_full + st, kCtas * M::kEntry);
            if constexpr (kPair) {
              const uint32_t bar = lead_bar<kPair>(v_full + st);
              tma_load_4d_pair(dst, &tmV, bar, 0, at, c.x.kvh * p.vh, c.x.b * p.vb);
              tma_load_4d_pair(dst + kHalf / 2, &tmV, bar, 64, at, c.x.kvh * p.vh, c.x.b * p.vb);
            } else {
              tma_load_4d(dst, &tmV, v_full + st, 0, at, c.x.kvh * p.vh, c.x.b * p.vb);
              tma_load_4d(dst + kHalf, &tmV, v_full + st, 64, at, c.x.kvh * p.vh, c.x.b * p.vb);
            }
          }
        }
      }
    } else if (lead) {
      // ------------------------------------------------------------------ MMA issuer (whole warp)
      const uint64_t dKk = smem_desc_sw128(sbase + M::kOffK, 16, 1024);      // K-major
      const uint64_t dKm = smem_desc_sw128(sbase + M::kOffK2, kHalf, 1024);  // MN-major
      const uint64_t dVk = smem_desc_sw128(sbase + M::kOffV, 16, 1024);
      const uint64_t dQk = smem_desc_sw128(sbase + M::kOffQ, 16, 1024), dDOk = smem_desc_sw128(sbase + M::kOffDO, 16, 1024);
      uint64_t* ks_full = kPair ? k_full : k2_full;  // K of the scores
      Cur sc, dc;                  // the steps whose S and dP, and whose dQ product come next
      int ks = 0, vs = 0, kd = 0;  // ring positions of their units' first chunks
      int qn = 0;                  // units before sc's
      int rs = 0;                  // region of S of the step whose dQ product comes next
      sc.start(p, begin, end);
      sc.settle(p);
      // S of sc's step, the G-th, into the region that dS(G - 2) held (its product was issued)
      auto issue_s = [&](int G, int region) -> bool {
        const int pos = ks + sc.t, st = pos % kK;
        const bool reuse = sc.reuse(kK), keep = sc.keep(p, kK);
        if (sc.t == 0 && !wait_lead<kPair>(q_full, qn & 1, abort, 180)) return false;
        if (!reuse && !wait_lead<kPair>(ks_full + st, (pos / kK) & 1, abort, 181)) return false;
        tc_fence_after();
        issue_qk<kPair>(tmem + col_s(region), dQk, desc_add(dKk, st * M::kEntry));
        commit<kPair>(s_full + (G & 1));
        if (kPair && !keep) commit<kPair>(k_empty + st);
        if (sc.t + 1 == sc.n) commit<kPair>(q_empty);
        return true;
      };
      // dP of the same step, into the region of S(G - 1), which has been loaded
      auto issue_dp = [&](int G, int region) -> bool {
        const int pos = vs + sc.t, st = pos % kV;
        const bool reuse = sc.reuse(kV), keep = sc.keep(p, kV);
        if (sc.t == 0 && !wait_lead<kPair>(do_full, qn & 1, abort, 182)) return false;
        if (!reuse && !wait_lead<kPair>(v_full + st, (pos / kV) & 1, abort, 183)) return false;
        if (G > 0 && !wait_lead<kPair>(s_read + ((G - 1) & 1), ((G - 1) >> 1) & 1, abort, 184)) return false;
        tc_fence_after();
        issue_qk<kPair>(tmem + col_dp(region), dDOk, desc_add(dVk, st * M::kEntry));
        commit<kPair>(dp_full + (G & 1));
        if (!keep) commit<kPair>(v_empty + st);
        if (sc.t + 1 == sc.n) {
          commit<kPair>(do_empty);
          ++qn;
          if (!sc.keep(p, kK)) ks += sc.n;
          if (!keep) vs += sc.n;
        }
        return true;
      };
      bool ok = true;
      if (sc.valid()) ok = issue_s(0, rs) && issue_dp(0, rs);
      dc = sc;
      if (sc.valid()) sc.next_chunk(p);
      for (int G = 0; ok && dc.valid(); ++G) {
        const int rn = next_region(rs);
        if (sc.valid()) ok = issue_s(G + 1, rn) && issue_dp(G + 1, rn);
        const int pos = kd + dc.t, st = pos % kK, n16 = (dc.keys(dc.t) + 15) >> 4;
        const bool keep = dc.keep(p, kK);
        if (ok && kPair && !dc.reuse(kK)) ok = wait_lead<kPair>(k2_full + st, (pos / kK) & 1, abort, 185);
        uint64_t k = desc_add(dKm, st * M::kEntry);
        fwd::opaque(k);
        const uint32_t t_ds = tmem + col_dp(rs);
        if (ok) ok = wait_lead<kPair>(ds_full + (G & 1), (G >> 1) & 1, abort, 186);
        if (!ok) break;
        tc_fence_after();
        if (n16 == 8) {
          mma_ts_128<kPair, 64>(tmem + kColDQ, t_ds, k, kPair ? idesc_bf16_f32(256, 128, 0, 1) : bdq::kIdescDQ, dc.t > 0);
        } else {  // the last chunk: only the sixteens that hold keys
#pragma unroll 1
          for (int kk = 0; kk < n16; ++kk) issue_dq<kPair>(tmem, t_ds, kk, k, dc.t > 0 || kk > 0);
        }
        if (!keep) commit<kPair>(k2_empty + st);
        if (dc.t + 1 == dc.n) {
          commit<kPair>(dq_done);
          if (!keep) kd += dc.n;
        }
        dc = sc;
        if (sc.valid()) sc.next_chunk(p);
        rs = rn;
      }
      if constexpr (kPair)
        mma_commit_pair_warp(drain, 1);
      else
        mma_commit_warp(drain);
      fwdp::drain_wait(drain, 0);
    }
  } else {
    setmaxnreg_inc<bdq::kRegsElem>();
    // ------------------------------------------------------------------ elementwise and output
    const int h = warp >> 2, quarter = warp & 3, r = 32 * quarter + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const float kLog2e = 1.4426950408889634f;
    int G = 0, un = 0, rs = 0;
    bool ok = true;
    crossf::Unit px = {};  // the unit whose dQ is still in TMEM
    // dQ = scale * accumulator, channels [64h, 64h + 64) of this thread's row of unit px
    auto write_out = [&](int unit) -> bool {
      if (!warp_wait(dq_done, unit & 1, abort, 190)) return false;
      tc_fence_after();
      const uint32_t tD = tmem + kColDQ + 64 * h + lane_off;
      if constexpr (kPair) {
        const uint32_t off = M::kOffOut + h * kHalf + quarter * 4096;
        if (lane == 0) tma_store_wait_read();  // the unit before has left the buffer
        __syncwarp();
        crossf::stage_o(tD, p.scale, sbase + off);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          const int r0 = px.row + 32 * quarter;
          if (r0 < p.Lq) {
            tma_store_5d(&tmDQ, smem + off, 64 * h, r0, px.g, px.kvh, px.b);
            tma_store_commit();
          }
        }
      } else {
        const crossf::Row y = crossf::unit_row(p, px, r);  // (single)
        if (p.n_split > 1) {
          const int64_t rows = static_cast<int64_t>(p.B) * p.heads * p.Lq;
          const int64_t row = (static_cast<int64_t>(px.b) * p.heads + y.head) * p.Lq + y.q;
          crossf::store_o_f32(tD, p.scale,
                              reinterpret_cast<float4*>(p.dq_part + (y.ok ? px.part * rows + row : 0) * 128) + 16 * h, y.ok);
        } else {
          const int64_t at = y.ok ? px.b * p.dq_s[0] + y.head * p.dq_s[1] + y.q * p.dq_s[2] : 0;
          fwd::store_o(tD, 2, p.scale, reinterpret_cast<uint4*>(p.dq + at) + 8 * h, y.ok);
        }
      }
      return true;
    };
    // the row statistics of a unit, loaded while the unit before is worked on
    float n_lse = 0.f, n_dd = 0.f;
    auto load_stats = [&](const Cur& u) {
      crossf::Unit x = u.x;
      x.row += 128 * rank;
      const crossf::Row y = crossf::unit_row(p, x, r);
      const int64_t at = (static_cast<int64_t>(x.b) * p.heads + y.head) * p.Lq + y.q;
      n_lse = y.ok ? p.lse[at] : 0.f;
      n_dd = y.ok ? p.delta[at] : 0.f;
    };
    Cur c, nx;
    c.start(p, begin, end);
    if (c.valid()) load_stats(c);
    for (; ok && c.valid(); c = nx) {
      crossf::Unit x = c.x;  // (row: this CTA's first)
      x.row += 128 * rank;
      const float neg_lse2 = -n_lse * kLog2e, dd = n_dd;
      nx = c;
      nx.advance(p);
      if (nx.valid()) load_stats(nx);
      if (c.n == 0) {  // no keys: no gradient
        const crossf::Row y = crossf::unit_row(p, x, r);
        if (y.ok) {
          if (p.n_split > 1) {
            const int64_t bh = static_cast<int64_t>(x.b) * p.heads + y.head;
            float4* dst = reinterpret_cast<float4*>(
                p.dq_part + (x.part * static_cast<int64_t>(p.B) * p.heads * p.Lq + bh * p.Lq + y.q) * 128) + 16 * h;
#pragma unroll
            for (int e = 0; e < 16; ++e) dst[e] = make_float4(0.f, 0.f, 0.f, 0.f);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(p.dq + x.b * p.dq_s[0] + y.head * p.dq_s[1] + y.q * p.dq_s[2]) + 8 * h;
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        continue;
      }
      // a warp without query rows works on nothing: its rows of dS and dQ reach no other row
      const bool act = p.pk > 1 ? 32 * quarter < p.pk * p.Lq : x.row + 32 * quarter < p.Lq;
      for (c.t = 0; c.t < c.n; ++c.t, ++G, rs = next_region(rs)) {
        const int e2 = G & 1;
        const int nv = c.keys(c.t) - 64 * h;  // keys of this thread's 64 columns
        const bool work = act && nv > 0;
        ok = warp_wait(s_full + e2, (G >> 1) & 1, abort, 192);
        if (!ok) break;
        tc_fence_after();
        float pf[64];
        if (work) {
          uint32_t s[64];
          tmem_ld64_wait(tmem + col_s(rs) + 64 * h + lane_off, s);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive<kPair>(lead_bar<kPair>(s_read + e2));
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            float x0, x1;
            ffma2(x0, x1, __uint_as_float(s[e]), __uint_as_float(s[e + 1]), p.scale_log2, p.scale_log2, neg_lse2,
                  neg_lse2);
            pf[e] = ex2_approx(x0);
            pf[e + 1] = ex2_approx(x1);
          }
        } else if (lane == 0) {
          arrive<kPair>(lead_bar<kPair>(s_read + e2));
        }
        ok = warp_wait(dp_full + e2, (G >> 1) & 1, abort, 193);
        if (!ok) break;
        tc_fence_after();
        if (work) {
          const uint32_t tDP = tmem + col_dp(rs) + 64 * h + lane_off;
          uint32_t dp[64];
          tmem_ld64_wait(tDP, dp);
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            float a0, a1, d0, d1;
            fadd2(a0, a1, __uint_as_float(dp[e]), __uint_as_float(dp[e + 1]), -dd, -dd);
            ffma2(d0, d1, a0, a1, pf[e], pf[e + 1], 0.f, 0.f);
            w[e >> 1] = pack_bf16x2(d0, d1);
          }
          if (nv < 64) {  // no key in these columns: their P and dP may be anything, dS is zero
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (2 * e >= nv) w[e] = 0u;
              else if (2 * e + 1 >= nv) w[e] &= 0xffffu;
            }
          }
          tmem_st32(tDP, w);
          tmem_wait_st();
        }
        if (c.t == 0 && un > 0) {  // this step's dQ product overwrites the previous unit's dQ
          ok = write_out(un - 1);
          if (!ok) break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive<kPair>(lead_bar<kPair>(ds_full + e2));
      }
      px = x;
      ++un;
    }
    if (ok && un > 0) write_out(un - 1);
    if (lane == 0) tma_store_wait_read();
  }

  tc_fence_before();
  __syncthreads();
  if (*abort && tid == 0) {
    // after a failed wait, give loads already issued time to land before the CTA leaves
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 100000ull) {
    }
  }
  __syncthreads();
  if constexpr (kPair) cluster_sync();  // neither CTA leaves while the other may still reach into it
  if (warp == kMmaWarp) {
    __syncwarp();
    if constexpr (kPair)
      tmem_dealloc_pair(tmem, bdq::kTmemCols);
    else
      tmem_dealloc(tmem, bdq::kTmemCols);
  }
}

}  // namespace dsa
