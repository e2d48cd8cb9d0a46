// dK and dV of the cross attention's backward, key-major: for key row m of a kv head, over the
// query rows n of every head that shares it
//   P_nm = exp(scale q_n.k_m - LSE_n),  dS_nm = P_nm (dO_n.v_m - D_n),
//   dV_m = sum_n P_nm dO_n,  dK_m = scale sum_n dS_nm q_n.
//
// A prompt gives few key units (128 keys of one kv head) and each has 10^4 to 10^5 query rows, so
// the query chunks (128 rows, or pk heads of Lq rows) of all units form one sequence that is cut
// into a range of equal length per CTA.  A unit inside one CTA's range is written by it; of a unit
// that is cut, each CTA writes its piece's fp32 sums to a slot (two per CTA) and
// cross_kv_combine adds them in CTA order: no atomics, the same bits from run to run.
//
// Per chunk the products take 2048 clocks: S^T = K Q^T and dP^T = V dO^T (128 x 128 each), dV +=
// P^T dO and dK += dS^T Q (P^T and dS^T from TMEM).  TMEM holds dV, dK, one S^T and one dP^T, so
// the schedule keeps the tensor pipe busy without a second buffer: P^T and dS^T are written over
// dP^T, which frees the scores' columns as soon as they are in registers, and the chunk's
// elementwise work is handed over in two halves of 64 queries:
//   tensor pipe   dP(c)      S(c+1)       grads A(c)  grads B(c)   dP(c+1) ...
//   elementwise   (exp of c) dS A, dS B(c)      exp of c+1 ...
// 24 heads x 35840 rows over 512 and 203 keys: 257 us, 3600 clocks per chunk.  What bounds it is
// that cycle: dP(c), dS (750 clocks), the four gradient products and dP(c + 1) follow one another,
// with 1250 clocks of exponentials and some 200 per hand-over beside them; running a quarter or
// three eighths of the exponentials on the FMA pipe changed nothing.  A second dP buffer would
// break it, for which TMEM has no columns left (dV, dK, S, dP: 512).
// (64-query chunks with two buffers, the window backward's form, run the score products at
// N = 64, two thirds of the pipe's rate, and twice the hand-overs: 1830 clocks per 64 queries.)
//
// Persistent and warp-specialised, one CTA per SM, 384 threads:
//   warp 8      TMA producer of K and V of a unit, and Q of its chunks (3 entries)
//   warp 10     TMA producer of dO (2 entries)
//   warp 11     -LSE log2 e and -D of a chunk's rows into shared memory (2 entries), and how many
//               of its rows exist (the others' P and dS are set to 0: against an infinite key the
//               score of a row of zeros is NaN)
//   warp 9      MMA issuer
//   warps 0-7   elementwise, two threads per key row: thread h takes queries [32h, 32h + 32) of
//               either half; at the end of a piece warps 0-3 write dV and warps 4-7 dK
#pragma once

#include <stdint.h>

#include "dsa_cross_fwd.cuh"
#include "sm100.cuh"

namespace dsa {

struct CrossKvParams : CrossShape {
  int per_unit;        // query chunks of a unit
  const float* lse;    // [B, heads, Lq]
  const float* delta;
  __nv_bfloat16 *dk, *dv;  // through strides (batch, head, row)
  int64_t dk_s[3], dv_s[3];
  float *dk_part, *dv_part;  // [2 * grid, 128, 128] fp32
  uint32_t q_bytes;    // bytes a chunk's Q (or dO) boxes load
  int qb, qk, qg, db, dkv, dg, kb, kh, vb, vh;  // 1, or 0 for a broadcast (stride 0) dimension of q, dO, k, v
  float scale, scale_log2;
};

namespace crosskv {
constexpr int kThreads = 384;
constexpr int kKWarp = 8, kMmaWarp = 9, kDoWarp = 10, kVecWarp = 11;
constexpr int kRegsElem = 216, kRegsAux = 72, kRegsAtLaunch = 168;
static_assert(2 * 128 * kRegsElem + 128 * kRegsAux == kThreads * kRegsAtLaunch, "split must use the launch registers");
constexpr int kQ = 3, kDo = 2;
constexpr uint32_t kTile = 128 * 128 * 2, kHalf = kTile / 2;
constexpr uint32_t kOffK = 0, kOffV = kTile, kOffQ = 2 * kTile, kOffDo = kOffQ + kQ * kTile;
constexpr uint32_t kOffVec = kOffDo + kDo * kTile;  // [kDo][2][128] floats
constexpr uint32_t kOffBar = kOffVec + kDo * 1024;
constexpr uint32_t kSmemUsed = kOffBar + 256;
constexpr uint32_t kSmemBytes = 227 * 1024;
static_assert(kSmemUsed <= kSmemBytes, "shared memory layout too large");
constexpr uint32_t kTmemCols = 512, kColDV = 0, kColDK = 128, kColS = 256, kColDP = 384;
constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, 0, 0), kIdescAcc = idesc_bf16_f32(128, 128, 0, 1);

__device__ __forceinline__ int kv_chunks(const CrossKvParams& p, int b) { return (crossf::kv_length(p, b) + 127) / 128; }

// Units in all (whole warp); their number fits 31 bits.
__device__ __forceinline__ int count_units(const CrossKvParams& p) {
  int all = 0;
  for (int i = threadIdx.x & 31; i < p.B; i += 32) all += kv_chunks(p, i) * p.kv_heads;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  return all;
}

// A unit: 128-key chunk kt of kv head kvh of batch entry b.
struct KvUnit {
  int b, kvh, kt;
};

// The v-th unit (whole warp, v below their number; a lane takes a batch entry of 32).
__device__ __forceinline__ KvUnit find_unit(const CrossKvParams& p, int v) {
  const int lane = threadIdx.x & 31;
  KvUnit x = {0, 0, 0};
  int before = 0;
#pragma unroll 1
  for (int first = 0; first < p.B; first += 32) {
    const int c = first + lane < p.B ? kv_chunks(p, first + lane) : 0;
    const int own = c * p.kv_heads;
    int end = own;  // (inclusive sums)
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int below = __shfl_up_sync(0xffffffffu, end, d);
      if (lane >= d) end += below;
    }
    end += before;
    const unsigned m = __ballot_sync(0xffffffffu, v < end);
    if (m) {
      const int at = __ffs(m) - 1, n = __shfl_sync(0xffffffffu, c, at);
      const int rem = v - __shfl_sync(0xffffffffu, end - own, at);
      x.b = first + at;
      x.kvh = rem / n;
      x.kt = rem - x.kvh * n;
      break;
    }
    before = __shfl_sync(0xffffffffu, end, 31);
  }
  return x;
}

// Walks the pieces of a CTA's range of the chunk sequence: unit, first query chunk, number of
// chunks (0: past the range).
struct Pieces : KvUnit {
  int chunks;  // key chunks of the batch entry
  int c0, n;
  int64_t left;
  __device__ __forceinline__ Pieces(const CrossKvParams& p, const KvUnit& first, int64_t lo, int64_t hi) : KvUnit(first) {
    chunks = kv_chunks(p, b);
    c0 = static_cast<int>(lo % max(p.per_unit, 1));
    left = hi - lo;
    n = static_cast<int>(min(static_cast<int64_t>(p.per_unit - c0), left));
  }
  __device__ __forceinline__ void next(const CrossKvParams& p) {
    left -= n;
    c0 = 0;
    n = static_cast<int>(min(static_cast<int64_t>(p.per_unit), left));
    if (n == 0 || ++kt < chunks) return;
    kt = 0;
    if (++kvh < p.kv_heads) return;
    kvh = 0;
    do {
      chunks = kv_chunks(p, ++b);  // (units are left: an entry with keys follows)
    } while (chunks == 0);
  }
};

// A query chunk of a kv head: rows from `row` of head g of the group (pk > 1: pk heads from g).
struct QChunk {
  int g, row;
  // Rows that exist: the first of the 128.
  __device__ __forceinline__ int rows(const CrossKvParams& p) const {
    return p.pk > 1 ? min(p.pk, p.group - g) * p.Lq : min(p.Lq - row, 128);
  }
  __device__ __forceinline__ void start(const CrossKvParams& p, int c) {
    if (p.pk > 1) {
      g = c * p.pk;
      row = 0;
    } else {
      const int per_head = (p.Lq + 127) / 128;
      g = c / per_head;
      row = 128 * (c % per_head);
    }
  }
  __device__ __forceinline__ void next(const CrossKvParams& p) {
    row += 128;
    if (row >= p.Lq) {
      row = 0;
      g += p.pk;
    }
  }
};

// D (+)= A B^T over 128 channels, both K-major tiles of two 64-channel halves.
__device__ __forceinline__ void issue_scores(uint32_t d_tmem, uint64_t a, uint64_t b) {
  mma_ss_128<false, kHalf, kHalf>(d_tmem, a, b, kIdescS, 0);
}

// D (+)= A B over 64 queries: A (P^T at +0, dS^T at +16 of each thread's 32 columns) from TMEM, B
// an MN-major tile of queries x channels.
__device__ __forceinline__ void issue_grad(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, bool accumulate) {
  mma_ts_64<32>(d_tmem, a_tmem, b, kIdescAcc, accumulate);
}
}  // namespace crosskv

__global__ void __launch_bounds__(crosskv::kThreads, 1)
    cross_kv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDO,
                    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, CrossKvParams p) {
  using namespace crosskv;
  using fwd::desc_add;
  using fwd::warp_wait;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
  if (pad + kSmemUsed > kSmemBytes) {  // uniform over the CTA: nothing has started yet
    if (threadIdx.x == 0) device_report(DSA_DEV_BOUNDS, 7);
    return;
  }
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw + pad;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* kv_full = bars;
  uint64_t* kv_free = bars + 1;
  uint64_t* q_full = bars + 2;           // [kQ]
  uint64_t* q_empty = q_full + kQ;       // [kQ]
  uint64_t* do_full = q_empty + kQ;      // [kDo]
  uint64_t* do_empty = do_full + kDo;    // [kDo]
  uint64_t* vec_full = do_empty + kDo;   // [kDo]
  uint64_t* vec_free = vec_full + kDo;   // [kDo] read (8)
  uint64_t* s_full = vec_free + kDo;     // S^T of a chunk ready
  uint64_t* s_read = s_full + 1;         // loaded (8)
  uint64_t* dp_full = s_full + 2;        // dP^T ready
  uint64_t* p_full = s_full + 3;         // [2] P^T and dS^T of a half written (8)
  uint64_t* dkv_full = s_full + 5;       // every product of a piece done
  uint64_t* dkv_free = s_full + 6;       // dK and dV read out (8)
  uint64_t* drain = s_full + 7;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_full + 8);
  volatile int* abort = reinterpret_cast<volatile int*>(s_full + 8) + 1;
  int64_t* range = reinterpret_cast<int64_t*>(s_full + 9);        // [2] of the chunk sequence
  KvUnit* first_unit = reinterpret_cast<KvUnit*>(s_full + 11);    // the one that it begins in
  int* n_rows = reinterpret_cast<int*>(s_full + 13);              // [kDo] rows of a chunk (with -LSE and -D)
  static_assert(2 + 2 * kQ + 4 * kDo + 13 + (kDo + 1) / 2 <= 256 / 8, "barriers must fit their 256 bytes");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    tma_prefetch_map(&tmQ);
    tma_prefetch_map(&tmDO);
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
    mbar_init(kv_full, 1);
    mbar_init(kv_free, 1);
    for (int s = 0; s < kQ; ++s) {
      mbar_init(q_full + s, 1);
      mbar_init(q_empty + s, 1);
    }
    for (int s = 0; s < kDo; ++s) {
      mbar_init(do_full + s, 1);
      mbar_init(do_empty + s, 1);
      mbar_init(vec_full + s, 1);
      mbar_init(vec_free + s, 8);
    }
    mbar_init(s_full, 1);
    mbar_init(s_read, 8);
    mbar_init(dp_full, 1);
    mbar_init(p_full, 8);
    mbar_init(p_full + 1, 8);
    mbar_init(dkv_full, 1);
    mbar_init(dkv_free, 8);
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    const int64_t all = static_cast<int64_t>(count_units(p)) * p.per_unit;
    const int64_t b = all * blockIdx.x / gridDim.x, e = all * (blockIdx.x + 1) / gridDim.x;
    const KvUnit x = find_unit(p, static_cast<int>(b / max(p.per_unit, 1)));
    if (lane == 0) {
      range[0] = b;
      range[1] = e;
      *first_unit = x;
    }
  }
  if (p.pk > 1) {
    // chunks of packed heads leave the rows from pk * Lq on unwritten, and the gradient products
    // read them against P = dS = 0: zeros, once
    for (uint32_t i = tid; i < (kQ + kDo) * kTile / 16; i += kThreads) st_shared_v4(sbase + kOffQ + 16 * i, 0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int64_t lo = range[0], hi = range[1];
  const KvUnit u0 = *first_unit;

  if (warp >= 8) {
    setmaxnreg_dec<kRegsAux>();
    if (warp == kKWarp) {
      // ------------------------------------------------------------------ TMA producer of K, V and Q
      if (lane == 0) {
        int ld = 0;
        bool ok = true;
        Pieces x(p, u0, lo, hi);
        for (int k = 0; ok && x.n > 0; ++k, x.next(p)) {
          ok = mbar_wait(kv_free, (k & 1) ^ 1, abort, 200);
          if (!ok) break;
          mbar_arrive_expect_tx(kv_full, 2 * kTile);
          tma_load_4d(smem + kOffK, &tmK, kv_full, 0, 128 * x.kt, x.kvh * p.kh, x.b * p.kb);
          tma_load_4d(smem + kOffK + kHalf, &tmK, kv_full, 64, 128 * x.kt, x.kvh * p.kh, x.b * p.kb);
          tma_load_4d(smem + kOffV, &tmV, kv_full, 0, 128 * x.kt, x.kvh * p.vh, x.b * p.vb);
          tma_load_4d(smem + kOffV + kHalf, &tmV, kv_full, 64, 128 * x.kt, x.kvh * p.vh, x.b * p.vb);
          QChunk q;
          q.start(p, x.c0);
          for (int c = 0; c < x.n; ++c, ++ld, q.next(p)) {
            const int st = ld % kQ;
            ok = mbar_wait(q_empty + st, ((ld / kQ) & 1) ^ 1, abort, 201);
            if (!ok) break;
            uint8_t* dst = smem + kOffQ + st * kTile;
            mbar_arrive_expect_tx(q_full + st, p.q_bytes);
            tma_load_5d(dst, &tmQ, q_full + st, 0, q.row, q.g * p.qg, x.kvh * p.qk, x.b * p.qb);
            tma_load_5d(dst + kHalf, &tmQ, q_full + st, 64, q.row, q.g * p.qg, x.kvh * p.qk, x.b * p.qb);
          }
        }
      }
    } else if (warp == kDoWarp) {
      // ------------------------------------------------------------------ TMA producer of dO
      if (lane == 0) {
        int ld = 0;
        bool ok = true;
        Pieces x(p, u0, lo, hi);
        for (int k = 0; ok && x.n > 0; ++k, x.next(p)) {
          QChunk q;
          q.start(p, x.c0);
          for (int c = 0; c < x.n; ++c, ++ld, q.next(p)) {
            const int st = ld % kDo;
            ok = mbar_wait(do_empty + st, ((ld / kDo) & 1) ^ 1, abort, 202);
            if (!ok) break;
            uint8_t* dst = smem + kOffDo + st * kTile;
            mbar_arrive_expect_tx(do_full + st, p.q_bytes);
            tma_load_5d(dst, &tmDO, do_full + st, 0, q.row, q.g * p.dg, x.kvh * p.dkv, x.b * p.db);
            tma_load_5d(dst + kHalf, &tmDO, do_full + st, 64, q.row, q.g * p.dg, x.kvh * p.dkv, x.b * p.db);
          }
        }
      }
    } else if (warp == kVecWarp) {
      // ------------------------------------------------------------------ -LSE log2 e and -D (whole warp)
      int ld = 0;
      bool ok = true;
      Pieces x(p, u0, lo, hi);
      for (int k = 0; ok && x.n > 0; ++k, x.next(p)) {
        QChunk q;
        q.start(p, x.c0);
        for (int c = 0; c < x.n; ++c, ++ld, q.next(p)) {
          const int st = ld % kDo;
          float nl[4], nd[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const crossf::Row y = crossf::unit_row(p, crossf::Unit{x.b, x.kvh, 0, q.g, q.row}, 32 * e + lane);
            const int64_t at = (static_cast<int64_t>(x.b) * p.heads + y.head) * p.Lq + y.q;
            nl[e] = y.ok ? -p.lse[at] * 1.4426950408889634f : -INFINITY;
            nd[e] = y.ok ? -p.delta[at] : 0.f;
          }
          ok = warp_wait(vec_free + st, ((ld / kDo) & 1) ^ 1, abort, 203);
          if (!ok) break;
          float* v = reinterpret_cast<float*>(smem + kOffVec + st * 1024);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[32 * e + lane] = nl[e];
            v[128 + 32 * e + lane] = nd[e];
          }
          if (lane == 0) n_rows[st] = q.rows(p);
          __syncwarp();
          if (lane == 0) mbar_arrive(vec_full + st);
        }
      }
    } else {
      // ------------------------------------------------------------------ MMA issuer (whole warp)
      const uint64_t dK = smem_desc_sw128(sbase + kOffK, 16, 1024), dV = smem_desc_sw128(sbase + kOffV, 16, 1024);
      const uint64_t dQk = smem_desc_sw128(sbase + kOffQ, 16, 1024), dQm = smem_desc_sw128(sbase + kOffQ, kHalf, 1024);
      const uint64_t dOk = smem_desc_sw128(sbase + kOffDo, 16, 1024), dOm = smem_desc_sw128(sbase + kOffDo, kHalf, 1024);
      int C = 0;  // chunks before
      bool ok = true;
      auto issue_s = [&](int c) -> bool {  // S^T of the CTA's c-th chunk, once that of chunk c - 1 has been loaded
        if (!warp_wait(q_full + c % kQ, (c / kQ) & 1, abort, 210)) return false;
        if (c > 0 && !warp_wait(s_read, (c - 1) & 1, abort, 211)) return false;
        tc_fence_after();
        issue_scores(tmem + kColS, dK, desc_add(dQk, c % kQ * kTile));
        mma_commit_warp(s_full);
        return true;
      };
      Pieces x(p, u0, lo, hi);
      for (int k = 0; ok && x.n > 0; ++k, x.next(p)) {
        const int n = x.n;
        ok = warp_wait(kv_full, k & 1, abort, 212) && issue_s(C);
        for (int c = 0; c < n && ok; ++c, ++C) {
          const int st = C % kDo;
          ok = warp_wait(do_full + st, (C / kDo) & 1, abort, 213);
          if (!ok) break;
          tc_fence_after();
          issue_scores(tmem + kColDP, dV, desc_add(dOk, st * kTile));
          mma_commit_warp(dp_full);
          if (c + 1 < n)
            ok = issue_s(C + 1);
          else
            mma_commit_warp(kv_free);
          if (ok && c == 0) ok = warp_wait(dkv_free, (k & 1) ^ 1, abort, 214);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (ok) ok = warp_wait(p_full + i, C & 1, abort, 215);
            if (!ok) break;
            tc_fence_after();
            issue_grad(tmem + kColDV, tmem + kColDP + 64 * i, desc_add(dOm, st * kTile + i * 8192), c > 0 || i > 0);
            issue_grad(tmem + kColDK, tmem + kColDP + 64 * i + 16, desc_add(dQm, C % kQ * kTile + i * 8192), c > 0 || i > 0);
          }
          if (!ok) break;
          mma_commit_warp(q_empty + C % kQ);
          mma_commit_warp(do_empty + st);
        }
        if (!ok) break;
        mma_commit_warp(dkv_full);
      }
      mma_commit_warp(drain);
      fwdp::drain_wait(drain, 0);
    }
  } else {
    setmaxnreg_inc<kRegsElem>();
    // ------------------------------------------------------------------ P^T, dS^T and dK / dV out
    const int h = warp >> 2, m = 32 * (warp & 3) + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int C = 0;
    bool ok = true;
    Pieces x(p, u0, lo, hi);
    for (int k = 0; ok && x.n > 0; ++k, x.next(p)) {
      const int len = crossf::kv_length(p, x.b);
      const bool k_ok = 128 * x.kt + m < len, tail = 128 * x.kt + 128 > len;
      for (int c = 0; c < x.n; ++c, ++C) {
        const int st = C % kDo;
        const float4* nl = reinterpret_cast<const float4*>(smem + kOffVec + st * 1024);
        ok = warp_wait(vec_full + st, (C / kDo) & 1, abort, 220);
        if (ok) ok = warp_wait(s_full, C & 1, abort, 221);
        if (!ok) break;
        tc_fence_after();
        const int nq = n_rows[st];
        float pf[64];  // P^T of queries [32h, 32h + 32) and [64 + 32h, 96 + 32h)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t s[32];
          const bool any = 64 * half + 32 * h < nq;  // of the rows there are
          if (any) tmem_ld32_wait(tmem + kColS + 64 * half + 32 * h + lane_off, s);
          if (half == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_read);
          }
          if (!any) continue;
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            const float4 l4 = nl[16 * half + 8 * h + g];
            const float lv[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const int i = 4 * g + e;
              float x0, x1;
              ffma2(x0, x1, __uint_as_float(s[i]), __uint_as_float(s[i + 1]), p.scale_log2, p.scale_log2, lv[e],
                    lv[e + 1]);
              pf[32 * half + i] = ex2_approx(x0);
              pf[32 * half + i + 1] = ex2_approx(x1);
            }
          }
        }
        ok = warp_wait(dp_full, C & 1, abort, 222);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t tD = tmem + kColDP + 64 * half + 32 * h + lane_off;
          uint32_t d[32], pk[16], ds[16];
          const int left = nq - 64 * half - 32 * h;  // rows there are
          if (left > 0) {
            tmem_ld32_wait(tD, d);
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              const float4 d4 = nl[32 + 16 * half + 8 * h + g];
              const float dv[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
              for (int e = 0; e < 4; e += 2) {
                const int i = 4 * g + e;
                const float p0 = pf[32 * half + i], p1 = pf[32 * half + i + 1];
                float a0, a1, d0, d1;
                fadd2(a0, a1, __uint_as_float(d[i]), __uint_as_float(d[i + 1]), dv[e], dv[e + 1]);
                ffma2(d0, d1, a0, a1, p0, p1, 0.f, 0.f);
                pk[i / 2] = pack_bf16x2(p0, p1);
                ds[i / 2] = pack_bf16x2(d0, d1);
              }
            }
            if (left < 32) {  // a missing row's P and dP may be anything: both are zero
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const uint32_t keep = 2 * e + 1 < left ? 0xffffffffu : 2 * e < left ? 0xffffu : 0u;
                pk[e] &= keep;
                ds[e] &= keep;
              }
            }
          }
          if (left <= 0 || (tail && !k_ok)) {  // and a padding key's
#pragma unroll
            for (int e = 0; e < 16; ++e) pk[e] = ds[e] = 0u;
          }
          __syncwarp();
          tmem_st16(tD, pk);  // over this thread's own dP columns
          tmem_st16(tD + 16, ds);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(p_full + half);
            if (half == 1) mbar_arrive(vec_free + st);
          }
        }
      }
      if (!ok) break;
      // dV (warps 0-3) or dK (warps 4-7) of the unit's 128 keys: bf16 of a whole unit, fp32 sums
      // (unscaled) of a piece; padding keys: zeros, or nothing
      ok = warp_wait(dkv_full, k & 1, abort, 223);
      if (!ok) break;
      tc_fence_after();
      const bool whole = x.n == p.per_unit, row_ok = 128 * x.kt + m < p.Lk;
      const int64_t* os = h ? p.dk_s : p.dv_s;
      __nv_bfloat16* out = (h ? p.dk : p.dv) + x.b * os[0] + x.kvh * os[1];
      uint4* dst = reinterpret_cast<uint4*>(out + (row_ok ? 128 * x.kt + m : 0) * os[2]);
      float4* slot = reinterpret_cast<float4*>((h ? p.dk_part : p.dv_part) +
                                               (2 * static_cast<int64_t>(blockIdx.x) + (k > 0)) * 16384 + m * 128);
      const float f = h ? p.scale : 1.f;
#pragma unroll 1
      for (int g = 0; g < 4; ++g) {
        uint32_t a[32];
        tmem_ld32_wait(tmem + (h ? kColDK : kColDV) + lane_off + g * 32, a);
        if (!k_ok) {
#pragma unroll
          for (int e = 0; e < 32; ++e) a[e] = 0u;
        }
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (k_ok)
              slot[8 * g + e] = make_float4(__uint_as_float(a[4 * e]), __uint_as_float(a[4 * e + 1]),
                                            __uint_as_float(a[4 * e + 2]), __uint_as_float(a[4 * e + 3]));
        } else if (row_ok) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint4 y;
            y.x = pack_bf16x2(__uint_as_float(a[8 * e + 0]) * f, __uint_as_float(a[8 * e + 1]) * f);
            y.y = pack_bf16x2(__uint_as_float(a[8 * e + 2]) * f, __uint_as_float(a[8 * e + 3]) * f);
            y.z = pack_bf16x2(__uint_as_float(a[8 * e + 4]) * f, __uint_as_float(a[8 * e + 5]) * f);
            y.w = pack_bf16x2(__uint_as_float(a[8 * e + 6]) * f, __uint_as_float(a[8 * e + 7]) * f);
            dst[4 * g + e] = y;
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(dkv_free);
    }
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
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// What the key-major pass leaves: dK and dV of the units that were cut between its n_cta CTAs,
// scale * (for dK) the sum of the pieces' fp32 sums, in CTA order, as bf16; and zeros for the
// padding's rows that no unit covers (without queries: for every row).  A block takes 16 rows
// (blockIdx.z) of dk or dv (blockIdx.y), of the unit that the end of CTA blockIdx.x's range cuts if
// its first piece is there, or (blockIdx.x >= n_cta) of a 128-key chunk of a kv head.
__global__ void __launch_bounds__(256) cross_kv_combine(CrossKvParams p, int n_cta) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = 16 * blockIdx.z + warp;  // this warp's rows: r and r + 8
  const bool is_dk = blockIdx.y == 0;
  const int64_t* s = is_dk ? p.dk_s : p.dv_s;
  __nv_bfloat16* out = is_dk ? p.dk : p.dv;
  if (blockIdx.x >= static_cast<unsigned>(n_cta)) {
    const int chunks = (p.Lk + 127) / 128, x = blockIdx.x - n_cta, kt = x % chunks, bh = x / chunks, b = bh / p.kv_heads;
    // (a whole unit's CTA, or the other blocks, write its chunk: the padding in it too)
    const int from = p.per_unit > 0 ? 128 * crosskv::kv_chunks(p, b) : 0;
    out += b * s[0] + (bh % p.kv_heads) * s[1];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int l = 128 * kt + r + 8 * j;
      if (l >= from && l < p.Lk) reinterpret_cast<uint2*>(out + l * s[2])[lane] = make_uint2(0u, 0u);
    }
    return;
  }
  if (p.per_unit == 0) return;
  const int64_t all = static_cast<int64_t>(crosskv::count_units(p)) * p.per_unit;
  // all * i / n_cta, with one wide division for all of them
  const int64_t per = all / n_cta;
  const int over = static_cast<int>(all - per * n_cta);
  auto bound = [&](int i) -> int64_t { return per * i + over * i / n_cta; };
  const int i0 = blockIdx.x;
  const int64_t lo0 = bound(i0), cut_at = bound(i0 + 1);
  if (lo0 >= cut_at || cut_at >= all) return;  // no range, or the last
  const int v = static_cast<int>(cut_at / p.per_unit);
  const int64_t start = static_cast<int64_t>(v) * p.per_unit, end = start + p.per_unit;
  if (cut_at == start || lo0 > start) return;  // no unit is cut here, or an earlier CTA holds its first piece
  const crosskv::KvUnit u = crosskv::find_unit(p, v);
  const int len = crossf::kv_length(p, u.b), l = 128 * u.kt + r;
  out += u.b * s[0] + u.kvh * s[1];
  const float f = is_dk ? p.scale : 1.f;
  const float* part = is_dk ? p.dk_part : p.dv_part;
  float4 a[2];
  a[0] = a[1] = make_float4(0.f, 0.f, 0.f, 0.f);
  int64_t lo = lo0;
#pragma unroll 1
  for (int i = i0; i < n_cta && lo < end; ++i) {
    const int64_t hi = bound(i + 1);
    if (lo < hi) {  // (a range is empty where there are fewer query chunks than CTAs)
      const float4* src =
          reinterpret_cast<const float4*>(part + (2 * static_cast<int64_t>(i) + (lo < start)) * 16384 + r * 128) + lane;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (l + 8 * j >= len) continue;
        const float4 x = src[8 * 32 * j];
        a[j].x += x.x;
        a[j].y += x.y;
        a[j].z += x.z;
        a[j].w += x.w;
      }
    }
    lo = hi;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int lj = l + 8 * j;
    if (lj >= p.Lk) continue;
    reinterpret_cast<uint2*>(out + lj * s[2])[lane] =
        make_uint2(pack_bf16x2(a[j].x * f, a[j].y * f), pack_bf16x2(a[j].z * f, a[j].w * f));
  }
}

}  // namespace dsa
