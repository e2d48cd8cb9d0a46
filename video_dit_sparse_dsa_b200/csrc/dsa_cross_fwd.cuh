// Cross attention, forward: every query row attends to an encoder's states, a key sequence of
// another length that the query rows of a batch entry share.
//
//   O_n = sum_{m < len_b} softmax_m(scale q_n k_m) v_m,   LSE_n = ln sum_{m < len_b} exp(scale q_n k_m)
//
// for the query rows n of batch entry b and head h, the keys and values of kv head
// h / (heads / kv_heads), and the first len_b of Lk states (the rest is the batch's padding and
// may hold anything: no value of it reaches a result).  len_b = 0 gives O = 0, LSE = -inf.
//
// A video's cross attention has many query rows (10^4 to 10^5) over few keys (a prompt of 77 to
// 512 states).  Per 128 query rows it moves 64 KB (Q, O) and, per 256 keys, takes 2048 clocks of
// products and 2048 of exponentials at the MUFU rate, so memory, tensor pipe and softmax all
// stand within a factor of two of each other at 256 to 512 keys, and what decides is how well the
// three overlap from one query tile to the next: a tile has one or two 256-key steps only.
//
// Two forms of one persistent, warp-specialised kernel.  Many rows (more than 128 per head) run on
// CTA pairs (kPair): a cluster of two CTAs holds 256 rows of one head, 128 each, and every product
// is one M = 256 tcgen05.mma.cta_group::2 issued by the even CTA; the scores take a step's 256
// keys as N, half from each CTA's shared memory, and P V the 128 channels as N, half from each.
// So a CTA holds half of K and V: up to 512 keys of both fit beside three Q tiles, and stay for
// all consecutive units of their kv head, where a single CTA re-reads V for every unit and has no
// room to load Q ahead (24 heads x 115200 rows over 512 keys: 694 us when built, and 953 as single
// CTAs).  Few rows over many keys (a single token over every state) run on single CTAs, with up to 128 / Lq heads of a kv head packed
// into a unit, so that K and V are read once for them, and with the keys cut into parts, one unit
// each, whose fp32 partial outputs cross_merge_kernel joins by their LSEs.
//
// A unit is 128 (pair: 256) query rows of one kv head over a range of its key chunks (128 keys),
// in steps of up to two chunks.  Roles (12 warps per CTA):
//   warp 8   TMA producer of K and Q
//   warp 10  TMA producer of V
//   warp 11  takes each V chunk as it lands, zeroes the rows past the last key that the product
//            will read (against P = 0, but 0 * NaN is NaN) and hands it to the MMA warp
//   warp 9   MMA issuer (pair: the even CTA's): the scores of step G + 1, which may be the next
//            unit's first, as soon as the softmax warps hold those of step G in registers, then
//            O += P(G) V(G)
//   warps 0-7  softmax of the CTA's own 128 rows: warpgroup i takes the step's chunk i (a single
//            chunk: half of its sixteens of columns), a thread per query row; the two threads of a
//            row agree on the row max through shared memory.
// The pipeline does not drain between units: a unit's output is read out of TMEM, divided and
// written during the next unit's first step, after that step's P is stored and before it is
// handed over (the products of that step overwrite O), when the last product of the unit has
// long finished.  The CTA's (pair's) units are a contiguous range of the unit sequence; ranges
// are cut at equal cost, as batch entries have their own lengths.
// Pair barriers: loads of K and Q count on the even CTA's barriers, products commit to both
// CTAs', and the softmax warps and V hand-overs of both arrive on the even CTA's.
//
// Measured in a loop of calls (one call on a cool GPU with L2 flushed in brackets): 24 heads x 115200
// rows over 512 keys 804 us, at the power cap, 901 TFLOP/s (686); 12 heads of 2 x 35840 rows over 512
// and 203 keys 214 us, 735 TFLOP/s (188); 24 x 16384 rows over 77 keys 63 us, 3.3 TB/s (64); one row of
// 24 heads, 6 of keys, over 115201 and 70007 keys 125 us, 4.5 TB/s (131).  With one or two steps per
// tile it is bound by the softmax of a step (2850 clocks per 256 keys, 2048 of them products) and by
// the 1200 to 1500 that a unit's read-out adds.
//
// TMEM (512 columns): as the window forward: regions R0 R1 R2 of 128 columns that scores and P
// rotate through (even steps: S in R0 R1, P in R0; odd: S in R1 R2, P in R2), O in the fourth.
#pragma once

#include <stdint.h>

#include "dsa_fwd_bf16.cuh"
#include "dsa_fwd_pair.cuh"
#include "sm100.cuh"

namespace dsa {

// What a cross attention's units are cut from (the forward's and the query-major backward's).
struct CrossShape {
  const int32_t* kv_len;  // [B] valid keys of each batch entry, or null: Lk
  int B, heads, kv_heads, group, Lq, Lk;
  int pk;                 // heads packed into a unit (Lq * pk <= 128), or 1
  int tiles;              // units per kv head and part
  int n_split;            // parts of the keys
  int n_units;            // B * kv_heads * n_split * tiles
  int unit_cost;          // a unit's fixed cost in eighths of a chunk, at least 1
};

struct CrossFwdParams : CrossShape {
  __nv_bfloat16* out;
  int64_t ob, oh, ol;     // strides of out in elements
  float* lse;             // [B, heads, Lq]
  float* part_o;          // n_split > 1: [n_split, B * heads * Lq, 128] and [n_split, B * heads * Lq]
  float* part_lse;
  uint32_t q_bytes;       // bytes a unit's Q boxes load
  int qb, qk, qg, kb, kh, vb, vh;  // 1, or 0 for a broadcast (stride 0) dimension
  float scale_log2;
};

namespace crossf {
constexpr int kThreads = 384;
constexpr int kKWarp = 8, kMmaWarp = 9, kVWarp = 10, kHandWarp = 11;
constexpr int kRegsSoftmax = 216, kRegsAux = 72;
constexpr int kRegsAtLaunch = (2 * 128 * kRegsSoftmax + 128 * kRegsAux) / kThreads;  // 168
static_assert(kRegsAtLaunch * kThreads == 2 * 128 * kRegsSoftmax + 128 * kRegsAux, "split must use the launch registers");
constexpr uint32_t kTile = 128 * 128 * 2, kHalf = kTile / 2;  // 128 rows x 128 channels; 64 channels
// Shared memory: 224 KB of tiles, the barriers, the exchange buffer.
// Single: Q 1, K 3 and V 3 chunks.  Pair (per CTA): Q 2; K 2 steps, this CTA's half of the keys of
// each; V 4 chunks of this CTA's 64 channels (both hold four chunks, 512 keys); 32 KB of output.
template <bool kPair>
struct Mem {
  static constexpr int kQ = kPair ? 2 : 1, kK = kPair ? 2 : 3, kV = kPair ? 4 : 3;
  static constexpr uint32_t kVBytes = kPair ? kHalf : kTile;
  static constexpr uint32_t kOffK = kQ * kTile, kOffV = kOffK + kK * kTile, kOffOut = kOffV + kV * kVBytes;
  // chunks of a unit whose K, and whose V, fit
  static constexpr int kKChunks = kPair ? 2 * kK : kK, kVChunks = kV;
  static_assert(kOffOut + (kPair ? kTile : 0) == 7 * kTile, "both forms use 224 KB");
};
constexpr uint32_t kOffBar = 7 * kTile;
constexpr uint32_t kOffX = kOffBar + 512;
constexpr uint32_t kSmemUsed = kOffX + 2 * 2 * 128 * 4;
constexpr uint32_t kSmemBytes = 227 * 1024;
static_assert(kSmemUsed <= kSmemBytes, "shared memory layout too large");
constexpr uint32_t kTmemCols = 512, kColO = 384;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: P <= 256, as in the window forward
// column pairs (bit e of the 8 pairs of every 16 columns) whose 2^x runs on the FMA pipe
constexpr uint32_t kPolyMask = 0x22u;

__device__ __forceinline__ int kv_length(const CrossShape& p, int b) {
  return p.kv_len == nullptr ? p.Lk : min(max(__ldg(p.kv_len + b), 0), p.Lk);
}

// Chunks per part of a sequence of `chunks`: even, so that parts are whole steps.
__device__ __forceinline__ int chunks_per_part(const CrossShape& p, int chunks) {
  const int per = (chunks + p.n_split - 1) / p.n_split;
  return p.n_split > 1 ? (per + 1) & ~1 : per;
}

// The CTA's units [begin, end): the sequence is cut at equal cost, a unit costing its chunks and a
// constant for its own start and end, in eighths of a chunk: unit_cost (chosen by each kernel's launch).
__device__ __forceinline__ int64_t unit_cost(const CrossShape& p, int b) {
  return 8 * static_cast<int64_t>(chunks_per_part(p, (kv_length(p, b) + 127) / 128)) + p.unit_cost;
}

// Called by a whole warp: a lane takes a batch entry of 32.
__device__ __forceinline__ void unit_range(const CrossShape& p, int cta, int n_cta, int& begin, int& end) {
  const int lane = threadIdx.x & 31;
  const int64_t per_b = static_cast<int64_t>(p.kv_heads) * p.n_split * p.tiles;
  int64_t total = 0;
  for (int b = lane; b < p.B; b += 32) total += per_b * unit_cost(p, b);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
  const int64_t x0 = total * cta / n_cta, x1 = total * (cta + 1) / n_cta;
  begin = end = p.n_units;
  int64_t acc = 0;
  for (int first = 0; first < p.B; first += 32) {
    const int b = first + lane;
    const int64_t c = b < p.B ? unit_cost(p, b) : 0;
    int64_t next = per_b * c;  // (inclusive sums)
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t below = __shfl_up_sync(0xffffffffu, next, d);
      if (lane >= d) next += below;
    }
    next += acc;
    const int64_t at = next - per_b * c;
    const unsigned m0 = __ballot_sync(0xffffffffu, at <= x0 && x0 < next);
    const unsigned m1 = __ballot_sync(0xffffffffu, at <= x1 && x1 < next);
    const int u0 = at <= x0 && x0 < next ? static_cast<int>(b * per_b + (x0 - at + c - 1) / c) : 0;
    const int u1 = at <= x1 && x1 < next ? static_cast<int>(b * per_b + (x1 - at + c - 1) / c) : 0;
    if (m0) begin = __shfl_sync(0xffffffffu, u0, __ffs(m0) - 1);
    if (m1) end = __shfl_sync(0xffffffffu, u1, __ffs(m1) - 1);
    acc = __shfl_sync(0xffffffffu, next, 31);
  }
}

// A unit: kRows (128, pair 256) rows from `row` of head g of a kv head's group (pk > 1: pk heads'
// rows from head g), over part `part` of the keys.
struct Unit {
  int b, kvh, part, g, row;
};

// Walks the CTA's units [begin, end) and their steps.  Consecutive units are neighbours in the
// sequence (row, head in the group, part, kv head, batch), so moving on needs no division.
template <int kRows>
struct Cursor {
  int u, end;
  Unit x;
  int len;      // keys of the unit's batch entry
  int c0, n;    // the unit's first chunk and number of chunks
  int t;        // step
  bool same;    // the previous unit of this CTA has the same keys

  __device__ __forceinline__ bool valid() const { return u < end; }
  __device__ __forceinline__ int in_step() const { return min(n - 2 * t, 2); }  // chunks of the step
  __device__ __forceinline__ bool last() const { return 2 * t + 2 >= n; }
  // A pair's step of one chunk: columns of the scores from each CTA (N in multiples of 32).
  __device__ __forceinline__ int half_columns() const { return ((keys(2 * t) + 31) & ~31) / 2; }
  // Keys present in the unit's chunk j.
  __device__ __forceinline__ int keys(int j) const { return min(len - 128 * (c0 + j), 128); }
  // The unit's K (or V) is still in the ring, which holds `chunks`, from the previous unit; the
  // next unit will find it there too.
  __device__ __forceinline__ bool reuse(int chunks) const { return same && n <= chunks; }
  __device__ __forceinline__ bool keep(const CrossShape& p, int chunks) const {
    return n <= chunks && u + 1 < end && (x.row + kRows < p.Lq || x.g + p.pk < p.group);
  }

  __device__ __forceinline__ void start(const CrossShape& p, int begin, int end_) {
    u = begin;
    end = end_;
    const int tile = u % p.tiles, slice = u / p.tiles;
    if (p.pk > 1) {
      x.g = tile * p.pk;
      x.row = 0;
    } else {
      const int per_head = (p.Lq + kRows - 1) / kRows;
      x.g = tile / per_head;
      x.row = kRows * (tile % per_head);
    }
    x.part = slice % p.n_split;
    x.kvh = slice / p.n_split % p.kv_heads;
    x.b = slice / p.n_split / p.kv_heads;
    same = false;
    t = 0;
    if (valid()) chunks(p);
  }
  __device__ __forceinline__ void chunks(const CrossShape& p) {
    len = kv_length(p, x.b);
    const int all = (len + 127) / 128, per = chunks_per_part(p, all);
    c0 = x.part * per;
    n = max(min(per, all - c0), 0);
  }
  // The next unit, with or without keys.
  __device__ __forceinline__ void advance(const CrossShape& p) {
    ++u;
    t = 0;
    same = true;
    x.row += kRows;
    if (x.row < p.Lq) return;
    x.row = 0;
    x.g += p.pk;
    if (x.g < p.group) return;
    x.g = 0;
    same = false;
    if (++x.part == p.n_split) {
      x.part = 0;
      if (++x.kvh == p.kv_heads) {
        x.kvh = 0;
        ++x.b;
      }
    }
    if (valid()) chunks(p);
  }
  // This unit, or the next one that has keys.
  __device__ __forceinline__ void settle(const CrossShape& p) {
    while (valid() && n == 0) advance(p);
  }
  __device__ __forceinline__ void next_unit(const CrossShape& p) {
    advance(p);
    settle(p);
  }
  // The next chunk (a user that counts t in chunks).
  __device__ __forceinline__ void next_chunk(const CrossShape& p) {
    if (t + 1 >= n)
      next_unit(p);
    else
      ++t;
  }
  __device__ __forceinline__ void next_step(const CrossShape& p) {
    if (last())
      next_unit(p);
    else
      ++t;
  }
};

// 2^x for a pair on the FMA pipe: as exp2_poly2, with a quartic for 2^f (minimax fit on
// [-0.5, 0.5], relative error 2.6e-6), because the row sums also give the fp32 LSE.  (That it keeps
// NaN costs nothing measurable; a max over the scores that keeps it took 1 to 2% more.)
__device__ __forceinline__ void exp2_quartic2(float x0, float x1, float& y0, float& y1) {
  constexpr float kRound = 12582912.0f;  // 1.5 * 2^23
  constexpr float c0 = 0.9999992847442627f, c1 = 0.6931217908859253f, c2 = 0.240247443318367f,
                  c3 = 0.05591785907745361f, c4 = 0.009570101276040077f;
  x0 = max_nan(x0, -126.f);
  x1 = max_nan(x1, -126.f);
  float t0, t1, n0, n1, f0, f1, q0, q1;
  fadd2(t0, t1, x0, x1, kRound, kRound);
  fadd2(n0, n1, t0, t1, -kRound, -kRound);
  ffma2(f0, f1, n0, n1, -1.f, -1.f, x0, x1);
  ffma2(q0, q1, c4, c4, f0, f1, c3, c3);
  ffma2(q0, q1, q0, q1, f0, f1, c2, c2);
  ffma2(q0, q1, q0, q1, f0, f1, c1, c1);
  ffma2(q0, q1, q0, q1, f0, f1, c0, c0);
  constexpr int kOne = 0x3f800000;
  fmul2_ftz(y0, y1, q0, q1, __int_as_float(kOne + (__float_as_int(t0) << 23)),
            __int_as_float(kOne + (__float_as_int(t1) << 23)));
}

// An arrival on the MMA warp's barrier: this CTA's, or the even CTA's of the pair (whose address
// `lead_bar` gives).
template <bool kPair>
__device__ __forceinline__ uint32_t lead_bar(uint64_t* bar) {
  if constexpr (kPair) return mapa_shared(smem_u32(bar), 0);
  return smem_u32(bar);
}
template <bool kPair>
__device__ __forceinline__ void arrive(uint32_t bar) {
  if constexpr (kPair)
    mbar_arrive_cluster(bar);
  else
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A barrier that the pair's other CTA arrives on too is acquired at cluster scope.
template <bool kPair>
__device__ __forceinline__ bool wait_lead(uint64_t* bar, uint32_t parity, volatile int* abort, int site) {
  if constexpr (kPair) return fwdp::warp_wait_cl(bar, parity, abort, site);
  return fwd::warp_wait(bar, parity, abort, site);
}

// The products so far arrive on `bar` (of both CTAs of a pair) when they are done.
template <bool kPair>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (kPair)
    mma_commit_pair_warp(bar, fwdp::kBoth);
  else
    mma_commit_warp(bar);
}

// O (+)= P V over 16 keys: P at tP, V at the descriptor.
template <bool kPair>
__device__ __forceinline__ void issue_pv(uint32_t tmem, uint32_t tP, uint64_t v, bool accumulate) {
  if constexpr (kPair)
    mma_ts_pair_warp(tmem + kColO, tP, v, idesc_bf16_f32(256, 128, 0, 1), accumulate);
  else
    mma_ts_warp(tmem + kColO, tP, v, idesc_bf16_f32(128, 128, 0, 1), accumulate);
}

// 2^x of 16 score columns (scaled, less the reference max) as packed bf16, added to the row sums.
__device__ __forceinline__ void exp_16(const uint32_t* s, float scale_log2, float neg_m, float (&sa)[4], float (&sb)[4],
                                       uint32_t (&pk)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float x0, x1, p0, p1;
    ffma2(x0, x1, __uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]), scale_log2, scale_log2, neg_m, neg_m);
    if ((kPolyMask >> e) & 1u) {
      exp2_quartic2(x0, x1, p0, p1);
    } else {
      p0 = ex2_approx(x0);
      p1 = ex2_approx(x1);
    }
    fadd2(sa[e & 3], sb[e & 3], sa[e & 3], sb[e & 3], p0, p1);
    pk[e] = pack_bf16x2(p0, p1);
  }
}

// A row's running softmax: the reference max, the row sum against it, and the factor that the old
// O and l take where the reference moved in the last step.
//
// The reference starts at fwd::kLowest, for scores that are not finite.
struct RowState {
  float m_used = fwd::kLowest, l = 0.f, alpha = 1.f;
  // Agrees with the partner thread on the row max, mx being this thread's; true: it moved.
  __device__ __forceinline__ bool update(bool ok, float mx, float scale_log2, float* xbuf, int& xe, int i, int r, int bar_id) {
    mx = fmaxf(mx, fwd::pair_exchange(xbuf, xe, i, r, bar_id, ok ? mx : -INFINITY));
    alpha = 1.f;
    if (!ok) return false;
    const float m_new = fmaxf(m_used, mx * scale_log2);
    const bool need = m_new > m_used + kRescaleThreshold;
    if (need) {
      alpha = ex2_approx(m_used - m_new);
      m_used = m_new;
    }
    l *= alpha;
    return need;
  }
};

// The scores are in registers: their columns may be overwritten.
template <bool kPair>
__device__ __forceinline__ void scores_loaded(bool ok, uint32_t loaded) {
  if (!ok) return;
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) arrive<kPair>(loaded);
}

// One step's softmax for this thread's 128 score columns at tS, of which the first nvalid hold
// keys: writes P as packed bf16 at tP; true: the reference max moved.  With !ok (an earlier wait
// failed) the thread only takes part in the exchange.
template <bool kPair>
__device__ __forceinline__ bool softmax_step(bool ok, uint32_t tS, uint32_t tP, uint32_t loaded, float scale_log2,
                                             RowState& st, float* xbuf, int& xe, int i, int r, int bar_id, int nvalid) {
  uint32_t s[128];
  tmem_ld128_wait(tS, s);
  if (nvalid < 128) {
#pragma unroll
    for (int c = 0; c < 128; ++c)
      if (c >= nvalid) s[c] = 0xff800000u;
  }
  scores_loaded<kPair>(ok, loaded);
  float mxs[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    mxs[e] = fmaxf(__uint_as_float(s[e]), __uint_as_float(s[120 + e]));
#pragma unroll
    for (int c = 8 + e; c < 120; c += 16)
      mxs[e] = max3f(mxs[e], __uint_as_float(s[c]), __uint_as_float(s[c + 8]));
  }
  const float mx = max3f(max3f(mxs[0], mxs[1], mxs[2]), max3f(mxs[3], mxs[4], mxs[5]), fmaxf(mxs[6], mxs[7]));
  const bool need = st.update(ok, mx, scale_log2, xbuf, xe, i, r, bar_id);
  if (!ok) return false;
  float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    uint32_t pk[8];
    exp_16(s + 16 * g, scale_log2, -st.m_used, sa, sb, pk);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[8 * g + e] = pk[e];
  }
  st.l += ((sa[0] + sb[0]) + (sa[1] + sb[1])) + ((sa[2] + sb[2]) + (sa[3] + sb[3]));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) w[e] = s[32 * h + e];
    tmem_st32(tP + 32 * h, w);
  }
  return need;
}

// The same over at most 64 columns, in sixteens: only those below n16 are worked on and written
// (a step's softmax costs by its keys; against one that masks a step's rest: a pair of
// prompts of 512 and 203 keys 205 -> 197 us, 77 keys 65.9 -> 64.8 us).
template <bool kPair>
__device__ __forceinline__ bool softmax_few(bool ok, uint32_t tS, uint32_t tP, uint32_t loaded, float scale_log2,
                                            RowState& st, float* xbuf, int& xe, int i, int r, int bar_id, int n16,
                                            int nvalid) {
  uint32_t s[64];
  tmem_ld64_wait(tS, s);
  float mx = -INFINITY;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    if (g >= n16) continue;
    if (16 * g + 16 > nvalid) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (16 * g + e >= nvalid) s[16 * g + e] = 0xff800000u;
    }
    float a = __uint_as_float(s[16 * g]), b = __uint_as_float(s[16 * g + 1]);
#pragma unroll
    for (int e = 2; e < 16; e += 4) {
      a = max3f(a, __uint_as_float(s[16 * g + e]), __uint_as_float(s[16 * g + e + 1]));
      if (e + 2 < 16) b = max3f(b, __uint_as_float(s[16 * g + e + 2]), __uint_as_float(s[16 * g + e + 3]));
    }
    mx = max3f(mx, a, b);
  }
  scores_loaded<kPair>(ok, loaded);
  const bool need = st.update(ok, mx, scale_log2, xbuf, xe, i, r, bar_id);
  if (!ok) return false;
  float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    if (g >= n16) continue;
    uint32_t pk[8];
    exp_16(s + 16 * g, scale_log2, -st.m_used, sa, sb, pk);
    tmem_st8(tP + 8 * g, pk);
  }
  st.l += ((sa[0] + sb[0]) + (sa[1] + sb[1])) + ((sa[2] + sb[2]) + (sa[3] + sb[3]));
  return need;
}

// O row columns [0, 64) from tO, times inv, as fp32 to dst where `write` (the TMEM loads are
// warp-collective: every lane takes part).
__device__ __forceinline__ void store_o_f32(uint32_t tO, float inv, float4* dst, bool write) {
#pragma unroll 1
  for (int g = 0; g < 2; ++g) {
    uint32_t o[32];
    tmem_ld32_wait(tO + 32 * g, o);
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (write)
        dst[8 * g + c] = make_float4(__uint_as_float(o[4 * c]) * inv, __uint_as_float(o[4 * c + 1]) * inv,
                                     __uint_as_float(o[4 * c + 2]) * inv, __uint_as_float(o[4 * c + 3]) * inv);
  }
}

// A warp's 32 rows x 64 channels of O, from TMEM times inv (of the lane's own row), as bf16 to
// shared memory, 128-byte swizzled (16-byte vector c of row r at c ^ (r % 8)) as a TMA store
// reads them.
__device__ __forceinline__ void stage_o(uint32_t tO, float inv, uint32_t stage) {
  const uint32_t lane = threadIdx.x & 31, row = stage + lane * 128;
#pragma unroll
  for (uint32_t g = 0; g < 2; ++g) {
    uint32_t o[32];
    tmem_ld32_wait(tO + 32 * g, o);
#pragma unroll
    for (uint32_t c = 0; c < 4; ++c) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = pack_bf16x2(__uint_as_float(o[8 * c + 2 * e]) * inv, __uint_as_float(o[8 * c + 2 * e + 1]) * inv);
      st_shared_v4(row + (((4 * g + c) ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
    }
  }
}

// Query row of thread r in a unit: its head and position, or no row.
struct Row {
  bool ok;
  int head, q;
};

__device__ __forceinline__ Row unit_row(const CrossShape& p, const Unit& x, int r) {
  Row y;
  int g = x.g;
  if (p.pk > 1) {  // row r = (head in the pack) * Lq + position
    g += r / p.Lq;
    y.q = r % p.Lq;
    y.ok = r < p.pk * p.Lq && g < p.group;
  } else {
    y.q = x.row + r;
    y.ok = y.q < p.Lq;
  }
  y.head = x.kvh * p.group + g;
  return y;
}
}  // namespace crossf

// kPair: launched as clusters of two.
template <bool kPair>
__global__ void __launch_bounds__(crossf::kThreads, 1)
    cross_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                     CrossFwdParams p) {
  using namespace crossf;
  using fwd::desc_add;
  using fwd::warp_wait;
  using M = Mem<kPair>;
  using Cur = Cursor<kPair ? 256 : 128>;
  constexpr int kCtas = kPair ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
  if (pad + kSmemUsed > kSmemBytes) {  // the same in every CTA: nothing has started yet
    if (threadIdx.x == 0) device_report(DSA_DEV_BOUNDS, 5);
    return;
  }
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw + pad;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* q_full = bars;                // [kQ]
  uint64_t* q_empty = q_full + M::kQ;
  uint64_t* k_full = q_empty + M::kQ;     // [kK]
  uint64_t* k_empty = k_full + M::kK;
  uint64_t* v_land = k_empty + M::kK;     // [kV] the chunk has landed in this CTA
  uint64_t* v_full = v_land + M::kV;      // [kV] handed over (by each CTA)
  uint64_t* v_empty = v_full + M::kV;
  uint64_t* s_full = v_empty + M::kV;     // [2] scores of a step of parity e ready
  uint64_t* s_read = s_full + 2;          // [2] loaded by the softmax warps (8 per CTA)
  uint64_t* p_full = s_full + 4;          // [2] P of a step of parity e written (8 per CTA)
  uint64_t* o_done = s_full + 6;          // the products of a step into O done
  uint64_t* o_final = s_full + 7;         // the products of a unit done
  uint64_t* o_free = s_full + 8;          // O of a unit read out (8 per CTA)
  uint64_t* drain = s_full + 9;           // every product issued has completed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_full + 10);
  volatile int* abort = reinterpret_cast<volatile int*>(s_full + 10) + 1;
  int* range = reinterpret_cast<int*>(s_full + 11);  // [2]
  static_assert(2 * M::kQ + 2 * M::kK + 3 * M::kV + 12 <= 512 / 8, "barriers must fit their 512 bytes");
  float* xbuf = reinterpret_cast<float*>(smem + kOffX);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = kPair ? static_cast<int>(cluster_ctarank()) : 0;
  const bool lead = rank == 0;
  if (tid == 0) {
    tma_prefetch_map(&tmQ);
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
    if constexpr (kPair) tma_prefetch_map(&tmO);
    for (int s = 0; s < M::kQ; ++s) {
      mbar_init(q_full + s, 1);
      mbar_init(q_empty + s, 1);
    }
    for (int s = 0; s < M::kK; ++s) {
      mbar_init(k_full + s, 1);
      mbar_init(k_empty + s, 1);
    }
    for (int s = 0; s < M::kV; ++s) {
      mbar_init(v_land + s, 1);
      mbar_init(v_full + s, kCtas);
      mbar_init(v_empty + s, 1);
    }
    for (int e = 0; e < 2; ++e) {
      mbar_init(s_full + e, 1);
      mbar_init(s_read + e, 8 * kCtas);
      mbar_init(p_full + e, 8 * kCtas);
    }
    mbar_init(o_done, 1);
    mbar_init(o_final, 1);
    mbar_init(o_free, 8 * kCtas);
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    int b, e;
    unit_range(p, blockIdx.x / kCtas, gridDim.x / kCtas, b, e);
    if (lane == 0) {
      range[0] = b;
      range[1] = e;
    }
  }
  if (warp == kMmaWarp) {
    if constexpr (kPair) {
      tmem_alloc_pair(tmem_slot, kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, kTmemCols);
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
    setmaxnreg_dec<kRegsAux>();
    if (warp == kKWarp) {
      // ------------------------------------------------------------------ TMA producer of K and Q
      if (lane == 0) {
        Cur c;
        c.start(p, begin, end);
        int ld = 0, un = 0;  // K ring entries loaded, units with keys
        bool ok = true;
        auto load_q = [&]() {
          const int st = un % M::kQ;
          ok = mbar_wait(q_empty + st, ((un / M::kQ) & 1) ^ 1, abort, 140);
          ++un;
          if (!ok) return;
          uint8_t* dst = smem + st * kTile;
          const int row = c.x.row + 128 * rank;  // (rows past Lq load as zeros)
          if (lead) mbar_arrive_expect_tx(q_full + st, kCtas * p.q_bytes);
          if constexpr (kPair) {
            const uint32_t bar = lead_bar<kPair>(q_full + st);
            tma_load_5d_pair(dst, &tmQ, bar, 0, row, c.x.g * p.qg, c.x.kvh * p.qk, c.x.b * p.qb);
            tma_load_5d_pair(dst + kHalf, &tmQ, bar, 64, row, c.x.g * p.qg, c.x.kvh * p.qk, c.x.b * p.qb);
          } else {
            tma_load_5d(dst, &tmQ, q_full + st, 0, row, c.x.g * p.qg, c.x.kvh * p.qk, c.x.b * p.qb);
            tma_load_5d(dst + kHalf, &tmQ, q_full + st, 64, row, c.x.g * p.qg, c.x.kvh * p.qk, c.x.b * p.qb);
          }
        };
        for (c.settle(p); ok && c.valid(); c.next_unit(p)) {
          if (c.reuse(M::kKChunks)) {  // K is still in shared memory
            load_q();
            continue;
          }
          // the first step's K, then Q (whose wait is for the previous unit's last scores, and K
          // of a step does not wait for it), then the other steps' K
          const int head = c.x.kvh * p.kh, b = c.x.b * p.kb;
          const int n_loads = kPair ? (c.n + 1) / 2 : c.n, n_first = kPair ? 1 : min(c.n, 2);
          for (int j = 0; j < n_loads && ok; ++j, ++ld) {
            if (j == n_first) load_q();
            const int st = ld % M::kK;
            if (ok) ok = mbar_wait(k_empty + st, ((ld / M::kK) & 1) ^ 1, abort, 141);
            if (!ok) break;
            uint8_t* dst = smem + M::kOffK + st * kTile;
            if constexpr (kPair) {
              // a step of two chunks: this CTA's chunk; of one: this CTA's half of its columns
              // (boxes of 64 keys)
              c.t = j;
              const bool two = c.in_step() == 2;
              const int row = 128 * (c.c0 + 2 * j) + (two ? 128 : c.half_columns()) * rank;
              if (lead) mbar_arrive_expect_tx(k_full + st, two ? 2 * kTile : kTile);
              const uint32_t bar = lead_bar<kPair>(k_full + st);
              for (int h = 0; h < (two ? 2 : 1); ++h) {
                tma_load_4d_pair(dst + h * (kHalf / 2), &tmK, bar, 0, row + 64 * h, head, b);
                tma_load_4d_pair(dst + kHalf + h * (kHalf / 2), &tmK, bar, 64, row + 64 * h, head, b);
              }
            } else {
              mbar_arrive_expect_tx(k_full + st, kTile);
              tma_load_4d(dst, &tmK, k_full + st, 0, 128 * (c.c0 + j), head, b);
              tma_load_4d(dst + kHalf, &tmK, k_full + st, 64, 128 * (c.c0 + j), head, b);
            }
          }
          if (ok && n_loads <= n_first) load_q();
        }
      }
    } else if (warp == kVWarp) {
      // ------------------------------------------------------------------ TMA producer of V
      if (lane == 0) {
        Cur c;
        int ld = 0;
        bool ok = true;
        c.start(p, begin, end);
        for (c.settle(p); ok && c.valid(); c.next_unit(p)) {
          if (c.reuse(M::kVChunks)) continue;
          const int head = c.x.kvh * p.vh, b = c.x.b * p.vb;
          for (int j = 0; j < c.n; ++j, ++ld) {
            const int st = ld % M::kV;
            ok = mbar_wait(v_empty + st, ((ld / M::kV) & 1) ^ 1, abort, 142);
            if (!ok) break;
            uint8_t* dst = smem + M::kOffV + st * M::kVBytes;
            mbar_arrive_expect_tx(v_land + st, M::kVBytes);
            tma_load_4d(dst, &tmV, v_land + st, 64 * rank, 128 * (c.c0 + j), head, b);
            if constexpr (!kPair) tma_load_4d(dst + kHalf, &tmV, v_land + st, 64, 128 * (c.c0 + j), head, b);
          }
        }
      }
    } else if (warp == kHandWarp) {
      // ------------------------------------------------------------------ V hand-over (whole warp)
      Cur c;
      int ld = 0;
      bool ok = true;
      c.start(p, begin, end);
      for (c.settle(p); ok && c.valid(); c.next_unit(p)) {
        if (c.reuse(M::kVChunks)) continue;
        for (int j = 0; j < c.n; ++j, ++ld) {
          const int st = ld % M::kV;
          ok = warp_wait(v_land + st, (ld / M::kV) & 1, abort, 143);
          if (!ok) break;
          const int keys = c.keys(j);
          if (keys & 15) {  // rows [keys, next multiple of 16): zeros, whatever the padding holds
            const int pad_rows = 16 - (keys & 15);
            if constexpr (kPair) {
              const uint32_t v0 = sbase + M::kOffV + st * M::kVBytes + (lane & 7) * 16;
              for (int rr = lane >> 3; rr < pad_rows; rr += 4) st_shared_v4(v0 + (keys + rr) * 128, 0u, 0u, 0u, 0u);
            } else {
              const uint32_t v0 = sbase + M::kOffV + st * M::kVBytes + (lane >> 3 & 1) * kHalf + (lane & 7) * 16;
              for (int rr = lane >> 4; rr < pad_rows; rr += 2) st_shared_v4(v0 + (keys + rr) * 128, 0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) {
            if constexpr (kPair)
              mbar_arrive_release_cluster(lead_bar<kPair>(v_full + st));
            else
              mbar_arrive(v_full + st);
          }
        }
      }
    } else if (lead) {
      // ------------------------------------------------------------------ MMA issuer (whole warp)
      const uint64_t dQ = smem_desc_sw128(sbase, 16, 1024);
      const uint64_t dK = smem_desc_sw128(sbase + M::kOffK, 16, 1024);     // K-major
      const uint64_t dV = smem_desc_sw128(sbase + M::kOffV, kHalf, 1024);  // MN-major
      Cur sc, pc;          // the steps whose scores and whose P V products come next
      int ks = 0, vs = 0;  // ring positions of the current units' first K stage and V entry
      int qn = 0, un = 0;  // units whose Q was taken, units whose products into O were issued
      sc.start(p, begin, end);
      sc.settle(p);
      pc = sc;
      // S of sc's step, the G-th, into the region pair of its parity; only columns that hold keys,
      // in sixteens (a pair's two-chunk step: all 256): the others are masked
      auto issue_s = [&](int G) -> bool {
        const int e = G & 1, qs = qn % M::kQ;
        if (sc.t == 0 && !wait_lead<kPair>(q_full + qs, (qn / M::kQ) & 1, abort, 150)) return false;
        const bool reuse = sc.reuse(M::kKChunks), keep = sc.keep(p, M::kKChunks);
        const int nb = sc.in_step(), loads = kPair ? 1 : nb;
        for (int b = 0; b < loads; ++b) {
          const int pos = ks + (kPair ? sc.t : 2 * sc.t + b), st = pos % M::kK;
          if (!reuse && !wait_lead<kPair>(k_full + st, (pos / M::kK) & 1, abort, 151)) return false;
          tc_fence_after();
          const uint32_t idesc = kPair ? idesc_bf16_f32(256, nb == 2 ? 256 : 2 * sc.half_columns(), 0, 0)
                                       : idesc_bf16_f32(128, (sc.keys(2 * sc.t + b) + 15) & ~15, 0, 0);
          mma_ss_128<kPair, kHalf, kHalf>(tmem + fwd::col_s(e) + 128 * b, desc_add(dQ, qs * kTile), desc_add(dK, st * kTile),
                                          idesc, 0);
          if (!keep) commit<kPair>(k_empty + st);
        }
        commit<kPair>(s_full + e);
        if (sc.last()) {
          commit<kPair>(q_empty + qs);
          ++qn;
          if (!keep) ks += kPair ? (sc.n + 1) / 2 : sc.n;
        }
        sc.next_step(p);
        return true;
      };
      bool ok = true;
      if (sc.valid()) ok = issue_s(0);
      for (int G = 0; ok && pc.valid(); ++G) {
        const int e = G & 1;
        ok = wait_lead<kPair>(s_read + e, (G >> 1) & 1, abort, 152);
        const Cur ahead = sc;  // the step after pc's
        if (ok && sc.valid()) ok = issue_s(G + 1);
        const int nb = pc.in_step();
        const bool reuse = pc.reuse(M::kVChunks), keep = pc.keep(p, M::kVChunks);
        if (ok && pc.t == 0) ok = wait_lead<kPair>(o_free, (un & 1) ^ 1, abort, 154);
        if (ok) ok = wait_lead<kPair>(p_full + e, (G >> 1) & 1, abort, 153);
        if (!ok) break;
        for (int b = 0; b < nb && ok; ++b) {
          const int pos = vs + 2 * pc.t + b, st = pos % M::kV;
          if (!reuse) ok = wait_lead<kPair>(v_full + st, (pos / M::kV) & 1, abort, 155);
          if (!ok) break;
          tc_fence_after();
          uint64_t v = desc_add(dV, st * M::kVBytes);
          fwd::opaque(v);
          const int kk_n = (pc.keys(2 * pc.t + b) + 15) >> 4;
          const bool first = pc.t == 0 && b == 0;
          const uint32_t tP = tmem + fwd::col_p(e) + 64 * b;
          if (kk_n == 8) {
            mma_ts_128<kPair, 32>(tmem + kColO, tP, v, idesc_bf16_f32(kPair ? 256 : 128, 128, 0, 1), !first);
          } else {  // the last chunk: only the sixteens that hold keys
#pragma unroll 1
            for (int kk = 0; kk < kk_n; ++kk) issue_pv<kPair>(tmem, tP + 8 * kk, desc_add(v, kk * 2048), !first || kk > 0);
          }
          if (!keep) commit<kPair>(v_empty + st);
        }
        if (!ok) break;
        commit<kPair>(o_done);
        if (pc.last()) {
          commit<kPair>(o_final);
          ++un;
          if (!keep) vs += pc.n;
        }
        pc = ahead;
      }
      // every product issued has completed before the TMEM is released
      if constexpr (kPair)
        mma_commit_pair_warp(drain, 1);
      else
        mma_commit_warp(drain);
      fwdp::drain_wait(drain, 0);
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // ------------------------------------------------------------------ softmax and output
    // Waits by parity are unambiguous: s_full[e] completes again only after this warp's s_read
    // and p_full arrivals for the step before; o_done completes once per step and o_final once
    // per unit, each again only after this warp's next p_full arrival.  A softmax warp never
    // leaves the loop early, so its partner finds it at every named barrier.
    const int i = warp >> 2, r = tid & 127, bar_id = 1 + (warp & 3);
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + kColO + 64 * i + lane_off;
    const int64_t rows = static_cast<int64_t>(p.B) * p.heads * p.Lq;
    int G = 0, un = 0, xe = 0;
    bool ok = true;
    // the unit whose output is still in TMEM
    bool pending = false;
    Unit px;  // (row: this CTA's first)
    float p_inv = 0.f, p_lse = 0.f;
    auto write_out = [&]() {  // the un-th unit's
      if constexpr (kPair) {
        if (lane == 0) tma_store_wait_read();  // the unit before has left the buffer
      }
      ok = warp_wait(o_final, un & 1, abort, 162);
      if (!ok) return;
      tc_fence_after();
      const Row y = unit_row(p, px, r);
      const int row = y.ok ? (px.b * p.heads + y.head) * p.Lq + y.q : 0;  // (rows in all fit 31 bits)
      if constexpr (kPair) {
        // through shared memory and a TMA store of the warp's 32 rows x 64 channels, 4 KB each
        const uint32_t off = M::kOffOut + warp * 4096;
        stage_o(tO, p_inv, sbase + off);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          arrive<kPair>(lead_bar<kPair>(o_free));
          const int r0 = px.row + 32 * (warp & 3);
          if (r0 < p.Lq) {  // (rows past Lq are not written)
            tma_store_5d(&tmO, smem + off, 64 * i, r0, px.g, px.kvh, px.b);
            tma_store_commit();
          }
        }
        if (i == 0 && y.ok) p.lse[row] = p_lse;
      } else {
        if (p.n_split > 1) {
          const int64_t at = px.part * rows + row;
          store_o_f32(tO, p_inv, reinterpret_cast<float4*>(p.part_o + at * 128) + 16 * i, y.ok);
          if (i == 0 && y.ok) p.part_lse[at] = p_lse;
        } else {
          const int64_t at = px.b * p.ob + (y.ok ? y.head * p.oh + y.q * p.ol : 0);
          fwd::store_o(tO, 2, p_inv, reinterpret_cast<uint4*>(p.out + at) + 8 * i, y.ok);
          if (i == 0 && y.ok) p.lse[row] = p_lse;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free);
      }
      ++un;
    };
    Cur c;
    c.start(p, begin, end);
    for (; c.valid(); c.advance(p)) {
      if (c.n == 0) {  // no keys: O = 0, LSE = ln 0
        Unit x = c.x;
        x.row += 128 * rank;
        const Row y = unit_row(p, x, r);
        if (y.ok) {
          const int64_t row = (static_cast<int64_t>(c.x.b) * p.heads + y.head) * p.Lq + y.q;
          if (p.n_split > 1) {
            // an empty part has weight 0 in the join, which does not read its values
            if (i == 0) p.part_lse[c.x.part * rows + row] = -INFINITY;
          } else {
            uint4* dst = reinterpret_cast<uint4*>(p.out + c.x.b * p.ob + y.head * p.oh + y.q * p.ol) + 8 * i;
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e] = make_uint4(0u, 0u, 0u, 0u);
            if (i == 0) p.lse[row] = -INFINITY;
          }
        }
        continue;
      }
      RowState st;
      // a warp without query rows (few rows, the last tile of a head) does no softmax: what its
      // rows of P and O hold reaches no other row (one token over 115201 + 70007 keys: 119 us
      // with all warps' exponentials in the way)
      const bool act = p.pk > 1 ? 32 * (warp & 3) < p.pk * p.Lq : c.x.row + 128 * rank + 32 * (warp & 3) < p.Lq;
      for (c.t = 0; 2 * c.t < c.n; ++c.t, ++G) {
        const int e = G & 1;
        if (ok) ok = warp_wait(s_full + e, (G >> 1) & 1, abort, 160);  // (committed to this CTA too)
        if (ok) tc_fence_after();
        bool need = false;
        const uint32_t tS = tmem + fwd::col_s(e) + lane_off, tP = tmem + fwd::col_p(e) + lane_off;
        const uint32_t loaded = lead_bar<kPair>(s_read + e);
        const bool two = c.in_step() == 2;
        const int keys = c.keys(2 * c.t + (two ? i : 0));  // of this warpgroup's chunk
        if (!act) {
          if (ok && lane == 0) arrive<kPair>(loaded);
        } else if (two && keys > 64) {
          need = softmax_step<kPair>(ok, tS + 128 * i, tP + 64 * i, loaded, p.scale_log2, st, xbuf, xe, i, r, bar_id, keys);
        } else {
          // a single chunk: this warpgroup's half of its sixteens; the second chunk, up to 64 keys
          const int n16 = two ? (keys + 15) >> 4 : (keys + 31) >> 5, first = two ? 0 : 16 * n16 * i;
          need = softmax_few<kPair>(ok, tS + (two ? 128 * i : first), tP + (two ? 64 * i : first / 2), loaded, p.scale_log2,
                                    st, xbuf, xe, i, r, bar_id, n16, keys - first);
        }
        if (ok && c.t == 0 && pending) write_out();
        if (ok && c.t > 0 && __any_sync(0xffffffffu, need)) {
          ok = warp_wait(o_done, (G - 1) & 1, abort, 161);
          if (ok) {
            tc_fence_after();
            fwd::rescale_o(tO, 2, st.alpha);
          }
        }
        if (ok) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive<kPair>(lead_bar<kPair>(p_full + e));
        }
      }
      const float l_all = act ? st.l + fwd::pair_exchange(xbuf, xe, i, r, bar_id, st.l) : 1.f;
      px = c.x;
      px.row += 128 * rank;
      p_inv = fwd::row_inverse(st.m_used, l_all);
      p_lse = fwd::row_lse(st.m_used, l_all);
      pending = true;
    }
    if (ok && pending) write_out();
    if (kPair && lane == 0) tma_store_wait_read();
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
      tmem_dealloc_pair(tmem, kTmemCols);
    else
      tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the n_part partial attentions of each row (fp32 O_j over disjoint keys, with LSE_j):
// L = ln sum_j e^LSE_j, O = sum_j e^(LSE_j - L) O_j, in part order.  A part with LSE = -inf has
// no keys, or none of any weight, and its O is not read; if all are so, O is 0 without keys and NaN
// (0 / 0) with them.  A block takes one row: 8 warps take the parts in turn, a lane four channels,
// and the warps' sums are added in warp order.
__global__ void __launch_bounds__(256) cross_merge_kernel(CrossFwdParams p) {
  __shared__ float4 acc[8][32];
  __shared__ float wsum[8], wmax[8];
  const int64_t rows = static_cast<int64_t>(p.B) * p.heads * p.Lq, row = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float m = -INFINITY;
  bool nan = false;
  for (int j = threadIdx.x; j < p.n_split; j += 256) {
    const float v = p.part_lse[j * rows + row];
    nan |= v != v;
    m = fmaxf(m, v);
  }
  if (nan) m = __int_as_float(0x7fc00000);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float v = __shfl_xor_sync(0xffffffffu, m, o);
    m = max_nan(m, v);
  }
  if (lane == 0) wmax[warp] = m;
  __syncthreads();
  m = wmax[0];
#pragma unroll
  for (int w = 1; w < 8; ++w) m = max_nan(m, wmax[w]);
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  float s = 0.f;
  if (m != -INFINITY) {
#pragma unroll 4
    for (int j = warp; j < p.n_split; j += 8) {
      const float l = p.part_lse[j * rows + row];
      if (l == -INFINITY) continue;
      const float w = __expf(l - m);
      const float4 v = reinterpret_cast<const float4*>(p.part_o + (j * rows + row) * 128)[lane];
      s += w;
      a.x = fmaf(w, v.x, a.x);
      a.y = fmaf(w, v.y, a.y);
      a.z = fmaf(w, v.z, a.z);
      a.w = fmaf(w, v.w, a.w);
    }
  }
  acc[warp][lane] = a;
  if (lane == 0) wsum[warp] = s;
  __syncthreads();
  if (warp != 0) return;
  s = 0.f;
  a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    s += wsum[w];
    a.x += acc[w][lane].x;
    a.y += acc[w][lane].y;
    a.z += acc[w][lane].z;
    a.w += acc[w][lane].w;
  }
  const int q = static_cast<int>(row % p.Lq), h = static_cast<int>(row / p.Lq % p.heads), b = static_cast<int>(row / p.Lq / p.heads);
  const bool none = m == -INFINITY && crossf::kv_length(p, b) == 0;
  const float inv = none ? 0.f : 1.f / s;
  reinterpret_cast<uint2*>(p.out + b * p.ob + h * p.oh + q * p.ol)[lane] =
      make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
  if (lane == 0) p.lse[row] = fabsf(m) < INFINITY ? m + __logf(s) : m;
}

}  // namespace dsa
