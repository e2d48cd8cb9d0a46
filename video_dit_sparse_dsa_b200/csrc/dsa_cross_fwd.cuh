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
// Persistent, warp-specialised, one CTA per SM.  A unit is 128 query rows of one kv head over a
// range of its key chunks (128 keys); it runs in steps of up to two chunks.  Roles:
//   warp 8   TMA producer of K (4-entry ring of 32 KB chunks)
//   warp 10  TMA producer of V (2 entries)
//   warp 11  TMA producer of Q (the next unit's, once the last scores of this one are done)
//   warp 9   MMA issuer: the scores of step G + 1, which may be the next unit's first, as soon
//            as the softmax warps hold those of step G in registers, then O += P(G) V(G)
//   warps 0-7  softmax: warpgroup i takes the step's chunk i (a single chunk: its half i), a
//            thread per query row; the two threads of a row agree on the row max through shared
//            memory.
// The pipeline does not drain between units: a unit's output is read out of TMEM, divided and
// written during the next unit's first step, after that step's P is stored and before it is
// handed over (the products of that step overwrite O), when the last product of the unit has
// long finished.
// K of up to 512 keys and V of up to 256 stay in shared memory for every consecutive unit of
// their kv head (the CTA's units are a contiguous range of the unit sequence): no reloads.
// Units are cut into ranges of equal cost over the CTAs (batch entries have their own lengths).
// Few query rows over many keys (a single token over every state): up to 128 / Lq heads of a kv
// head are packed into a unit, so K and V are read once for them, and the keys are cut into
// parts, one unit each, whose fp32 partial outputs cross_merge_kernel joins by their LSEs.
//
// TMEM (512 columns): as the window forward: regions R0 R1 R2 of 128 columns that scores and P
// rotate through (even steps: S in R0 R1, P in R0; odd: S in R1 R2, P in R2), O in the fourth.
#pragma once

#include <stdint.h>

#include "dsa_fwd_bf16.cuh"
#include "sm100.cuh"

namespace dsa {

struct CrossFwdParams {
  const int32_t* kv_len;  // [B] valid keys of each batch entry, or null: Lk
  __nv_bfloat16* out;
  int64_t ob, oh, ol;     // strides of out in elements
  float* lse;             // [B, heads, Lq]
  float* part_o;          // n_split > 1: [n_split, B * heads * Lq, 128] and [n_split, B * heads * Lq]
  float* part_lse;
  int B, heads, kv_heads, group, Lq, Lk;
  int pk;                 // heads packed into a unit (Lq * pk <= 128), or 1
  int tiles;              // units per kv head and part
  int n_split;
  int n_units;            // B * kv_heads * n_split * tiles
  uint32_t q_bytes;       // bytes a unit's Q boxes load
  int qb, qk, qg, kb, kh, vb, vh;  // 1, or 0 for a broadcast (stride 0) dimension
  float scale_log2;
};

namespace crossf {
constexpr int kThreads = 384;
constexpr int kKWarp = 8, kMmaWarp = 9, kVWarp = 10, kQWarp = 11;
constexpr int kRegsSoftmax = 216, kRegsAux = 72;
constexpr int kRegsAtLaunch = (2 * 128 * kRegsSoftmax + 128 * kRegsAux) / kThreads;  // 168
static_assert(kRegsAtLaunch * kThreads == 2 * 128 * kRegsSoftmax + 128 * kRegsAux, "split must use the launch registers");
constexpr int kKStages = 4, kVStages = 2;
constexpr uint32_t kTile = 128 * 128 * 2, kHalf = kTile / 2;  // 128 rows x 128 channels; 64 channels
constexpr uint32_t kOffQ = 0, kOffK = kTile, kOffV = kOffK + kKStages * kTile;
constexpr uint32_t kOffBar = kOffV + kVStages * kTile;
constexpr uint32_t kOffX = kOffBar + 256;
constexpr uint32_t kSmemUsed = kOffX + 2 * 2 * 128 * 4;
constexpr uint32_t kSmemBytes = 227 * 1024;
static_assert(kSmemUsed <= kSmemBytes, "shared memory layout too large");
constexpr uint32_t kTmemCols = 512, kColO = 384;
constexpr uint32_t kIdescPV = idesc_bf16_f32(128, 128, 0, 1);
constexpr float kRescaleThreshold = 8.0f;  // log2 units: P <= 256, as in the window forward
// column pairs (bit e of the 8 pairs of every 16 columns) whose 2^x runs on the FMA pipe
constexpr uint32_t kPolyMask = 0x22u;

__device__ __forceinline__ int kv_length(const CrossFwdParams& p, int b) {
  return p.kv_len == nullptr ? p.Lk : min(max(__ldg(p.kv_len + b), 0), p.Lk);
}

// Chunks per part of a sequence of `chunks`: even, so that parts are whole steps.
__device__ __forceinline__ int chunks_per_part(const CrossFwdParams& p, int chunks) {
  const int per = (chunks + p.n_split - 1) / p.n_split;
  return p.n_split > 1 ? (per + 1) & ~1 : per;
}

// The CTA's units [begin, end): the sequence is cut at equal cost, a unit costing its chunks and
// a constant (about half a chunk's) for its own start and end.
__device__ __forceinline__ int64_t unit_cost(const CrossFwdParams& p, int b) {
  return 2 * static_cast<int64_t>(chunks_per_part(p, (kv_length(p, b) + 127) / 128)) + 1;
}

__device__ __forceinline__ void unit_range(const CrossFwdParams& p, int cta, int n_cta, int& begin, int& end) {
  const int64_t per_b = static_cast<int64_t>(p.kv_heads) * p.n_split * p.tiles;
  int64_t total = 0;
  for (int b = 0; b < p.B; ++b) total += per_b * unit_cost(p, b);
  const int64_t x0 = total * cta / n_cta, x1 = total * (cta + 1) / n_cta;
  int64_t acc = 0;
  begin = end = p.n_units;
  bool b0 = false, b1 = false;
  for (int b = 0; b < p.B; ++b) {
    const int64_t c = unit_cost(p, b), next = acc + per_b * c;
    if (!b0 && x0 < next) {
      begin = static_cast<int>(b * per_b + (x0 - acc + c - 1) / c);
      b0 = true;
    }
    if (!b1 && x1 < next) {
      end = static_cast<int>(b * per_b + (x1 - acc + c - 1) / c);
      b1 = true;
    }
    acc = next;
  }
}

// A unit: 128 rows from `row` of head g of a kv head's group (pk > 1: pk heads' rows from head
// g), over part `part` of the keys.
struct Unit {
  int b, kvh, part, g, row;
};

// Walks the CTA's units [begin, end) and their steps.  Consecutive units are neighbours in the
// sequence (row, head in the group, part, kv head, batch), so moving on needs no division.
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
  // Keys present in the unit's chunk j.
  __device__ __forceinline__ int keys(int j) const { return min(len - 128 * (c0 + j), 128); }
  // The unit's K (or V) chunks are still in the `stages` ring entries that the previous unit
  // used; the next unit will find them there too.
  __device__ __forceinline__ bool reuse(int stages) const { return same && n <= stages; }
  __device__ __forceinline__ bool keep(const CrossFwdParams& p, int stages) const {
    return n <= stages && u + 1 < end && (x.row + 128 < p.Lq || x.g + p.pk < p.group);
  }

  __device__ __forceinline__ void start(const CrossFwdParams& p, int begin, int end_) {
    u = begin;
    end = end_;
    const int tile = u % p.tiles, slice = u / p.tiles;
    if (p.pk > 1) {
      x.g = tile * p.pk;
      x.row = 0;
    } else {
      const int per_head = (p.Lq + 127) / 128;
      x.g = tile / per_head;
      x.row = 128 * (tile % per_head);
    }
    x.part = slice % p.n_split;
    x.kvh = slice / p.n_split % p.kv_heads;
    x.b = slice / p.n_split / p.kv_heads;
    same = false;
    t = 0;
    if (valid()) chunks(p);
  }
  __device__ __forceinline__ void chunks(const CrossFwdParams& p) {
    len = kv_length(p, x.b);
    const int all = (len + 127) / 128, per = chunks_per_part(p, all);
    c0 = x.part * per;
    n = max(min(per, all - c0), 0);
  }
  // The next unit, with or without keys.
  __device__ __forceinline__ void advance(const CrossFwdParams& p) {
    ++u;
    t = 0;
    same = true;
    x.row += 128;
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
  __device__ __forceinline__ void settle(const CrossFwdParams& p) {
    while (valid() && n == 0) advance(p);
  }
  __device__ __forceinline__ void next_unit(const CrossFwdParams& p) {
    advance(p);
    settle(p);
  }
  __device__ __forceinline__ void next_step(const CrossFwdParams& p) {
    if (last())
      next_unit(p);
    else
      ++t;
  }
};

// 2^x for a pair on the FMA pipe: as exp2_poly2, with a quartic for 2^f (minimax fit on
// [-0.5, 0.5], relative error 2.6e-6), because the row sums also give the fp32 LSE.
__device__ __forceinline__ void exp2_quartic2(float x0, float x1, float& y0, float& y1) {
  constexpr float kRound = 12582912.0f;  // 1.5 * 2^23
  constexpr float c0 = 0.9999992847442627f, c1 = 0.6931217908859253f, c2 = 0.240247443318367f,
                  c3 = 0.05591785907745361f, c4 = 0.009570101276040077f;
  x0 = fmaxf(x0, -126.f);
  x1 = fmaxf(x1, -126.f);
  float t0, t1, n0, n1, f0, f1, q0, q1;
  fadd2(t0, t1, x0, x1, kRound, kRound);
  fadd2(n0, n1, t0, t1, -kRound, -kRound);
  ffma2(f0, f1, n0, n1, -1.f, -1.f, x0, x1);
  ffma2(q0, q1, c4, c4, f0, f1, c3, c3);
  ffma2(q0, q1, q0, q1, f0, f1, c2, c2);
  ffma2(q0, q1, q0, q1, f0, f1, c1, c1);
  ffma2(q0, q1, q0, q1, f0, f1, c0, c0);
  y0 = __int_as_float(__float_as_int(q0) + (__float_as_int(t0) << 23));
  y1 = __int_as_float(__float_as_int(q1) + (__float_as_int(t1) << 23));
}

// One step's softmax for this thread's NC score columns at tS: agrees on the row max with the
// partner thread, writes P as packed bf16 at tP, updates the reference max and the row sum, and
// returns whether the reference moved (alpha: the factor that the old O and l take).  Columns
// from nvalid on hold no key.  With !ok (an earlier wait failed) the thread only takes part in
// the exchange.
template <int NC>
__device__ __forceinline__ bool softmax_step(bool ok, uint32_t tS, uint32_t tP, uint64_t* loaded, float scale_log2,
                                             float& m_used, float& l, float& alpha, float* xbuf, int& xe, int i, int r,
                                             int bar_id, int nvalid) {
  uint32_t s[NC];
  if constexpr (NC == 128)
    tmem_ld128_wait(tS, s);
  else
    tmem_ld64_wait(tS, s);
  if (nvalid < NC) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (c >= nvalid) s[c] = 0xff800000u;
  }
  if (ok) {
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(loaded);
  }
  float mxs[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    mxs[e] = fmaxf(__uint_as_float(s[e]), __uint_as_float(s[NC - 8 + e]));
#pragma unroll
    for (int c = 8 + e; c < NC - 8; c += 16)
      mxs[e] = max3f(mxs[e], __uint_as_float(s[c]), __uint_as_float(s[c + 8]));
  }
  float mx = max3f(max3f(mxs[0], mxs[1], mxs[2]), max3f(mxs[3], mxs[4], mxs[5]), fmaxf(mxs[6], mxs[7]));
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
  const float neg_m = -m_used;
  float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int g = 0; g < NC / 16; ++g) {
    uint32_t pk[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float x0, x1, p0, p1;
      ffma2(x0, x1, __uint_as_float(s[16 * g + 2 * e]), __uint_as_float(s[16 * g + 2 * e + 1]), scale_log2, scale_log2,
            neg_m, neg_m);
      if ((kPolyMask >> e) & 1u) {
        exp2_quartic2(x0, x1, p0, p1);
      } else {
        p0 = ex2_approx(x0);
        p1 = ex2_approx(x1);
      }
      fadd2(sa[e & 3], sb[e & 3], sa[e & 3], sb[e & 3], p0, p1);
      pk[e] = pack_bf16x2(p0, p1);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s[8 * g + e] = pk[e];
  }
  l += ((sa[0] + sb[0]) + (sa[1] + sb[1])) + ((sa[2] + sb[2]) + (sa[3] + sb[3]));
#pragma unroll
  for (int h = 0; h < NC / 64; ++h) {
    uint32_t w[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) w[e] = s[32 * h + e];
    tmem_st32(tP + 32 * h, w);
  }
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

// Writes a warp's 32 rows x 64 channels of O, from TMEM times inv (of the lane's own row), as
// bf16 to rows dst + r * ld, r < n_rows.  A lane holds one row as eight 16-byte vectors; three
// exchanges within groups of 8 lanes transpose them, so that 8 lanes write one row's 128 bytes
// together: stores of a lane's own vectors, 32 rows to an instruction, took 22 of 90 us of the
// 77-key and 86 of 343 us of the 203 + 512-key workload.
__device__ __forceinline__ void store_o_rows(uint32_t tO, float inv, __nv_bfloat16* dst, int64_t ld, int n_rows) {
  const int lane = threadIdx.x & 31;
  uint32_t w[8][4];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    uint32_t o[32];
    tmem_ld32_wait(tO + 32 * g, o);
#pragma unroll
    for (int e = 0; e < 16; ++e)
      w[4 * g + e / 4][e % 4] = pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
  }
#pragma unroll
  for (int k = 1; k < 8; k <<= 1) {
    const bool hi = lane & k;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (c & k) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? w[c][e] : w[c | k][e], k);
        if (hi)
          w[c][e] = got;
        else
          w[c | k][e] = got;
      }
    }
  }
  // w[i]: vector (lane & 7) of row (lane & ~7) + i
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = (lane & ~7) + i;
    if (r < n_rows)
      *(reinterpret_cast<uint4*>(dst + r * ld) + (lane & 7)) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
  }
}

// Query row of thread r in a unit: its head and position, or no row.
struct Row {
  bool ok;
  int head, q;
};

__device__ __forceinline__ Row unit_row(const CrossFwdParams& p, const Unit& x, int r) {
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

__global__ void __launch_bounds__(crossf::kThreads, 1)
    cross_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, CrossFwdParams p) {
  using namespace crossf;
  using fwd::desc_add;
  using fwd::warp_wait;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
  if (pad + kSmemUsed > kSmemBytes) {  // uniform over the CTA: nothing has started yet
    if (threadIdx.x == 0) device_report(DSA_DEV_BOUNDS, 5);
    return;
  }
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw + pad;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* q_full = bars;
  uint64_t* q_empty = bars + 1;
  uint64_t* k_full = bars + 2;              // [kKStages]
  uint64_t* k_empty = k_full + kKStages;
  uint64_t* v_full = k_empty + kKStages;    // [kVStages]
  uint64_t* v_empty = v_full + kVStages;
  uint64_t* s_full = v_empty + kVStages;    // [2] scores of a step of parity e ready
  uint64_t* s_read = s_full + 2;            // [2] loaded by the softmax warps (8)
  uint64_t* p_full = s_full + 4;            // [2] P of a step of parity e written (8)
  uint64_t* o_done = s_full + 6;            // the products of a step into O done
  uint64_t* o_final = s_full + 7;           // the products of a unit done
  uint64_t* o_free = s_full + 8;            // O of a unit read out (8)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_full + 9);
  volatile int* abort = reinterpret_cast<volatile int*>(s_full + 10);
  int* range = reinterpret_cast<int*>(s_full + 11);  // [2]
  static_assert(2 * (1 + kKStages + kVStages) + 12 <= 256 / 8, "barriers must fit their 256 bytes");
  float* xbuf = reinterpret_cast<float*>(smem + kOffX);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    tma_prefetch_map(&tmQ);
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(k_full + s, 1);
      mbar_init(k_empty + s, 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(v_full + s, 1);
      mbar_init(v_empty + s, 1);
    }
    for (int e = 0; e < 2; ++e) {
      mbar_init(s_full + e, 1);
      mbar_init(s_read + e, 8);
      mbar_init(p_full + e, 8);
    }
    mbar_init(o_done, 1);
    mbar_init(o_final, 1);
    mbar_init(o_free, 8);
    *abort = 0;
    fence_mbar_init();
    int b, e;
    unit_range(p, blockIdx.x, gridDim.x, b, e);
    range[0] = b;
    range[1] = e;
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int begin = range[0], end = range[1];

  if (warp >= 8) {
    setmaxnreg_dec<kRegsAux>();
    if (warp == kQWarp) {
      // ------------------------------------------------------------------ TMA producer of Q
      if (lane == 0) {
        Cursor c;
        c.start(p, begin, end);
        int n = 0;
        for (c.settle(p); c.valid(); c.next_unit(p), ++n) {
          if (!mbar_wait(q_empty, (n & 1) ^ 1, abort, 140)) break;
          mbar_arrive_expect_tx(q_full, p.q_bytes);
          tma_load_5d(smem + kOffQ, &tmQ, q_full, 0, c.x.row, c.x.g * p.qg, c.x.kvh * p.qk, c.x.b * p.qb);
          tma_load_5d(smem + kOffQ + kHalf, &tmQ, q_full, 64, c.x.row, c.x.g * p.qg, c.x.kvh * p.qk, c.x.b * p.qb);
        }
      }
    } else if (warp == kKWarp || warp == kVWarp) {
      // ------------------------------------------------------------------ TMA producers of K and V
      if (lane == 0) {
        const bool is_k = warp == kKWarp;
        const CUtensorMap* map = is_k ? &tmK : &tmV;
        const int stages = is_k ? kKStages : kVStages;
        uint64_t* full0 = is_k ? k_full : v_full;
        uint64_t* empty0 = is_k ? k_empty : v_empty;
        uint8_t* base = smem + (is_k ? kOffK : kOffV);
        Cursor c;
        int ld = 0;
        bool ok = true;
        c.start(p, begin, end);
        for (c.settle(p); ok && c.valid(); c.next_unit(p)) {
          if (c.reuse(stages)) continue;  // still in shared memory
          const int head = c.x.kvh * (is_k ? p.kh : p.vh), b = c.x.b * (is_k ? p.kb : p.vb);
          for (int j = 0; j < c.n; ++j, ++ld) {
            const int st = ld % stages;
            ok = mbar_wait(empty0 + st, ((ld / stages) & 1) ^ 1, abort, is_k ? 141 : 142);
            if (!ok) break;
            mbar_arrive_expect_tx(full0 + st, kTile);
            tma_load_4d(base + st * kTile, map, full0 + st, 0, 128 * (c.c0 + j), head, b);
            tma_load_4d(base + st * kTile + kHalf, map, full0 + st, 64, 128 * (c.c0 + j), head, b);
          }
        }
      }
    } else {
      // ------------------------------------------------------------------ MMA issuer (whole warp)
      const uint64_t dQ = smem_desc_sw128(sbase + kOffQ, 16, 1024);
      const uint64_t dK = smem_desc_sw128(sbase + kOffK, 16, 1024);     // K-major
      const uint64_t dV = smem_desc_sw128(sbase + kOffV, kHalf, 1024);  // MN-major
      Cursor sc, pc;   // the steps whose scores and whose P V products come next
      int ks = 0, vs = 0;  // ring positions of the current units' first chunks
      int qn = 0;          // units whose Q was taken
      int un = 0;          // units whose products into O were issued
      sc.start(p, begin, end);
      sc.settle(p);
      pc = sc;
      // S of sc's step, the G-th, into the region pair of its parity
      auto issue_s = [&](int G) -> bool {
        const int e = G & 1;
        if (sc.t == 0 && !warp_wait(q_full, qn & 1, abort, 150)) return false;
        const int nb = sc.in_step();
        const bool reuse = sc.reuse(kKStages), keep = sc.keep(p, kKStages);
        for (int b = 0; b < nb; ++b) {
          const int pos = ks + 2 * sc.t + b, st = pos % kKStages;
          if (!reuse && !warp_wait(k_full + st, (pos / kKStages) & 1, abort, 151)) return false;
          tc_fence_after();
          // only the columns that hold keys, in sixteens: the others are masked
          const uint32_t idesc = idesc_bf16_f32(128, (sc.keys(2 * sc.t + b) + 15) & ~15, 0, 0);
          uint64_t q = dQ, k = desc_add(dK, st * kTile);
          fwd::opaque(q);
          fwd::opaque(k);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ss_warp(tmem + fwd::col_s(e) + 128 * b, desc_add(q, (kk >> 2) * kHalf + (kk & 3) * 32),
                        desc_add(k, (kk >> 2) * kHalf + (kk & 3) * 32), idesc, kk > 0);
          if (!keep) mma_commit_warp(k_empty + st);
        }
        mma_commit_warp(s_full + e);
        if (sc.last()) {
          mma_commit_warp(q_empty);
          ++qn;
          if (!keep) ks += sc.n;
        }
        sc.next_step(p);
        return true;
      };
      bool ok = true;
      if (sc.valid()) ok = issue_s(0);
      for (int G = 0; ok && pc.valid(); ++G) {
        const int e = G & 1;
        ok = warp_wait(s_read + e, (G >> 1) & 1, abort, 152);
        if (ok && sc.valid()) ok = issue_s(G + 1);
        if (ok) ok = warp_wait(p_full + e, (G >> 1) & 1, abort, 153);
        if (ok && pc.t == 0) ok = warp_wait(o_free, (un & 1) ^ 1, abort, 154);
        if (!ok) break;
        const int nb = pc.in_step();
        const bool reuse = pc.reuse(kVStages), keep = pc.keep(p, kVStages);
        for (int b = 0; b < nb && ok; ++b) {
          const int pos = vs + 2 * pc.t + b, st = pos % kVStages;
          const int keys = pc.keys(2 * pc.t + b);
          if (!reuse) {
            ok = warp_wait(v_full + st, (pos / kVStages) & 1, abort, 155);
            if (!ok) break;
            if (keys & 15) {
              // rows past the last key up to the next multiple of 16 meet P = 0 in the product:
              // zeros there, whatever the padding holds (0 * NaN is NaN)
              const int pad_rows = 16 - (keys & 15);
              const uint32_t v0 = sbase + kOffV + st * kTile + (lane >> 3 & 1) * kHalf + (lane & 7) * 16;
              for (int rr = lane >> 4; rr < pad_rows; rr += 2) st_shared_v4(v0 + (keys + rr) * 128, 0u, 0u, 0u, 0u);
              fence_proxy_async_smem();
              __syncwarp();
            }
          }
          tc_fence_after();
          uint64_t v = desc_add(dV, st * kTile);
          fwd::opaque(v);
          const int kk_n = (keys + 15) >> 4;
          const bool first = pc.t == 0 && b == 0;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            if (kk < kk_n)
              mma_ts_warp(tmem + kColO, tmem + fwd::col_p(e) + 64 * b + 8 * kk, desc_add(v, kk * 2048), kIdescPV,
                          !first || kk > 0);
          if (!keep) mma_commit_warp(v_empty + st);
        }
        if (!ok) break;
        mma_commit_warp(o_done);
        if (pc.last()) {
          mma_commit_warp(o_final);
          ++un;
          if (!keep) vs += pc.n;
        }
        pc.next_step(p);
      }
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
    Unit px;
    float p_inv = 0.f, p_lse = 0.f;
    auto write_out = [&]() {  // the un-th unit's
      ok = warp_wait(o_final, un & 1, abort, 162);
      if (!ok) return;
      tc_fence_after();
      const Row y = unit_row(p, px, r);
      const int64_t row = (static_cast<int64_t>(px.b) * p.heads + (y.ok ? y.head : 0)) * p.Lq + (y.ok ? y.q : 0);
      if (p.n_split > 1) {
        const int64_t at = px.part * rows + row;
        store_o_f32(tO, p_inv, reinterpret_cast<float4*>(p.part_o + at * 128) + 16 * i, y.ok);
        if (i == 0 && y.ok) p.part_lse[at] = p_lse;
      } else {
        if (p.pk > 1) {
          const int64_t at = px.b * p.ob + (y.ok ? y.head * p.oh + y.q * p.ol : 0);
          fwd::store_o(tO, 2, p_inv, reinterpret_cast<uint4*>(p.out + at) + 8 * i, y.ok);
        } else {
          const int r0 = px.row + (r & ~31);  // the warp's first row
          store_o_rows(tO, p_inv, p.out + px.b * p.ob + y.head * p.oh + r0 * p.ol + 64 * i, p.ol, p.Lq - r0);
        }
        if (i == 0 && y.ok) p.lse[row] = p_lse;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
      ++un;
    };
    Cursor c;
    c.start(p, begin, end);
    for (; c.valid(); c.advance(p)) {
      if (c.n == 0) {  // no keys: O = 0, LSE = ln 0
        const Row y = unit_row(p, c.x, r);
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
      float m_used = -INFINITY, l = 0.f;
      for (c.t = 0; 2 * c.t < c.n; ++c.t, ++G) {
        const int e = G & 1;
        if (ok) ok = warp_wait(s_full + e, (G >> 1) & 1, abort, 160);
        if (ok) tc_fence_after();
        float alpha;
        bool need;
        if (c.in_step() == 2)
          need = softmax_step<128>(ok, tmem + fwd::col_s(e) + 128 * i + lane_off, tmem + fwd::col_p(e) + 64 * i + lane_off,
                                   s_read + e, p.scale_log2, m_used, l, alpha, xbuf, xe, i, r, bar_id,
                                   c.keys(2 * c.t + i));
        else
          need = softmax_step<64>(ok, tmem + fwd::col_s(e) + 64 * i + lane_off, tmem + fwd::col_p(e) + 32 * i + lane_off,
                                  s_read + e, p.scale_log2, m_used, l, alpha, xbuf, xe, i, r, bar_id,
                                  min(max(c.keys(2 * c.t) - 64 * i, 0), 64));
        if (ok && c.t == 0 && pending) write_out();
        if (ok && c.t > 0 && __any_sync(0xffffffffu, need)) {
          ok = warp_wait(o_done, (G - 1) & 1, abort, 161);
          if (ok) {
            tc_fence_after();
            fwd::rescale_o(tO, 2, alpha);
          }
        }
        if (ok) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full + e);
        }
      }
      const float l_all = l + fwd::pair_exchange(xbuf, xe, i, r, bar_id, l);
      px = c.x;
      p_inv = 1.f / l_all;
      p_lse = (m_used + __log2f(l_all)) * 0.69314718055994531f;
      pending = true;
    }
    if (ok && pending) write_out();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the n_part partial attentions of each row (fp32 O_j over disjoint keys, with LSE_j):
// L = ln sum_j e^LSE_j, O = sum_j e^(LSE_j - L) O_j, in part order.  A part with LSE = -inf has
// no keys and its O is not read.  A block takes one row: 8 warps take the parts in turn, a lane
// four channels, and the warps' sums are added in warp order.
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
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(m), "f"(v));
  }
  if (lane == 0) wmax[warp] = m;
  __syncthreads();
  m = wmax[0];
#pragma unroll
  for (int w = 1; w < 8; ++w) asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(m), "f"(wmax[w]));
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
  const bool none = m == -INFINITY;
  const float inv = none ? 0.f : 1.f / s;
  const int q = static_cast<int>(row % p.Lq), h = static_cast<int>(row / p.Lq % p.heads), b = static_cast<int>(row / p.Lq / p.heads);
  reinterpret_cast<uint2*>(p.out + b * p.ob + h * p.oh + q * p.ol)[lane] =
      make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
  if (lane == 0) p.lse[row] = none ? -INFINITY : m + __logf(s);
}

}  // namespace dsa
