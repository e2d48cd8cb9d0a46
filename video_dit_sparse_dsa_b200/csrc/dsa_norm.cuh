// Root-mean-square norm of rows, with the addition of a residual before it, in the type of
// its input or in 8 bits (e4m3) with a scale for every 128 channels, and its backward.
//
//   h = x + r,   y_c = w_c h_c / sqrt(mean_c h_c^2 + eps)
//   8 bits: s_g = max_{c in g} |y_c| / 448 over each group g of 128 channels, y8_c = rn(y_c / s_g)
//   backward, with rho = 1 / sqrt(mean h^2 + eps) and g = w dy:
//     dx = rho g - h rho^3 mean_c(g_c h_c) + dh,   dw_c = sum over rows of dy_c h_c rho
//
// Everything between the loads and the one rounding of each output is fp32: y is taken from
// the unrounded sum x + r, which is also what h rounds.
//
// Bound by memory: a row is read once, kept in registers (kVec = 8 consecutive channels per
// thread and vector, NV vectors per thread, tpr threads per row: whole warps, or 16 lanes up to
// 128 channels) while its sums are taken, and written from there.  C channels are ceil(C / 8)
// vectors; vector i * tpr + t belongs to thread t of the row, so a warp's loads are contiguous and
// a group of 128 channels is 16 consecutive lanes.  Rows whose address, length or stride is not a
// multiple of 16 bytes go through the same kernel with element-wise loads (kAligned = false; about
// a quarter of the rate: 40000 x 1537 bf16 with a residual 295 us, 1.7 TB/s, backward with dh 330).
// Times of one call with L2 flushed, and the share of a copy's rate: bf16 with a residual, 71680 x
// 1536: 133 us, 100%; to e4m3 150, 79%; 35840 x 5120 to e4m3: 244, 81%; 860160 x 128 without a
// residual: 88, 77%; fp32 with a residual, 35840 x 1536: 135, 100%.  Backward, bf16 with dh, 35840 x
// 5120: 256, 88%; 860160 x 128 without: 149, 68%; fp32 with dh, 35840 x 1536: 146, 92%; 17920 x 5120
// (too wide for the ring, read twice): 235, 96%.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "sm100.cuh"

namespace dsa {
namespace norm {

constexpr int kVec = 8;        // channels per vector
constexpr int kMaxNV = 4;      // vectors per thread
constexpr int kMaxWarps = 16;  // warps per row: C <= 16 * 32 * 4 * 8 = 16384
constexpr int kMaxC = kMaxWarps * 32 * kMaxNV * kVec;
constexpr int kMaxRows = 8;    // rows of several warps per block
constexpr int kGroup = 128;    // channels per 8-bit scale
constexpr int kMaxStages = 4;  // of the backward's ring
constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126: the reciprocal of a scale stays finite

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& d, float x) { d = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }

// Eight consecutive channels as loaded (bf16: 4 registers, fp32: 8), and as fp32 values.
template <typename T>
struct Raw8 {
  uint32_t u[2 * sizeof(T)];
};

// Channels [c, c + 8) of a row of C (past the end: zeros).
template <bool kAligned, typename T>
__device__ __forceinline__ void load_raw(const T* row, int c, int C, Raw8<T>& v) {
  if constexpr (kAligned) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
      const uint4 x = reinterpret_cast<const uint4*>(row + c)[i];
      v.u[4 * i] = x.x;
      v.u[4 * i + 1] = x.y;
      v.u[4 * i + 2] = x.z;
      v.u[4 * i + 3] = x.w;
    }
  } else if constexpr (sizeof(T) == 2) {
    const uint16_t* r = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = c + 2 * e < C ? r[c + 2 * e] : 0u, hi = c + 2 * e + 1 < C ? r[c + 2 * e + 1] : 0u;
      v.u[e] = lo | (hi << 16);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v.u[e] = c + e < C ? __float_as_uint(row[c + e]) : 0u;
  }
}

template <typename T>
__device__ __forceinline__ void zero_raw(Raw8<T>& v) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(2 * sizeof(T)); ++i) v.u[i] = 0u;
}

template <typename T>
__device__ __forceinline__ void expand(const Raw8<T>& r, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (sizeof(T) == 2)
      v[e] = __uint_as_float(e & 1 ? r.u[e >> 1] & 0xffff0000u : r.u[e >> 1] << 16);
    else
      v[e] = __uint_as_float(r.u[e]);
  }
}

template <bool kAligned, typename T>
__device__ __forceinline__ void load8(const T* row, int c, int C, float (&v)[8]) {
  Raw8<T> r;
  load_raw<kAligned>(row, c, C, r);
  expand(r, v);
}

template <bool kAligned>
__device__ __forceinline__ void store8(__nv_bfloat16* row, int c, int C, const float (&v)[8]) {
  if constexpr (kAligned) {
    uint32_t u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
      u[e] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(row + c) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < C) from_f(row[c + e], v[e]);
  }
}

template <bool kAligned>
__device__ __forceinline__ void store8(float* row, int c, int C, const float (&v)[8]) {
  if constexpr (kAligned) {
    reinterpret_cast<float4*>(row + c)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(row + c)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < C) row[c + e] = v[e];
  }
}

// The weight's channels, or ones.
template <bool kAligned, typename T>
__device__ __forceinline__ void load_weight(const T* w, int c, int C, float (&v)[8]) {
  if (w != nullptr) {
    load8<kAligned>(w, c, C, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 1.f;
  }
}

// Eight values as e4m3 (round to nearest even, saturating; NaN stays NaN).
template <bool kAligned>
__device__ __forceinline__ void store8_e4m3(uint8_t* row, int c, int C, const float (&v)[8]) {
  uint32_t u[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h], v[4 * h + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h + 2], v[4 * h + 3]), __NV_SATFINITE, __NV_E4M3);
    u[h] = lo | (hi << 16);
  }
  if constexpr (kAligned) {
    *reinterpret_cast<uint2*>(row + c) = make_uint2(u[0], u[1]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < C) row[c + e] = static_cast<uint8_t>(u[e >> 2] >> (8 * (e & 3)));
  }
}

// Sum over the lanes of a row within a warp (16 or 32).
__device__ __forceinline__ float lane_sum(float s, int tpr) {
  if (tpr > 16) s += __shfl_xor_sync(0xffffffffu, s, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// One sum per warp of a row: rows of kMaxWarps floats, those that no warp writes zero.
using Slots = float[kMaxRows][kMaxWarps];

__device__ __forceinline__ void clear_slots(Slots& s) {
  for (int i = threadIdx.x; i < kMaxRows * kMaxWarps; i += blockDim.x) (&s[0][0])[i] = 0.f;
}

// The sum over a row's warps, in order (four at a time; a loop over the warps took longer than
// the rest of the reduction).
__device__ __forceinline__ float slot_sum(const float (&s)[kMaxWarps]) {
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxWarps / 4; ++i) {
    const float4 v = reinterpret_cast<const float4*>(s)[i];
    t += (v.x + v.y) + (v.z + v.w);
  }
  return t;
}
}  // namespace norm

struct NormParams {
  const void* x;
  const void* r;   // residual or null
  const void* w;   // [C] or null (ones)
  void* y;         // [rows, C]: the input's type, or e4m3
  void* h;         // [rows, C] x + r (with a residual)
  float* scales;   // 8 bits: [rows, ceil(C / 128)]
  int64_t rows, x_ld, r_ld;  // row strides of x and r in elements; y and h are contiguous
  int C, tpr;      // tpr threads per row
  float eps;
};

// A block takes blockDim / tpr rows.
template <typename T, int NV, bool kAligned, bool kFp8>
__global__ void __launch_bounds__(512) rmsnorm_kernel(NormParams p) {
  using namespace norm;
  __shared__ __align__(16) Slots slot;
  const int tpr = p.tpr, t = threadIdx.x % tpr;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
  const bool live = row < p.rows;
  const int64_t row0 = live ? row : 0;
  const T* x = static_cast<const T*>(p.x) + row0 * p.x_ld;
  const T* r = p.r != nullptr ? static_cast<const T*>(p.r) + row0 * p.r_ld : nullptr;
  if (tpr > 32) {
    clear_slots(slot);
    __syncthreads();
  }
  // every load of the row before its first store: h may be the residual's or x's own buffer, so
  // the compiler keeps loads behind stores
  Raw8<T> xr[NV], rr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = kVec * (i * tpr + t);
    zero_raw(xr[i]);
    if (live && c < p.C) load_raw<kAligned>(x, c, p.C, xr[i]);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = kVec * (i * tpr + t);
    zero_raw(rr[i]);
    if (r != nullptr && live && c < p.C) load_raw<kAligned>(r, c, p.C, rr[i]);
  }
  float v[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    expand(xr[i], v[i]);
    if (r != nullptr) {
      const int c = kVec * (i * tpr + t);
      float a[8];
      expand(rr[i], a);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] += a[e];
      if (live && c < p.C) store8<kAligned>(static_cast<T*>(p.h) + row * p.C, c, p.C, v[i]);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e], v[i][e], ss);
  }
  ss = lane_sum(ss, tpr);
  if (tpr > 32) {
    if ((threadIdx.x & 31) == 0) slot[threadIdx.x / tpr][t >> 5] = ss;
    __syncthreads();
    ss = slot_sum(slot[threadIdx.x / tpr]);
  }
  const float rho = rsqrtf(ss / static_cast<float>(p.C) + p.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = kVec * (i * tpr + t);
    const bool in = live && c < p.C;
    float y[8];
    if (in && p.w != nullptr) {
      float w[8];
      load8<kAligned>(static_cast<const T*>(p.w), c, p.C, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = v[i][e] * rho * w[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = v[i][e] * rho;  // past the end: 0
    }
    if constexpr (kFp8) {
      // a group's 16 vectors are 16 consecutive lanes of one warp
      float m = 0.f;
      if (in) {
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max_nan(m, c + e < p.C ? fabsf(y[e]) : 0.f);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      // NaN in the group: NaN scale; nothing but zeros: 1
      const float s = m == 0.f ? 1.f : max_nan(m / kE4m3Max, kMinScale);
      // y / s as y times 1 / s in two terms (Brisebarre, Muller, Raina, "Accelerating correctly rounded
      // floating-point division when the divisor is known in advance"): one term's product puts a
      // value next to a tie on its other side, a division of each value takes a fifth more time
      // (71680 x 1536 with a residual: 176 us against 147)
      const float hi = 1.f / s, lo = s < INFINITY ? fmaf(-hi, s, 1.f) * hi : 0.f;
      if (in) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          float a, b;
          fmul2(a, b, y[e], y[e + 1], lo, lo);
          ffma2(y[e], y[e + 1], y[e], y[e + 1], hi, hi, a, b);
        }
        store8_e4m3<kAligned>(static_cast<uint8_t*>(p.y) + row * p.C, c, p.C, y);
        if ((t & 15) == 0) p.scales[row * ((p.C + kGroup - 1) / kGroup) + c / kGroup] = s;
      }
    } else {
      if (in) store8<kAligned>(static_cast<T*>(p.y) + row * p.C, c, p.C, y);
    }
  }
}

struct NormBwdParams {
  const void* h;
  const void* w;    // or null
  const void* dy;
  const void* dh;   // gradient that reaches h beside the norm, or null
  void* dx;         // [rows, C]
  float* dw_part;   // [gridDim.x, C] sums over the block's rows, or null
  int64_t rows, h_ld, dy_ld, dh_ld;
  int C, tpr;
  int J;            // rows per thread and iteration (1 unless a row is within a warp)
  int stages;       // ring form: stages of the shared-memory ring
  float eps;
};

// Persistent: block b takes row groups (J rows for each of its R row slots) b, b + gridDim.x, ...;
// each thread keeps the sums of
// its channels' dw over the rows it sees in registers, so dw needs no atomics: the block's row
// slots add theirs in order at the end, and rmsnorm_dw_kernel adds the blocks' in order.
//
// kRing (aligned rows, of which the ring holds two groups or more): one more warp brings the
// block's rows through a ring of bulk copies into shared memory, so the next row groups are in
// flight while one is worked on; the rows are read from there twice, for the sums and for the
// outputs, so nothing of a row stays in registers and two blocks of 352 threads share an SM.
// (35840 x 5120 bf16 with dh: 299 us with loads at the head of each iteration, 355 us prefetching
// into registers, 262 to 301 us from a ring that the working warps fill themselves.)  Without the
// ring the second reading comes from L1 or L2.
// kWarpRow: a row is within a warp (tpr <= 32), J rows per thread and iteration; else J = 1.
// (The launch bounds stand for 88 and 120 registers.)
template <typename T, int NV, bool kAligned, bool kDw, bool kRing, bool kWarpRow>
__global__ void __launch_bounds__(NV <= 2 ? 736 : 544) rmsnorm_bwd_kernel(NormBwdParams p) {
  using namespace norm;
  __shared__ __align__(16) Slots slot[2][2];  // [iteration parity][sum]
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages];
  __shared__ int abort;
  // ring: [C] T of the weight, [stages][h, dy, dh][J R rows][C] T; kDw with several rows per block:
  // [C] floats at the end
  extern __shared__ __align__(16) uint8_t norm_smem[];
  const int workers = kRing ? blockDim.x - 32 : blockDim.x;
  const int tpr = p.tpr, R = workers / tpr;
  const T* w = static_cast<const T*>(p.w);
  const int G = kWarpRow ? R * p.J : R;  // rows of a group
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  const int n_tens = p.dh != nullptr ? 3 : 2;
  const uint32_t row_bytes = static_cast<uint32_t>(p.C) * sizeof(T);
  uint8_t* ring = norm_smem + (w != nullptr ? row_bytes : 0u);
  if constexpr (!kWarpRow) {
#pragma unroll
    for (int i = 0; i < 4; ++i) clear_slots(slot[i >> 1][i & 1]);
    __syncthreads();
  }
  if constexpr (kRing) {
    if (w != nullptr) {
      for (uint32_t i = threadIdx.x; i < row_bytes / 16; i += blockDim.x)
        reinterpret_cast<uint4*>(norm_smem)[i] = reinterpret_cast<const uint4*>(w)[i];
      w = reinterpret_cast<const T*>(norm_smem);
    }
    if (threadIdx.x == 0) {
      abort = 0;
      for (int i = 0; i < p.stages; ++i) {
        mbar_init(full + i, 1);
        mbar_init(empty + i, workers / 32);
      }
      fence_mbar_init();
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) >= workers) {
      // the loading warp: per tensor one copy where its rows follow one another in memory, else
      // one per row
      const int lane = threadIdx.x & 31;
      int st = 0, phase = 1;
      for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * G; r0 < p.rows; r0 += step) {
        const int n = static_cast<int>(min(static_cast<int64_t>(G), p.rows - r0));
        if (!__all_sync(0xffffffffu, mbar_wait(empty + st, phase, &abort, 231))) break;
        if (lane == 0) mbar_arrive_expect_tx(full + st, n * n_tens * row_bytes);
        __syncwarp();
        for (int k = 0; k < n_tens; ++k) {
          const T* src = static_cast<const T*>(k == 0 ? p.h : k == 1 ? p.dy : p.dh);
          const int64_t ld = k == 0 ? p.h_ld : k == 1 ? p.dy_ld : p.dh_ld;
          uint8_t* dst = ring + static_cast<size_t>(st * n_tens + k) * G * row_bytes;
          if (ld == p.C) {
            if (lane == 0) bulk_load(dst, src + r0 * ld, n * row_bytes, full + st);
          } else {
            for (int r = lane; r < n; r += 32) bulk_load(dst + r * row_bytes, src + (r0 + r) * ld, row_bytes, full + st);
          }
        }
        if (++st == p.stages) {
          st = 0;
          phase ^= 1;
        }
      }
    }
  }
  float acc[kDw ? NV : 1][8];
#pragma unroll
  for (int i = 0; i < (kDw ? NV : 1); ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[i][e] = 0.f;
  }
  const int t = threadIdx.x % tpr, rs = threadIdx.x / tpr;
  const float inv_c = 1.f / static_cast<float>(p.C);
  // a failed wait (in the status word) writes nothing more, but takes part in every barrier
  bool ok = static_cast<int>(threadIdx.x) < workers;
  int par = 0, st = 0, phase = 0;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * G; r0 < p.rows && static_cast<int>(threadIdx.x) < workers; r0 += step) {
    if constexpr (kRing) ok = mbar_wait(full + st, phase, &abort, 230) && ok;
    for (int j = 0; j < (kWarpRow ? p.J : 1); ++j) {
      const int64_t row = r0 + j * R + rs;
      const bool live = row < p.rows;
      const int64_t row0 = live ? row : 0;
      const T *h, *dy, *dh;
      if constexpr (kRing) {
        const int tens = G * p.C;
        h = reinterpret_cast<const T*>(ring) + st * n_tens * tens + (j * R + rs) * p.C;
        dy = h + tens;
        dh = n_tens == 3 ? dy + tens : nullptr;
      } else {
        h = static_cast<const T*>(p.h) + row0 * p.h_ld;
        dy = static_cast<const T*>(p.dy) + row0 * p.dy_ld;
        dh = p.dh != nullptr ? static_cast<const T*>(p.dh) + row0 * p.dh_ld : nullptr;
      }
      float ss2[2] = {0.f, 0.f}, gh2[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = kVec * (i * tpr + t);
        if (!live || c >= p.C) continue;
        float wv[8], hv[8], gv[8];
        load8<kAligned>(h, c, p.C, hv);
        load8<kAligned>(dy, c, p.C, gv);
        load_weight<kAligned>(w, c, p.C, wv);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          float g0, g1;
          ffma2(ss2[0], ss2[1], hv[e], hv[e + 1], hv[e], hv[e + 1], ss2[0], ss2[1]);
          ffma2(g0, g1, gv[e], gv[e + 1], wv[e], wv[e + 1], 0.f, 0.f);
          ffma2(gh2[0], gh2[1], g0, g1, hv[e], hv[e + 1], gh2[0], gh2[1]);
        }
      }
      float ss = lane_sum(ss2[0] + ss2[1], tpr), gh = lane_sum(gh2[0] + gh2[1], tpr);
      if constexpr (!kWarpRow) {
        // the slots alternate, so one barrier per row suffices: a warp that writes slot[par] again
        // has passed the other parity's barrier, which every reader of slot[par] reached after
        // reading
        if ((threadIdx.x & 31) == 0) {
          slot[par][0][rs][t >> 5] = ss;
          slot[par][1][rs][t >> 5] = gh;
        }
        named_bar_sync(1, workers);
        ss = slot_sum(slot[par][0][rs]);
        gh = slot_sum(slot[par][1][rs]);
        par ^= 1;
      }
      const float rho = rsqrtf(ss * inv_c + p.eps);
      // dx = rho (g - h rho^2 mean(g h)) + dh, rho taken in one factor at a time: rho^3 alone leaves
      // fp32's range for rows of 1e13 and above or 1e-13 and below, whose gradient does not
      const float k = rho * (gh * inv_c) * rho;
      if (!live || !ok) continue;  // no barrier follows for this row
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = kVec * (i * tpr + t);
        if (c >= p.C) continue;
        float wv[8], hv[8], gv[8], o[8];
        load_weight<kAligned>(w, c, p.C, wv);
        load8<kAligned>(h, c, p.C, hv);
        load8<kAligned>(dy, c, p.C, gv);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = 0.f;
        if (dh != nullptr) load8<kAligned>(dh, c, p.C, o);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          float g0, g1;
          ffma2(g0, g1, gv[e], gv[e + 1], wv[e], wv[e + 1], 0.f, 0.f);
          ffma2(g0, g1, hv[e], hv[e + 1], -k, -k, g0, g1);
          ffma2(o[e], o[e + 1], g0, g1, rho, rho, o[e], o[e + 1]);
          if constexpr (kDw) {
            ffma2(g0, g1, hv[e], hv[e + 1], rho, rho, 0.f, 0.f);
            ffma2(acc[i][e], acc[i][e + 1], gv[e], gv[e + 1], g0, g1, acc[i][e], acc[i][e + 1]);
          }
        }
        store8<kAligned>(static_cast<T*>(p.dx) + row * p.C, c, p.C, o);
      }
    }
    if constexpr (kRing) {
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(empty + st);
      if (++st == p.stages) {
        st = 0;
        phase ^= 1;
      }
    }
  }
  if constexpr (kRing) {
    __syncthreads();
    if (abort) {  // copies already issued land before the block leaves
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 100000ull) {
      }
    }
  }
  if constexpr (kDw) {
    float* part = p.dw_part + static_cast<int64_t>(blockIdx.x) * p.C;
    float* dw_smem = reinterpret_cast<float*>(norm_smem);  // (the ring's copies have all been read)
    for (int s = 0; s < R; ++s) {  // the row slots' sums in order
      __syncthreads();
      if (rs != s) continue;  // (the loading warp: rs = R)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = kVec * (i * tpr + t);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (c + e >= p.C) continue;
          const float sum = (s > 0 ? dw_smem[c + e] : 0.f) + acc[i][e];
          if (s + 1 < R)
            dw_smem[c + e] = sum;
          else
            part[c + e] = sum;
        }
      }
    }
  }
}

// dw_c = sum of n_part partial sums, in order: a block of 8 warps takes 32 channels, warp w the
// parts w, w + 8, ..., and the warps' sums are added in warp order.
template <typename T>
__global__ void __launch_bounds__(256) rmsnorm_dw_kernel(const float* __restrict__ part, int n_part, int C, T* dw) {
  __shared__ float s[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < C) {
#pragma unroll 4
    for (int i = warp; i < n_part; i += 8) a += part[static_cast<int64_t>(i) * C + c];
  }
  s[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && c < C) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += s[i][lane];
    norm::from_f(dw[c], t);
  }
}

}  // namespace dsa
