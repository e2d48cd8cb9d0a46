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
// thread and vector, NV vectors per thread, W warps per row) while its sums are taken, and
// written from there.  C channels are ceil(C / 8) vectors; vector i * 32 W + t belongs to
// thread t of the row, so a warp's loads are contiguous and a group of 128 channels is 16
// consecutive lanes.  Rows whose address, length or stride is not a multiple of 16 bytes go
// through the same kernel with element-wise loads (kAligned = false).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace dsa {
namespace norm {

constexpr int kVec = 8;        // channels per vector
constexpr int kMaxNV = 4;      // vectors per thread
constexpr int kMaxWarps = 16;  // warps per row: C <= 16 * 32 * 4 * 8 = 16384
constexpr int kMaxC = kMaxWarps * 32 * kMaxNV * kVec;
constexpr int kGroup = 128;    // channels per 8-bit scale
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

// max that keeps NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// Sum over the W warps of a row; every thread of the block calls it.  `slot` holds one float
// per warp of the block and is free again after the next __syncthreads.
__device__ __forceinline__ float row_sum(float s, int W, float* slot) {
  s = warp_sum(s);
  if (W == 1) return s;
  const int warp = threadIdx.x >> 5, first = warp / W * W;
  if ((threadIdx.x & 31) == 0) slot[warp] = s;
  __syncthreads();
  float t = 0.f;
  for (int i = 0; i < W; ++i) t += slot[first + i];
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
  int C, W;        // W warps per row
  float eps;
};

// A block takes blockDim / (32 W) rows.
template <typename T, int NV, bool kAligned, bool kFp8>
__global__ void __launch_bounds__(512) rmsnorm_kernel(NormParams p) {
  using namespace norm;
  __shared__ float slot[kMaxWarps];
  const int tpr = 32 * p.W, t = threadIdx.x % tpr;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
  const bool live = row < p.rows;
  const int64_t row0 = live ? row : 0;
  const T* x = static_cast<const T*>(p.x) + row0 * p.x_ld;
  const T* r = p.r != nullptr ? static_cast<const T*>(p.r) + row0 * p.r_ld : nullptr;
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
  ss = row_sum(ss, p.W, slot);
  const float rho = 1.f / sqrtf(ss / static_cast<float>(p.C) + p.eps);
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
      const float inv = 1.f / s;
      if (in) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= inv;
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
  int C, W;
  float eps;
};

// Persistent: block b takes row groups b, b + gridDim.x, ...; each thread keeps the sums of
// its channels' dw over the rows it sees in registers, so dw needs no atomics: the block's row
// slots add theirs in order at the end, and rmsnorm_dw_kernel adds the blocks' in order.
template <typename T, int NV, bool kAligned, bool kDw>
__global__ void __launch_bounds__(512) rmsnorm_bwd_kernel(NormBwdParams p) {
  using namespace norm;
  __shared__ float slot[2][2][kMaxWarps];  // [iteration parity][sum][warp]
  extern __shared__ float dw_smem[];       // kDw and several rows per block: [C]
  const int tpr = 32 * p.W, t = threadIdx.x % tpr, R = blockDim.x / tpr, rs = threadIdx.x / tpr;
  const T* w = static_cast<const T*>(p.w);
  float acc[kDw ? NV : 1][8];
#pragma unroll
  for (int i = 0; i < (kDw ? NV : 1); ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[i][e] = 0.f;
  }
  int par = 0;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * R; r0 < p.rows; r0 += static_cast<int64_t>(gridDim.x) * R, par ^= 1) {
    const int64_t row = r0 + rs;
    const bool live = row < p.rows;
    const int64_t row0 = live ? row : 0;
    const T* h = static_cast<const T*>(p.h) + row0 * p.h_ld;
    const T* dy = static_cast<const T*>(p.dy) + row0 * p.dy_ld;
    const T* dh = p.dh != nullptr ? static_cast<const T*>(p.dh) + row0 * p.dh_ld : nullptr;
    Raw8<T> hr[NV], gr[NV], dr[NV];  // h, dy, dh
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = kVec * (i * tpr + t);
      zero_raw(hr[i]);
      zero_raw(gr[i]);
      zero_raw(dr[i]);
      if (live && c < p.C) {
        load_raw<kAligned>(h, c, p.C, hr[i]);
        load_raw<kAligned>(dy, c, p.C, gr[i]);
        if (dh != nullptr) load_raw<kAligned>(dh, c, p.C, dr[i]);
      }
    }
    float ss = 0.f, gh = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = kVec * (i * tpr + t);
      float wv[8];
      if (w != nullptr && c < p.C) {
        load8<kAligned>(w, c, p.C, wv);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) wv[e] = 1.f;
      }
      float hv[8], gv[8];
      expand(hr[i], hv);
      expand(gr[i], gv);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss = fmaf(hv[e], hv[e], ss);
        gh = fmaf(gv[e] * wv[e], hv[e], gh);
      }
    }
    ss = warp_sum(ss);
    gh = warp_sum(gh);
    if (p.W > 1) {
      // the slots alternate, so one barrier per iteration suffices: a warp that writes
      // slot[par] again has passed the other parity's barrier, which every reader of
      // slot[par] reached after reading
      const int warp = threadIdx.x >> 5, first = warp / p.W * p.W;
      if ((threadIdx.x & 31) == 0) {
        slot[par][0][warp] = ss;
        slot[par][1][warp] = gh;
      }
      __syncthreads();
      ss = gh = 0.f;
      for (int i = 0; i < p.W; ++i) {
        ss += slot[par][0][first + i];
        gh += slot[par][1][first + i];
      }
    }
    const float inv_c = 1.f / static_cast<float>(p.C);
    const float rho = 1.f / sqrtf(ss * inv_c + p.eps);
    const float k = rho * rho * rho * (gh * inv_c);
    if (!live) continue;  // no barrier follows in this iteration
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = kVec * (i * tpr + t);
      if (c >= p.C) continue;
      float wv[8], hv[8], gv[8], o[8];
      if (w != nullptr) {
        load8<kAligned>(w, c, p.C, wv);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) wv[e] = 1.f;
      }
      expand(hr[i], hv);
      expand(gr[i], gv);
      expand(dr[i], o);  // zeros without dh
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        o[e] += rho * (gv[e] * wv[e]) - k * hv[e];
        if constexpr (kDw) acc[i][e] = fmaf(gv[e], hv[e] * rho, acc[i][e]);
      }
      store8<kAligned>(static_cast<T*>(p.dx) + row * p.C, c, p.C, o);
    }
  }
  if constexpr (kDw) {
    float* part = p.dw_part + static_cast<int64_t>(blockIdx.x) * p.C;
    for (int s = 0; s < R; ++s) {  // the row slots' sums in order
      __syncthreads();
      if (rs != s) continue;
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
