// The cross attention's backward around its two tensor-core passes (cross_kv_kernel, key-major,
// for dK and dV, and cross_dq_kernel, query-major, for dQ): D = rowsum(dO * O) before them and the
// sum of dQ's parts after them.  Both bound by memory.
#pragma once

#include <stdint.h>

#include "sm100.cuh"

namespace dsa {

struct CrossPrepParams {
  const __nv_bfloat16* o;
  const __nv_bfloat16* dout;
  int64_t o_s[3], do_s[3];  // strides (batch, head, row) in elements
  float* delta;             // [B, heads, Lq]
  int B, heads, Lq;
};

// D.  16 threads per row, 8 channels each, four rows a thread, all loads first (24 heads x
// 35840 rows, 440 MB: 88 us with L2 flushed, 5.0 TB/s; one row at a time took 14% more).
__global__ void __launch_bounds__(256) cross_preprocess(CrossPrepParams p) {
  constexpr int kRows = 4;
  const int part = threadIdx.x % 16;
  const int64_t id0 = static_cast<int64_t>(blockIdx.x) * (16 * kRows) + threadIdx.x / 16;
  const int64_t all = static_cast<int64_t>(p.B) * p.heads * p.Lq;
  uint4 x[kRows], y[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t id = id0 + 16 * i, bh = id / p.Lq, b = bh / p.heads, h = bh % p.heads, q = id % p.Lq;
    x[i] = y[i] = make_uint4(0u, 0u, 0u, 0u);
    if (id < all) {
      x[i] = reinterpret_cast<const uint4*>(p.o + b * p.o_s[0] + h * p.o_s[1] + q * p.o_s[2])[part];
      y[i] = reinterpret_cast<const uint4*>(p.dout + b * p.do_s[0] + h * p.do_s[1] + q * p.do_s[2])[part];
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const uint32_t xs[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, ys[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s = fmaf(__uint_as_float(xs[e] << 16), __uint_as_float(ys[e] << 16), s);
      s = fmaf(__uint_as_float(xs[e] & 0xffff0000u), __uint_as_float(ys[e] & 0xffff0000u), s);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int64_t id = id0 + 16 * i;
    if (part == 0 && id < all) p.delta[id] = s;
  }
}

struct CrossDqCombineParams {
  const float* part;         // [n_part, rows, 128] fp32
  __nv_bfloat16* dq;         // through strides (batch, head, row)
  int64_t s[3];
  int n_part;
  int B, heads, Lq;
};

// dQ = the sum of the parts in part order, as bf16 (no parts: zeros).  A thread takes 4 channels
// of one row.
__global__ void __launch_bounds__(256) cross_dq_combine(CrossDqCombineParams p) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t row = id / 32, bh = row / p.Lq, rows = static_cast<int64_t>(p.B) * p.heads * p.Lq;
  if (row >= rows) return;
  const int c = static_cast<int>(id % 32), q = static_cast<int>(row % p.Lq);
  const int64_t b = bh / p.heads, h = bh % p.heads;
  const float4* src = reinterpret_cast<const float4*>(p.part + row * 128) + c;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int j = 0; j < p.n_part; ++j) {
    const float4 x = src[j * rows * 32];
    a.x += x.x;
    a.y += x.y;
    a.z += x.z;
    a.w += x.w;
  }
  reinterpret_cast<uint2*>(p.dq + b * p.s[0] + h * p.s[1] + q * p.s[2])[c] =
      make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
}

}  // namespace dsa
