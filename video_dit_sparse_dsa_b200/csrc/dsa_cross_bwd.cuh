// The kernels around the two tensor-core passes of the cross attention's backward (the cross
// modes of bwd_bf16_kernel, key-major, for dK and dV, and of bwd_dq_kernel, query-major, for dQ):
// D = rowsum(dO * O) before them, and the sums of their parts after them.  All bound by memory.
#pragma once

#include <stdint.h>

#include "sm100.cuh"

namespace dsa {

struct CrossPrepParams {
  const __nv_bfloat16* o;
  const __nv_bfloat16* dout;
  int64_t o_s[3], do_s[3];  // strides (batch, head, row) in elements
  const float* lse;         // [B, heads, Lq]
  float* delta_pad;         // [B * heads, Lp]
  float* lse_pad;
  int B, heads, Lq, Lp;     // Lp: Lq rounded up to 64
};

// D, and a copy of the LSE, in rows of Lp values, zeros past Lq: every 64-row TMA box of the
// key-major pass starts on 16 bytes and lies inside.  16 threads per row, 8 channels each.
__global__ void __launch_bounds__(256) cross_preprocess(CrossPrepParams p) {
  const int64_t id = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / 16;
  const int part = threadIdx.x % 16;
  const int64_t bh = id / p.Lp;
  const int q = static_cast<int>(id % p.Lp);
  const bool in = bh < static_cast<int64_t>(p.B) * p.heads, live = in && q < p.Lq;
  float s = 0.f;
  if (live) {
    const int64_t b = bh / p.heads, h = bh % p.heads;
    const uint4 x = reinterpret_cast<const uint4*>(p.o + b * p.o_s[0] + h * p.o_s[1] + q * p.o_s[2])[part];
    const uint4 y = reinterpret_cast<const uint4*>(p.dout + b * p.do_s[0] + h * p.do_s[1] + q * p.do_s[2])[part];
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s = fmaf(__uint_as_float(xs[e] << 16), __uint_as_float(ys[e] << 16), s);
      s = fmaf(__uint_as_float(xs[e] & 0xffff0000u), __uint_as_float(ys[e] & 0xffff0000u), s);
    }
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (in && part == 0) {
    p.delta_pad[id] = s;
    p.lse_pad[id] = live ? p.lse[bh * p.Lq + q] : 0.f;
  }
}

struct CrossCombineParams {
  const float* part[2];      // [n_part, rows, 128] fp32
  __nv_bfloat16* out[2];     // through strides (batch, head, row)
  int64_t s[2][3];
  float scale[2];
  int n_part, n_out;         // n_out: 1 or 2 tensors
  int64_t part_stride;       // rows * 128
  int B, heads, L;
  const int32_t* len;        // rows from len[b] on are zero and have no parts; null: L
};

// out = scale * sum of the parts in part order, as bf16 (no parts: zeros).  A thread takes 4
// channels of one row; blockIdx.y is the tensor.
__global__ void __launch_bounds__(256) cross_combine(CrossCombineParams p) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t row = id / 32, bh = row / p.L;
  if (bh >= static_cast<int64_t>(p.B) * p.heads) return;
  const int c = static_cast<int>(id % 32), l = static_cast<int>(row % p.L), k = blockIdx.y;
  const int64_t b = bh / p.heads, h = bh % p.heads;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.len == nullptr || l < p.len[b]) {
    const float4* src = reinterpret_cast<const float4*>((k ? p.part[1] : p.part[0]) + row * 128) + c;
#pragma unroll 4
    for (int j = 0; j < p.n_part; ++j) {
      const float4 x = src[j * (p.part_stride / 4)];
      a.x += x.x;
      a.y += x.y;
      a.z += x.z;
      a.w += x.w;
    }
  }
  const float f = k ? p.scale[1] : p.scale[0];
  __nv_bfloat16* out = k ? p.out[1] + b * p.s[1][0] + h * p.s[1][1] + l * p.s[1][2]
                         : p.out[0] + b * p.s[0][0] + h * p.s[0][1] + l * p.s[0][2];
  reinterpret_cast<uint2*>(out)[c] =
      make_uint2(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f));
}

}  // namespace dsa
