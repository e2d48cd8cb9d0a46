// The kernels around the two tensor-core passes of the cross attention's backward (the cross
// mode of bwd_bf16_kernel, key-major, for dK and dV, and cross_dq_kernel, query-major, for dQ):
// D = rowsum(dO * O) before them, and the sums of their parts after them.  All bound by memory.
#pragma once

#include <stdint.h>

#include "dsa_bwd_bf16.cuh"
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

// dK and dV of the 128-key units that were cut between CTAs: scale * (for dK) the sum of the
// pieces' fp32 sums, in CTA order, as bf16; and zeros for the padding's rows.  A block takes one
// 128-key chunk of one kv head (blockIdx.x) of dk or dv (blockIdx.y); n_cta: the key-major pass'
// grid.
__global__ void __launch_bounds__(256) cross_kv_combine(BwdBf16Params p, int n_cta) {
  const int chunks = (p.Lk + 127) / 128, kt = blockIdx.x % chunks, bh = blockIdx.x / chunks, b = bh / p.kv_heads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, len = bwd_kv_length(p, b), kv_c = (len + 127) / 128;
  const bool is_dk = blockIdx.y == 0;
  const int64_t* s = is_dk ? p.dk_s : p.dv_s;
  __nv_bfloat16* out = (is_dk ? p.dk : p.dv) + b * s[0] + (bh % p.kv_heads) * s[1];
  // units before this one, and in all (every warp adds them up)
  int64_t before = 0, units = 0;
  for (int i = lane; i < p.B; i += 32) {
    const int64_t n = static_cast<int64_t>(bwd_kv_chunks(p, i)) * p.kv_heads;
    units += n;
    if (i < b) before += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    units += __shfl_xor_sync(0xffffffffu, units, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  int i0 = 0, i1 = -1;  // the CTAs that hold pieces of this unit
  int64_t start = 0, all = units * p.per_unit;
  if (kt < kv_c && p.per_unit > 0) {
    start = (before + static_cast<int64_t>(bh % p.kv_heads) * kv_c + kt) * p.per_unit;
    i0 = static_cast<int>(((start + 1) * n_cta - 1) / all);
    i1 = static_cast<int>(((start + p.per_unit) * n_cta - 1) / all);
  }
  const float f = is_dk ? p.scale : 1.f;
  const float* part = is_dk ? p.dk_part : p.dv_part;
  for (int r = warp; r < 128; r += 8) {
    const int l = 128 * kt + r;
    if (l >= p.Lk) break;
    if (l < len && i0 == i1) continue;  // one CTA's own: written by it
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = i0; i <= i1 && l < len; ++i) {
      const int64_t lo = all * i / n_cta;
      if (lo == all * (i + 1) / n_cta) continue;  // an empty range (fewer query chunks than CTAs)
      const float4 x = reinterpret_cast<const float4*>(part + (2 * static_cast<int64_t>(i) + (lo < start)) * 16384 + r * 128)[lane];
      a.x += x.x;
      a.y += x.y;
      a.z += x.z;
      a.w += x.w;
    }
    reinterpret_cast<uint2*>(out + l * s[2])[lane] =
        make_uint2(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f));
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
