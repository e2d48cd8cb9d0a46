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
// key-major pass starts on 16 bytes and lies inside.  16 threads per row, 8 channels each, four
// rows a thread, all loads first (one row at a time took 96 us for 440 MB, 4.6 TB/s).
__global__ void __launch_bounds__(256) cross_preprocess(CrossPrepParams p) {
  constexpr int kRows = 4;
  const int part = threadIdx.x % 16;
  const int64_t id0 = static_cast<int64_t>(blockIdx.x) * (16 * kRows) + threadIdx.x / 16;
  const int64_t all = static_cast<int64_t>(p.B) * p.heads * p.Lp;
  uint4 x[kRows], y[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t id = id0 + 16 * i, bh = id / p.Lp, b = bh / p.heads, h = bh % p.heads;
    const int q = static_cast<int>(id % p.Lp);
    x[i] = y[i] = make_uint4(0u, 0u, 0u, 0u);
    if (id < all && q < p.Lq) {
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
    if (part == 0 && id < all) {
      const int q = static_cast<int>(id % p.Lp);
      p.delta_pad[id] = s;
      p.lse_pad[id] = q < p.Lq ? p.lse[id / p.Lp * p.Lq + q] : 0.f;
    }
  }
}

// dK and dV of the 128-key units that were cut between CTAs: scale * (for dK) the sum of the
// pieces' fp32 sums, in CTA order, as bf16; and zeros for the padding's rows.  A block takes 16
// rows (blockIdx.z) of one 128-key chunk of one kv head (blockIdx.x) of dk or dv (blockIdx.y);
// n_cta: the key-major pass' grid.
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
  const int r = 16 * blockIdx.z + warp, l = 128 * kt + r;  // this warp's rows: l and l + 8
  const bool cut = i0 != i1;  // (otherwise one CTA's own: its valid rows are written)
  float4 a[2];
  a[0] = a[1] = make_float4(0.f, 0.f, 0.f, 0.f);
  int64_t lo = i1 >= i0 ? all * i0 / n_cta : 0;
  for (int i = i0; i <= i1 && cut; ++i) {
    const int64_t hi = all * (i + 1) / n_cta;
    if (lo < hi) {  // (a range is empty where there are fewer query chunks than CTAs)
      const float4* src = reinterpret_cast<const float4*>(part + (2 * static_cast<int64_t>(i) + (lo < start)) * 16384 + r * 128) + lane;
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
    if (lj >= p.Lk || (lj < len && !cut)) continue;
    reinterpret_cast<uint2*>(out + lj * s[2])[lane] =
        make_uint2(pack_bf16x2(a[j].x * f, a[j].y * f), pack_bf16x2(a[j].z * f, a[j].w * f));
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
