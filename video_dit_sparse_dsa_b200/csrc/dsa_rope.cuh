// Rotary positions over the three axes (time, height, width) of the token grid.
//
// A head's first R = d_t + d_h + d_w channels are R / 2 pairs: d_t / 2 of the time axis, then
// d_h / 2 of the height, d_w / 2 of the width; the channels past R pass through.  Pair j of an
// axis turns by the angle a = (start + i * step) * theta^(-2j / d_axis) at coordinate i:
//   (x, y) -> (x cos a - y sin a, x sin a + y cos a),
// and the inverse turns by -a, which is also the backward (a rotation's transpose).  A pair is
// channels (2j, 2j + 1) (interleaved) or (j, j + R / 2) (halves).
//
// The angles depend on one coordinate of one axis each, so cos and sin of a grid are a table
// of T d_t / 2 + H d_h / 2 + W d_w / 2 entries (27 KB for a 30 x 48 x 80 grid and 128
// channels, where one entry per token and pair would be 59 MB): rope_table_kernel fills it,
// angles in fp64 (a far position times a frequency keeps its fraction of a turn), and the
// rotation reads it through L1.
//
// The rotation is bound by memory: q and k are read and written once.  A thread takes one
// 16-byte vector (halves: the vector pair) of one token, looks its four (eight) angles up once
// and applies them to that token's heads in turn, so the table reads and index arithmetic are
// spread over the heads; the heads' loads are independent and kept in flight together.  Input
// and output have their own strides: the call also moves the projection's token-major rows into
// the attention's head-major layout (or the gradients back).  24 heads x 115200 tokens of q and k
// in bf16: 444 us, 6.4 TB/s or 98% of a copy's rate; 10 heads x 34503 tokens of q and k in fp32,
// halves: 119 us, 91%.  A frame of 256 tokens is one short launch: its call is host time.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "dsa_norm.cuh"

namespace dsa {

struct RopeTableParams {
  int n[3], pairs[3];  // coordinates and pairs of each axis
  double start[3], step[3];
  double log_theta;
  float2* table;
};

__global__ void __launch_bounds__(256) rope_table_kernel(RopeTableParams p) {
  int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  float2* out = p.table;
#pragma unroll
  for (int a = 0; a < 3; ++a) {
    const int64_t n = static_cast<int64_t>(p.n[a]) * p.pairs[a];
    if (i < n) {
      const int j = static_cast<int>(i % p.pairs[a]);
      const double pos = p.start[a] + static_cast<double>(i / p.pairs[a]) * p.step[a];
      double s, c;
      sincos(pos * exp(-p.log_theta * j / p.pairs[a]), &s, &c);
      out[i] = make_float2(static_cast<float>(c), static_cast<float>(s));
      return;
    }
    i -= n;
    out += n;
  }
}

struct RopeView {
  int64_t b, h, n;  // strides of batch, head and token in elements
};

struct RopeParams {
  const void* in[2];   // q and k (k may be null)
  void* out[2];
  RopeView si[2], so[2];
  const float2* table;
  int H, W, N;         // token grid (T is N / (H W))
  int heads, hpt;      // heads per thread
  int d;
  int pairs[3];        // pairs of each axis
  int off[3];          // first table entry of each axis
  int inverse;
};

namespace rope {
// (cos, sin) of pair j of the token at (t, h, w).
__device__ __forceinline__ float2 angle(const RopeParams& p, int j, int t, int h, int w) {
  int a = 0, i = t;
  if (j >= p.pairs[0]) {
    j -= p.pairs[0];
    a = 1;
    i = h;
    if (j >= p.pairs[1]) {
      j -= p.pairs[1];
      a = 2;
      i = w;
    }
  }
  float2 cs = p.table[p.off[a] + static_cast<int64_t>(i) * p.pairs[a] + j];
  if (p.inverse) cs.y = -cs.y;
  return cs;
}
}  // namespace rope

// Vector form: d, R (halves: R / 2), every stride and address in whole 16-byte vectors of 8
// channels.  A token's work items are its d / 8 vectors (interleaved), or its R / 16 vector
// pairs and (d - R) / 8 vectors that pass through (halves).  The grid is (token items, head
// groups, batch); n_tens = 1 or 2 tensors.
template <typename T, bool kHalves>
__global__ void __launch_bounds__(256) rope_kernel(RopeParams p, int items, int n_tens) {
  using namespace norm;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t n = id / items;
  if (n >= p.N) return;
  const int item = static_cast<int>(id % items);
  const int w = static_cast<int>(n % p.W), h = static_cast<int>(n / p.W) % p.H, t = static_cast<int>(n / p.W / p.H);
  const int half = p.pairs[0] + p.pairs[1] + p.pairs[2], n_rot = kHalves ? half / 8 : half / 4;
  const bool rot = item < n_rot;
  // channels of this item: c0 (and c0 + half)
  const int c0 = kHalves && !rot ? 2 * half + 8 * (item - n_rot) : 8 * item;
  constexpr int NA = kHalves ? 8 : 4, kHeads = 4;
  float2 cs[NA];
  if (rot) {
#pragma unroll
    for (int i = 0; i < NA; ++i) cs[i] = rope::angle(p, NA * item + i, t, h, w);
  }
  const int h0 = blockIdx.y * p.hpt, h1 = min(h0 + p.hpt, p.heads);
  for (int k = 0; k < n_tens; ++k) {
    const T* src = static_cast<const T*>(p.in[k]) + blockIdx.z * p.si[k].b + n * p.si[k].n + c0;
    T* dst = static_cast<T*>(p.out[k]) + blockIdx.z * p.so[k].b + n * p.so[k].n + c0;
    // kHeads heads at a time, every load before the first store: the call may work in place, so
    // the compiler keeps loads behind stores
    for (int hb = h0; hb < h1; hb += kHeads) {
      Raw8<T> x[kHeads], y[kHalves ? kHeads : 1];
#pragma unroll
      for (int u = 0; u < kHeads; ++u) {
        if (hb + u >= h1) continue;
        load_raw<true>(src + (hb + u) * p.si[k].h, 0, 8, x[u]);
        if constexpr (kHalves) {
          if (rot) load_raw<true>(src + (hb + u) * p.si[k].h + half, 0, 8, y[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kHeads; ++u) {
        if (hb + u >= h1) continue;
        T* o = dst + (hb + u) * p.so[k].h;
        float a[8];
        expand(x[u], a);
        if constexpr (kHalves) {
          if (rot) {
            float b[8], z[8];
            expand(y[u], b);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              z[i] = a[i] * cs[i].y + b[i] * cs[i].x;
              a[i] = a[i] * cs[i].x - b[i] * cs[i].y;
            }
            store8<true>(o + half, 0, 8, z);
          }
        } else {
          if (rot) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float f = a[2 * i], g = a[2 * i + 1];
              a[2 * i] = f * cs[i].x - g * cs[i].y;
              a[2 * i + 1] = f * cs[i].y + g * cs[i].x;
            }
          }
        }
        store8<true>(o, 0, 8, a);
      }
    }
  }
}

// Any d, R, strides and alignment: one pair, or one channel past R, per thread and head.
template <typename T, bool kHalves>
__global__ void __launch_bounds__(256) rope_any_kernel(RopeParams p, int items, int n_tens) {
  using namespace norm;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t n = id / items;
  if (n >= p.N) return;
  const int item = static_cast<int>(id % items);
  const int w = static_cast<int>(n % p.W), h = static_cast<int>(n / p.W) % p.H, t = static_cast<int>(n / p.W / p.H);
  const int half = p.pairs[0] + p.pairs[1] + p.pairs[2];
  const bool rot = item < half;
  const int c0 = rot ? (kHalves ? item : 2 * item) : item + half, c1 = rot ? (kHalves ? item + half : c0 + 1) : c0;
  const float2 cs = rot ? rope::angle(p, item, t, h, w) : make_float2(1.f, 0.f);
  const int h0 = blockIdx.y * p.hpt, h1 = min(h0 + p.hpt, p.heads);
  for (int k = 0; k < n_tens; ++k) {
    const T* src = static_cast<const T*>(p.in[k]) + blockIdx.z * p.si[k].b + n * p.si[k].n;
    T* dst = static_cast<T*>(p.out[k]) + blockIdx.z * p.so[k].b + n * p.so[k].n;
#pragma unroll 4
    for (int hh = h0; hh < h1; ++hh) {
      const T* s = src + hh * p.si[k].h;
      T* o = dst + hh * p.so[k].h;
      if (rot) {
        const float a = to_f(s[c0]), b = to_f(s[c1]);
        from_f(o[c0], a * cs.x - b * cs.y);
        from_f(o[c1], a * cs.y + b * cs.x);
      } else {
        o[c0] = s[c0];
      }
    }
  }
}

}  // namespace dsa
