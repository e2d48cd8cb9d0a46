// C entry points of the operators around the sliding attention in a transformer block (declared
// in include/dsa.h): cross attention to an encoder's states, rotary positions, and the
// root-mean-square norm.  Included by dsa_api.cu (the library is one translation unit), whose
// status, alignment and tensor-map helpers these use.
#pragma once

namespace {

// SMs that the splits below are planned for (a B200); other counts only change the balance.
constexpr int kPlanSms = 148;

// ---------------------------------------------------------------- views
// A [B, heads, rows, 128] view: strides in elements, each a whole number of 16-byte vectors; a
// broadcast (stride 0) batch or head dimension is fine for an input.
bool view_ok(const dsa_view_t* v, int64_t B, int64_t heads, int64_t rows, bool output) {
  if (v == nullptr || v->data == nullptr || !aligned(v->data, 16)) return false;
  const int64_t n[3] = {B, heads, rows};
  for (int a = 0; a < 3; ++a) {
    if (n[a] <= 1) continue;
    const int64_t s = v->stride[a];
    if (s < 0 || s % 8 != 0 || s >= (int64_t(1) << 39)) return false;
    if (s == 0 ? (output || a == 2) : s < 128) return false;
  }
  return true;
}

// Rank-4 or rank-5 map of a view: (channel, row[, head in the group], head, batch), boxes of 64
// channels x box_rows rows (x box_heads heads of the group), 128-byte swizzled; rows and heads
// past the end load as zeros.  A broadcast dimension gets extent 1; m[0..2] (group, head, batch)
// is 0 for it, the factor of its coordinate, and 1 otherwise.
bool make_view_map(CUtensorMap* map, const dsa_view_t* v, int64_t B, int64_t heads, int64_t group, int64_t rows,
                   int box_rows, int box_heads, int m[3]) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const int rank = group > 0 ? 5 : 4;
  const int64_t g = group > 0 ? group : 1;
  // extents and strides in elements of row, head in the group, head (of heads / g), batch
  int64_t n[4] = {rows, g, heads / g, B}, s[4] = {v->stride[2], v->stride[1], v->stride[1] * g, v->stride[0]};
  for (int a = 0; a < 4; ++a) {
    if (n[a] <= 1 || s[a] == 0) {  // one entry: its stride is never taken
      if (a > 0) m[a - 1] = n[a] <= 1 ? 1 : 0;
      n[a] = 1;
      s[a] = 128;
    } else if (a > 0) {
      m[a - 1] = 1;
    }
  }
  cuuint64_t dims[5] = {128}, strides[4];
  cuuint32_t box[5] = {64, static_cast<cuuint32_t>(box_rows), 1, 1, 1}, estr[5] = {1, 1, 1, 1, 1};
  int r = 1;
  for (int a = 0; a < 4; ++a) {
    if (a == 1) {
      if (rank == 4) continue;
      box[r] = static_cast<cuuint32_t>(box_heads);
    }
    dims[r] = static_cast<cuuint64_t>(n[a]);
    strides[r - 1] = static_cast<cuuint64_t>(s[a]) * 2;
    ++r;
  }
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, v->data, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---------------------------------------------------------------- cross attention
struct CrossPlan {
  int group, pk, tiles;   // heads per kv head; heads packed into a 128-row unit; units per kv head
  bool pair;              // the forward runs on CTA pairs
  int64_t units;          // B * kv_heads * tiles
  int chunks;             // 128-key chunks of Lk
  int64_t rows;           // B * heads * Lq
  int split_q;            // parts of the keys (forward, and dQ)
  int64_t kv_units;       // 128-key units of kv heads (dK, dV), at most; `tiles` query chunks each
};

// pack: a kv head's heads may share a unit.  (Not packing takes more units, so at most as many
// parts of the keys and as much workspace.)
dsa_status_t cross_plan(const dsa_cross_t* p, CrossPlan* c, bool pack = true) {
  if (p == nullptr) return DSA_ERR_INVALID_ARG;
  if (p->B <= 0 || p->heads <= 0 || p->kv_heads <= 0 || p->heads % p->kv_heads != 0 || p->Lq < 0 || p->Lk < 0)
    return DSA_ERR_INVALID_ARG;
  if (!(p->scale > 0.f) || !std::isfinite(p->scale)) return DSA_ERR_INVALID_ARG;
  if (p->dtype != DSA_F32 && p->dtype != DSA_BF16) return DSA_ERR_INVALID_ARG;
  if (p->dtype != DSA_BF16 || p->d != 128) return DSA_ERR_UNSUPPORTED;
  c->group = p->heads / p->kv_heads;
  c->pk = pack && c->group > 1 && p->Lq > 0 && p->Lq <= 64 ? (c->group < 128 / p->Lq ? c->group : 128 / p->Lq) : 1;
  const int64_t tiles = c->pk > 1 ? (c->group + c->pk - 1) / c->pk
                                  : static_cast<int64_t>(c->group) * ((static_cast<int64_t>(p->Lq) + 127) / 128);
  const int64_t slices = static_cast<int64_t>(p->B) * p->kv_heads;
  c->rows = static_cast<int64_t>(p->B) * p->heads * p->Lq;
  // unit and row indices are 32 bits in the kernels
  if (p->Lq > INT32_MAX - 128 || p->Lk > INT32_MAX - 128 || tiles > INT32_MAX || slices > INT32_MAX ||
      slices * tiles > INT32_MAX || c->rows > INT32_MAX)
    return DSA_ERR_UNSUPPORTED;
  c->tiles = static_cast<int>(tiles);
  c->units = slices * tiles;
  c->chunks = (p->Lk + 127) / 128;
  // Too few units to fill the GPU: the keys are cut into parts of at least four chunks (two
  // steps), for about four units per SM.
  c->split_q = 1;
  if (c->units > 0 && c->units < kPlanSms && c->chunks >= 8) {
    int64_t s = 4 * kPlanSms / c->units;
    if (s > c->chunks / 4) s = c->chunks / 4;
    int64_t per = (c->chunks + s - 1) / s;
    per = (per + 1) / 2 * 2;
    c->split_q = static_cast<int>((c->chunks + per - 1) / per);
  }
  // more than one 128-row tile per head, and not in parts: a cluster of two CTAs per 256 rows
  c->pair = c->split_q == 1 && p->Lq > 128;
  c->kv_units = slices * c->chunks;
  if (c->kv_units > INT32_MAX - kPlanSms) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

// Several heads of a unit come in one TMA box, which cannot repeat a head: a view whose heads are
// one (stride 0) is not packed.
bool heads_broadcast(const dsa_view_t* v, const CrossPlan& c) { return c.pk > 1 && v->stride[1] == 0; }

struct CrossWorkspace {
  float *part_o, *part_lse;                       // forward, split_q > 1
  float *delta, *dq_part, *dk_part, *dv_part;     // backward
  size_t bytes;
};

CrossWorkspace cross_workspace(const dsa_cross_t* p, const CrossPlan& c, int kind, void* base) {
  CrossWorkspace w;
  std::memset(&w, 0, sizeof(w));
  uint8_t* b = static_cast<uint8_t*>(base);
  size_t off = 0;
  auto take = [&](size_t floats) {
    float* at = reinterpret_cast<float*>(b + off);
    off += round_up(sizeof(float) * floats, kAlign);
    return at;
  };
  if (kind == DSA_WS_FWD) {
    if (c.split_q > 1) {
      w.part_o = take(static_cast<size_t>(c.split_q) * c.rows * 128);
      w.part_lse = take(static_cast<size_t>(c.split_q) * c.rows);
    }
  } else {
    w.delta = take(static_cast<size_t>(c.rows));
    if (c.split_q > 1) w.dq_part = take(static_cast<size_t>(c.split_q) * c.rows * 128);
    // the pieces of the 128-key units that are cut between CTAs: at most two per CTA
    w.dk_part = take(2 * kPlanSms * 128 * 128);
    w.dv_part = take(2 * kPlanSms * 128 * 128);
  }
  w.bytes = off;
  return w;
}

// Grid of a persistent kernel, one CTA per SM; checks the registers its setmaxnreg split needs.
template <typename K>
dsa_status_t persistent_grid(K kernel, uint32_t smem, int regs, int64_t units, unsigned* grid) {
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return DSA_ERR_CUDA;
  if (regs > 0) {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess) return DSA_ERR_CUDA;
    if (fa.numRegs < regs) return DSA_ERR_UNSUPPORTED;
  }
  int sms = 0;
  if (sm_count(&sms) != DSA_OK) return DSA_ERR_CUDA;
  *grid = static_cast<unsigned>(units < sms ? units : sms);
  return DSA_OK;
}

// A persistent kernel over CTA pairs: as many clusters of two as stay resident (looked up once per
// device), no more than units.
template <auto kKernel, typename... Args>
dsa_status_t launch_pairs(uint32_t smem, int threads, int regs, int64_t units, cudaStream_t s, const Args&... args) {
  static std::atomic<int> cache[kPairMaxDevices] = {};
  unsigned grid = 0;
  dsa_status_t st = persistent_grid(kKernel, smem, regs, INT32_MAX, &grid);
  if (st != DSA_OK) return st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(grid / 2 * 2, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSA_ERR_CUDA;
  const bool cached = dev >= 0 && dev < kPairMaxDevices;
  if (cached) n = cache[dev].load(std::memory_order_relaxed);
  if (n <= 0) {
    if (cudaOccupancyMaxActiveClusters(&n, kKernel, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      return DSA_ERR_CUDA;
    }
    if (cached) cache[dev].store(n, std::memory_order_relaxed);
  }
  cfg.gridDim.x = 2u * static_cast<unsigned>(units < n ? units : n);
  if (cudaLaunchKernelEx(&cfg, kKernel, args...) != cudaSuccess) {
    cudaGetLastError();
    return DSA_ERR_CUDA;
  }
  return launch_status();
}

dsa_status_t launch_dq_combine(const dsa::CrossDqCombineParams& cp, cudaStream_t s) {
  const int64_t threads = static_cast<int64_t>(cp.B) * cp.heads * cp.Lq * 32;
  dsa::cross_dq_combine<<<static_cast<unsigned>((threads + 255) / 256), 256, 0, s>>>(cp);
  return launch_status();
}

void copy_strides(int64_t (&d)[3], const dsa_view_t* v) {
  for (int a = 0; a < 3; ++a) d[a] = v->stride[a];
}

// ---------------------------------------------------------------- rotary positions
bool rope_axes_ok(const int32_t* axes) {
  for (int a = 0; a < 3; ++a)
    if (axes[a] < 0 || axes[a] % 2 != 0) return false;
  return static_cast<int64_t>(axes[0]) + axes[1] + axes[2] > 0;
}

// ---------------------------------------------------------------- norm
dsa_status_t check_norm(const dsa_norm_t* p) {
  if (p == nullptr || p->rows < 0 || p->C <= 0) return DSA_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f) || !std::isfinite(p->eps)) return DSA_ERR_INVALID_ARG;
  if (p->dtype != DSA_F32 && p->dtype != DSA_BF16) return DSA_ERR_INVALID_ARG;
  if (p->C > dsa::norm::kMaxC || p->rows > (int64_t(1) << 30)) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

// Row stride of a [rows, C] operand: at least C unless there is one row.
bool ld_ok(int64_t ld, const dsa_norm_t* p) { return p->rows <= 1 || ld >= p->C; }

// Whole 16-byte vectors of 8 channels: address and row stride (C is checked apart).
bool vec_ok(const void* ptr, int64_t ld, const dsa_norm_t* p) {
  return ptr == nullptr || (aligned(ptr, 16) && (p->rows <= 1 || ld % (p->dtype == DSA_BF16 ? 8 : 4) == 0));
}

struct NormShape {
  int NV, tpr, R;  // vectors per thread, threads per row, rows per block
};

// Fewest idle lanes; among equals the widest NV up to nv_pref (fewer warps meet at the row's
// barrier).
NormShape norm_shape(int C, int nv_pref, int threads) {
  const int nvec = (C + dsa::norm::kVec - 1) / dsa::norm::kVec;
  NormShape best = {1, 16, threads / 16};
  if (nvec <= 16) return best;  // up to 128 channels: two rows to a warp
  best.NV = 0;
  int waste = INT32_MAX;
  for (int pass = 0; pass < 2 && best.NV == 0; ++pass) {
    for (int nv = pass == 0 ? nv_pref : dsa::norm::kMaxNV; nv >= 1; --nv) {
      const int W = (nvec + 32 * nv - 1) / (32 * nv);
      if (W > dsa::norm::kMaxWarps) continue;
      const int idle = 32 * nv * W - nvec;
      if (idle < waste) {
        waste = idle;
        best.NV = nv;
        best.tpr = 32 * W;
      }
    }
  }
  best.R = threads / best.tpr > 1 ? threads / best.tpr : 1;
  return best;
}

template <typename T, bool kFp8>
dsa_status_t launch_norm(const dsa::NormParams& np, const NormShape& sh, bool vec, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((np.rows + sh.R - 1) / sh.R), threads = sh.tpr * sh.R;
#define DSA_NORM_CASE(NV)                                                              \
  case NV:                                                                             \
    if (vec)                                                                           \
      dsa::rmsnorm_kernel<T, NV, true, kFp8><<<grid, threads, 0, s>>>(np);             \
    else                                                                               \
      dsa::rmsnorm_kernel<T, NV, false, kFp8><<<grid, threads, 0, s>>>(np);            \
    break;
  switch (sh.NV) {
    DSA_NORM_CASE(1)
    DSA_NORM_CASE(2)
    DSA_NORM_CASE(3)
    DSA_NORM_CASE(4)
  }
#undef DSA_NORM_CASE
  return launch_status();
}

dsa_status_t norm_fwd(const dsa_norm_t* p, const void* x, int64_t x_ld, const void* r, int64_t r_ld, const void* w,
                      void* y, float* scales, void* h, bool fp8, void* stream) {
  dsa_status_t st = check_norm(p);
  if (st != DSA_OK) return st;
  if (!ld_ok(x_ld, p) || (r != nullptr && !ld_ok(r_ld, p))) return DSA_ERR_INVALID_ARG;
  if ((r != nullptr) != (h != nullptr)) return DSA_ERR_INVALID_ARG;
  const size_t elem = p->dtype == DSA_BF16 ? 2 : 4;
  if (!aligned(x, elem) || !aligned(r, elem) || !aligned(w, elem) || !aligned(h, elem) ||
      !aligned(y, fp8 ? 1 : elem) || !aligned(scales, 4))
    return DSA_ERR_INVALID_ARG;
  if (p->rows == 0) return DSA_OK;
  if (!x || !y || (fp8 && !scales)) return DSA_ERR_INVALID_ARG;
  dsa::NormParams np;
  np.x = x;
  np.r = r;
  np.w = w;
  np.y = y;
  np.h = h;
  np.scales = scales;
  np.rows = p->rows;
  np.x_ld = x_ld;
  np.r_ld = r_ld;
  np.C = p->C;
  np.eps = p->eps;
  const NormShape sh = norm_shape(p->C, 4, 256);
  np.tpr = sh.tpr;
  const bool vec = p->C % 8 == 0 && vec_ok(x, x_ld, p) && vec_ok(r, r_ld, p) && vec_ok(w, 0, p) && vec_ok(h, 0, p) &&
                   (fp8 ? aligned(y, 8) : aligned(y, 16));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p->dtype == DSA_BF16)
    return fp8 ? launch_norm<__nv_bfloat16, true>(np, sh, vec, s) : launch_norm<__nv_bfloat16, false>(np, sh, vec, s);
  return fp8 ? launch_norm<float, true>(np, sh, vec, s) : launch_norm<float, false>(np, sh, vec, s);
}

// The backward's launch: block shape, blocks (each with a partial dw), and the stages of the
// shared-memory ring for `tensors` inputs (0: they do not fit twice, the kernel loads directly).
// Resident blocks: what 88 registers a thread allow, up to four, and each with two stages or more
// (both sides of these are measured beside the kernel).
struct NormBwdShape {
  NormShape sh;
  int blocks_per_sm, stages, J;
  size_t smem;
  unsigned grid;
};

NormBwdShape norm_bwd_shape(const dsa_norm_t* p, int tensors, bool vec) {
  NormBwdShape b;
  b.sh = norm_shape(p->C, 2, 256);
  const size_t elem = p->dtype == DSA_BF16 ? 2 : 4, rows = elem * p->C * tensors * b.sh.R;
  // rows within a warp: as many per thread and iteration as make a stage of about 24 KB
  b.J = 1;
  while (b.sh.tpr <= 32 && b.J < 16 && 2 * b.J * rows <= 24 * 1024) b.J *= 2;
  const size_t stage = b.J * rows;
  const int threads = b.sh.tpr * b.sh.R;
  b.stages = 0;
  b.blocks_per_sm = threads > 336 ? 1 : threads > 224 ? 2 : threads > 168 ? 3 : 4;
  for (int n = b.blocks_per_sm; n >= 1 && vec && b.stages == 0; --n) {
    const size_t room = size_t(220) * 1024 / n, need = 2048 + elem * p->C + 2 * stage;
    if (room < need) continue;
    const size_t fit = 2 + (room - need) / stage;
    b.stages = static_cast<int>(fit < dsa::norm::kMaxStages ? fit : dsa::norm::kMaxStages);
    b.blocks_per_sm = n;
  }
  const size_t dw = b.sh.R > 1 ? sizeof(float) * p->C : 0;  // the row slots' sums meet here
  const size_t ring = b.stages > 0 ? b.stages * stage + elem * p->C : 0;  // and the weight
  b.smem = ring > dw ? ring : dw;
  const int64_t G = static_cast<int64_t>(b.sh.R) * b.J, groups = (p->rows + G - 1) / G;
  b.grid = static_cast<unsigned>(groups < b.blocks_per_sm * kPlanSms ? groups : b.blocks_per_sm * kPlanSms);
  return b;
}

template <typename T, int NV, bool kDw, bool kWarpRow>
dsa_status_t launch_norm_bwd_nv(const dsa::NormBwdParams& np, const NormBwdShape& b, bool vec, cudaStream_t s) {
  const unsigned threads = b.sh.tpr * b.sh.R;
  if (b.stages > 0) {
    auto kernel = dsa::rmsnorm_bwd_kernel<T, NV, true, kDw, true, kWarpRow>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(b.smem)) != cudaSuccess)
      return DSA_ERR_CUDA;
    kernel<<<b.grid, threads + 32, b.smem, s>>>(np);
  } else if (vec) {
    // (rows within a warp always fit the ring)
    if constexpr (!kWarpRow)
      dsa::rmsnorm_bwd_kernel<T, NV, true, kDw, false, false><<<b.grid, threads, b.smem, s>>>(np);
  } else {
    dsa::rmsnorm_bwd_kernel<T, NV, false, kDw, false, kWarpRow><<<b.grid, threads, b.smem, s>>>(np);
  }
  return launch_status();
}

template <typename T, bool kDw>
dsa_status_t launch_norm_bwd(const dsa::NormBwdParams& np, const NormBwdShape& b, bool vec, cudaStream_t s) {
  if (b.sh.tpr <= 32)  // at most two vectors a thread
    return b.sh.NV == 1 ? launch_norm_bwd_nv<T, 1, kDw, true>(np, b, vec, s) : launch_norm_bwd_nv<T, 2, kDw, true>(np, b, vec, s);
  switch (b.sh.NV) {
    case 1: return launch_norm_bwd_nv<T, 1, kDw, false>(np, b, vec, s);
    case 2: return launch_norm_bwd_nv<T, 2, kDw, false>(np, b, vec, s);
    case 3: return launch_norm_bwd_nv<T, 3, kDw, false>(np, b, vec, s);
    default: return launch_norm_bwd_nv<T, 4, kDw, false>(np, b, vec, s);
  }
}

}  // namespace

extern "C" {

size_t dsa_cross_workspace_size(const dsa_cross_t* p, int32_t kind) {
  CrossPlan c;
  if (cross_plan(p, &c) != DSA_OK || (kind != DSA_WS_FWD && kind != DSA_WS_BWD)) return 0;
  return cross_workspace(p, c, kind, nullptr).bytes;
}

dsa_status_t dsa_fwd_cross(const dsa_cross_t* p, const dsa_view_t* q, const dsa_view_t* k, const dsa_view_t* v,
                           const int32_t* kv_len, const dsa_view_t* out, float* lse, void* workspace, size_t ws_bytes,
                           void* stream) {
  CrossPlan c;
  dsa_status_t st = cross_plan(p, &c);
  if (st != DSA_OK) return st;
  if (p->Lq == 0) return DSA_OK;
  if (!view_ok(q, p->B, p->heads, p->Lq, false) || !view_ok(out, p->B, p->heads, p->Lq, true) || lse == nullptr ||
      !aligned(lse, 4) || !aligned(kv_len, 4))
    return DSA_ERR_INVALID_ARG;
  if (p->Lk > 0 && (!view_ok(k, p->B, p->kv_heads, p->Lk, false) || !view_ok(v, p->B, p->kv_heads, p->Lk, false)))
    return DSA_ERR_INVALID_ARG;
  if (heads_broadcast(q, c)) cross_plan(p, &c, false);
  const CrossWorkspace ws = cross_workspace(p, c, DSA_WS_FWD, workspace);
  if (ws.bytes > 0 && (workspace == nullptr || ws_bytes < ws.bytes || !aligned(workspace, kAlign)))
    return DSA_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  dsa::CrossFwdParams fp;
  std::memset(&fp, 0, sizeof(fp));
  fp.kv_len = kv_len;
  fp.out = static_cast<__nv_bfloat16*>(out->data);
  fp.ob = out->stride[0];
  fp.oh = out->stride[1];
  fp.ol = out->stride[2];
  fp.lse = lse;
  fp.part_o = ws.part_o;
  fp.part_lse = ws.part_lse;
  fp.B = p->B;
  fp.heads = p->heads;
  fp.kv_heads = p->kv_heads;
  fp.group = c.group;
  fp.Lq = p->Lq;
  fp.Lk = p->Lk;
  fp.pk = c.pk;
  fp.tiles = c.tiles;
  fp.n_split = p->Lk > 0 ? c.split_q : 0;
  fp.n_units = static_cast<int>(c.units * c.split_q);
  fp.scale_log2 = p->scale * 1.4426950408889634f;
  fp.unit_cost = 4;
  if (p->Lk > 0) {
    CUtensorMap tq, tk, tv;
    int mq[3], mk[3], mv[3];
    const int box_rows = c.pk > 1 ? p->Lq : 128;
    if (!make_view_map(&tq, q, p->B, p->heads, c.group, p->Lq, box_rows, c.pk, mq) ||
        !make_view_map(&tk, k, p->B, p->kv_heads, 0, p->Lk, c.pair ? 64 : 128, 1, mk) ||
        !make_view_map(&tv, v, p->B, p->kv_heads, 0, p->Lk, 128, 1, mv))
      return DSA_ERR_CUDA;
    fp.q_bytes = static_cast<uint32_t>(box_rows * c.pk) * 256;  // per CTA
    fp.qg = mq[0];
    fp.qk = mq[1];
    fp.qb = mq[2];
    fp.kh = mk[1];
    fp.kb = mk[2];
    fp.vh = mv[1];
    fp.vb = mv[2];
    if (c.pair) {
      fp.tiles = static_cast<int>(c.group * ((static_cast<int64_t>(p->Lq) + 255) / 256));
      fp.n_units = p->B * p->kv_heads * fp.tiles;
      // measured on a 512 + 203-key pair alone: units of four and of two chunks take times of 9 : 5.7
      // (with a cost of 4 the CTAs of the short entry ran 212 us, those of the long one 186); a line
      // through those two lengths, other pairs of lengths are not measured
      fp.unit_cost = 12;
      CUtensorMap to;
      int mo[3];
      if (!make_view_map(&to, out, p->B, p->heads, c.group, p->Lq, 32, 1, mo)) return DSA_ERR_CUDA;
      return launch_pairs<dsa::cross_fwd_kernel<true>>(dsa::crossf::kSmemBytes, dsa::crossf::kThreads,
                                                       dsa::crossf::kRegsAtLaunch, fp.n_units, s, tq, tk, tv, to, fp);
    }
    unsigned grid = 0;
    st = persistent_grid(dsa::cross_fwd_kernel<false>, dsa::crossf::kSmemBytes, dsa::crossf::kRegsAtLaunch, fp.n_units,
                         &grid);
    if (st != DSA_OK) return st;
    dsa::cross_fwd_kernel<false><<<grid, dsa::crossf::kThreads, dsa::crossf::kSmemBytes, s>>>(tq, tk, tv, tq, fp);
    st = launch_status();
    if (st != DSA_OK || c.split_q == 1) return st;
  }
  dsa::cross_merge_kernel<<<static_cast<unsigned>(c.rows), 256, 0, s>>>(fp);  // without keys: O = 0, LSE = -inf
  return launch_status();
}

dsa_status_t dsa_bwd_cross(const dsa_cross_t* p, const dsa_view_t* q, const dsa_view_t* k, const dsa_view_t* v,
                           const dsa_view_t* out, const float* lse, const dsa_view_t* dout, const int32_t* kv_len,
                           const dsa_view_t* dq, const dsa_view_t* dk, const dsa_view_t* dv, void* workspace,
                           size_t ws_bytes, void* stream) {
  CrossPlan c;
  dsa_status_t st = cross_plan(p, &c);
  if (st != DSA_OK) return st;
  if (p->Lq > 0 && (!view_ok(q, p->B, p->heads, p->Lq, false) || !view_ok(out, p->B, p->heads, p->Lq, false) ||
                    !view_ok(dout, p->B, p->heads, p->Lq, false) || !view_ok(dq, p->B, p->heads, p->Lq, true) ||
                    lse == nullptr))
    return DSA_ERR_INVALID_ARG;
  if (p->Lk > 0 && (!view_ok(k, p->B, p->kv_heads, p->Lk, false) || !view_ok(v, p->B, p->kv_heads, p->Lk, false) ||
                    !view_ok(dk, p->B, p->kv_heads, p->Lk, true) || !view_ok(dv, p->B, p->kv_heads, p->Lk, true)))
    return DSA_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(kv_len, 4)) return DSA_ERR_INVALID_ARG;
  if (heads_broadcast(q, c) || heads_broadcast(dout, c)) cross_plan(p, &c, false);
  const CrossWorkspace ws = cross_workspace(p, c, DSA_WS_BWD, workspace);
  if (ws.bytes > 0 && (workspace == nullptr || ws_bytes < ws.bytes || !aligned(workspace, kAlign)))
    return DSA_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  dsa::CrossDqCombineParams cq;
  std::memset(&cq, 0, sizeof(cq));
  cq.B = p->B;
  cq.heads = p->heads;
  cq.Lq = p->Lq;
  cq.part = ws.dq_part;
  if (p->Lq > 0) {
    cq.dq = static_cast<__nv_bfloat16*>(dq->data);
    copy_strides(cq.s, dq);
  }
  if (p->Lk == 0) return p->Lq > 0 ? launch_dq_combine(cq, s) : DSA_OK;  // no keys: dq = 0

  dsa::CrossShape shape;
  std::memset(&shape, 0, sizeof(shape));
  shape.kv_len = kv_len;
  shape.B = p->B;
  shape.heads = p->heads;
  shape.kv_heads = p->kv_heads;
  shape.group = c.group;
  shape.Lq = p->Lq;
  shape.Lk = p->Lk;
  shape.pk = c.pk;
  shape.tiles = c.tiles;
  shape.n_split = c.split_q;
  shape.n_units = static_cast<int>(c.units * c.split_q);
  shape.unit_cost = 4;

  dsa::CrossKvParams kp;
  std::memset(&kp, 0, sizeof(kp));
  static_cast<dsa::CrossShape&>(kp) = shape;
  kp.per_unit = c.tiles;
  kp.lse = lse;
  kp.delta = ws.delta;
  kp.dk = static_cast<__nv_bfloat16*>(dk->data);
  kp.dv = static_cast<__nv_bfloat16*>(dv->data);
  copy_strides(kp.dk_s, dk);
  copy_strides(kp.dv_s, dv);
  kp.dk_part = ws.dk_part;
  kp.dv_part = ws.dv_part;
  kp.scale = p->scale;
  kp.scale_log2 = p->scale * 1.4426950408889634f;
  if (p->Lq == 0) {  // no queries: dk = dv = 0
    dsa::cross_kv_combine<<<dim3(static_cast<unsigned>(c.kv_units), 2, 8), 256, 0, s>>>(kp, 0);
    return launch_status();
  }

  dsa::CrossPrepParams pp;
  pp.o = static_cast<const __nv_bfloat16*>(out->data);
  pp.dout = static_cast<const __nv_bfloat16*>(dout->data);
  copy_strides(pp.o_s, out);
  copy_strides(pp.do_s, dout);
  pp.delta = ws.delta;
  pp.B = p->B;
  pp.heads = p->heads;
  pp.Lq = p->Lq;
  dsa::cross_preprocess<<<static_cast<unsigned>((c.rows + 63) / 64), 256, 0, s>>>(pp);
  st = launch_status();
  if (st != DSA_OK) return st;

  CUtensorMap tq, tdo, tk, tv, tdq;
  int mq[3], mdo[3], mk[3], mv[3], mdq[3];
  const int box_rows = c.pk > 1 ? p->Lq : 128;
  if (!make_view_map(&tq, q, p->B, p->heads, c.group, p->Lq, box_rows, c.pk, mq) ||
      !make_view_map(&tdo, dout, p->B, p->heads, c.group, p->Lq, box_rows, c.pk, mdo) ||
      !make_view_map(&tk, k, p->B, p->kv_heads, 0, p->Lk, 128, 1, mk) ||
      !make_view_map(&tv, v, p->B, p->kv_heads, 0, p->Lk, 128, 1, mv) ||
      !make_view_map(&tdq, dq, p->B, p->heads, c.group, p->Lq, 32, 1, mdq))
    return DSA_ERR_CUDA;
  {
    kp.q_bytes = static_cast<uint32_t>(box_rows * c.pk) * 256;
    kp.qg = mq[0];
    kp.qk = mq[1];
    kp.qb = mq[2];
    kp.dg = mdo[0];
    kp.dkv = mdo[1];
    kp.db = mdo[2];
    kp.kh = mk[1];
    kp.kb = mk[2];
    kp.vh = mv[1];
    kp.vb = mv[2];
    // one CTA per SM (two slots of the workspace each), no more than query chunks
    const int64_t work = c.kv_units * c.tiles;
    unsigned grid = 0;
    st = persistent_grid(dsa::cross_kv_kernel, dsa::crosskv::kSmemBytes, dsa::crosskv::kRegsAtLaunch,
                         work < kPlanSms ? work : kPlanSms, &grid);
    if (st != DSA_OK) return st;
    dsa::cross_kv_kernel<<<grid, dsa::crosskv::kThreads, dsa::crosskv::kSmemBytes, s>>>(tq, tdo, tk, tv, kp);
    st = launch_status();
    if (st != DSA_OK) return st;
    dsa::cross_kv_combine<<<dim3(static_cast<unsigned>(c.kv_units) + grid, 2, 8), 256, 0, s>>>(kp, static_cast<int>(grid));
    st = launch_status();
    if (st != DSA_OK) return st;
  }
  dsa::CrossDqParams dp;
  std::memset(&dp, 0, sizeof(dp));
  static_cast<dsa::CrossShape&>(dp) = shape;
  dp.lse = lse;
  dp.delta = ws.delta;
  dp.dq = static_cast<__nv_bfloat16*>(dq->data);
  copy_strides(dp.dq_s, dq);
  dp.dq_part = ws.dq_part;
  dp.scale = p->scale;
  dp.scale_log2 = p->scale * 1.4426950408889634f;
  dp.q_bytes = kp.q_bytes;
  dp.qg = mq[0];
  dp.qk = mq[1];
  dp.qb = mq[2];
  dp.dg = mdo[0];
  dp.dk = mdo[1];
  dp.db = mdo[2];
  dp.kh = mk[1];
  dp.kb = mk[2];
  dp.vh = mv[1];
  dp.vb = mv[2];
  if (c.pair) {
    CUtensorMap tk64, tv64;
    if (!make_view_map(&tk64, k, p->B, p->kv_heads, 0, p->Lk, 64, 1, mk) ||
        !make_view_map(&tv64, v, p->B, p->kv_heads, 0, p->Lk, 64, 1, mv))
      return DSA_ERR_CUDA;
    dp.tiles = static_cast<int>(c.group * ((static_cast<int64_t>(p->Lq) + 255) / 256));
    dp.n_units = p->B * p->kv_heads * dp.tiles;
    // measured on the same pair of lengths: units of four and of two chunks take times of 14.2 : 7.0
    // (with a cost of 4 the CTAs of the long entry ran 510 thousand clocks, those of the short one
    // 441).  It is not a unit's own start and end alone, which take longer: the two chunks stay in
    // the K and V rings from unit to unit, the four do not
    dp.unit_cost = 1;
    return launch_pairs<dsa::cross_dq_kernel<true>>(dsa::crossdq::kSmemBytes, dsa::crossdq::kThreads,
                                                    dsa::bdq::kRegsAtLaunch, dp.n_units, s, tq, tdo, tk64, tk, tv64, tdq, dp);
  }
  unsigned grid = 0;
  st = persistent_grid(dsa::cross_dq_kernel<false>, dsa::crossdq::kSmemBytes, dsa::bdq::kRegsAtLaunch, dp.n_units, &grid);
  if (st != DSA_OK) return st;
  dsa::cross_dq_kernel<false><<<grid, dsa::crossdq::kThreads, dsa::crossdq::kSmemBytes, s>>>(tq, tdo, tk, tk, tv, tdq, dp);
  st = launch_status();
  if (st != DSA_OK || c.split_q == 1) return st;
  cq.n_part = c.split_q;
  return launch_dq_combine(cq, s);
}

dsa_status_t dsa_rope_table(const int32_t* grid, const int32_t* axes, const double* start, const double* step,
                            double theta, float* table, void* stream) {
  if (!grid || !axes || !start || !step || !table || !aligned(table, 8)) return DSA_ERR_INVALID_ARG;
  if (!rope_axes_ok(axes) || !(theta > 0.0) || !std::isfinite(theta)) return DSA_ERR_INVALID_ARG;
  dsa::RopeTableParams rp;
  int64_t n = 0;
  for (int a = 0; a < 3; ++a) {
    if (grid[a] <= 0 || !std::isfinite(start[a]) || !std::isfinite(step[a])) return DSA_ERR_INVALID_ARG;
    rp.n[a] = grid[a];
    rp.pairs[a] = axes[a] / 2;
    rp.start[a] = start[a];
    rp.step[a] = step[a];
    n += static_cast<int64_t>(rp.n[a]) * rp.pairs[a];
  }
  if (n > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  rp.log_theta = std::log(theta);
  rp.table = reinterpret_cast<float2*>(table);
  dsa::rope_table_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, static_cast<cudaStream_t>(stream)>>>(rp);
  return launch_status();
}

dsa_status_t dsa_rope(const dsa_rope_t* p, const float* table, const dsa_view_t* q, const dsa_view_t* q_out,
                      const dsa_view_t* k, const dsa_view_t* k_out, void* stream) {
  if (p == nullptr || p->B <= 0 || p->heads <= 0 || p->d <= 0 || p->T <= 0 || p->H <= 0 || p->W <= 0)
    return DSA_ERR_INVALID_ARG;
  if (p->dtype != DSA_F32 && p->dtype != DSA_BF16) return DSA_ERR_INVALID_ARG;
  if ((p->interleaved & ~1) != 0 || (p->inverse & ~1) != 0) return DSA_ERR_INVALID_ARG;
  if (!rope_axes_ok(p->axes)) return DSA_ERR_INVALID_ARG;
  const int64_t R = static_cast<int64_t>(p->axes[0]) + p->axes[1] + p->axes[2];
  if (R > p->d) return DSA_ERR_INVALID_ARG;
  if (!table || !aligned(table, 8) || !q || !q_out || (k == nullptr) != (k_out == nullptr)) return DSA_ERR_INVALID_ARG;
  const int64_t N = static_cast<int64_t>(p->T) * p->H * p->W;
  const int64_t entries = static_cast<int64_t>(p->T) * (p->axes[0] / 2) + static_cast<int64_t>(p->H) * (p->axes[1] / 2) +
                          static_cast<int64_t>(p->W) * (p->axes[2] / 2);
  if (N > INT32_MAX || entries > INT32_MAX || p->B > 65535 || p->d > 65536 || N * p->d > (int64_t(1) << 38))
    return DSA_ERR_UNSUPPORTED;
  const size_t elem = p->dtype == DSA_BF16 ? 2 : 4;
  const int64_t vec = 16 / elem;  // elements of 16 bytes
  const bool halves = p->interleaved == 0;
  bool vector = p->d % 8 == 0 && (halves ? R / 2 : R) % 8 == 0;
  dsa::RopeParams rp;
  std::memset(&rp, 0, sizeof(rp));
  const dsa_view_t* in[2] = {q, k};
  const dsa_view_t* out[2] = {q_out, k_out};
  const int n_tens = k != nullptr ? 2 : 1;
  for (int t = 0; t < n_tens; ++t) {
    for (int io = 0; io < 2; ++io) {
      const dsa_view_t* v = io ? out[t] : in[t];
      if (v->data == nullptr || !aligned(v->data, elem)) return DSA_ERR_INVALID_ARG;
      const int64_t n[3] = {p->B, p->heads, N};
      dsa::RopeView& rv = io ? rp.so[t] : rp.si[t];
      int64_t s[3];
      for (int a = 0; a < 3; ++a) {
        s[a] = n[a] <= 1 ? 0 : v->stride[a];
        if (s[a] < 0 || (n[a] > 1 && io && s[a] < p->d)) return DSA_ERR_INVALID_ARG;
        if (s[a] % vec != 0) vector = false;
      }
      rv.b = s[0];
      rv.h = s[1];
      rv.n = s[2];
      if (!aligned(v->data, 16)) vector = false;
    }
    rp.in[t] = in[t]->data;
    rp.out[t] = out[t]->data;
  }
  rp.table = reinterpret_cast<const float2*>(table);
  rp.H = p->H;
  rp.W = p->W;
  rp.N = static_cast<int>(N);
  rp.heads = p->heads;
  rp.d = p->d;
  rp.inverse = p->inverse;
  for (int a = 0; a < 3; ++a) rp.pairs[a] = p->axes[a] / 2;
  rp.off[1] = p->T * rp.pairs[0];
  rp.off[2] = rp.off[1] + p->H * rp.pairs[1];
  const int half = static_cast<int>(R / 2);
  const int items = vector ? (halves ? half / 8 + (p->d - 2 * half) / 8 : p->d / 8) : half + (p->d - 2 * half);
  // heads per thread: all of them when the tokens alone fill the GPU, fewer for small grids
  const int64_t blocks = (N * items + 255) / 256;
  int64_t groups = (8 * kPlanSms + blocks * p->B - 1) / (blocks * p->B);
  const int64_t most = (p->heads + 3) / 4;  // at least the four heads a thread loads together
  if (groups > most) groups = most;
  rp.hpt = static_cast<int>((p->heads + groups - 1) / groups);
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((p->heads + rp.hpt - 1) / rp.hpt),
                  static_cast<unsigned>(p->B));
  if (blocks > INT32_MAX || grid.y > 65535) return DSA_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
#define DSA_ROPE_LAUNCH(K, T)                                    \
  if (halves)                                                    \
    dsa::K<T, true><<<grid, 256, 0, s>>>(rp, items, n_tens);     \
  else                                                           \
    dsa::K<T, false><<<grid, 256, 0, s>>>(rp, items, n_tens);
  if (vector) {
    if (p->dtype == DSA_BF16) {
      DSA_ROPE_LAUNCH(rope_kernel, __nv_bfloat16)
    } else {
      DSA_ROPE_LAUNCH(rope_kernel, float)
    }
  } else {
    if (p->dtype == DSA_BF16) {
      DSA_ROPE_LAUNCH(rope_any_kernel, __nv_bfloat16)
    } else {
      DSA_ROPE_LAUNCH(rope_any_kernel, float)
    }
  }
#undef DSA_ROPE_LAUNCH
  return launch_status();
}

dsa_status_t dsa_rmsnorm(const dsa_norm_t* p, const void* x, int64_t x_ld, const void* residual, int64_t r_ld,
                         const void* weight, void* y, void* sum, void* stream) {
  return norm_fwd(p, x, x_ld, residual, r_ld, weight, y, nullptr, sum, false, stream);
}

dsa_status_t dsa_rmsnorm_fp8(const dsa_norm_t* p, const void* x, int64_t x_ld, const void* residual, int64_t r_ld,
                             const void* weight, void* y8, float* scales, void* sum, void* stream) {
  return norm_fwd(p, x, x_ld, residual, r_ld, weight, y8, scales, sum, true, stream);
}

size_t dsa_rmsnorm_bwd_workspace_size(const dsa_norm_t* p) {
  if (check_norm(p) != DSA_OK) return 0;
  // the most blocks any of its forms launches (four per SM, or one per row group)
  const int64_t groups = p->rows < 4 * kPlanSms ? p->rows : 4 * kPlanSms;
  return round_up(sizeof(float) * static_cast<size_t>(groups > 0 ? groups : 1) * p->C, kAlign);
}

dsa_status_t dsa_rmsnorm_bwd(const dsa_norm_t* p, const void* h, int64_t h_ld, const void* weight, const void* dy,
                             int64_t dy_ld, const void* dh, int64_t dh_ld, void* dx, void* dweight, void* workspace,
                             size_t ws_bytes, void* stream) {
  dsa_status_t st = check_norm(p);
  if (st != DSA_OK) return st;
  if (!ld_ok(h_ld, p) || !ld_ok(dy_ld, p) || (dh != nullptr && !ld_ok(dh_ld, p))) return DSA_ERR_INVALID_ARG;
  if (dweight != nullptr && weight == nullptr) return DSA_ERR_INVALID_ARG;
  const size_t elem = p->dtype == DSA_BF16 ? 2 : 4;
  if (!aligned(h, elem) || !aligned(dy, elem) || !aligned(dh, elem) || !aligned(weight, elem) || !aligned(dx, elem) ||
      !aligned(dweight, elem))
    return DSA_ERR_INVALID_ARG;
  if (p->rows > 0 && (!h || !dy || !dx)) return DSA_ERR_INVALID_ARG;
  const bool vec = p->C % 8 == 0 && vec_ok(h, h_ld, p) && vec_ok(dy, dy_ld, p) && vec_ok(dh, dh_ld, p) &&
                   vec_ok(weight, 0, p) && vec_ok(dx, 0, p);
  const NormBwdShape b = norm_bwd_shape(p, dh != nullptr ? 3 : 2, vec);
  if (dweight != nullptr && p->rows > 0 &&
      (workspace == nullptr || ws_bytes < dsa_rmsnorm_bwd_workspace_size(p) || !aligned(workspace, kAlign)))
    return DSA_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* part = static_cast<float*>(workspace);
  if (p->rows > 0) {
    dsa::NormBwdParams np;
    np.h = h;
    np.w = weight;
    np.dy = dy;
    np.dh = dh;
    np.dx = dx;
    np.dw_part = part;
    np.rows = p->rows;
    np.h_ld = h_ld;
    np.dy_ld = dy_ld;
    np.dh_ld = dh_ld;
    np.C = p->C;
    np.tpr = b.sh.tpr;
    np.J = b.J;
    np.stages = b.stages;
    np.eps = p->eps;
    if (p->dtype == DSA_BF16)
      st = dweight ? launch_norm_bwd<__nv_bfloat16, true>(np, b, vec, s) : launch_norm_bwd<__nv_bfloat16, false>(np, b, vec, s);
    else
      st = dweight ? launch_norm_bwd<float, true>(np, b, vec, s) : launch_norm_bwd<float, false>(np, b, vec, s);
    if (st != DSA_OK) return st;
  }
  if (dweight == nullptr) return DSA_OK;
  const unsigned blocks = static_cast<unsigned>((p->C + 31) / 32);
  if (p->dtype == DSA_BF16)
    dsa::rmsnorm_dw_kernel<__nv_bfloat16><<<blocks, 256, 0, s>>>(part, static_cast<int>(b.grid), p->C,
                                                                 static_cast<__nv_bfloat16*>(dweight));
  else
    dsa::rmsnorm_dw_kernel<float><<<blocks, 256, 0, s>>>(part, static_cast<int>(b.grid), p->C,
                                                         static_cast<float*>(dweight));
  return launch_status();
}

}  // extern "C"
