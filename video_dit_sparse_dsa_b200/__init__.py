"""3D Deformable Slide Attention (3D-DSA) on NVIDIA B200 (sm_100a).

Thin Python binding of the C ABI in ``include/dsa.h`` (argument marshalling only: every
step of the computation runs in the library's CUDA kernels).  PyTorch provides device
memory and streams.  The library is built in-tree by ``video_dit_sparse_dsa_b200.build``;
if it is missing, every entry point raises: there is no CPU fallback.

Operator ("MegaSlide-DiT: Memory-Centric Adaptation and Deformable Local Attention for
Efficient Video Diffusion", abstract; tile-granular window as in "Fast Video Generation
with Sliding Tile Attention", abstract): for query tile i with integer offset o, the
window of w' = min(w, G) tiles per axis starts at clamp(i + o - floor(w'/2), 0, G - w');
each query token attends with softmax(scale q K^T) V to exactly the tokens of those tiles.

Tensors: q, k, v, out, dout, dq, dk, dv are ``[B, heads, T, H, W, d]`` contiguous CUDA
tensors (bf16 with d = 128, or fp32 with d in {64, 128} for the forward); lse is
``[B, heads, T, H, W]`` fp32; tile offsets are int32 ``[nTiles, 3]`` in tile units.

Around it in a transformer block: ``forward_cross`` / ``backward_cross`` (cross attention to an
encoder's states), ``rope_table`` / ``rope`` (rotary positions over the token grid) and
``rms_norm`` / ``rms_norm_fp8`` / ``rms_norm_backward`` (root-mean-square norm with the
residual's addition).  These take strided tensors (views of a projection).

Calls run on the device of their tensors, whichever device is current, and on ``stream`` (default:
that device's current stream).  A call on another stream than the current one is ordered after
what is on that stream, as its kernels would be, and allocates what it needs there: the caller
orders it after the work that makes its inputs, and what reads its results after it.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libdsa_b200.so")

DSA_F32, DSA_BF16 = 0, 1
DSA_WS_FWD, DSA_WS_BWD = 0, 1
_STATUS = {0: "DSA_OK", 1: "DSA_ERR_INVALID_ARG", 2: "DSA_ERR_UNSUPPORTED", 3: "DSA_ERR_CUDA",
           4: "DSA_ERR_TIMEOUT", 5: "DSA_ERR_WORKSPACE", 6: "DSA_ERR_DEVICE"}

# kernel launches of one dsa_fwd call (planner, forward) and of one dsa_bwd call (planner,
# the inverse map's count, scan and fill, D preprocess, backward, dQ conversion)
FWD_LAUNCHES = 2
BWD_LAUNCHES = 7

# every symbol include/dsa.h declares
EXPORTS = ("dsa_version", "dsa_status_string", "dsa_plan_shape", "dsa_workspace_size", "dsa_plan", "dsa_fwd",
           "dsa_fwd_host_bytes", "dsa_fwd_host", "dsa_bwd", "dsa_device_status", "dsa_fwd_noalloc",
           "dsa_list_workspace_size", "dsa_fwd_list", "dsa_bwd_list", "dsa_plan_heads", "dsa_block_map",
           "dsa_lstsq_workspace_size", "dsa_lstsq_factor", "dsa_lstsq_solve", "dsa_prefix_workspace_size",
           "dsa_fwd_prefix", "dsa_bwd_prefix_workspace_size", "dsa_bwd_prefix", "dsa_selftest_wait",
           "dsa_cross_workspace_size", "dsa_fwd_cross", "dsa_bwd_cross", "dsa_rope_table", "dsa_rope", "dsa_rmsnorm",
           "dsa_rmsnorm_fp8", "dsa_rmsnorm_bwd_workspace_size", "dsa_rmsnorm_bwd")


class DsaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_STATUS.get(status, status)}")


class Problem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("heads", ctypes.c_int32), ("d", ctypes.c_int32), ("T", ctypes.c_int32),
                ("H", ctypes.c_int32), ("W", ctypes.c_int32), ("tile", ctypes.c_int32 * 3),
                ("window", ctypes.c_int32 * 3), ("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


class View(ctypes.Structure):
    """dsa_view_t: a [B, heads, rows, d] tensor through its strides."""
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64 * 3)]


class Cross(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("d", ctypes.c_int32),
                ("Lq", ctypes.c_int32), ("Lk", ctypes.c_int32), ("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


class Rope(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("heads", ctypes.c_int32), ("d", ctypes.c_int32), ("T", ctypes.c_int32),
                ("H", ctypes.c_int32), ("W", ctypes.c_int32), ("axes", ctypes.c_int32 * 3),
                ("interleaved", ctypes.c_int32), ("inverse", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class Norm(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("C", ctypes.c_int32), ("eps", ctypes.c_float), ("dtype", ctypes.c_int32)]


_lib = None


def load_library(path: Optional[str] = None):
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"3D-DSA CUDA library not built ({p}); run python -m video_dit_sparse_dsa_b200.build")
    lib = ctypes.CDLL(p)
    vp, sz, i32, i32p = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)
    pp = ctypes.POINTER(Problem)
    lib.dsa_version.restype = i32
    lib.dsa_version.argtypes = []
    lib.dsa_status_string.restype = ctypes.c_char_p
    lib.dsa_status_string.argtypes = [ctypes.c_int]
    lib.dsa_plan_shape.argtypes = [pp, i32p, i32p]
    lib.dsa_workspace_size.restype = sz
    lib.dsa_workspace_size.argtypes = [pp, i32]
    lib.dsa_plan.argtypes = [pp, vp, vp, vp, vp, vp, vp]
    lib.dsa_fwd.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.dsa_fwd_host_bytes.restype = sz
    lib.dsa_fwd_host_bytes.argtypes = [pp]
    lib.dsa_fwd_host.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.dsa_bwd.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.dsa_device_status.argtypes = [vp, i32p, i32p]
    lib.dsa_fwd_noalloc.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp]
    lib.dsa_list_workspace_size.restype = sz
    lib.dsa_list_workspace_size.argtypes = [pp, i32, i32, i32]
    lib.dsa_fwd_list.argtypes = [pp, vp, vp, vp, vp, vp, i32, i32, vp, vp, vp]
    lib.dsa_bwd_list.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, vp, vp, vp, vp, sz, vp]
    lib.dsa_plan_heads.argtypes = [pp, vp, vp, vp, vp]
    lib.dsa_block_map.argtypes = [pp, vp, vp, vp, vp, vp, i32, i32, vp, vp]
    lib.dsa_lstsq_workspace_size.restype = sz
    lib.dsa_lstsq_workspace_size.argtypes = [i32, i32, i32]
    lib.dsa_lstsq_factor.argtypes = [i32, i32, vp, ctypes.c_float, vp, vp]
    lib.dsa_lstsq_solve.argtypes = [i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
    lib.dsa_prefix_workspace_size.restype = sz
    lib.dsa_prefix_workspace_size.argtypes = [pp, i32]
    lib.dsa_fwd_prefix.argtypes = [pp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.dsa_selftest_wait.argtypes = [vp]
    lib.dsa_bwd_prefix_workspace_size.restype = sz
    lib.dsa_bwd_prefix_workspace_size.argtypes = [pp, i32]
    lib.dsa_bwd_prefix.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                   vp, vp, sz, vp]
    cp, wp, rp, np_, i64 = ctypes.POINTER(Cross), ctypes.POINTER(View), ctypes.POINTER(Rope), ctypes.POINTER(Norm), ctypes.c_int64
    i32x3, f64x3 = ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_double)
    lib.dsa_cross_workspace_size.restype = sz
    lib.dsa_cross_workspace_size.argtypes = [cp, i32]
    lib.dsa_fwd_cross.argtypes = [cp, wp, wp, wp, vp, wp, vp, vp, sz, vp]
    lib.dsa_bwd_cross.argtypes = [cp, wp, wp, wp, wp, vp, wp, vp, wp, wp, wp, vp, sz, vp]
    lib.dsa_rope_table.argtypes = [i32x3, i32x3, f64x3, f64x3, ctypes.c_double, vp, vp]
    lib.dsa_rope.argtypes = [rp, vp, wp, wp, wp, wp, vp]
    lib.dsa_rmsnorm.argtypes = [np_, vp, i64, vp, i64, vp, vp, vp, vp]
    lib.dsa_rmsnorm_fp8.argtypes = [np_, vp, i64, vp, i64, vp, vp, vp, vp, vp]
    lib.dsa_rmsnorm_bwd_workspace_size.restype = sz
    lib.dsa_rmsnorm_bwd_workspace_size.argtypes = [np_]
    lib.dsa_rmsnorm_bwd.argtypes = [np_, vp, i64, vp, vp, i64, vp, i64, vp, vp, vp, sz, vp]
    for name in ("dsa_plan_shape", "dsa_plan", "dsa_fwd", "dsa_fwd_host", "dsa_bwd", "dsa_device_status",
                 "dsa_fwd_noalloc", "dsa_fwd_list", "dsa_bwd_list", "dsa_plan_heads", "dsa_block_map",
                 "dsa_lstsq_factor", "dsa_lstsq_solve", "dsa_fwd_prefix", "dsa_bwd_prefix",
                 "dsa_selftest_wait", "dsa_fwd_cross", "dsa_bwd_cross", "dsa_rope_table", "dsa_rope", "dsa_rmsnorm",
                 "dsa_rmsnorm_fp8", "dsa_rmsnorm_bwd"):
        getattr(lib, name).restype = ctypes.c_int
    if path is None:
        _lib = lib
    return lib


def head_range(n_slices: int, rank: int, world: int):
    """The (batch, head) slices [lo, hi) of a problem with n_slices = B * heads that rank
    `rank` of `world` takes when one problem is split over GPUs by heads.  Slices are
    independent problems (each has its own softmax), so ranks run the same calls on their
    slices with no collective; contiguous ranges of near-equal size, the first
    n_slices % world ranks one slice longer."""
    if world <= 0 or not 0 <= rank < world:
        raise ValueError(f"rank {rank} of {world}")
    base, extra = divmod(int(n_slices), world)
    lo = rank * base + min(rank, extra)
    return lo, lo + base + (1 if rank < extra else 0)


def make_problem(B, heads, d, grid, tile, window, scale=None, dtype=DSA_BF16) -> Problem:
    p = Problem()
    p.B, p.heads, p.d = int(B), int(heads), int(d)
    p.T, p.H, p.W = (int(x) for x in grid)
    for a in range(3):
        p.tile[a] = int(tile[a])
        p.window[a] = int(window[a])
    p.scale = float(1.0 / math.sqrt(d)) if scale is None else float(scale)
    p.dtype = int(dtype)
    return p


def _problem_of(q: torch.Tensor, tile, window, scale) -> Problem:
    if q.dim() != 6:
        raise ValueError("q must be [B, heads, T, H, W, d]")
    if q.dtype == torch.bfloat16:
        dt = DSA_BF16
    elif q.dtype == torch.float32:
        dt = DSA_F32
    else:
        raise ValueError(f"unsupported dtype {q.dtype}")
    B, heads, T, H, W, d = q.shape
    return make_problem(B, heads, d, (T, H, W), tile, window, scale, dt)


def _check(st: int, what: str):
    if st != 0:
        raise DsaError(st, what)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t: torch.Tensor, name: str, like: torch.Tensor, dtype=None, numel: Optional[int] = None):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, q on {like.device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")


def _need_workspace(ws: torch.Tensor, device: torch.device) -> int:
    """The bytes of a workspace (whether they suffice, the library checks)."""
    if not ws.is_contiguous() or ws.device != device:
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return ws.numel() * ws.element_size()


class _On:
    """Runs a call on a device and on ``stream`` (default: that device's current stream).  What the
    call allocates comes from that stream's memory: a block of another stream's (the current
    one's) may still be in use by work queued there, which nothing orders before this call.
    (The raw stream and device lookups: a Stream object and a device guard cost a small call more
    host time than its kernel takes.)"""
    __slots__ = ("device", "index", "guard", "ptr", "side")

    def __init__(self, device: torch.device, stream):
        if device.type != "cuda":
            raise ValueError("tensors must be CUDA tensors")
        self.device, self.index = device, device.index
        own = torch._C._cuda_getCurrentRawStream(self.index)
        self.ptr = own if stream is None else _stream(stream)
        self.side = None  # the call's stream, where it is not the current one
        if self.ptr != own:
            self.side = (torch.cuda.ExternalStream(self.ptr, device=device) if self.ptr else
                         torch.cuda.default_stream(device))

    def __enter__(self):
        self.guard = None
        if torch._C._cuda_getDevice() != self.index:
            self.guard = torch.cuda.device(self.index)
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def scratch(self, n_bytes: int):
        """Memory of the call's own (freed after it on the host, so reused on its stream alone)."""
        return self._make(torch.empty, n_bytes, dtype=torch.uint8, device=self.device) if n_bytes else None

    def empty(self, shape, dtype: torch.dtype) -> torch.Tensor:
        if self.side is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        return self._result(torch.empty, shape, dtype=dtype, device=self.device)

    def empty_like(self, t: torch.Tensor) -> torch.Tensor:
        return torch.empty_like(t) if self.side is None else self._result(torch.empty_like, t)

    def _make(self, f, *args, **kw) -> torch.Tensor:
        if self.side is None:
            return f(*args, **kw)
        with torch.cuda.stream(self.side):
            return f(*args, **kw)

    def _result(self, f, *args, **kw) -> torch.Tensor:
        """On another stream: a tensor that the caller gets, and may use and drop on its current one."""
        t = self._make(f, *args, **kw)
        t.record_stream(torch.cuda.current_stream(self.device))
        return t


def plan_shape(problem: Problem):
    lib = load_library()
    n, wt = ctypes.c_int32(), ctypes.c_int32()
    _check(lib.dsa_plan_shape(ctypes.byref(problem), ctypes.byref(n), ctypes.byref(wt)), "dsa_plan_shape")
    return n.value, wt.value


def workspace_size(problem: Problem, backward: bool = False) -> int:
    return int(load_library().dsa_workspace_size(ctypes.byref(problem), DSA_WS_BWD if backward else DSA_WS_FWD))


def workspace(problem: Problem, device, backward: bool = False) -> torch.Tensor:
    """A device workspace of the right size (torch's caching allocator returns 512-byte
    aligned blocks)."""
    return torch.empty(max(workspace_size(problem, backward), 256), dtype=torch.uint8, device=device)


def plan(problem: Problem, offsets: torch.Tensor, inverse: bool = True, stream=None):
    """Run the window planner.  Returns (starts, kv_tiles[, row_ptr, q_tiles]) on the device."""
    lib = load_library()
    n, wt = plan_shape(problem)
    if not offsets.is_cuda or offsets.dtype != torch.int32 or not offsets.is_contiguous() or offsets.numel() != 3 * n:
        raise ValueError("offsets must be a contiguous int32 CUDA tensor [nTiles, 3]")
    on = _On(offsets.device, stream)
    starts = on.empty((n, 3), torch.int32)
    kv = on.empty((n, wt), torch.int32)
    row_ptr = on.empty((n + 1,), torch.int32) if inverse else None
    q_tiles = on.empty((n * wt,), torch.int32) if inverse else None
    with on:
        _check(lib.dsa_plan(ctypes.byref(problem), _ptr(offsets), _ptr(starts), _ptr(kv), _ptr(row_ptr), _ptr(q_tiles),
                            ctypes.c_void_p(on.ptr)), "dsa_plan")
    return (starts, kv, row_ptr, q_tiles) if inverse else (starts, kv)


def forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, offsets: torch.Tensor, tile: Sequence[int],
            window: Sequence[int], scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
            lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
    """3D-DSA forward.  Returns (out, lse)."""
    lib = load_library()
    p = _problem_of(q, tile, window, scale)
    for t, name in ((k, "k"), (v, "v")):
        _need(t, name, q, q.dtype)
        if t.shape != q.shape:
            raise ValueError(f"{name} shape {tuple(t.shape)} != q shape {tuple(q.shape)}")
    _need(q, "q", q)
    _need(offsets, "offsets", q, torch.int32, 3 * plan_shape(p)[0])
    on = _On(q.device, stream)
    if out is None:
        out = on.empty_like(q)
    if lse is None:
        lse = on.empty(q.shape[:5], torch.float32)
    _need(out, "out", q, q.dtype, q.numel())
    _need(lse, "lse", q, torch.float32, q.shape[:5].numel())
    if ws is None:
        ws = on.scratch(max(workspace_size(p), 256))
    n_ws = _need_workspace(ws, q.device)
    with on:
        _check(lib.dsa_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(offsets), _ptr(out), _ptr(lse), _ptr(ws),
                           n_ws, ctypes.c_void_p(on.ptr)), "dsa_fwd")
    return out, lse


def prefix_workspace_size(problem: Problem, L_text: int) -> int:
    return int(load_library().dsa_prefix_workspace_size(ctypes.byref(problem), int(L_text)))


def forward_prefix(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, offsets: torch.Tensor, q_text: torch.Tensor,
                   k_text: torch.Tensor, v_text: torch.Tensor, tile: Sequence[int], window: Sequence[int],
                   scale: Optional[float] = None, ws: Optional[torch.Tensor] = None, stream=None):
    """3D-DSA with a text prefix: video queries over their windows and every text key, text
    queries over every key.  q, k, v: [B, heads, T, H, W, 128]; q_text, k_text, v_text:
    [B, heads, L_text, 128].  Returns (out, lse, out_text, lse_text)."""
    lib = load_library()
    p = _problem_of(q, tile, window, scale)
    for t, name in ((k, "k"), (v, "v")):
        _need(t, name, q, q.dtype)
        if t.shape != q.shape:
            raise ValueError(f"{name} shape {tuple(t.shape)} != q shape {tuple(q.shape)}")
    _need(q, "q", q)
    _need(offsets, "offsets", q, torch.int32, 3 * plan_shape(p)[0])
    if q_text.dim() != 4 or tuple(q_text.shape[:2]) != tuple(q.shape[:2]) or q_text.shape[3] != q.shape[5]:
        raise ValueError(f"q_text shape {tuple(q_text.shape)} does not match q {tuple(q.shape)}")
    for t, name in ((q_text, "q_text"), (k_text, "k_text"), (v_text, "v_text")):
        _need(t, name, q, q.dtype)
        if t.shape != q_text.shape:
            raise ValueError(f"{name} shape {tuple(t.shape)} != q_text shape {tuple(q_text.shape)}")
    L_text = int(q_text.shape[2])
    on = _On(q.device, stream)
    out = on.empty_like(q)
    lse = on.empty(q.shape[:5], torch.float32)
    out_text = on.empty_like(q_text)
    lse_text = on.empty(q_text.shape[:3], torch.float32)
    if ws is None:
        ws = on.scratch(max(prefix_workspace_size(p, L_text), 256))
    n_ws = _need_workspace(ws, q.device)
    with on:
        _check(lib.dsa_fwd_prefix(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(offsets), L_text, _ptr(q_text),
                                  _ptr(k_text), _ptr(v_text), _ptr(out), _ptr(lse), _ptr(out_text), _ptr(lse_text),
                                  _ptr(ws), n_ws, ctypes.c_void_p(on.ptr)), "dsa_fwd_prefix")
    return out, lse, out_text, lse_text


def selftest_wait(stream=None):
    """Enqueue the failure-path self-test (a bounded wait that runs out after 2 s and records
    DSA_ERR_TIMEOUT at site 99); read the result with device_status()."""
    _check(load_library().dsa_selftest_wait(ctypes.c_void_p(_stream(stream))), "dsa_selftest_wait")


def prefix_bwd_workspace_size(problem: Problem, L_text: int) -> int:
    return int(load_library().dsa_bwd_prefix_workspace_size(ctypes.byref(problem), int(L_text)))


def backward_prefix(q, k, v, out, lse, dout, offsets, q_text, k_text, v_text, out_text, lse_text, dout_text,
                    tile: Sequence[int], window: Sequence[int], scale: Optional[float] = None,
                    ws: Optional[torch.Tensor] = None, stream=None):
    """Backward of forward_prefix (gradients of sum(out * dout) + sum(out_text * dout_text)).
    Returns (dq, dk, dv, dq_text, dk_text, dv_text)."""
    lib = load_library()
    p = _problem_of(q, tile, window, scale)
    for t, name in ((k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _need(t, name, q, q.dtype)
        if t.shape != q.shape:
            raise ValueError(f"{name} shape {tuple(t.shape)} != q shape {tuple(q.shape)}")
    _need(q, "q", q)
    _need(lse, "lse", q, torch.float32, q.shape[:5].numel())
    _need(offsets, "offsets", q, torch.int32, 3 * plan_shape(p)[0])
    if q_text.dim() != 4 or tuple(q_text.shape[:2]) != tuple(q.shape[:2]) or q_text.shape[3] != q.shape[5]:
        raise ValueError(f"q_text shape {tuple(q_text.shape)} does not match q {tuple(q.shape)}")
    for t, name in ((q_text, "q_text"), (k_text, "k_text"), (v_text, "v_text"), (out_text, "out_text"),
                    (dout_text, "dout_text")):
        _need(t, name, q, q.dtype)
        if t.shape != q_text.shape:
            raise ValueError(f"{name} shape {tuple(t.shape)} != q_text shape {tuple(q_text.shape)}")
    _need(lse_text, "lse_text", q, torch.float32, q_text.shape[:3].numel())
    L_text = int(q_text.shape[2])
    on = _On(q.device, stream)
    dq, dk, dv = on.empty_like(q), on.empty_like(q), on.empty_like(q)
    dqt, dkt, dvt = on.empty_like(q_text), on.empty_like(q_text), on.empty_like(q_text)
    if ws is None:
        ws = on.scratch(max(prefix_bwd_workspace_size(p, L_text), 256))
    n_ws = _need_workspace(ws, q.device)
    with on:
        _check(lib.dsa_bwd_prefix(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout),
                                  _ptr(offsets), L_text, _ptr(q_text), _ptr(k_text), _ptr(v_text), _ptr(out_text),
                                  _ptr(lse_text), _ptr(dout_text), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dqt), _ptr(dkt),
                                  _ptr(dvt), _ptr(ws), n_ws, ctypes.c_void_p(on.ptr)), "dsa_bwd_prefix")
    return dq, dk, dv, dqt, dkt, dvt


def forward_host_bytes(problem: Problem) -> int:
    return int(load_library().dsa_fwd_host_bytes(ctypes.byref(problem)))


def forward_host(problem: Problem, q_host: torch.Tensor, k_host: torch.Tensor, v_host: torch.Tensor,
                 offsets_host: torch.Tensor, out_host: torch.Tensor, lse_host: torch.Tensor, dev: torch.Tensor,
                 stream=None):
    """3D-DSA forward from pinned host tensors through the caller's device buffer ``dev``
    (uint8, at least forward_host_bytes(problem) bytes); asynchronous on ``stream``."""
    lib = load_library()
    for t in (q_host, k_host, v_host, offsets_host, out_host, lse_host):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("host tensors must be contiguous CPU tensors")
    rows = problem.B * problem.heads * problem.T * problem.H * problem.W
    row_bytes = problem.d * (2 if problem.dtype == DSA_BF16 else 4)
    for t, name, n in ((q_host, "q_host", rows * row_bytes), (k_host, "k_host", rows * row_bytes),
                       (v_host, "v_host", rows * row_bytes), (out_host, "out_host", rows * row_bytes),
                       (lse_host, "lse_host", 4 * rows), (offsets_host, "offsets_host", 12 * plan_shape(problem)[0])):
        if t.numel() * t.element_size() != n:
            raise ValueError(f"{name} has {t.numel() * t.element_size()} bytes, expected {n}")
    if not dev.is_cuda:
        raise ValueError("dev must be a CUDA tensor")
    n_dev = _need_workspace(dev, dev.device)
    _check(lib.dsa_fwd_host(ctypes.byref(problem), _ptr(q_host), _ptr(k_host), _ptr(v_host), _ptr(offsets_host),
                            _ptr(out_host), _ptr(lse_host), _ptr(dev), n_dev, ctypes.c_void_p(_stream(stream))),
           "dsa_fwd_host")


def backward(q, k, v, out, lse, dout, offsets, tile, window, scale=None, dq=None, dk=None, dv=None, ws=None,
             stream=None):
    """3D-DSA backward of sum(out * dout).  Returns (dq, dk, dv)."""
    lib = load_library()
    p = _problem_of(q, tile, window, scale)
    for t, name in ((k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _need(t, name, q, q.dtype)
        if t.shape != q.shape:
            raise ValueError(f"{name} shape {tuple(t.shape)} != q shape {tuple(q.shape)}")
    _need(q, "q", q)
    _need(lse, "lse", q, torch.float32, q.shape[:5].numel())
    _need(offsets, "offsets", q, torch.int32, 3 * plan_shape(p)[0])
    on = _On(q.device, stream)
    dq = on.empty_like(q) if dq is None else dq
    dk = on.empty_like(q) if dk is None else dk
    dv = on.empty_like(q) if dv is None else dv
    for t, name in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        _need(t, name, q, q.dtype, q.numel())
    if ws is None:
        ws = on.scratch(max(workspace_size(p, backward=True), 256))
    n_ws = _need_workspace(ws, q.device)
    with on:
        _check(lib.dsa_bwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(offsets),
                           _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), n_ws, ctypes.c_void_p(on.ptr)),
               "dsa_bwd")
    return dq, dk, dv


def _list_args(q: torch.Tensor, row_ptr: torch.Tensor, kv_list: torch.Tensor, n_tiles: int):
    """-> (list pointer, nnz, per_head): row_ptr [nTiles + 1] is one list for every head,
    [B * heads, nTiles + 1] one list per (batch, head)."""
    _need(row_ptr, "row_ptr", q, torch.int32)
    BH = q.shape[0] * q.shape[1]
    if row_ptr.numel() == n_tiles + 1 and row_ptr.dim() == 1:
        per_head = 0
    elif tuple(row_ptr.shape) == (BH, n_tiles + 1):
        per_head = 1
    else:
        raise ValueError(f"row_ptr must be [nTiles + 1] or [B * heads, nTiles + 1], got {tuple(row_ptr.shape)}")
    if kv_list is not None and kv_list.numel() > 0:
        _need(kv_list, "kv_list", q, torch.int32)
        return _ptr(kv_list), int(kv_list.numel()), per_head
    return None, 0, per_head


def forward_list(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, row_ptr: torch.Tensor, kv_list: torch.Tensor,
                 tile: Sequence[int], scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, stream=None):
    """Block-sparse forward over key-tile lists: query tile i attends to the key tiles
    kv_list[row_ptr[i]:row_ptr[i+1]] (int32 CUDA tensors; tiles in raster order of the tile
    grid); row_ptr [nTiles + 1] is one list for every head, [B * heads, nTiles + 1] one per
    (batch, head) with absolute positions in kv_list.  Returns (out, lse); an empty row
    gives out = 0 and lse = -inf."""
    lib = load_library()
    p = _problem_of(q, tile, (1, 1, 1), scale)
    for t, name in ((k, "k"), (v, "v")):
        _need(t, name, q, q.dtype)
        if t.shape != q.shape:
            raise ValueError(f"{name} shape {tuple(t.shape)} != q shape {tuple(q.shape)}")
    _need(q, "q", q)
    n_tiles, _ = plan_shape(p)
    lst, nnz, per_head = _list_args(q, row_ptr, kv_list, n_tiles)
    on = _On(q.device, stream)
    if out is None:
        out = on.empty_like(q)
    if lse is None:
        lse = on.empty(q.shape[:5], torch.float32)
    _need(out, "out", q, q.dtype, q.numel())
    _need(lse, "lse", q, torch.float32, q.shape[:5].numel())
    with on:
        _check(lib.dsa_fwd_list(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(row_ptr), lst, nnz, per_head, _ptr(out),
                                _ptr(lse), ctypes.c_void_p(on.ptr)), "dsa_fwd_list")
    return out, lse


def backward_list(q, k, v, out, lse, dout, row_ptr, kv_list, tile, scale=None, dq=None, dk=None, dv=None, ws=None,
                  stream=None):
    """Backward of sum(out * dout) for forward_list.  Returns (dq, dk, dv)."""
    lib = load_library()
    p = _problem_of(q, tile, (1, 1, 1), scale)
    for t, name in ((k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _need(t, name, q, q.dtype)
        if t.shape != q.shape:
            raise ValueError(f"{name} shape {tuple(t.shape)} != q shape {tuple(q.shape)}")
    _need(q, "q", q)
    _need(lse, "lse", q, torch.float32, q.shape[:5].numel())
    n_tiles, _ = plan_shape(p)
    lst, nnz, per_head = _list_args(q, row_ptr, kv_list, n_tiles)
    on = _On(q.device, stream)
    dq = on.empty_like(q) if dq is None else dq
    dk = on.empty_like(q) if dk is None else dk
    dv = on.empty_like(q) if dv is None else dv
    for t, name in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        _need(t, name, q, q.dtype, q.numel())
    if ws is None:
        size = int(lib.dsa_list_workspace_size(ctypes.byref(p), nnz, per_head, DSA_WS_BWD))
        ws = on.scratch(max(size, 256))
    n_ws = _need_workspace(ws, q.device)
    with on:
        _check(lib.dsa_bwd_list(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout),
                                _ptr(row_ptr), lst, nnz, per_head, _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), n_ws,
                                ctypes.c_void_p(on.ptr)), "dsa_bwd_list")
    return dq, dk, dv


def block_map(q: torch.Tensor, k: torch.Tensor, lse: torch.Tensor, row_ptr: torch.Tensor, kv_list: torch.Tensor,
              tile: Sequence[int], scale: Optional[float] = None, out: Optional[torch.Tensor] = None, stream=None):
    """Block attention mass [B * heads, nTiles, nTiles] (fp32): mean attention probability
    of each query tile's tokens on each key tile, against the LSE forward_list wrote for
    the same lists."""
    lib = load_library()
    p = _problem_of(q, tile, (1, 1, 1), scale)
    _need(q, "q", q)
    _need(k, "k", q, q.dtype, q.numel())
    _need(lse, "lse", q, torch.float32, q.shape[:5].numel())
    n_tiles, _ = plan_shape(p)
    lst, nnz, per_head = _list_args(q, row_ptr, kv_list, n_tiles)
    BH = q.shape[0] * q.shape[1]
    on = _On(q.device, stream)
    if out is None:
        out = on.empty((BH, n_tiles, n_tiles), torch.float32)
    _need(out, "out", q, torch.float32, BH * n_tiles * n_tiles)
    with on:
        _check(lib.dsa_block_map(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(lse), _ptr(row_ptr), lst, nnz, per_head,
                                 _ptr(out), ctypes.c_void_p(on.ptr)), "dsa_block_map")
    return out


def lstsq_factor(M: torch.Tensor, lam: float, stream=None) -> torch.Tensor:
    """Cholesky factor (fp64 [p, p], lower) of M^T M + lam I for a design matrix M (fp32
    CUDA [m, p], p <= 32), to be reused by lstsq_solve across heads and steps."""
    lib = load_library()
    if not M.is_cuda or M.dtype != torch.float32 or not M.is_contiguous() or M.dim() != 2:
        raise ValueError("M must be a contiguous fp32 CUDA tensor [m, p]")
    m, p = M.shape
    on = _On(M.device, stream)
    L = on.empty((p, p), torch.float64)
    with on:
        _check(lib.dsa_lstsq_factor(m, p, _ptr(M), float(lam), _ptr(L), ctypes.c_void_p(on.ptr)),
               "dsa_lstsq_factor")
    return L


def lstsq_solve(M: torch.Tensor, L: torch.Tensor, S: torch.Tensor, X: Optional[torch.Tensor] = None, ws=None,
                stream=None) -> torch.Tensor:
    """X [batch, p] (fp32) with (M^T M + lam I) x_b = M^T s_b for every row s_b of S
    [batch, m] (fp32 CUDA), L from lstsq_factor."""
    lib = load_library()
    m, p = M.shape
    if not S.is_cuda or S.dtype != torch.float32 or not S.is_contiguous() or S.dim() != 2 or S.shape[1] != m:
        raise ValueError("S must be a contiguous fp32 CUDA tensor [batch, m]")
    batch = S.shape[0]
    _need(M, "M", S, torch.float32)
    _need(L, "L", S, torch.float64, p * p)
    on = _On(S.device, stream)
    if X is None:
        X = on.empty((batch, p), torch.float32)
    _need(X, "X", S, torch.float32, batch * p)
    n_ws = int(lib.dsa_lstsq_workspace_size(m, p, batch))
    if ws is None and n_ws > 0:
        ws = on.scratch(n_ws)
    with on:
        _check(lib.dsa_lstsq_solve(m, p, batch, _ptr(M), _ptr(L), _ptr(S), _ptr(X), _ptr(ws),
                                   0 if ws is None else ws.numel(), ctypes.c_void_p(on.ptr)), "dsa_lstsq_solve")
    return X


def plan_heads(problem: Problem, offsets: torch.Tensor, stream=None):
    """Per-(batch, head) window offsets [B * heads, nTiles, 3] (int32 CUDA) as per-head
    key-tile lists: returns (row_ptr [B * heads, nTiles + 1], kv_list) for forward_list /
    backward_list."""
    lib = load_library()
    n, wt = plan_shape(problem)
    BH = problem.B * problem.heads
    if not offsets.is_cuda or offsets.dtype != torch.int32 or not offsets.is_contiguous() or \
            offsets.numel() != BH * n * 3:
        raise ValueError("offsets must be a contiguous int32 CUDA tensor [B * heads, nTiles, 3]")
    on = _On(offsets.device, stream)
    row_ptr = on.empty((BH, n + 1), torch.int32)
    kv_list = on.empty((BH * n * wt,), torch.int32)
    with on:
        _check(lib.dsa_plan_heads(ctypes.byref(problem), _ptr(offsets), _ptr(row_ptr), _ptr(kv_list),
                                  ctypes.c_void_p(on.ptr)), "dsa_plan_heads")
    return row_ptr, kv_list


# ---------------------------------------------------------------- around the sliding attention
def _dtype_of(t: torch.Tensor, name: str) -> int:
    if t.dtype == torch.bfloat16:
        return DSA_BF16
    if t.dtype == torch.float32:
        return DSA_F32
    raise ValueError(f"{name}: unsupported dtype {t.dtype}")


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _like(t: torch.Tensor, name: str, ref: torch.Tensor, shape=None, dtype=None):
    if t.device != ref.device:
        raise ValueError(f"{name} is on {t.device}, expected {ref.device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} shape {tuple(t.shape)} != {tuple(shape)}")


def _ws(ws: Optional[torch.Tensor], n_bytes: int, on: _On, ref: torch.Tensor):
    if ws is None:
        return on.scratch(n_bytes), n_bytes
    if ws.device != ref.device or not ws.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {ref.device}")
    return ws, ws.numel() * ws.element_size()


def _fit(sizes: int):
    """Sizes (their bits in one number, which costs a call least) that the C structures' 32 bits hold:
    ctypes would keep the low bits of larger ones."""
    if sizes > 2 ** 31 - 1:
        raise DsaError(2, "a size of 2^31 or more")


def _rows_view(t: torch.Tensor, name: str) -> View:
    """A [B, heads, rows, d] tensor as dsa_view_t."""
    s = t.stride()
    if s[3] != 1 and t.shape[3] > 1 and t.numel() > 0:
        raise ValueError(f"{name}: the channels must be contiguous")
    return View(t.data_ptr(), s[:3])


def _cross(q, k, v, kv_len, scale) -> Cross:
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B, heads, Lq, d], k and v [B, kv_heads, Lk, d]")
    B, heads, Lq, d = q.shape
    _, kv_heads, Lk, _ = k.shape
    _fit(B | heads | kv_heads | Lq | Lk | d)
    _like(k, "k", q, (B, kv_heads, Lk, d), q.dtype)
    _like(v, "v", q, k.shape, q.dtype)
    if kv_len is not None:
        _like(kv_len, "kv_len", q, (B,), torch.int32)
        if not kv_len.is_contiguous():
            raise ValueError("kv_len must be contiguous")
    return Cross(B, heads, kv_heads, d, Lq, Lk, 1.0 / math.sqrt(d) if scale is None else scale, _dtype_of(q, "q"))


def _out_like(t: Optional[torch.Tensor], name: str, ref: torch.Tensor, on: _On) -> torch.Tensor:
    """`t`, or a new tensor of ref's shape and dimension order."""
    if t is None:
        return on.empty_like(ref)
    _like(t, name, ref, ref.shape, ref.dtype)
    return t


def cross_workspace_size(problem: Cross, backward: bool = False) -> int:
    return int(load_library().dsa_cross_workspace_size(ctypes.byref(problem), DSA_WS_BWD if backward else DSA_WS_FWD))


def forward_cross(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, kv_len: Optional[torch.Tensor] = None,
                  scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
    """Cross attention to an encoder's states.  q: [B, heads, Lq, 128] bf16; k, v: [B, kv_heads,
    Lk, 128] (kv_heads divides heads), strided views with contiguous channels; kv_len: int32
    [B] on the device, the valid states of each batch entry (the rest is padding that reaches no
    result; 0 gives out = 0 and lse = -inf).  Returns (out, lse), out in q's dimension order."""
    lib = load_library()
    p = _cross(q, k, v, kv_len, scale)
    with _On(q.device, stream) as on:
        out = _out_like(out, "out", q, on)
        if lse is None:
            lse = on.empty(q.shape[:3], torch.float32)
        _like(lse, "lse", q, q.shape[:3], torch.float32)
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")
        ws, n_ws = _ws(ws, cross_workspace_size(p), on, q)
        _check(lib.dsa_fwd_cross(p, _rows_view(q, "q"), _rows_view(k, "k"), _rows_view(v, "v"), _addr(kv_len),
                                 _rows_view(out, "out"), lse.data_ptr(), _addr(ws), n_ws, on.ptr), "dsa_fwd_cross")
    return out, lse


def backward_cross(q, k, v, out, lse, dout, kv_len: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                   dq=None, dk=None, dv=None, ws: Optional[torch.Tensor] = None, stream=None):
    """Backward of forward_cross (gradients of sum(out * dout)).  Returns (dq, dk, dv), in the
    dimension orders of q, k and v; a shared kv head's gradient is summed over its heads, rows
    past kv_len are zero."""
    lib = load_library()
    p = _cross(q, k, v, kv_len, scale)
    for t, name in ((out, "out"), (dout, "dout")):
        _like(t, name, q, q.shape, q.dtype)
    _like(lse, "lse", q, q.shape[:3], torch.float32)
    if not lse.is_contiguous():
        raise ValueError("lse must be contiguous")
    with _On(q.device, stream) as on:
        dq, dk, dv = _out_like(dq, "dq", q, on), _out_like(dk, "dk", k, on), _out_like(dv, "dv", v, on)
        ws, n_ws = _ws(ws, cross_workspace_size(p, backward=True), on, q)
        _check(lib.dsa_bwd_cross(p, _rows_view(q, "q"), _rows_view(k, "k"), _rows_view(v, "v"), _rows_view(out, "out"),
                                 lse.data_ptr(), _rows_view(dout, "dout"), _addr(kv_len), _rows_view(dq, "dq"),
                                 _rows_view(dk, "dk"), _rows_view(dv, "dv"), _addr(ws), n_ws, on.ptr), "dsa_bwd_cross")
    return dq, dk, dv


def _axes(axes: Sequence[int]):
    if len(axes) != 3:
        raise ValueError("axes must be the channels of (time, height, width)")
    return [int(a) for a in axes]


def rope_table(grid: Sequence[int], axes: Sequence[int], theta: float = 10000.0, start=(0, 0, 0), step=(1, 1, 1),
               device="cuda", stream=None) -> torch.Tensor:
    """(cos, sin) of every coordinate and channel pair of each axis of a (T, H, W) token grid,
    fp32 [T axes[0]/2 + H axes[1]/2 + W axes[2]/2, 2]: the angle of coordinate i and pair j of
    axis a is (start[a] + i step[a]) theta^(-2j / axes[a]).  Kept by the caller for rope()."""
    lib = load_library()
    axes = _axes(axes)
    if len(grid) != 3 or len(start) != 3 or len(step) != 3:
        raise ValueError("grid, start and step must have three entries")
    _fit(max(*(int(g) for g in grid), *axes))
    n = sum(int(g) * (a // 2) for g, a in zip(grid, axes))
    device = torch.device(device)
    if device.type == "cuda":
        current = torch.cuda.current_device()  # (this may be the process' first call to CUDA)
        device = torch.device("cuda", current if device.index is None else device.index)
    with _On(device, stream) as on:
        table = on.empty((max(n, 0), 2), torch.float32)
        i3, d3 = ctypes.c_int32 * 3, ctypes.c_double * 3
        _check(lib.dsa_rope_table(i3(*(int(g) for g in grid)), i3(*axes), d3(*(float(x) for x in start)),
                                  d3(*(float(x) for x in step)), float(theta), table.data_ptr(), on.ptr),
               "dsa_rope_table")
    return table


def _grid_view(t: torch.Tensor, name: str) -> View:
    """A [B, heads, T, H, W, d] tensor whose (T, H, W) are one token dimension."""
    _, _, T, H, W, d = t.shape
    sb, sh, st, sy, sx, sd = t.stride()
    if sd != 1 and d > 1 and t.numel() > 0:
        raise ValueError(f"{name}: the channels must be contiguous")
    token = sx if W > 1 else sy if H > 1 else st if T > 1 else 0
    if (H > 1 and sy != W * token) or (T > 1 and st != H * W * token):
        raise ValueError(f"{name}: (T, H, W) must be one dimension of tokens in raster order")
    return View(t.data_ptr(), (sb, sh, token))


def rope(q: torch.Tensor, k: Optional[torch.Tensor], table: torch.Tensor, axes: Sequence[int],
         interleaved: bool = True, inverse: bool = False, q_out: Optional[torch.Tensor] = None,
         k_out: Optional[torch.Tensor] = None, stream=None):
    """Rotary positions over the token grid, q and k in one launch (k may be None).  q, k:
    [B, heads, T, H, W, d] bf16 or fp32, contiguous channels, tokens in raster order, any other
    strides (a projection's token-major rows as a view).  axes: channels of (time, height, width);
    interleaved: pairs (2j, 2j + 1), else (j, j + R / 2).  inverse=True turns back, which is also
    the backward.  Returns (q_out, k_out): contiguous unless given (an output may be its input)."""
    lib = load_library()
    if q.dim() != 6:
        raise ValueError("q must be [B, heads, T, H, W, d]")
    axes = _axes(axes)
    B, heads, T, H, W, d = q.shape
    _fit(B | heads | T | H | W | d)
    p = Rope(B, heads, d, T, H, W, tuple(axes), 1 if interleaved else 0, 1 if inverse else 0, _dtype_of(q, "q"))
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    _like(table, "table", q, (T * (axes[0] // 2) + H * (axes[1] // 2) + W * (axes[2] // 2), 2), torch.float32)
    if not table.is_contiguous():
        raise ValueError("table must be contiguous")

    def result(x, y, name):
        _like(x, name, q, q.shape, q.dtype)
        if y is None:
            return on.empty(x.shape, x.dtype)
        _like(y, name + "_out", q, q.shape, q.dtype)
        return y

    with _On(q.device, stream) as on:
        q_out = result(q, q_out, "q")
        kv = ko = None
        if k is not None:
            k_out = result(k, k_out, "k")
            kv, ko = _grid_view(k, "k"), _grid_view(k_out, "k_out")
        _check(lib.dsa_rope(p, table.data_ptr(), _grid_view(q, "q"), _grid_view(q_out, "q_out"), kv, ko, on.ptr),
               "dsa_rope")
    return q_out, k_out


def _rows(t: torch.Tensor, name: str):
    """(rows, C, row stride) of a [..., C] tensor whose leading dimensions are one of rows."""
    if t.dim() == 0:
        raise ValueError(f"{name}: a tensor of rows has at least one dimension")
    C = t.shape[-1]
    if t.is_contiguous():
        return (t.numel() // C if C else 0), C, C
    if C > 1 and t.numel() > 0 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the channels must be contiguous")
    rows, ld = 1, 0
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n != 1 and t.numel() > 0:
            if rows > 1 and s != rows * ld:
                raise ValueError(f"{name}: the leading dimensions must be one dimension of rows")
            if rows == 1:
                ld = s
        rows *= n
    return rows, C, ld if rows > 1 else C


def _norm(x: torch.Tensor, weight, eps: float):
    rows, C, ld = _rows(x, "x")
    _fit(C)
    if weight is not None:
        _like(weight, "weight", x, (C,), x.dtype)
        if not weight.is_contiguous():
            raise ValueError("weight must be contiguous")
    return Norm(rows, C, eps, _dtype_of(x, "x")), ld


def _contiguous_out(t, name: str, ref: torch.Tensor, on: _On, dtype=None):
    dtype = dtype or ref.dtype
    if t is None:
        return on.empty(ref.shape, dtype)
    _like(t, name, ref, ref.shape, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
             residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
             sum_out: Optional[torch.Tensor] = None, stream=None):
    """Root-mean-square norm over the last dimension (C <= 16384), after the residual's addition:
    h = x + residual, y = weight * h / sqrt(mean h^2 + eps).  x, residual: [..., C] bf16 or fp32
    rows of any row stride; weight: [C] of the same type, or None.  Returns (y, h); h is x itself
    without a residual.  sum_out may be the residual (updated in place)."""
    y, h, _ = _rms_norm(x, weight, eps, residual, out, None, sum_out, None, stream)
    return y, h


def rms_norm_fp8(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 scales: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None, stream=None):
    """rms_norm with y as e4m3 and an fp32 scale for every 128 channels of a row.  Returns (y8,
    scales, h): y8 [..., C] float8_e4m3fn, scales [..., ceil(C / 128)], y = y8 * scale."""
    y, h, s = _rms_norm(x, weight, eps, residual, out, scales, sum_out, torch.float8_e4m3fn, stream)
    return y, s, h


def _rms_norm(x, weight, eps, residual, out, scales, sum_out, dtype8, stream):
    lib = load_library()
    p, x_ld = _norm(x, weight, eps)
    r_ld = 0
    if residual is not None:
        _like(residual, "residual", x, x.shape, x.dtype)
        r_ld = _rows(residual, "residual")[2]
    elif sum_out is not None:
        raise ValueError("sum_out without a residual")
    with _On(x.device, stream) as on:
        y = _contiguous_out(out, "out", x, on, dtype8)
        h = _contiguous_out(sum_out, "sum_out", x, on) if residual is not None else None
        args = (p, x.data_ptr(), x_ld, _addr(residual), r_ld, _addr(weight), y.data_ptr())
        if dtype8 is None:
            _check(lib.dsa_rmsnorm(*args, _addr(h), on.ptr), "dsa_rmsnorm")
        else:
            shape = x.shape[:-1] + ((p.C + 127) // 128,)
            if scales is None:
                scales = on.empty(shape, torch.float32)
            _like(scales, "scales", x, shape, torch.float32)
            if not scales.is_contiguous():
                raise ValueError("scales must be contiguous")
            _check(lib.dsa_rmsnorm_fp8(*args, scales.data_ptr(), _addr(h), on.ptr), "dsa_rmsnorm_fp8")
    return y, x if h is None else h, scales


def rms_norm_backward(h: torch.Tensor, weight: Optional[torch.Tensor], dy: torch.Tensor,
                      dh: Optional[torch.Tensor] = None, eps: float = 1e-6, dx: Optional[torch.Tensor] = None,
                      dweight: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
    """Backward of rms_norm, given its h (= x without a residual), the gradient dy of y and,
    optionally, the gradient dh that reaches h beside the norm.  Returns (dx, dweight): dx is
    the gradient of x and of the residual; dweight is None without a weight."""
    lib = load_library()
    p, h_ld = _norm(h, weight, eps)
    _like(dy, "dy", h, h.shape, h.dtype)
    dy_ld, dh_ld = _rows(dy, "dy")[2], 0
    if dh is not None:
        _like(dh, "dh", h, h.shape, h.dtype)
        dh_ld = _rows(dh, "dh")[2]
    if weight is None and dweight is not None:
        raise ValueError("dweight without a weight")
    with _On(h.device, stream) as on:
        dx = _contiguous_out(dx, "dx", h, on)
        if weight is not None:
            dweight = _contiguous_out(dweight, "dweight", weight, on)
        size = int(lib.dsa_rmsnorm_bwd_workspace_size(p)) if weight is not None else 0
        ws, n_ws = _ws(ws, size, on, h)
        _check(lib.dsa_rmsnorm_bwd(p, h.data_ptr(), h_ld, _addr(weight), dy.data_ptr(), dy_ld, _addr(dh), dh_ld,
                                   dx.data_ptr(), _addr(dweight), _addr(ws), n_ws, on.ptr), "dsa_rmsnorm_bwd")
    return dx, dweight


def device_status(stream=None):
    """Synchronise ``stream`` and read/clear the device status word: (status, site, block)."""
    lib = load_library()
    site, block = ctypes.c_int32(), ctypes.c_int32()
    st = lib.dsa_device_status(ctypes.c_void_p(_stream(stream)), ctypes.byref(site), ctypes.byref(block))
    return st, site.value, block.value
