"""RMS norm with the residual's addition (own type and e4m3), forward and backward, against the
fp64 definition with bounds counted from the documented roundings."""
import pytest
import torch

from tests import _block_ref as ref
import video_dit_sparse_dsa_b200 as dsa

pytestmark = pytest.mark.gpu
EPS = 1e-6
DEV = "cuda"


def draw(seed, rows, C, dtype, residual, weight):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, C, generator=g).to(dtype)
    r = torch.randn(rows, C, generator=g).to(dtype) if residual else None
    w = (1 + 0.3 * torch.randn(C, generator=g)).to(dtype) if weight else None
    dy = torch.randn(rows, C, generator=g).to(dtype)
    return x, r, w, dy


def dev(*ts):
    return [t if t is None else t.to(DEV) for t in ts]


# one channel, odd channels, a vector's and a warp's borders, several warps per row, the widest
SHAPES = [(1, 1), (3, 7), (5, 8), (2, 100), (17, 128), (33, 129), (4, 256), (9, 1000), (65, 1536), (7, 2048), (3, 4096),
          (300, 5120), (2, 8192), (2, 8200), (1, 16384), (2, 12345)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,C", SHAPES)
def test_forward(rows, C, dtype):
    for residual, weight in ((False, True), (True, True), (True, False)):
        x, r, w, _ = draw(rows * 7 + C, rows, C, dtype, residual, weight)
        y, h = dsa.rms_norm(*dev(x, w), eps=EPS, residual=dev(r)[0])
        ry, rh = ref.norm(x, r, w, EPS)
        u = ref.U[dtype]
        ref.close(y, ry, (u + ref.NORM_ERR) * ry.abs(), f"y {rows}x{C}")
        if residual:
            ref.close(h, rh, u * rh.abs() + 2.0 ** -24 * rh.abs(), "h")
        else:
            assert h.shape == x.shape and torch.equal(h.cpu(), x)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,C", SHAPES)
def test_fp8(rows, C, dtype):
    x, r, w, _ = draw(rows * 11 + C, rows, C, dtype, True, True)
    x[0] = x[0] * 1e-3
    r[0] = r[0] * 1e-3
    y8, s, h = dsa.rms_norm_fp8(*dev(x, w), eps=EPS, residual=dev(r)[0])
    ry, rh = ref.norm(x, r, w, EPS)
    n = -(-C // 128)
    assert y8.dtype == torch.float8_e4m3fn and s.shape == (rows, n)
    amax = torch.nn.functional.pad(ry.abs(), (0, n * 128 - C)).view(rows, n, 128).amax(-1)
    ref.close(s, amax / 448, 2 * ref.NORM_ERR * amax / 448, "scales")
    full = s.cpu().double().repeat_interleave(128, 1)[:, :C]
    got = y8.float().cpu().double() * full
    # e4m3: half a step of 2^-3 of the value, or of the smallest step 2^-9 of the scale
    ref.close(got, ry, (2.0 ** -4 + ref.NORM_ERR) * ry.abs() + 2.0 ** -10 * full, "values")
    ref.close(h, rh, (ref.U[dtype] + 2.0 ** -24) * rh.abs(), "h")


def test_fp8_zero_tiny_and_nonfinite_rows():
    x = torch.randn(6, 300)
    x[1] = 0
    x[2] = 1e-30
    x[3, 5] = float("nan")
    x[4, 200] = float("inf")
    w = torch.ones(300)
    w[128:256] = 0  # a group of zeros beside others
    y8, s, _ = dsa.rms_norm_fp8(*dev(x, w), eps=EPS)
    y8, s = y8.float().cpu(), s.cpu()
    assert (y8[1] == 0).all() and (s[1] == 1).all()
    assert (s[[0, 2], 1] == 1).all() and (y8[[0, 2], 128:256] == 0).all()
    assert torch.isnan(y8[3]).all() and torch.isnan(s[3]).all()
    # inf: rho = 0, the other channels 0, the channel itself NaN (0 * inf)
    assert torch.isnan(s[4, 1]) and (y8[4, :128] == 0).all() and (s[4, 0] == 1).all()
    ry, _ = ref.norm(x[[0, 5]], None, w, EPS)
    full = s[[0, 5]].double().repeat_interleave(128, 1)[:, :300]
    ref.close(y8[[0, 5]].double() * full, ry, (2.0 ** -4 + ref.NORM_ERR) * ry.abs() + 2.0 ** -10 * full, "neighbours")


def test_nonfinite_rows_stay_alone():
    x, r, w, dy = draw(5, 4, 520, torch.bfloat16, True, True)
    x[1, 3], x[2, 7] = float("nan"), float("inf")
    y, h = dsa.rms_norm(*dev(x, w), eps=EPS, residual=dev(r)[0])
    assert torch.isnan(y[1]).all() and torch.isnan(y[2, 7]) and (y[2].nan_to_num() == 0).all()
    ry, _ = ref.norm(x, r, w, EPS)
    ref.close(y[[0, 3]], ry[[0, 3]], (2.0 ** -8 + ref.NORM_ERR) * ry[[0, 3]].abs(), "y")
    dx, _ = dsa.rms_norm_backward(*dev(x, w, dy), eps=EPS)
    rx = ref.norm_bwd(x, w, dy, None, EPS)
    ref.close(dx[[0, 3]], rx[0][[0, 3]], (rx[2] + 2.0 ** -8 * rx[0].abs())[[0, 3]], "dx")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,C", SHAPES + [(2000, 64), (1500, 520), (700, 1536)])
def test_backward(rows, C, dtype):
    for with_dh, weight in ((False, True), (True, True), (True, False)):
        h, dh, w, dy = draw(rows * 13 + C, rows, C, dtype, with_dh, weight)
        dx, dw = dsa.rms_norm_backward(*dev(h, w, dy), dh=dev(dh)[0], eps=EPS)
        rx, rw, tx, tw = ref.norm_bwd(h, w, dy, dh, EPS)
        u = ref.U[dtype]
        ref.close(dx, rx, tx + u * rx.abs(), f"dx {rows}x{C}")
        if weight:
            ref.close(dw, rw, tw + u * rw.abs(), f"dw {rows}x{C}")
        else:
            assert dw is None


def test_backward_against_differences():
    """<dx, u> and <dw, t> against central differences of the fp64 forward."""
    h, _, w, dy = draw(3, 5, 200, torch.float32, False, True)
    dx, dw = dsa.rms_norm_backward(*dev(h, w, dy), eps=EPS)
    g = torch.Generator().manual_seed(9)
    u, t = torch.randn(5, 200, generator=g).double(), torch.randn(200, generator=g).double()
    f = lambda hh, ww: float((ref.norm(hh, None, ww, EPS)[0] * dy.double()).sum())  # noqa: E731
    e = 1e-4
    num = (f(h.double() + e * u, w) - f(h.double() - e * u, w)) / (2 * e)
    numw = (f(h, w.double() + e * t) - f(h, w.double() - e * t)) / (2 * e)
    _, _, tx, tw = ref.norm_bwd(h, w, dy, None, EPS)
    # the kernel's bound against the direction, and the differences' own error (third derivative * e^2)
    assert abs(float((dx.cpu().double() * u).sum()) - num) <= float((tx * u.abs()).sum()) + 2e-5 * (1 + abs(num))
    assert abs(float((dw.cpu().double() * t).sum()) - numw) <= float((tw * t.abs()).sum()) + 2e-5 * (1 + abs(numw))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_alignment_and_leading_dimensions(dtype):
    g = torch.Generator().manual_seed(1)
    buf = torch.randn(2, 9, 3, 264, generator=g).to(dtype).to(DEV)
    x, r = buf[:, :, 1], buf[:, :, 2, :]           # rows of a fused projection, stride 792
    w = (1 + torch.randn(264, generator=g)).to(dtype).to(DEV)
    y, h = dsa.rms_norm(x, w, residual=r)
    ry, rh = ref.norm(x.cpu(), r.cpu(), w.cpu(), EPS)
    ref.close(y, ry, (ref.U[dtype] + ref.NORM_ERR) * ry.abs(), "strided y")
    ref.close(h, rh, (ref.U[dtype] + 2.0 ** -24) * rh.abs(), "strided h")
    odd = buf.view(-1)[1:1 + 9 * 264].view(9, 264)  # not 16-byte aligned
    y, _ = dsa.rms_norm(odd, w)
    ry, _ = ref.norm(odd.cpu(), None, w.cpu(), EPS)
    ref.close(y, ry, (ref.U[dtype] + ref.NORM_ERR) * ry.abs(), "unaligned y")
    dx, dw = dsa.rms_norm_backward(x, w, r, dh=r)
    rx, rw, tx, tw = ref.norm_bwd(x.cpu(), w.cpu(), r.cpu(), r.cpu(), EPS)
    ref.close(dx, rx, tx + ref.U[dtype] * rx.abs(), "strided dx")
    ref.close(dw, rw, tw + ref.U[dtype] * rw.abs(), "strided dw")


def test_residual_updated_in_place_and_neighbours_untouched():
    x, r, w, _ = draw(2, 37, 1536, torch.bfloat16, True, True)
    want, _ = dsa.rms_norm(*dev(x, w), residual=dev(r)[0])
    buf = torch.full((39, 1536), 7.0, dtype=torch.bfloat16, device=DEV)
    buf[1:38] = r.to(DEV)
    y, h = dsa.rms_norm(*dev(x, w), residual=buf[1:38], sum_out=buf[1:38])
    assert torch.equal(y, want) and h.data_ptr() == buf[1:38].data_ptr()
    assert torch.equal(buf[1:38].cpu(), (x.float() + r.float()).to(torch.bfloat16))
    assert (buf[[0, 38]] == 7).all()


def test_no_rows():
    x = torch.empty(0, 256, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    assert dsa.rms_norm(x, w)[0].shape == (0, 256)
    assert dsa.rms_norm_fp8(x, w)[1].shape == (0, 2)
    dx, dw = dsa.rms_norm_backward(x, w, x)
    assert dx.shape == (0, 256) and (dw == 0).all()


def test_same_bits_and_graph_replay():
    h, dh, w, dy = dev(*draw(4, 4099, 1536, torch.bfloat16, True, True))
    first = dsa.rms_norm_backward(h, w, dy, dh=dh)
    second = dsa.rms_norm_backward(h, w, dy, dh=dh)
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    dx, dw = torch.empty_like(h), torch.empty_like(w)
    y, s = torch.empty(h.shape, dtype=torch.bfloat16, device=DEV), torch.empty_like(h)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            dsa.rms_norm_backward(h, w, dy, dh=dh, dx=dx, dweight=dw)
            dsa.rms_norm(h, w, residual=dh, out=y, sum_out=s)
    for seed in (11, 12):
        h2, dh2, _, dy2 = dev(*draw(seed, 4099, 1536, torch.bfloat16, True, True))
        h.copy_(h2), dh.copy_(dh2), dy.copy_(dy2)
        graph.replay()
        want = dsa.rms_norm_backward(h2, w, dy2, dh=dh2)
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
        yy, ss = dsa.rms_norm(h2, w, residual=dh2)
        assert torch.equal(y, yy) and torch.equal(s, ss)
