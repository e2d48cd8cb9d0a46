"""Rotary positions over the token grid against the fp64 definition."""
import pytest
import torch

from tests import _block_ref as ref
import video_dit_sparse_dsa_b200 as dsa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def check(got, x, grid, axes, table, interleaved, inverse, what):
    want, tol = ref.rope(x, grid, axes, table, interleaved, inverse)
    ref.close(got, want, tol + ref.U[x.dtype] * want.abs(), what)


@pytest.mark.parametrize("grid,axes,kw", [
    ((1, 1, 1), (2, 0, 0), {}),
    ((30, 48, 80), (44, 42, 42), {}),
    ((5, 7, 9), (16, 56, 56), dict(theta=256.0, start=(100000, -3, 0.5), step=(1, 0.25, 2))),
    ((3, 1, 4), (0, 8, 0), {}),
    ((200001, 1, 1), (44, 0, 0), dict(start=(10 ** 6, 0, 0))),
])
def test_table(grid, axes, kw):
    t = dsa.rope_table(grid, axes, **kw)
    want = ref.rope_table(grid, axes, **kw)
    # fp32 rounding of a cosine, and the fp64 angle's own error (a few steps of up to 1.2e6)
    ref.close(t, want, 2.0 ** -25 + 1e-9, "table")


GRIDS = [((1, 1, 1), 1, 1), ((1, 16, 16), 1, 12), ((3, 5, 7), 2, 3), ((4, 9, 11), 1, 5), ((2, 2, 3), 3, 24)]
# (d, axes): 16-byte vectors, pass-through channels, odd pair counts, an axis without channels
SHAPES = [(128, (44, 42, 42)), (128, (16, 56, 56)), (64, (16, 24, 24)), (96, (32, 16, 16)), (128, (0, 32, 32)),
          (10, (2, 4, 2)), (7, (2, 2, 2)), (40, (6, 4, 4)), (256, (64, 96, 96))]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("d,axes", SHAPES)
def test_rope(d, axes, interleaved, dtype):
    for i, (grid, B, heads) in enumerate(GRIDS):
        g = torch.Generator().manual_seed(i)
        q, k = (torch.randn(B, heads, *grid, d, generator=g).to(dtype) for _ in range(2))
        table = dsa.rope_table(grid, axes)
        for inverse in (False, True):
            qo, ko = dsa.rope(q.to(DEV), k.to(DEV), table, axes, interleaved=interleaved, inverse=inverse)
            check(qo, q, grid, axes, table, interleaved, inverse, f"q {grid}")
            check(ko, k, grid, axes, table, interleaved, inverse, f"k {grid}")
        qo, none = dsa.rope(q.to(DEV), None, table, axes, interleaved=interleaved)
        check(qo, q, grid, axes, table, interleaved, False, "q alone")
        assert none is None


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_projection_views_and_back(dtype, interleaved):
    """Token-major rows of a fused projection into the head-major layout, and the gradients back
    into the fused gradient, whose other columns stay as they were."""
    B, heads, grid, d, axes = 2, 5, (3, 4, 6), 64, (16, 24, 24)
    N = grid[0] * grid[1] * grid[2]
    g = torch.Generator().manual_seed(0)
    buf = torch.randn(B, N, 3, heads, d, generator=g).to(dtype).to(DEV)
    view = lambda t, i: t[:, :, i].view(B, *grid, heads, d).permute(0, 4, 1, 2, 3, 5)  # noqa: E731
    table = dsa.rope_table(grid, axes)
    q, k = dsa.rope(view(buf, 0), view(buf, 1), table, axes, interleaved=interleaved)
    assert q.is_contiguous() and k.is_contiguous()
    check(q, view(buf, 0).cpu(), grid, axes, table, interleaved, False, "q")
    check(k, view(buf, 1).cpu(), grid, axes, table, interleaved, False, "k")
    dbuf = torch.full_like(buf, 3.0)
    dsa.rope(q, k, table, axes, interleaved=interleaved, inverse=True, q_out=view(dbuf, 0), k_out=view(dbuf, 1))
    check(view(dbuf, 0), q.cpu(), grid, axes, table, interleaved, True, "dq")
    check(view(dbuf, 1), k.cpu(), grid, axes, table, interleaved, True, "dk")
    assert (dbuf[:, :, 2] == 3).all()
    one = q.clone()
    dsa.rope(one, None, table, axes, interleaved=interleaved, inverse=True, q_out=one)  # in place
    assert torch.equal(one, view(dbuf, 0))
    # not 16-byte aligned
    odd = torch.randn(B * heads * N * d + 1, device=DEV, dtype=torch.float32).to(dtype)[1:].view(B, heads, *grid, d)
    y, _ = dsa.rope(odd, None, table, axes, interleaved=interleaved)
    check(y, odd.cpu(), grid, axes, table, interleaved, False, "unaligned")
    # one entry broadcast over batch and heads
    x = torch.randn(1, 1, *grid, d, device=DEV).to(dtype).expand(B, heads, *grid, d)
    y, _ = dsa.rope(x, None, table, axes, interleaved=interleaved)
    check(y, x.cpu(), grid, axes, table, interleaved, False, "broadcast")


def test_gradient_is_the_inverse():
    """<rope(x), dy> is linear in x: its derivative along u (also a difference, exactly) is
    <u, inverse(dy)>."""
    grid, axes = (2, 3, 5), (16, 24, 24)
    g = torch.Generator().manual_seed(2)
    x, u, dy = (torch.randn(1, 2, *grid, 64, generator=g) for _ in range(3))
    table = dsa.rope_table(grid, axes)
    for inter in (True, False):
        dx, _ = dsa.rope(dy.to(DEV), None, table, axes, interleaved=inter, inverse=True)
        f = lambda v: float((ref.rope(v, grid, axes, table, inter, False)[0] * dy.double()).sum())  # noqa: E731
        num = f(x.double() + 0.5 * u.double()) - f(x.double() - 0.5 * u.double())
        _, tol = ref.rope(dy, grid, axes, table, inter, True)
        bound = float(((tol + 2.0 ** -24 * dy.double().abs() * 2) * u.double().abs()).sum()) + 1e-9
        # the table's fp32 cos and sin are a rotation up to 2^-24
        assert abs(float((dx.cpu().double() * u.double()).sum()) - num) <= bound


def test_nonfinite_pairs_stay_alone_and_rest_passes():
    grid, axes = (1, 2, 2), (8, 8, 8)
    x = torch.randn(1, 2, *grid, 32).to(torch.bfloat16)
    x[0, 0, 0, 0, 0, 0] = float("nan")
    x[0, 1, 0, 0, 0, 30] = float("inf")  # past the rotated channels
    table = dsa.rope_table(grid, axes)
    y, _ = dsa.rope(x.to(DEV), None, table, axes)
    y = y.cpu()
    assert torch.isnan(y[0, 0, 0, 0, 0, :2]).all() and torch.isfinite(y[0, 0, 0, 0, 0, 2:]).all()
    assert torch.equal(y[..., 24:], x[..., 24:])


def test_graph_replay_and_side_stream():
    grid, axes = (3, 8, 8), (44, 42, 42)
    table = dsa.rope_table(grid, axes)
    q = torch.randn(1, 4, *grid, 128, device=DEV).to(torch.bfloat16)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.rope(q, None, table, axes, q_out=out)
    q.normal_()
    graph.replay()
    want, _ = dsa.rope(q, None, table, axes)
    assert torch.equal(out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = dsa.rope(q, None, table, axes, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
