"""NaN and infinities at keys of the sliding attention's forward: where its window covers the grid it
is attention over every token, so the fp64 definition of that gives what is finite, NaN and
infinite, and the finite values, at every column of a tile's softmax."""
import math

import pytest
import torch

from tests import _block_ref as ref
import video_dit_sparse_dsa_b200 as dsa

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
GRID, N = (4, 8, 16), 512
# tiles of one 128-token chunk (single CTAs) and of two (CTA pairs)
TILES = [(2, 8, 8), (4, 8, 8)]


def draw(seed, B, h, n):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn(B, h, n, 128, generator=g, device=DEV).to(BF) for _ in range(3)]


def token(r):
    """Token of row r of the first tile's first chunk (two planes of 8 x 8)."""
    t, y, x = r // 64, r // 8 % 8, r % 8
    return (t * GRID[1] + y) * GRID[2] + x


def compare(got, lse, q, k, v, extra=0.0, what=""):
    ro, rl, tol = ref.cross(q, k, v, None)
    # the FMA pipe's cubic (2^-13.6 of an exponential, in P and in the sum) beside the bound of P's rounding
    mag = tol / ref.P_ERR
    ref.close(lse, rl, ref.LSE_TOL + 2.0 ** -13, f"lse {what}")
    ref.close(got, ro, tol + (2.0 ** -12 + extra) * mag, f"out {what}")
    assert dsa.device_status()[0] == 0


def grid(x):
    return x.view(*x.shape[:2], *GRID, 128)


def tiles_of(tile):
    return (GRID[0] // tile[0]) * (GRID[1] // tile[1]) * (GRID[2] // tile[2])


def forward(q, k, v, tile):
    off = torch.zeros(tiles_of(tile), 3, dtype=torch.int32, device=DEV)
    out, lse = dsa.forward(grid(q), grid(k), grid(v), off, tile, GRID)
    return out.reshape(q.shape), lse.reshape(q.shape[:3])


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("tile", TILES)
def test_window(tile, bad):
    q, k, v = draw(1, 128, 1, N)
    for r in range(128):  # one entry of the batch for each row of the tile
        k[r, 0, token(r), r] = bad
    compare(*forward(q, k, v, tile), q, k, v, what=f"{bad}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_window_fp32(bad, d):
    """The fp32 path: one key, and from entry 8 on every key of a tile, of the grid, of all tiles but one."""
    g = torch.Generator(device=DEV).manual_seed(6)
    q, k, v = (torch.randn(12, 2, N, d, generator=g, device=DEV) for _ in range(3))
    x = torch.arange(N, device=DEV) % GRID[2] < 8
    for b in range(8):
        k[b, :, token(17 * b), b] = bad
    q[8:, :, :, 9] = q[8:, :, :, 9].abs() + 0.1
    k[8, :, x, 9] = k[9, :, :, 9] = k[10, :, ~x, 9] = k[11, :, 1:, 9] = bad
    off = torch.zeros(tiles_of((2, 8, 8)), 3, dtype=torch.int32, device=DEV)
    out, lse = dsa.forward(*(t.view(12, 2, *GRID, d) for t in (q, k, v)), off, (2, 8, 8), GRID)
    ro, rl, tol = ref.cross(q, k, v, None)
    # a score: at most 66 roundings of 2^-24 of a magnitude below 16, 2^-14 with the exponential's own; a
    # sum of 512 weights in a chain: 2^-15; the output has both in its numerator and its denominator
    ref.close(lse.view(12, 2, N), rl, 2.0 ** -13, "lse")
    ref.close(out.reshape(q.shape), ro, 2.0 ** -12 * tol / ref.P_ERR, "out")
    assert dsa.device_status()[0] == 0


@pytest.mark.parametrize("tile", TILES)
def test_whole_steps_of_minus_infinity(tile):
    q, k, v = draw(2, 4, 2, N)
    q[:, :, :, 9] = 1.0
    q[0, :, ::2, 9] = -1.0
    x = torch.arange(N, device=DEV) % GRID[2] < 8  # the first column of tiles: 256 keys
    k[0, :, :, 9] = -math.inf
    k[1, :, x, 9] = -math.inf
    k[2, :, ~x, 9] = -math.inf
    k[3, :, 1:, 9] = -math.inf
    compare(*forward(q, k, v, tile), q, k, v)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("tile", TILES)
def test_lists(tile, bad):
    n = tiles_of(tile)
    q, k, v = draw(3, 16, 1, N)
    for b in range(16):
        k[b, 0, token(48 + b), b] = bad
    rp = torch.arange(n + 1, dtype=torch.int32, device=DEV) * n
    kv = torch.arange(n, dtype=torch.int32, device=DEV).repeat(n)
    out, lse = dsa.forward_list(grid(q), grid(k), grid(v), rp, kv, tile)
    compare(out.reshape(q.shape), lse.reshape(q.shape[:3]), q, k, v, what=f"{bad}")


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("L", [77, 300])
@pytest.mark.parametrize("tile", TILES)
def test_prefix(tile, L, bad):
    """Keys among the video's and the text's; the text rows' parts are rounded to bf16 and joined."""
    q, k, v = draw(4, 16, 1, N + L)
    for b in range(16):
        k[b, 0, (token(48 + b), N + 45 + b)[b % 2], b] = bad
    if bad == -math.inf:
        q[15, :, :, 9], k[15, :, :, 9] = 1.0, bad  # nothing has a weight
    off = torch.zeros(tiles_of(tile), 3, dtype=torch.int32, device=DEV)
    video, text = [grid(t[:, :, :N].contiguous()) for t in (q, k, v)], [t[:, :, N:].contiguous() for t in (q, k, v)]
    out, lse, out_t, lse_t = dsa.forward_prefix(*video, off, *text, tile, GRID)
    got, got_lse = torch.cat((out.reshape(16, 1, N, 128), out_t), 2), torch.cat((lse.reshape(16, 1, N), lse_t), 2)
    compare(got, got_lse, q, k, v, extra=2.0 ** -8, what=f"{bad}")


@pytest.mark.parametrize("tile", TILES)
def test_block_map(tile):
    """A key whose scores are NaN makes the mass of its tile NaN, whichever of its columns it is in."""
    n = tiles_of(tile)
    q, k, v = draw(5, 16, 1, N)
    rp = torch.arange(n + 1, dtype=torch.int32, device=DEV) * n
    kv = torch.arange(n, dtype=torch.int32, device=DEV).repeat(n)
    _, lse = dsa.forward_list(grid(q), grid(k), grid(v), rp, kv, tile)
    clean = dsa.block_map(grid(q), grid(k), lse, rp, kv, tile)
    for b in range(16):
        k[b, 0, token(b), b] = math.nan
    m = dsa.block_map(grid(q), grid(k), lse, rp, kv, tile)
    assert torch.isnan(m[:, :, 0]).all() and torch.equal(m[:, :, 1:], clean[:, :, 1:])
    assert dsa.device_status()[0] == 0
