"""The sliding attention's calls on another stream than the current one: what they allocate is never
memory that work queued on the current stream still uses."""
import pytest
import torch

import video_dit_sparse_dsa_b200 as dsa
from tests import test_block_streams_gpu as block

pytestmark = pytest.mark.gpu
DEV = "cuda"
GRID, TILE, WINDOW, TILES = (8, 16, 24), (4, 8, 8), (3, 3, 3), 12
SHAPE = (1, 2, *GRID, 128)


def args(n=4):
    off = torch.randint(-1, 2, (TILES, 3), generator=torch.Generator().manual_seed(1), dtype=torch.int32).to(DEV)
    return [block.rn(10 + i, *SHAPE) for i in range(n)] + [off]


def problem():
    return dsa.make_problem(1, 2, 128, GRID, TILE, WINDOW)


def _forward():
    q, k, v, _, off = args()
    return lambda s: dsa.forward(q, k, v, off, TILE, WINDOW, stream=s), max(dsa.workspace_size(problem()), 256)


def _backward():
    q, k, v, do, off = args()
    out, lse = dsa.forward(q, k, v, off, TILE, WINDOW)
    return (lambda s: dsa.backward(q, k, v, out, lse, do, off, TILE, WINDOW, stream=s),
            dsa.workspace_size(problem(), backward=True))


def lists():
    rp = torch.arange(TILES + 1, dtype=torch.int32, device=DEV) * 5
    kv = torch.cat([torch.randperm(TILES, generator=torch.Generator().manual_seed(i))[:5] for i in range(TILES)])
    return rp, kv.to(torch.int32).to(DEV)


def _forward_list():
    q, k, v, _, _ = args()
    rp, kv = lists()
    return lambda s: dsa.forward_list(q, k, v, rp, kv, TILE, stream=s), 0


def _backward_list():
    q, k, v, do, _ = args()
    rp, kv = lists()
    out, lse = dsa.forward_list(q, k, v, rp, kv, TILE)
    n = dsa.load_library().dsa_list_workspace_size(problem(), kv.numel(), 0, dsa.DSA_WS_BWD)
    return lambda s: dsa.backward_list(q, k, v, out, lse, do, rp, kv, TILE, stream=s), n


def _forward_prefix():
    q, k, v, _, off = args()
    t = [block.rn(20 + i, 1, 2, 300, 128) for i in range(3)]
    return (lambda s: dsa.forward_prefix(q, k, v, off, *t, TILE, WINDOW, stream=s),
            dsa.prefix_workspace_size(problem(), 300))


def _backward_prefix():
    q, k, v, do, off = args()
    t = [block.rn(20 + i, 1, 2, 300, 128) for i in range(4)]
    out, lse, ot, lt = dsa.forward_prefix(q, k, v, off, *t[:3], TILE, WINDOW)
    return (lambda s: dsa.backward_prefix(q, k, v, out, lse, do, off, *t[:3], ot, lt, t[3], TILE, WINDOW, stream=s),
            dsa.prefix_bwd_workspace_size(problem(), 300))


def _block_map():
    q, k, v, _, _ = args()
    rp, kv = lists()
    _, lse = dsa.forward_list(q, k, v, rp, kv, TILE)
    return lambda s: (dsa.block_map(q, k, lse, rp, kv, TILE, stream=s),), 0


def _plan():
    off = args()[-1]
    return lambda s: dsa.plan(problem(), off, stream=s), 0


def _plan_heads():
    off = args()[-1].repeat(2, 1, 1)
    return lambda s: dsa.plan_heads(problem(), off, stream=s), 0


def _lstsq():
    M, S = block.rn(30, 4000, 3, dtype=torch.float32), block.rn(31, 24, 4000, dtype=torch.float32)

    def call(s):
        L = dsa.lstsq_factor(M, 0.5, stream=s)
        return L, dsa.lstsq_solve(M, L, S, stream=s)

    return call, 0


OPS = [_forward, _backward, _forward_list, _backward_list, _forward_prefix, _backward_prefix, _block_map, _plan,
       _plan_heads, _lstsq]


@pytest.mark.parametrize("queued", ["reads", "writes"])
@pytest.mark.parametrize("op", OPS, ids=lambda f: f.__name__[1:])
def test_memory_in_use_on_the_current_stream(op, queued):
    block.test_memory_in_use_on_the_current_stream(op, queued)


@pytest.mark.parametrize("op", OPS, ids=lambda f: f.__name__[1:])
def test_results_dropped_with_reads_queued(op):
    block.test_results_dropped_with_reads_queued(op)
