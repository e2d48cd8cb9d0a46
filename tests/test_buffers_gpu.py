"""Buffers of another size than the problem's are refused before anything is launched."""
import pytest
import torch

import video_dit_sparse_dsa_b200 as dsa

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
GRID, TILE, WINDOW, TILES, N = (4, 8, 16), (4, 8, 8), (1, 1, 1), 2, 512


def new(*shape, dtype=BF, device=DEV):
    return torch.zeros(*shape, dtype=dtype, device=device)


def video(n):
    return [new(1, 2, *GRID, 128) for _ in range(n)]


OFF = lambda n=TILES: new(n, 3, dtype=torch.int32)  # noqa: E731
LSE = lambda *s: new(*(s or (1, 2, *GRID)), dtype=torch.float32)  # noqa: E731
SMALL = lambda: new(1, 2, 4, 8, 8, 128)  # noqa: E731
LISTS = lambda: (torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV), torch.tensor([0, 1], dtype=torch.int32, device=DEV))  # noqa: E731


def refuses(f, *args, **kw):
    with pytest.raises((ValueError, dsa.DsaError)):
        f(*args, **kw)
    assert dsa.device_status()[0] == 0


def test_forward():
    q, k, v = video(3)
    f = lambda off=None, **kw: dsa.forward(q, k, v, OFF() if off is None else off, TILE, WINDOW, **kw)  # noqa: E731
    refuses(f, OFF(1))
    refuses(f, out=SMALL())
    refuses(f, lse=LSE(1, 2, 4, 8, 8))
    refuses(f, ws=new(64, dtype=torch.uint8))
    refuses(f, ws=new(16, dtype=torch.float32))
    assert f(ws=new(1 << 16, dtype=torch.float32))[0].shape == q.shape
    refuses(f, ws=new(1 << 16, 2, dtype=torch.uint8)[:, 0])
    assert f()[0].shape == q.shape


def test_backward():
    q, k, v, out, do = video(5)
    f = lambda off=None, lse=None, **kw: dsa.backward(q, k, v, out, LSE() if lse is None else lse, do,  # noqa: E731
                                                      OFF() if off is None else off, TILE, WINDOW, **kw)
    refuses(f, OFF(1))
    refuses(f, lse=LSE(1, 2, 4, 8, 8))
    for name in ("dq", "dk", "dv"):
        refuses(f, **{name: SMALL()})
    refuses(f, ws=new(64, dtype=torch.uint8))
    assert f()[0].shape == q.shape


def test_lists_and_map():
    q, k, v, out, do = video(5)
    refuses(dsa.forward_list, q, k, v, *LISTS(), TILE, out=SMALL())
    refuses(dsa.forward_list, q, k, v, *LISTS(), TILE, lse=LSE(1, 2, 4, 8, 8))
    refuses(dsa.backward_list, q, k, v, out, LSE(1, 2, 4, 8, 8), do, *LISTS(), TILE)
    refuses(dsa.backward_list, q, k, v, out, LSE(), do, *LISTS(), TILE, dk=SMALL())
    refuses(dsa.backward_list, q, k, v, out, LSE(), do, *LISTS(), TILE, ws=new(64, dtype=torch.uint8))
    refuses(dsa.block_map, q, SMALL(), LSE(), *LISTS(), TILE)
    refuses(dsa.block_map, q, k, LSE(1, 2, 4, 8, 8), *LISTS(), TILE)
    refuses(dsa.block_map, q, k, LSE(), *LISTS(), TILE, out=LSE(2, 2, 1))


def test_prefix():
    q, k, v, out, do = video(5)
    t = [new(1, 2, 30, 128) for _ in range(5)]
    refuses(dsa.forward_prefix, q, k, v, OFF(1), *t[:3], TILE, WINDOW)
    refuses(dsa.forward_prefix, q, k, v, OFF(), *t[:3], TILE, WINDOW, ws=new(64, dtype=torch.uint8))
    b = lambda off, lse, lse_t: dsa.backward_prefix(q, k, v, out, lse, do, off, *t[:3], t[3], lse_t, t[4], TILE, WINDOW)  # noqa: E731
    refuses(b, OFF(1), LSE(), LSE(1, 2, 30))
    refuses(b, OFF(), LSE(1, 2, 4, 8, 8), LSE(1, 2, 30))
    refuses(b, OFF(), LSE(), LSE(1, 2, 29))


def test_least_squares():
    M, S, L = LSE(100, 3), LSE(4, 100), new(3, 3, dtype=torch.float64)
    refuses(dsa.lstsq_solve, M, L[:2].contiguous(), S)
    refuses(dsa.lstsq_solve, M, L.float(), S)
    refuses(dsa.lstsq_solve, M.to(BF), L, S)
    refuses(dsa.lstsq_solve, M, L, S, X=LSE(3, 3))


@pytest.mark.parametrize("which", range(7))
def test_host(which):
    p = dsa.make_problem(1, 2, 128, GRID, TILE, WINDOW)
    host = [new(1, 2, *GRID, 128, device="cpu") for _ in range(3)] + [new(TILES, 3, dtype=torch.int32, device="cpu")]
    host += [new(1, 2, *GRID, 128, device="cpu"), new(1, 2, *GRID, dtype=torch.float32, device="cpu")]
    host += [new(dsa.forward_host_bytes(p), dtype=torch.uint8)]
    host[which] = host[which].flatten()[1:].clone() if which < 6 else host[which][:-256]
    refuses(dsa.forward_host, p, *host)


def test_host_without_a_device_buffer():
    p = dsa.make_problem(1, 2, 128, GRID, TILE, WINDOW)
    x = new(1, 2, *GRID, 128, device="cpu")
    refuses(dsa.forward_host, p, x, x, x, new(TILES, 3, dtype=torch.int32, device="cpu"), x.clone(),
            new(1, 2, *GRID, dtype=torch.float32, device="cpu"), new(dsa.forward_host_bytes(p), dtype=torch.uint8, device="cpu"))
