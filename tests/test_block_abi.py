"""CPU checks of the operators around the sliding attention: refusals at the C boundary and in
the binding, workspace sizes, and the tests' own fp64 gradients against autograd."""
import ctypes

import pytest
import torch

from tests import _block_ref as ref
import video_dit_sparse_dsa_b200 as dsa
from video_dit_sparse_dsa_b200 import build as dsa_build

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return dsa.load_library()


def view(data=FAKE, s=(1 << 16, 1 << 12, 128)):
    v = dsa.View()
    v.data = data
    for a in range(3):
        v.stride[a] = s[a]
    return ctypes.byref(v)


def cross(**kw):
    a = dict(B=2, heads=4, kv_heads=2, d=128, Lq=10, Lk=30, scale=0.1, dtype=dsa.DSA_BF16)
    a.update(kw)
    return dsa.Cross(**a)


BIG = 1 << 40


def fwd(lib, p, **kw):
    a = dict(q=view(), k=view(), v=view(), n=FAKE, out=view(), lse=FAKE, ws=FAKE, size=BIG)
    a.update(kw)
    return lib.dsa_fwd_cross(ctypes.byref(p), a["q"], a["k"], a["v"], a["n"], a["out"], a["lse"], a["ws"], a["size"], None)


def bwd(lib, p, **kw):
    a = dict(q=view(), k=view(), v=view(), out=view(), lse=FAKE, do=view(), n=FAKE, dq=view(), dk=view(), dv=view(),
             ws=FAKE, size=BIG)
    a.update(kw)
    return lib.dsa_bwd_cross(ctypes.byref(p), a["q"], a["k"], a["v"], a["out"], a["lse"], a["do"], a["n"], a["dq"],
                             a["dk"], a["dv"], a["ws"], a["size"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(heads=0), 1), (dict(kv_heads=3), 1), (dict(kv_heads=0), 1), (dict(Lq=-1), 1), (dict(Lk=-1), 1),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(dtype=7), 1), (dict(dtype=dsa.DSA_F32), 2), (dict(d=64), 2), (dict(d=0), 2),
    (dict(B=1 << 15, heads=1 << 15, kv_heads=1 << 15), 2),          # more units than 32 bits
    (dict(Lq=2 ** 31 - 1), 2), (dict(Lk=2 ** 31 - 1), 2), (dict(heads=64, kv_heads=64, Lq=1 << 26), 2),
])
def test_cross_refuses_problems(lib, kw, status):
    p = cross(**kw)
    assert fwd(lib, p) == status and bwd(lib, p) == status
    assert dsa.cross_workspace_size(p) == 0 and dsa.cross_workspace_size(p, backward=True) == 0


BAD_VIEWS = [None, view(data=None), view(data=FAKE + 8), view(s=(1 << 16, 1 << 12, 132)), view(s=(1 << 16, -128, 128)),
             view(s=(1 << 16, 64, 128)), view(s=(1 << 16, 1 << 12, 0)), view(s=(1 << 39, 1 << 12, 128))]


def test_cross_refuses_views_and_workspaces(lib):
    p = cross()
    for bad in BAD_VIEWS:
        for name in ("q", "k", "v", "out"):
            assert fwd(lib, p, **{name: bad}) == 1, name
        for name in ("q", "k", "v", "out", "do", "dq", "dk", "dv"):
            assert bwd(lib, p, **{name: bad}) == 1, name
    over = view(s=(0, 1 << 12, 128))  # a broadcast output
    assert fwd(lib, p, out=over) == 1 and bwd(lib, p, dk=over) == 1
    assert fwd(lib, p, lse=None) == 1 and fwd(lib, p, lse=FAKE + 2) == 1 and fwd(lib, p, n=FAKE + 2) == 1
    assert bwd(lib, p, lse=None) == 1 and bwd(lib, p, n=FAKE + 2) == 1
    assert lib.dsa_fwd_cross(None, *[view()] * 3, FAKE, view(), FAKE, FAKE, BIG, None) == 1
    long = cross(Lq=1, Lk=100000)
    need = dsa.cross_workspace_size(long)
    assert need > 0 and dsa.cross_workspace_size(p) == 0
    assert fwd(lib, long, ws=None) == 5 and fwd(lib, long, size=need - 1) == 5 and fwd(lib, long, ws=FAKE + 64) == 5
    need = dsa.cross_workspace_size(p, backward=True)
    assert need >= 2 * 4 * 2 * 4 * 64
    assert bwd(lib, p, ws=None) == 5 and bwd(lib, p, size=need - 1) == 5 and bwd(lib, p, ws=FAKE + 64) == 5
    assert lib.dsa_cross_workspace_size(ctypes.byref(p), 5) == 0
    assert fwd(lib, cross(Lq=0), q=None, out=None, lse=None) == 0  # nothing to do


def rope(lib, table=FAKE, q=None, qo=None, k=None, ko=None, **kw):
    a = dict(B=1, heads=2, d=64, T=2, H=3, W=4, interleaved=1, inverse=0, dtype=dsa.DSA_BF16)
    axes = kw.pop("axes", (16, 24, 24))
    a.update(kw)
    p = dsa.Rope(**a)
    for i in range(3):
        p.axes[i] = axes[i]
    return lib.dsa_rope(ctypes.byref(p), table, q or view(), qo or view(), k, ko, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(T=0), 1), (dict(d=0), 1), (dict(axes=(16, 24, 25)), 1), (dict(axes=(-2, 24, 24)), 1),
    (dict(axes=(0, 0, 0)), 1), (dict(axes=(16, 24, 26)), 1), (dict(dtype=2), 1), (dict(interleaved=2), 1),
    (dict(inverse=-1), 1), (dict(table=None), 1), (dict(table=FAKE + 4), 1), (dict(q=view(data=None)), 1),
    (dict(q=view(data=FAKE + 1)), 1), (dict(k=view()), 1), (dict(ko=view()), 1), (dict(q=view(s=(0, -64, 64))), 1),
    (dict(qo=view(s=(0, 0, 64))), 1), (dict(qo=view(s=(0, 4096, 32))), 1), (dict(B=70000), 2),
    (dict(T=1 << 20, H=1 << 10, W=8), 2),
])
def test_rope_refuses(lib, kw, status):
    assert rope(lib, **kw) == status


def test_rope_table_refuses(lib):
    i3, d3 = ctypes.c_int32 * 3, ctypes.c_double * 3

    def call(grid=(2, 3, 4), axes=(4, 4, 4), start=(0, 0, 0), step=(1, 1, 1), theta=1e4, table=FAKE):
        return lib.dsa_rope_table(i3(*grid), i3(*axes), d3(*start), d3(*step), theta, table, None)

    assert call(table=None) == 1 and call(theta=0.0) == 1 and call(theta=float("nan")) == 1
    assert call(grid=(0, 3, 4)) == 1 and call(axes=(3, 4, 4)) == 1 and call(axes=(0, 0, 0)) == 1
    assert call(start=(float("inf"), 0, 0)) == 1 and call(step=(float("nan"), 1, 1)) == 1 and call(table=FAKE + 4) == 1
    assert call(grid=(1 << 30, 1, 1), axes=(64, 2, 2)) == 2
    assert lib.dsa_rope_table(None, i3(4, 4, 4), d3(0, 0, 0), d3(1, 1, 1), 1e4, FAKE, None) == 1


def test_norm_refuses(lib):
    def fwd(x=FAKE, x_ld=256, r=None, r_ld=0, w=FAKE, y=FAKE, h=None, **kw):
        a = dict(rows=4, C=256, eps=1e-6, dtype=dsa.DSA_BF16)
        a.update(kw)
        p = dsa.Norm(**a)
        st = lib.dsa_rmsnorm(ctypes.byref(p), x, x_ld, r, r_ld, w, y, h, None)
        assert lib.dsa_rmsnorm_fp8(ctypes.byref(p), x, x_ld, r, r_ld, w, y, FAKE, h, None) in (st, 1)
        return st

    assert fwd(rows=-1) == 1 and fwd(C=0) == 1 and fwd(eps=-1.0) == 1 and fwd(eps=float("nan")) == 1
    assert fwd(dtype=3) == 1 and fwd(C=16385, x_ld=1 << 20) == 2 and fwd(rows=1 << 31) == 2
    assert fwd(x=None) == 1 and fwd(y=None) == 1 and fwd(x_ld=255) == 1 and fwd(x=FAKE + 1) == 1
    assert fwd(r=FAKE, r_ld=256) == 1 and fwd(h=FAKE) == 1 and fwd(r=FAKE, r_ld=100, h=FAKE) == 1
    assert fwd(rows=0, x=None, y=None, w=None) == 0
    p = dsa.Norm(rows=4, C=256, eps=1e-6, dtype=dsa.DSA_F32)
    assert lib.dsa_rmsnorm_fp8(ctypes.byref(p), FAKE, 256, None, 0, None, FAKE, None, None, None) == 1  # no scales

    def bwd(h=FAKE, h_ld=256, w=FAKE, dy=FAKE, dy_ld=256, dh=None, dh_ld=0, dx=FAKE, dw=FAKE, ws=FAKE, size=BIG):
        return lib.dsa_rmsnorm_bwd(ctypes.byref(p), h, h_ld, w, dy, dy_ld, dh, dh_ld, dx, dw, ws, size, None)

    need = lib.dsa_rmsnorm_bwd_workspace_size(ctypes.byref(p))
    assert need >= 256 * 4
    assert bwd(h=None) == 1 and bwd(dy=None) == 1 and bwd(dx=None) == 1 and bwd(w=None) == 1 and bwd(dy_ld=3) == 1
    assert bwd(dh=FAKE, dh_ld=9) == 1 and bwd(dx=FAKE + 2) == 1
    assert bwd(ws=None) == 5 and bwd(size=need - 1) == 5 and bwd(ws=FAKE + 32) == 5


def test_binding_refuses():
    t = torch.zeros(1, 2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dsa.forward_cross(t, t, t)  # not on a GPU
    with pytest.raises(ValueError):
        dsa.forward_cross(t, t[:, :, :, :64], t)
    with pytest.raises(ValueError):
        dsa.forward_cross(t, t, t.float())
    with pytest.raises(ValueError):
        dsa.forward_cross(t, t, t, kv_len=torch.zeros(1))
    with pytest.raises(ValueError):
        dsa.forward_cross(t.half(), t.half(), t.half())
    x = torch.zeros(1, 2, 2, 3, 4, 64)
    with pytest.raises(ValueError):
        dsa.rope(x, None, torch.zeros(3, 2), (16, 24, 24))  # a table of another grid
    with pytest.raises(ValueError):
        dsa.rope(x, None, torch.zeros(1, 2), (16, 24))
    with pytest.raises(ValueError):
        dsa._grid_view(x.transpose(2, 4).contiguous().transpose(2, 4), "x")  # not raster order
    with pytest.raises(ValueError):
        dsa.rms_norm(torch.zeros(4, 8, 16).transpose(0, 1))  # rows without one stride
    with pytest.raises(ValueError):
        dsa.rms_norm(torch.zeros(8, 16).t())
    with pytest.raises(ValueError):
        dsa.rms_norm(torch.zeros(4, 8), torch.zeros(7))
    assert dsa._rows(torch.zeros(2, 5, 3, 8)[:, :, 1], "x") == (10, 8, 24)
    assert dsa._rows(torch.zeros(8), "x") == (1, 8, 8)


def test_reference_gradients_are_autograds():
    """The fp64 gradients that the GPU tests compare with, against autograd of the definitions."""
    g = torch.Generator().manual_seed(0)
    rn = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64, requires_grad=True)  # noqa: E731
    q, k, v = rn(2, 4, 5, 8), rn(2, 2, 7, 8), rn(2, 2, 7, 8)
    do = torch.randn(2, 4, 5, 8, generator=g, dtype=torch.float64)
    lens = (7, 3)
    parts = []
    for b in range(2):
        kk, vv = (t[b, :, :lens[b]].repeat_interleave(2, 0) for t in (k, v))
        parts.append(torch.softmax(q[b] @ kk.transpose(1, 2) / 8 ** 0.5, -1) @ vv)
    torch.stack(parts).mul(do).sum().backward()
    with torch.no_grad():
        out, lse, _ = ref.cross(q, k, v, lens)
        grads, _ = ref.cross_bwd(q, k, v, out, lse, do, lens)
    assert torch.allclose(out, torch.stack(parts), atol=1e-12)
    for a, t in zip(grads, (q, k, v)):
        assert torch.allclose(a, t.grad, atol=1e-12)
    x, w = rn(6, 9), rn(9)
    dy, dh = (torch.randn(6, 9, generator=g, dtype=torch.float64) for _ in range(2))
    y, h = ref.norm(x, None, w, 1e-3)
    ((y * dy).sum() + (h * dh).sum()).backward()
    with torch.no_grad():
        dx, dw, _, _ = ref.norm_bwd(x, w, dy, dh, 1e-3)
    assert torch.allclose(dx, x.grad, atol=1e-12) and torch.allclose(dw, w.grad, atol=1e-12)
