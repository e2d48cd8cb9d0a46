"""Cross attention with NaN and infinities at valid keys and values: what is finite, NaN and infinite,
and the finite values, as the fp64 definition gives them, at every position of sixteen consecutive
keys (a batch entry has the odd value at one of them)."""
import math

import pytest
import torch

from tests import _block_ref as ref
import video_dit_sparse_dsa_b200 as dsa

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16

# (heads, kv_heads, Lq, Lk, first of the sixteen keys): row pairs over one chunk, one chunk's end, two
# steps and the last of them; single tiles; heads packed into a tile; keys in parts (the last in a
# part of one key more than whole steps)
FORMS = [(2, 2, 300, 77, 3), (1, 1, 257, 130, 114), (2, 1, 200, 512, 300), (1, 1, 150, 461, 445), (2, 2, 40, 77, 61),
         (1, 1, 90, 300, 130), (4, 1, 3, 200, 100), (2, 2, 1, 3000, 1500), (4, 2, 5, 2817, 2801)]


def draw(seed, B, h, hk, Lq, Lk):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn(B, n, L, 128, generator=g, device=DEV).to(BF) for n, L in ((h, Lq), (hk, Lk), (hk, Lk), (h, Lq))]


def check(q, k, v, do=None, what="", grads=("dq", "dk", "dv")):
    out, lse = dsa.forward_cross(q, k, v)
    ro, rl, tol = ref.cross(q, k, v, None)
    ref.close(lse, rl, ref.LSE_TOL, f"lse {what}")
    ref.close(out, ro, tol, f"out {what}")
    if do is not None:
        got = dsa.backward_cross(q, k, v, out, lse, do)
        rg, rt = ref.cross_bwd(q, k, v, out, lse, do, None)
        for name, a, b, t in zip(("dq", "dk", "dv"), got, rg, rt):
            if name in grads:
                ref.close(a, b, t, f"{name} {what}")
    assert dsa.device_status()[0] == 0
    return out, lse


def parts_of(h, hk, Lq, Lk):
    p = dsa.Cross(B=16, heads=h, kv_heads=hk, d=128, Lq=Lq, Lk=Lk, scale=1.0, dtype=dsa.DSA_BF16)
    return dsa.cross_workspace_size(p) > 0


def test_forms_cover_keys_in_parts():
    assert [parts_of(*f[:4]) for f in FORMS] == [f[3] >= 2800 for f in FORMS]


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: "x".join(str(x) for x in f[:4]))
def test_one_key(form, bad):
    """An infinite key gives rows of scores +inf and rows of -inf, by the sign of q's channel."""
    h, hk, Lq, Lk, first = form
    q, k, v, _ = draw(Lk, 16, h, hk, Lq, Lk)
    for b in range(16):
        k[b, hk - 1, first + b, 7 * b] = bad
    check(q, k, v, what=f"{bad}")


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: "x".join(str(x) for x in f[:4]))
def test_one_value(form, bad):
    h, hk, Lq, Lk, first = form
    q, k, v, _ = draw(Lk + 1, 16, h, hk, Lq, Lk)
    for b in range(16):
        v[b, hk - 1, first + b, 5 * b] = bad
    check(q, k, v, what=f"{bad}")


@pytest.mark.parametrize("form", FORMS, ids=lambda f: "x".join(str(x) for x in f[:4]))
def test_whole_steps_of_minus_infinity(form):
    """Scores of -inf at every key of some steps (a weight of 0), or at all keys (LSE -inf, no
    output), +inf for the rows on the other side."""
    h, hk, Lq, Lk, first = form
    q, k, v, _ = draw(Lk + 2, 16, h, hk, Lq, Lk)
    half = (torch.arange(Lq, device=DEV) % 2).bool()
    q[:, :, :, 9] = torch.where(half, 1.0, -1.0).to(BF)
    q[4:, :, :, 9] = 1.0
    for b in range(16):
        lo, hi = ((0, Lk), (0, min(256, Lk - 1)), (Lk // 2, Lk), (1, Lk))[b % 4]
        k[b, :, lo:hi, 9] = -math.inf
    check(q, k, v)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: "x".join(str(x) for x in f[:4]))
def test_dq_one_key(form, bad):
    """A weight of 0 against an infinite key is NaN: dS of that key is 0, not a small number."""
    h, hk, Lq, Lk, first = form
    q, k, v, do = draw(Lk + 3, 16, h, hk, Lq, Lk)
    for b in range(16):
        k[b, hk - 1, first + b, 7 * b] = bad
        if bad == -math.inf:
            q[b, :, :, 7 * b] = q[b, :, :, 7 * b].abs() + 0.25  # scores of -inf only
    check(q, k, v, do, what=f"{bad}", grads=("dq",))


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: "x".join(str(x) for x in f[:4]))
def test_backward_one_row(form, bad):
    """A row of dout, or a value, that is not finite."""
    h, hk, Lq, Lk, first = form
    q, k, v, do = draw(Lk + 4, 16, h, hk, Lq, Lk)
    for b in range(16):
        if b % 2:
            v[b, hk - 1, first + b, 5 * b] = bad
        else:
            do[b, h - 1, (7 * b) % Lq, 5 * b] = bad
    check(q, k, v, do, what=f"{bad}")


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: "x".join(str(x) for x in f[:4]))
def test_dk_dv_one_key(form, bad):
    """A tile's missing rows (zeros, whose score with an infinite key is NaN) add nothing."""
    h, hk, Lq, Lk, first = form
    q, k, v, do = draw(Lk + 5, 16, h, hk, Lq, Lk)
    for b in range(16):
        k[b, hk - 1, first + b, 7 * b] = bad
        if bad == -math.inf:
            q[b, :, :, 7 * b] = q[b, :, :, 7 * b].abs() + 0.25  # scores of -inf only
    check(q, k, v, do, what=f"{bad}", grads=("dk", "dv"))
