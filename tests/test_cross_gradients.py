"""The cross attention's gradients against central differences of the fp64 forward, along directions
of one row or key each, with bounds well below the derivative: gradients of zero and of the other
sign have to fail.

A direction is the sign of the expected gradient on its row, so that <grad, u> is the sum of its
magnitudes, where a bound's worst case is the sum of its elements' (a random direction over all of a
tensor sums the magnitudes of the errors against a derivative that mostly cancels)."""
import math

import pytest
import torch

from tests import _block_ref as ref
import video_dit_sparse_dsa_b200 as dsa

BF = torch.bfloat16
STEP = 1e-4  # the differences' own error: STEP^2 of the third derivative, 1e-15 / STEP of the value


def draw(seed, B, h, hk, Lq, Lk, device, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    q, k, v, do = (torch.randn(B, n, L, 128, generator=g) for n, L in ((h, Lq), (hk, Lk), (hk, Lk), (h, Lq)))
    return [t.to(BF).to(device) for t in (spread * q, k, v, do)]


def per_row(q, k, v, do, lens):
    """sum over channels of out * dout: [B, h, Lq] (a row of q changes its own entry only)."""
    return (ref.cross(q, k, v, lens)[0] * do.double()).sum(-1)


def differences(which, q, k, v, do, lens, u, at=None):
    """Derivatives along u: of every row's own entry (q, all rows at once), or of the sum of all
    along row `at` = (b, kv head, key) of u (k, v)."""
    x = [t.double() for t in (q, k, v)]
    i = "qkv".index(which)
    d = u
    if at is not None:
        d = torch.zeros_like(u)
        d[at] = u[at]
    up, dn = list(x), list(x)
    up[i], dn[i] = x[i] + STEP * d, x[i] - STEP * d
    r = (per_row(*up, do, lens) - per_row(*dn, do, lens)) / (2 * STEP)
    return r if at is None else float(r.sum())


def keys_of(B, hk, lens):
    return [(b, j, m) for b in range(B) for j in sorted({0, hk - 1}) for m in sorted({0, lens[b] // 2, lens[b] - 1})]


def test_formula():
    """The formula that the kernels are compared with, without any rounding."""
    B, h, hk, Lq, lens = 2, 4, 2, 9, (21, 8)
    q, k, v, do = draw(1, B, h, hk, Lq, 21, "cpu")
    out, lse, _ = ref.cross(q, k, v, lens)
    (dq, dk, dv), _ = ref.cross_bwd(q, k, v, out, lse, do, lens)
    num = differences("q", q, k, v, do, lens, torch.sign(dq))
    assert ((num - dq.abs().sum(-1)).abs() <= 1e-6 * dq.abs().sum(-1)).all() and (dq.abs().sum(-1) > 1e-3).all()
    for which, g in (("k", dk), ("v", dv)):
        for at in keys_of(B, hk, lens):
            want = float(g[at].abs().sum())
            assert abs(differences(which, q, k, v, do, lens, torch.sign(g), at) - want) <= 1e-6 * want and want > 1e-3


def out_rounding(q, k, v, do, lens):
    """What the rounding of the out that D is taken from adds to the bounds of dq and dk: |dD_n| is at
    most sum_c |dout_nc| tol_nc, and dS_nm is off by P_nm dD_n."""
    B, h, Lq, d = q.shape
    g = h // k.shape[1]
    _, lse, tol = ref.cross(q, k, v, lens)
    dD = (do.double().abs() * tol).sum(-1)
    tq, tk = torch.zeros_like(q, dtype=torch.float64), torch.zeros_like(k, dtype=torch.float64)
    for b, n in enumerate(lens):
        for i in range(h):
            qq, kk = q[b, i].double(), k[b, i // g, :n].double()
            e = torch.exp(qq @ kk.T / math.sqrt(d) - lse[b, i][:, None]) * dD[b, i][:, None] / math.sqrt(d)
            tq[b, i] = e @ kk.abs()
            tk[b, i // g, :n] += e.T @ qq.abs()
    return tq, tk, 0.0


# row pairs, single tiles, heads packed into a tile, keys in parts (with scores of a larger spread, so
# that the errors of a thousand keys are not summed in the worst case)
@pytest.mark.gpu
@pytest.mark.parametrize("B,h,hk,Lq,lens,spread", [(1, 1, 1, 260, (70,), 1.0), (2, 2, 1, 60, (200, 33), 1.0),
                                                   (2, 4, 2, 5, (70, 129), 1.0), (1, 2, 2, 3, (1400,), 3.0)])
def test_kernels(B, h, hk, Lq, lens, spread):
    q, k, v, do = draw(2, B, h, hk, Lq, max(lens), "cuda", spread)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = dsa.forward_cross(q, k, v, kv_len=n)
    grads = dsa.backward_cross(q, k, v, out, lse, do, kv_len=n)
    assert dsa.device_status()[0] == 0
    want, tols = ref.cross_bwd(q, k, v, out, lse, do, lens)
    extra = out_rounding(q, k, v, do, lens)
    # the derivative that the bounds stand against, where they are the largest part of it
    worst = 0.0
    for i, which in enumerate("qkv"):
        u = torch.sign(want[i])
        got, tol = (grads[i].double() * u).sum(-1), (tols[i] + extra[i]).sum(-1)
        if which == "q":
            num = differences("q", q, k, v, do, lens, u)
            pairs = list(zip(num.flatten().tolist(), got.flatten().tolist(), tol.flatten().tolist()))
        else:
            pairs = [(differences(which, q, k, v, do, lens, u, at), float(got[at]), float(tol[at])) for at in keys_of(B, hk, lens)]
        for num, g, t in pairs:
            assert abs(g - num) <= t + 1e-5 * abs(num), (which, g, num, t)
            assert abs(num) > t, (which, num, t)  # zero fails, and so does -g (further off)
            worst = max(worst, t / abs(num))
    assert worst < 0.75
