"""fp64 definitions of cross attention, rotary positions and the RMS norm, with the error bounds
that the kernels' roundings allow, for the tests of those operators.

Every bound counts the roundings that the kernels document, worst case, element by element:
  U[t]     half a step of type t relative to the value (bf16 2^-8, fp32 2^-24, e4m3 2^-4);
  cross attention: P (and dS) is rounded to bf16 before its products: relative 2^-8 of each term.
    A score adds 8 groups of 16 products, each addition off by at most 2^-22 of the sum of the
    magnitudes, which scaled is below 80 for the inputs here: 8 * 80 * 2^-22 < 2^-12, and with it
    the relative error of the exponential (itself good to 2^-18); the LSE's error is the same.
    dP - D is a difference of fp32 sums of 128 terms: 2^-16 of the sum of their magnitudes;
  norm: a sum of squares is a chain of at most 32 terms per lane and a tree of at most 5 + 16
    steps, each off by 2^-24: 2^-18 covers it and the few roundings after it; dweight sums `rows`
    terms in chains of at most rows / blocks + blocks: 2^-17.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
P_ERR = 2.0 ** -8 + 2.0 ** -12   # bf16 rounding of P or dS, and its own fp32 error
SCORE_ERR = 2.0 ** -12
DP_ERR = 2.0 ** -16
LSE_TOL = 2.0 ** -12
NORM_ERR = 2.0 ** -18


def close(got, ref, tol, what):
    """Element-wise |got - ref| <= tol, with non-finite references met exactly."""
    got, ref = got.double().cpu(), ref.double().cpu()
    tol = torch.as_tensor(tol, dtype=torch.float64).cpu().expand_as(ref)
    assert got.shape == ref.shape, f"{what}: shape {tuple(got.shape)} != {tuple(ref.shape)}"
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    inf = ~fin & ~torch.isnan(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    err = (got - ref).abs()[fin]
    assert torch.isfinite(err).all(), f"{what}: non-finite values"
    bad = err > tol[fin] + 1e-30
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {err.numel()} outside, worst "
                           f"{float((err / (tol[fin] + 1e-30)).max()):.2f} times the bound, error {float(err.max()):.3e}")


def cross(q, k, v, lens, scale=None):
    """-> out, lse, bound of out (fp64, on the inputs' device)."""
    B, h, Lq, d = q.shape
    hk, Lk = k.shape[1], k.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.zeros(B, h, Lq, d, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    lse = torch.full((B, h, Lq), -math.inf, dtype=torch.float64, device=q.device)
    for b in range(B):
        n = Lk if lens is None else min(max(int(lens[b]), 0), Lk)
        if n == 0 or Lq == 0:
            continue
        for i in range(h):
            j = i // (h // hk)
            kk, vv = k[b, j, :n].double(), v[b, j, :n].double()
            s = scale * (q[b, i].double() @ kk.T)
            lse[b, i] = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[b, i][:, None])
            out[b, i] = p @ vv
            tol[b, i] = P_ERR * (p @ vv.abs())
    tol += (U[torch.bfloat16] + SCORE_ERR) * out.abs()
    return out, lse, tol


def cross_bwd(q, k, v, out, lse, dout, lens, scale=None):
    """-> (dq, dk, dv), and their bounds, given the forward's rounded out and lse."""
    B, h, Lq, d = q.shape
    hk, Lk = k.shape[1], k.shape[2]
    g = h // hk
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    z = lambda t: torch.zeros(t.shape, dtype=torch.float64, device=q.device)  # noqa: E731
    dq, dk, dv, tq, tk, tv = z(q), z(k), z(v), z(q), z(k), z(v)
    for b in range(B):
        n = Lk if lens is None else min(max(int(lens[b]), 0), Lk)
        if n == 0 or Lq == 0:
            continue
        for i in range(h):
            j = i // g
            qq, kk, vv = q[b, i].double(), k[b, j, :n].double(), v[b, j, :n].double()
            do, oo = dout[b, i].double(), out[b, i].double()
            p = torch.exp(scale * (qq @ kk.T) - lse[b, i].double()[:, None])
            ds = p * (do @ vv.T - (do * oo).sum(-1, keepdim=True))
            mag = do.abs() @ vv.abs().T + (do * oo).abs().sum(-1, keepdim=True)
            e = P_ERR * ds.abs() + SCORE_ERR * ds.abs() + DP_ERR * p * mag
            dq[b, i] = scale * (ds @ kk)
            tq[b, i] = scale * (e @ kk.abs())
            dk[b, j, :n] += scale * (ds.T @ qq)
            tk[b, j, :n] += scale * (e.T @ qq.abs())
            dv[b, j, :n] += p.T @ do
            tv[b, j, :n] += P_ERR * (p.T @ do.abs()) + SCORE_ERR * (p.T @ do.abs())
    ub = U[torch.bfloat16]
    return (dq, dk, dv), (tq + ub * dq.abs(), tk + ub * dk.abs(), tv + ub * dv.abs())


def rope_angles(grid, axes, theta=10000.0, start=(0, 0, 0), step=(1, 1, 1)):
    """Angles [T, H, W, R / 2] in fp64."""
    T, H, W = grid
    idx = torch.meshgrid(*(torch.arange(n, dtype=torch.float64) for n in grid), indexing="ij")
    parts = []
    for a in range(3):
        pos = start[a] + idx[a] * step[a]
        for j in range(axes[a] // 2):
            parts.append(pos * theta ** (-2.0 * j / axes[a]))
    return torch.stack(parts, -1)


def rope_table(grid, axes, **kw):
    """The table's values in fp64: angles of each axis alone."""
    parts = []
    for a in range(3):
        one, ax = [1, 1, 1], [0, 0, 0]
        one[a], ax[a] = grid[a], axes[a]
        if axes[a]:
            ang = rope_angles(one, ax, **kw).reshape(-1)
            parts.append(torch.stack((ang.cos(), ang.sin()), -1))
    return torch.cat(parts)


def rope(x, grid, axes, table, interleaved, inverse):
    """-> y and its bound (fp64), with the fp32 table's values as they are."""
    T, H, W = grid
    x = x.double().cpu()
    R = sum(axes)
    cs, at = [], 0
    for a in range(3):
        n, m = grid[a], axes[a] // 2
        shape = [1, 1, 1, m, 2]
        shape[a] = n
        cs.append(table[at:at + n * m].double().cpu().view(shape).expand(T, H, W, m, 2))
        at += n * m
    cs = torch.cat(cs, 3)
    c, s = cs[..., 0], cs[..., 1] * (-1.0 if inverse else 1.0)
    y, tol = x.clone(), torch.zeros_like(x)
    even, odd = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    p, q = x[..., even], x[..., odd]
    y[..., even], y[..., odd] = p * c - q * s, p * s + q * c
    tol[..., even] = tol[..., odd] = 2.0 ** -22 * (p.abs() + q.abs())
    return y, tol


def norm(x, r, w, eps):
    """-> y, h (fp64, unrounded)."""
    h = x.double() if r is None else x.double() + r.double()
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    return (y if w is None else y * w.double()), h


def norm_bwd(h, w, dy, dh, eps):
    """-> dx, dw, bounds of both before the outputs' rounding (fp64)."""
    h, dy = h.double(), dy.double()
    rho = 1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    g = dy if w is None else dy * w.double()
    m = (g * h).mean(-1, keepdim=True)
    dx = rho * g - rho ** 3 * h * m
    tol = NORM_ERR * (rho * g.abs() + rho ** 3 * h.abs() * (g * h).abs().mean(-1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
        tol = tol + 2.0 ** -23 * (dh.double().abs() + dx.abs())
    t = dy * h * rho
    return dx, t.reshape(-1, t.shape[-1]).sum(0), tol, 2.0 ** -17 * t.abs().reshape(-1, t.shape[-1]).sum(0)
