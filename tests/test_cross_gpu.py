"""Cross attention to an encoder's states, forward and backward, against the fp64 definition with
element-wise bounds counted from the documented roundings."""
import math

import pytest
import torch

from tests import _block_ref as ref
import video_dit_sparse_dsa_b200 as dsa

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def draw(seed, B, h, hk, Lq, Lk, token_major=False, spread=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    if token_major:
        q = (spread * rn(B, Lq, h, 128)).to(BF).permute(0, 2, 1, 3)
        kv = rn(B, Lk, 2, hk, 128).to(BF)
        k, v = kv[:, :, 0].permute(0, 2, 1, 3), kv[:, :, 1].permute(0, 2, 1, 3)
        do = rn(B, Lq, h, 128).to(BF).permute(0, 2, 1, 3)
    else:
        q, k, v = (spread * rn(B, h, Lq, 128)).to(BF), rn(B, hk, Lk, 128).to(BF), rn(B, hk, Lk, 128).to(BF)
        do = rn(B, h, Lq, 128).to(BF)
    return q, k, v, do


def lens_of(lens):
    return None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)


def ok():
    st = dsa.device_status()
    assert st[0] == 0, f"device status {st}"


def check(q, k, v, do, lens, scale=None, backward=True, what=""):
    n = lens_of(lens)
    out, lse = dsa.forward_cross(q, k, v, kv_len=n, scale=scale)
    ok()
    ro, rl, tol = ref.cross(q, k, v, lens, scale)
    ref.close(out, ro, tol, f"out {what}")
    ref.close(lse, rl, ref.LSE_TOL, f"lse {what}")
    if backward:
        grads = dsa.backward_cross(q, k, v, out, lse, do, kv_len=n, scale=scale)
        ok()
        rg, rt = ref.cross_bwd(q, k, v, out, lse, do, lens, scale)
        for name, a, b, t in zip(("dq", "dk", "dv"), grads, rg, rt):
            ref.close(a, b, t, f"{name} {what}")
    return out, lse


# more batch entries than a warp has lanes, most of them without keys, units cut between CTAs
def many_lens(B, Lk):
    return tuple((Lk, 0, 0, 1, 0, Lk // 2, 0, 130)[b % 8] if b not in (0, B - 1) else 0 for b in range(B))


@pytest.mark.parametrize("B,h,hk,Lq,Lk", [(70, 2, 1, 3, 200), (45, 1, 1, 300, 260), (200, 1, 1, 1, 140)])
def test_many_batch_entries(B, h, hk, Lq, Lk):
    q, k, v, do = draw(19, B, h, hk, Lq, Lk)
    check(q, k, v, do, many_lens(B, Lk))
    check(q, k, v, do, (0,) * B)


# (B, heads, kv_heads, Lq, Lk, lens): one key and one row, chunk and step borders of the keys
# (16, 64, 128, 256), lengths of zero, shared kv heads, several tiles per CTA
CASES = [
    (1, 1, 1, 1, 1, None),
    (1, 2, 2, 5, 2, None),
    (2, 3, 1, 130, 77, (77, 1)),
    (3, 4, 2, 64, 128, (128, 0, 127)),
    (2, 2, 2, 257, 129, (129, 128)),
    (1, 3, 3, 128, 256, None),
    (2, 2, 1, 300, 257, (257, 255)),
    (1, 2, 2, 511, 512, (383,)),
    (4, 2, 2, 100, 513, (0, 513, 400, 16)),
    (2, 8, 1, 7, 40, (40, 33)),
    (2, 6, 2, 33, 200, (200, 17)),
    (1, 5, 5, 3000, 77, None),
    (2, 7, 7, 2111, 300, (300, 130)),
    (1, 20, 4, 1500, 700, None),
]


@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(str(x) for x in c[:5]))
def test_cross(case, token_major):
    B, h, hk, Lq, Lk, lens = case
    check(*draw(Lq + Lk, B, h, hk, Lq, Lk, token_major), lens)


# few rows over many keys: the keys are cut into parts
LONG = [(1, 1, 1, 1, 5000, None), (2, 8, 2, 1, 40001, (40001, 777)), (1, 4, 4, 130, 9999, (9000,)),
        (3, 2, 1, 3, 1024, (1024, 0, 1)), (1, 24, 24, 2, 3000, None), (2, 12, 3, 17, 20000, (1, 20000))]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "x".join(str(x) for x in c[:5]))
def test_long_keys(case):
    B, h, hk, Lq, Lk, lens = case
    p = dsa.Cross(B=B, heads=h, kv_heads=hk, d=128, Lq=Lq, Lk=Lk, scale=1.0, dtype=dsa.DSA_BF16)
    assert dsa.cross_workspace_size(p) > 0  # in parts
    check(*draw(Lk, B, h, hk, Lq, Lk), lens)


@pytest.mark.parametrize("spread", [0.01, 8.0])
def test_flat_and_peaked_scores(spread):
    check(*draw(3, 2, 2, 1, 200, 500, spread=spread), (500, 260))


def test_scores_that_grow_along_the_keys():
    """The running maximum moves at every step (rescaled sums)."""
    q, k, v, do = draw(4, 1, 2, 2, 150, 1100)
    k = (k.float() * torch.linspace(0.1, 6, 1100, device=DEV)[None, None, :, None]).to(BF)
    check(q, k, v, do, None)
    check(q, k.flip(2).contiguous(), v, do, (1000,))


def test_scale():
    check(*draw(5, 1, 2, 2, 100, 90), None, scale=0.3)


@pytest.mark.parametrize("case", [(2, 3, 3, 200, 300, (130, 299)), (2, 4, 2, 70, 600, (1, 513)), (2, 4, 1, 1, 3000, (100, 2570))])
def test_padding_may_hold_anything(case):
    """NaN, infinities and the type's extremes past kv_len reach nothing."""
    B, h, hk, Lq, Lk, lens = case
    q, k, v, do = draw(6, B, h, hk, Lq, Lk)
    n = lens_of(lens)
    out, lse = dsa.forward_cross(q, k, v, kv_len=n)
    grads = dsa.backward_cross(q, k, v, out, lse, do, kv_len=n)
    for bad in (math.nan, math.inf, -math.inf, torch.finfo(BF).min, torch.finfo(BF).max):
        k2, v2 = k.clone(), v.clone()
        for b, m in enumerate(lens):
            k2[b, :, m:], v2[b, :, m:] = bad, bad
        out2, lse2 = dsa.forward_cross(q, k2, v2, kv_len=n)
        assert torch.equal(out, out2) and torch.equal(lse, lse2), bad
        for name, a, c in zip(("dq", "dk", "dv"), grads, dsa.backward_cross(q, k2, v2, out, lse, do, kv_len=n)):
            assert torch.equal(a, c), (name, bad)
    ok()
    for b, m in enumerate(lens):
        assert (grads[1][b, :, m:] == 0).all() and (grads[2][b, :, m:] == 0).all()


def test_nonfinite_rows_stay_alone():
    q, k, v, do = draw(7, 1, 2, 2, 140, 100)
    want, _ = dsa.forward_cross(q, k, v)
    q2 = q.clone()
    q2[0, 1, 130, 5] = math.nan
    out, lse = dsa.forward_cross(q2, k, v)
    assert torch.isnan(out[0, 1, 130]).all() and torch.isnan(lse[0, 1, 130])
    keep = torch.ones(140, dtype=torch.bool)
    keep[130] = False
    assert torch.equal(out[0, 0], want[0, 0]) and torch.equal(out[0, 1, keep], want[0, 1, keep])
    ok()


def test_lengths_outside_are_limited():
    q, k, v, do = draw(8, 3, 2, 2, 60, 150)
    out, lse = dsa.forward_cross(q, k, v, kv_len=lens_of((-5, 150, 2 ** 31 - 1)))
    ro, rl, tol = ref.cross(q, k, v, (0, 150, 150))
    ref.close(out, ro, tol, "out")
    ref.close(lse, rl, ref.LSE_TOL, "lse")
    ok()


@pytest.mark.parametrize("Lq,Lk", [(0, 40), (40, 0), (0, 0), (0, 5000), (1, 0)])
def test_no_rows_or_keys(Lq, Lk):
    q, k, v, do = draw(9, 2, 4, 2, Lq, Lk)
    out, lse = dsa.forward_cross(q, k, v)
    assert (out == 0).all() and (lse == -math.inf).all()
    dq, dk, dv = dsa.backward_cross(q, k, v, out, lse, do)
    assert dq.shape == q.shape and dk.shape == k.shape
    assert (dq == 0).all() and (dk == 0).all() and (dv == 0).all()
    ok()


def test_broadcast_inputs():
    """Stride-0 batch and head dimensions (one prompt for a batch, one kv head seen by all)."""
    q, k, v, do = draw(10, 1, 1, 1, 90, 200)
    qe, ke, ve = q.expand(2, 6, 90, 128), k.expand(2, 3, 200, 128), v[:, 0:1].expand(2, 3, 200, 128)
    doe = do.expand(2, 6, 90, 128)
    out, lse = dsa.forward_cross(qe, ke, ve)
    full = [t.contiguous() for t in (qe, ke, ve, doe)]
    want = dsa.forward_cross(*full[:3])
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    grads = dsa.backward_cross(qe, ke, ve, out, lse, doe)
    for a, b in zip(grads, dsa.backward_cross(*full[:3], out, lse, full[3])):
        assert torch.equal(a, b)
    ok()


@pytest.mark.parametrize("Lq,Lk", [(7, 200), (1, 1300), (64, 77)])
@pytest.mark.parametrize("which", ["q", "dout", "both"])
def test_broadcast_heads_of_a_shared_kv_head(Lq, Lk, which):
    """Few rows, whose heads are packed into one tile unless they are one head by a stride of 0."""
    q, k, v, do = draw(18, 2, 6, 2, Lq, Lk)
    if which != "dout":
        q = q[:, 2:3].expand(2, 6, Lq, 128)
    if which != "q":
        do = do[:, 1:2].expand(2, 6, Lq, 128)
    check(q, k, v, do, (Lk, Lk // 2), what=which)


def test_outputs_through_strides_leave_neighbours():
    B, h, Lq, Lk = 2, 3, 150, 200
    q, k, v, do = draw(11, B, h, h, Lq, Lk)
    lens = lens_of((200, 90))
    want, lse = dsa.forward_cross(q, k, v, kv_len=lens)
    buf = torch.full((B, Lq + 3, h, 2, 128), 5.0, dtype=BF, device=DEV)
    out = buf[:, 1:1 + Lq, :, 0].permute(0, 2, 1, 3)
    dsa.forward_cross(q, k, v, kv_len=lens, out=out)
    assert torch.equal(out, want)
    assert (buf[:, :, :, 1] == 5).all() and (buf[:, 0] == 5).all() and (buf[:, 1 + Lq:] == 5).all()
    g = dsa.backward_cross(q, k, v, want, lse, do, kv_len=lens)
    dqb = torch.full_like(buf, 5.0)
    dkvb = torch.full((B, Lk + 1, 3, h, 128), 5.0, dtype=BF, device=DEV)
    dq = dqb[:, 1:1 + Lq, :, 0].permute(0, 2, 1, 3)
    dk, dv = dkvb[:, :Lk, 0].permute(0, 2, 1, 3), dkvb[:, :Lk, 2].permute(0, 2, 1, 3)
    dsa.backward_cross(q, k, v, want, lse, do, kv_len=lens, dq=dq, dk=dk, dv=dv)
    assert torch.equal(dq, g[0]) and torch.equal(dk, g[1]) and torch.equal(dv, g[2])
    assert (dqb[:, :, :, 1] == 5).all() and (dqb[:, 0] == 5).all() and (dqb[:, 1 + Lq:] == 5).all()
    assert (dkvb[:, :, 1] == 5).all() and (dkvb[:, Lk:] == 5).all()
    ok()


def test_gradients_against_differences():
    """<grad, u> against central differences of the fp64 forward, for q, k and v."""
    q, k, v, do = draw(12, 2, 4, 2, 40, 70)
    lens = (70, 33)
    out, lse = dsa.forward_cross(q, k, v, kv_len=lens_of(lens))
    grads = dsa.backward_cross(q, k, v, out, lse, do, kv_len=lens_of(lens))
    _, tols = ref.cross_bwd(q, k, v, out, lse, do, lens)
    f = lambda *t: float((ref.cross(*t, lens)[0] * do.double()).sum())  # noqa: E731
    g = torch.Generator(device=DEV).manual_seed(1)
    e = 1e-3
    for i, (x, grad, tol) in enumerate(zip((q, k, v), grads, tols)):
        u = torch.randn(x.shape, generator=g, device=DEV, dtype=torch.float64)
        up, dn = [t.double() for t in (q, k, v)], [t.double() for t in (q, k, v)]
        up[i], dn[i] = up[i] + e * u, dn[i] - e * u
        num = (f(*up) - f(*dn)) / (2 * e)
        # the bound along u; D comes from the rounded out (2^-8 of sum |dO O| in each dS)
        _, _, to = ref.cross(q, k, v, lens)
        slack = 0.0
        if i < 2:
            p_max = float((do.double().abs() * to).sum(-1).max())
            other = (k if i == 0 else q).double().abs().max()
            slack = float(u.abs().sum()) / math.sqrt(128) * p_max * float(other) / 70
        assert abs(float((grad.double() * u).sum()) - num) <= float((tol * u.abs()).sum()) + slack + 1e-3 * abs(num) + 1e-2


def test_same_bits_graphs_and_shared_workspace():
    """Two captured graphs that share one workspace, replayed in turn on new inputs."""
    q, k, v, do = draw(13, 2, 4, 2, 5, 4000)
    n = lens_of((4000, 1234))
    p = dsa.Cross(B=2, heads=4, kv_heads=2, d=128, Lq=5, Lk=4000, scale=1 / math.sqrt(128), dtype=dsa.DSA_BF16)
    size = max(dsa.cross_workspace_size(p), dsa.cross_workspace_size(p, backward=True))
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    out, lse = dsa.forward_cross(q, k, v, kv_len=n, ws=ws)
    g1 = dsa.backward_cross(q, k, v, out, lse, do, kv_len=n, ws=ws)
    g2 = dsa.backward_cross(q, k, v, out, lse, do, kv_len=n)
    assert all(torch.equal(a, b) for a, b in zip(g1, g2))
    dq, dk, dv = (torch.empty_like(t) for t in g1)
    fwd, bwd = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(fwd):
        dsa.forward_cross(q, k, v, kv_len=n, out=out, lse=lse, ws=ws)
    with torch.cuda.graph(bwd):
        dsa.backward_cross(q, k, v, out, lse, do, kv_len=n, dq=dq, dk=dk, dv=dv, ws=ws)
    for seed, lens in ((20, (0, 4000)), (21, (3999, 7))):
        new = draw(seed, 2, 4, 2, 5, 4000)
        for a, b in zip((q, k, v, do), new):
            a.copy_(b)
        n.copy_(lens_of(lens))
        fwd.replay()
        bwd.replay()
        wo, wl = dsa.forward_cross(*new[:3], kv_len=n)
        assert torch.equal(out, wo) and torch.equal(lse, wl)
        for a, b in zip((dq, dk, dv), dsa.backward_cross(*new[:3], wo, wl, new[3], kv_len=n)):
            assert torch.equal(a, b)
    ok()


def test_two_streams_at_once():
    a, b = draw(14, 1, 4, 4, 3000, 300), draw(15, 2, 8, 2, 2, 9000)
    want = [dsa.forward_cross(*x[:3]) for x in (a, b)]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [dsa.forward_cross(*x[:3], stream=st) for x, st in zip((a, b) * 3, s * 3)]
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])
    ok()
