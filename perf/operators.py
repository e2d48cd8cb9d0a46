"""Cases, inputs and plain forms of the operators around 3D-DSA in a video transformer block.

The operators are cross attention from video tokens to an encoder's states (forward and
backward), rotary positions over (time, height, width), and the root-mean-square norm with
the residual's addition (forward in bf16 / fp32 or e4m3 with scales, and backward).  With
``own`` false every operator runs in its plain form (elementary torch operations in fp32,
rounded once); with ``own`` true through the library's public calls.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LOG_THETA = math.log(10000.0)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one denoising step's cross attention of a small latent grid to a 77-token prompt
        {"name": "cross_fwd_16x32x32_text77", "op": "cross_fwd", "B": 1, "heads": 24, "kv_heads": 24, "Lq": 16384,
         "Lk": 77, "lens": "77", "token_major": False},
        # a guidance pair (prompt and negative prompt of different lengths, padded to 512) at 480p,
        # straight from the projections (token-major rows, k and v in one buffer)
        {"name": "cross_fwd_480p_pair_text512", "op": "cross_fwd", "B": 2, "heads": 12, "kv_heads": 12, "Lq": 35840,
         "Lk": 512, "lens": "512,203", "token_major": True},
        # the largest forward: 720p latents over a full 512-token prompt
        {"name": "cross_fwd_720p_text512", "op": "cross_fwd", "B": 1, "heads": 24, "kv_heads": 24, "Lq": 115200,
         "Lk": 512, "lens": "512", "token_major": False},
        # one new token (a register or caption token) over every state of a 720p clip, shared kv heads
        {"name": "cross_fwd_one_token_720p", "op": "cross_fwd", "B": 2, "heads": 24, "kv_heads": 6, "Lq": 1,
         "Lk": 115201, "lens": "115201,70007", "token_major": False},
        # the adaptation step's cross attention backward: batch of two, padded prompts
        {"name": "cross_bwd_480p_b2_text512", "op": "cross_bwd", "B": 2, "heads": 12, "kv_heads": 12, "Lq": 35840,
         "Lk": 512, "lens": "512,203", "token_major": True},
        # odd lengths, shared kv heads: image and text states of one encoder sequence
        {"name": "cross_bwd_gqa_odd", "op": "cross_bwd", "B": 2, "heads": 16, "kv_heads": 4, "Lq": 4099, "Lk": 1337,
         "lens": "1337,1", "token_major": False},
        # one latent frame, where the launch counts
        {"name": "rope_one_frame", "op": "rope", "B": 1, "heads": 12, "d": 128, "T": 1, "H": 16, "W": 16,
         "axes": "44,42,42", "pairs": "interleaved", "dtype": "bf16", "inverse": False},
        # q and k of a 720p clip out of the fused projection into the attention's layout
        {"name": "rope_720p", "op": "rope", "B": 1, "heads": 24, "d": 128, "T": 30, "H": 48, "W": 80,
         "axes": "44,42,42", "pairs": "interleaved", "dtype": "bf16", "inverse": False},
        # its backward at 480p: gradients of q and k back into the fused projection's gradient
        {"name": "rope_bwd_480p_halves_f32", "op": "rope", "B": 2, "heads": 5, "d": 128, "T": 21, "H": 31, "W": 53,
         "axes": "16,56,56", "pairs": "halves", "dtype": "f32", "inverse": True},
        # the norm before a projection in 8 bits for a handful of conditioning rows
        {"name": "norm_fp8_few_rows", "op": "norm", "rows": 3, "C": 5120, "dtype": "bf16", "residual": True,
         "weight": True, "fp8": True},
        # the block's norm with the residual's addition over a 480p batch of two
        {"name": "norm_480p_b2_residual", "op": "norm", "rows": 71680, "C": 1536, "dtype": "bf16", "residual": True,
         "weight": True, "fp8": False},
        # its backward in the adaptation step, wide rows
        {"name": "norm_bwd_480p_wide", "op": "norm_bwd", "rows": 35840, "C": 5120, "dtype": "bf16", "residual": True,
         "weight": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    """One more case of the listed ranges: sizes spread over their logarithm, odd ones among them."""
    op = rng.choice(["cross_fwd", "cross_fwd", "cross_bwd", "rope", "norm", "norm_bwd"])
    if op in ("cross_fwd", "cross_bwd"):
        B = rng.randint(1, 3)
        kv_heads = rng.choice([1, 2, 3, 5, 8, 12])
        heads = kv_heads * rng.choice([1, 1, 2, 4])
        if op == "cross_fwd" and rng.random() < 0.35:  # few rows over a long memory
            Lq, Lk = _log_int(rng, 1, 300), _log_int(rng, 2000, 120000)
        else:
            Lq, Lk = _log_int(rng, 1, 60000), _log_int(rng, 1 if op == "cross_fwd" else 8, 1500)
        # no dearer than the largest listed one (24 heads x 115200 rows x 512 keys; backward: 480p pair)
        cap = 24 * 115200 * 512 if op == "cross_fwd" else 12 * 35840 * 715
        while B * heads * Lq * Lk > cap:
            Lq = max(1, Lq // 2)
        lens = [Lk] + [rng.choice([Lk, rng.randint(0, Lk)]) for _ in range(B - 1)]  # the padding's length is the longest
        rng.shuffle(lens)
        return {"op": op, "B": B, "heads": heads, "kv_heads": kv_heads, "Lq": Lq, "Lk": Lk,
                "lens": ",".join(str(n) for n in lens), "token_major": rng.random() < 0.5}
    if op == "rope":
        while True:
            d = rng.choice([64, 96, 128, 128, 128])
            c = {"op": op, "B": rng.randint(1, 2), "heads": rng.randint(1, 24), "d": d, "T": rng.randint(1, 31),
                 "H": rng.randint(1, 60), "W": rng.randint(1, 90),
                 "axes": {64: "16,24,24", 96: "32,32,32", 128: rng.choice(["44,42,42", "16,56,56", "32,40,40"])}[d],
                 "pairs": rng.choice(["interleaved", "halves"]), "dtype": rng.choice(["bf16", "bf16", "f32"]),
                 "inverse": rng.random() < 0.5}
            if c["B"] * c["heads"] * d * c["T"] * c["H"] * c["W"] <= 24 * 128 * 60000:
                return c
    C = rng.choice([128, 256, 1024, 1536, 2048, 5120, _log_int(rng, 1, 8192)])
    rows = _log_int(rng, 1, 80000)
    while rows * C > 120_000_000:
        rows //= 2
    c = {"op": op, "rows": rows, "C": C, "dtype": rng.choice(["bf16", "bf16", "f32"]), "residual": rng.random() < 0.6,
         "weight": rng.random() < 0.8}
    if op == "norm":
        c["fp8"] = rng.random() < 0.4
    return c


def work(case):
    op = case["op"]
    if op in ("cross_fwd", "cross_bwd"):
        lens = _lens(case)
        qrows = case["B"] * case["heads"] * case["Lq"]
        krows = case["kv_heads"] * sum(lens)
        flops = 4.0 * case["heads"] * case["Lq"] * sum(lens) * 128
        if op == "cross_fwd":  # q, out, lse; k, v
            return {"bytes": qrows * (2 * 256 + 4) + krows * 2 * 256, "flops": flops}
        # q, out, dout, lse, dq; k, v of the real keys; dk, dv of every row
        return {"bytes": qrows * (4 * 256 + 4) + krows * 2 * 256 + 2 * 256 * case["B"] * case["kv_heads"] * case["Lk"],
                "flops": 2.5 * flops}
    if op == "rope":
        n = case["B"] * case["heads"] * case["T"] * case["H"] * case["W"] * case["d"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * 2 * n * size, "flops": 2 * 3.0 * n}
    n, size = case["rows"] * case["C"], 2 if case["dtype"] == "bf16" else 4
    w = case["C"] * size if case["weight"] else 0
    if op == "norm":  # x (and the residual, and their sum), y or its 8 bits and scales
        moved = n * size * (3 if case["residual"] else 1) + w
        moved += n + case["rows"] * -(-case["C"] // 128) * 4 if case["fp8"] else n * size
        return {"bytes": moved, "flops": 5.0 * n}
    # h, dy (and the residual stream's gradient), dx; weight and its gradient
    return {"bytes": n * size * (4 if case["residual"] else 3) + 2 * w, "flops": 9.0 * n}


# ---------------------------------------------------------------- inputs
def _lens(case):
    return [int(n) for n in case["lens"].split(",")]


def _axes(case):
    return tuple(int(n) for n in case["axes"].split(","))


def _randn(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _heads_of(gen, B, heads, L, n, token_major):
    """n tensors [B, heads, L, 128]: of one token-major projection buffer, or head-major each."""
    if token_major:
        buf = _randn(gen, B, L, n, heads, 128)
        return [buf[:, :, i].permute(0, 2, 1, 3) for i in range(n)]
    return [_randn(gen, B, heads, L, 128) for _ in range(n)]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if op in ("cross_fwd", "cross_bwd"):
        B, h, hk, Lq, Lk = (case[n] for n in ("B", "heads", "kv_heads", "Lq", "Lk"))
        (st["q"],) = _heads_of(gen, B, h, Lq, 1, case["token_major"])
        st["k"], st["v"] = _heads_of(gen, B, hk, Lk, 2, case["token_major"])
        st["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=DEV)
        if op == "cross_bwd":  # what a training step keeps of its forward
            st["out"], st["lse"] = _plain_cross(st)
            (st["dout"],) = _heads_of(gen, B, h, Lq, 1, case["token_major"])
    elif op == "rope":
        B, h, d, T, H, W = (case[n] for n in ("B", "heads", "d", "T", "H", "W"))
        dt = DTYPES[case["dtype"]]
        fused = lambda buf, i: buf[:, :, i].view(B, T, H, W, h, d).permute(0, 4, 1, 2, 3, 5)  # noqa: E731
        st["table"] = _table((T, H, W), _axes(case))
        if case["inverse"]:  # gradients in the attention's layout, back into the projection's gradient
            st["q"], st["k"] = (_randn(gen, B, h, T, H, W, d, dtype=dt) for _ in range(2))
            buf = torch.zeros(B, T * H * W, 3, h, d, dtype=dt, device=DEV)
            st["q_out"], st["k_out"] = fused(buf, 0), fused(buf, 1)
        else:
            buf = _randn(gen, B, T * H * W, 3, h, d, dtype=dt)
            st["q"], st["k"] = fused(buf, 0), fused(buf, 1)
            st["q_out"] = st["k_out"] = None
    else:
        rows, C, dt = case["rows"], case["C"], DTYPES[case["dtype"]]
        st["x"] = _randn(gen, rows, C, dtype=dt)
        st["w"] = (1.0 + 0.2 * torch.randn(C, generator=gen, device=DEV)).to(dt) if case["weight"] else None
        st["res"] = _randn(gen, rows, C, dtype=dt) if case["residual"] else None  # norm_bwd: the stream's gradient
        if op == "norm_bwd":
            st["dy"] = _randn(gen, rows, C, dtype=dt)
    return st


def _table(grid, axes):
    """(cos, sin) of every axis coordinate and pair, fp32 [sum n_a d_a / 2, 2], angles in fp64."""
    parts = []
    for n, da in zip(grid, axes):
        freq = torch.exp(-LOG_THETA * torch.arange(0, da, 2, dtype=torch.float64, device=DEV) / max(da, 1))
        ang = torch.arange(n, dtype=torch.float64, device=DEV)[:, None] * freq[None]
        parts.append(torch.stack((ang.cos(), ang.sin()), -1).reshape(-1, 2))
    return torch.cat(parts).float().contiguous()


# ---------------------------------------------------------------- one pass
EPS = 1e-6


def run(st):
    case, op = st["case"], st["case"]["op"]
    if own:
        import video_dit_sparse_dsa_b200 as dsa

        if op == "cross_fwd":
            return dsa.forward_cross(st["q"], st["k"], st["v"], kv_len=st["lens"])
        if op == "cross_bwd":
            return dsa.backward_cross(st["q"], st["k"], st["v"], st["out"], st["lse"], st["dout"], kv_len=st["lens"])
        if op == "rope":
            return dsa.rope(st["q"], st["k"], st["table"], _axes(case), interleaved=case["pairs"] == "interleaved",
                            inverse=case["inverse"], q_out=st["q_out"], k_out=st["k_out"])
        if op == "norm":
            if case["fp8"]:
                y8, scales, h = dsa.rms_norm_fp8(st["x"], st["w"], eps=EPS, residual=st["res"])
                return (y8, scales, h) if case["residual"] else (y8, scales)
            y, h = dsa.rms_norm(st["x"], st["w"], eps=EPS, residual=st["res"])
            return (y, h) if case["residual"] else y
        dx, dw = dsa.rms_norm_backward(st["x"], st["w"], st["dy"], dh=st["res"], eps=EPS)
        return (dx, dw) if case["weight"] else dx
    if op == "cross_fwd":
        return _plain_cross(st)
    if op == "cross_bwd":
        return _plain_cross_bwd(st)
    if op == "rope":
        return _plain_rope(st)
    return _plain_norm(st) if op == "norm" else _plain_norm_bwd(st)


# ---------------------------------------------------------------- plain forms (fp32)
def _head_chunks(heads, group, elems):
    """Ranges of query heads of whole kv groups whose score matrices stay near 2^28 values."""
    step = max(1, (1 << 28) // max(elems * group, 1)) * group
    return [(a, min(a + step, heads)) for a in range(0, heads, step)]


def _plain_cross(st):
    q, k, v = st["q"], st["k"], st["v"]
    B, h, Lq, d = q.shape
    g = h // k.shape[1]
    out, lse = torch.zeros_like(q), torch.full((B, h, Lq), -math.inf, device=DEV)
    for b, n in enumerate(_lens(st["case"])):
        if n == 0:
            continue
        for a, e in _head_chunks(h, g, Lq * n):
            kk = k[b, a // g:e // g, :n].float().repeat_interleave(g, dim=0)
            vv = v[b, a // g:e // g, :n].float().repeat_interleave(g, dim=0)
            s = (q[b, a:e].float() @ kk.transpose(1, 2)).mul_(1.0 / math.sqrt(d))
            m = s.amax(-1, keepdim=True)
            p = s.sub_(m).exp_()
            l = p.sum(-1, keepdim=True)
            out[b, a:e] = ((p @ vv) / l).to(q.dtype)
            lse[b, a:e] = (m + l.log())[..., 0]
    return out, lse


def _plain_cross_bwd(st):
    q, k, v, out, lse, dout = (st[n] for n in ("q", "k", "v", "out", "lse", "dout"))
    B, h, Lq, d = q.shape
    hk = k.shape[1]
    g, scale = h // hk, 1.0 / math.sqrt(d)
    dq = torch.zeros_like(q)
    dk, dv = (torch.zeros(k.shape, dtype=k.dtype, device=DEV) for _ in range(2))
    for b, n in enumerate(_lens(st["case"])):
        if n == 0:
            continue
        for a, e in _head_chunks(h, g, 2 * Lq * n):
            kk = k[b, a // g:e // g, :n].float().repeat_interleave(g, dim=0)
            vv = v[b, a // g:e // g, :n].float().repeat_interleave(g, dim=0)
            qq, do = q[b, a:e].float(), dout[b, a:e].float()
            D = (do * out[b, a:e].float()).sum(-1, keepdim=True)
            p = (qq @ kk.transpose(1, 2)).mul_(scale).sub_(lse[b, a:e, :, None]).exp_()
            ds = (do @ vv.transpose(1, 2)).sub_(D).mul_(p).mul_(scale)
            dq[b, a:e] = (ds @ kk).to(q.dtype)
            fold = lambda x: x.view(-1, g, n, d).sum(1)  # noqa: E731
            dk[b, a // g:e // g, :n] = fold(ds.transpose(1, 2) @ qq).to(k.dtype)
            dv[b, a // g:e // g, :n] = fold(p.transpose(1, 2) @ do).to(k.dtype)
    return dq, dk, dv


def _token_angles(st):
    """cos and sin [T, H, W, pairs] of the grid's tokens, out of the table."""
    case, axes = st["case"], _axes(st["case"])
    grid = (case["T"], case["H"], case["W"])
    cs, at = [], 0
    for i, (n, da) in enumerate(zip(grid, axes)):
        part = st["table"][at:at + n * da // 2].view(n, da // 2, 2)
        at += n * da // 2
        shape = [1, 1, 1, da // 2, 2]
        shape[i] = n
        cs.append(part.view(shape).expand(*grid, da // 2, 2))
    cs = torch.cat(cs, dim=3)
    return cs[..., 0], cs[..., 1]


def _plain_rope(st):
    case = st["case"]
    cos, sin = _token_angles(st)
    if case["inverse"]:
        sin = -sin
    r2 = cos.shape[-1]
    outs = []
    for x, into in ((st["q"], st["q_out"]), (st["k"], st["k_out"])):
        y = torch.empty(x.shape, dtype=x.dtype, device=DEV) if into is None else into
        step = max(1, (1 << 28) // x[:, 0].numel())  # heads at a time, so that the fp32 copies stay small
        for i in range(0, x.shape[1], step):
            h = slice(i, i + step)
            f = x[:, h].float()
            if case["pairs"] == "interleaved":
                a, b = f[..., 0:2 * r2:2], f[..., 1:2 * r2:2]
                z = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
            else:
                a, b = f[..., :r2], f[..., r2:2 * r2]
                z = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
            y[:, h, ..., :2 * r2] = z.to(x.dtype)
            y[:, h, ..., 2 * r2:] = x[:, h, ..., 2 * r2:]
        outs.append(y)
    return tuple(outs)


def _plain_norm(st):
    case, w = st["case"], st["w"]
    h = st["x"].float()
    if st["res"] is not None:
        h = h + st["res"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    if w is not None:
        y = y * w.float()
    total = h.to(st["x"].dtype)
    if case["fp8"]:
        rows, C = y.shape
        n = -(-C // 128)
        pad = torch.nn.functional.pad(y, (0, 128 * n - C)).view(rows, n, 128)
        scales = pad.abs().amax(-1) / 448.0
        scales = torch.where(scales > 0, scales, torch.ones_like(scales))
        y8 = (pad / scales[..., None]).view(rows, 128 * n)[:, :C].to(torch.float8_e4m3fn)
        return (y8, scales, total) if st["res"] is not None else (y8, scales)
    y = y.to(st["x"].dtype)
    return (y, total) if st["res"] is not None else y


def _plain_norm_bwd(st):
    h, dy, w, dh = st["x"].float(), st["dy"].float(), st["w"], st["res"]
    rstd = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    g = dy if w is None else dy * w.float()
    dx = rstd * (g - h * (rstd * rstd * (g * h).mean(-1, keepdim=True)))
    if dh is not None:
        dx = dx + dh.float()
    dx = dx.to(st["x"].dtype)
    if w is None:
        return dx
    return dx, (dy * (h * rstd)).sum(0).to(w.dtype)


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The outputs of ``run`` from the definitions in fp64 (for the 8-bit values: the quotients that they round)."""
    st = prepare(case, seed)
    f8 = torch.float64
    op = case["op"]
    if op in ("cross_fwd", "cross_bwd"):
        q, k, v = st["q"], st["k"], st["v"]
        B, h, Lq, d = q.shape
        hk, scale = k.shape[1], 1.0 / math.sqrt(d)
        o = torch.zeros(B, h, Lq, d, dtype=f8, device=DEV)
        lse = torch.full((B, h, Lq), -math.inf, dtype=f8, device=DEV)
        dk, dv = (torch.zeros(k.shape, dtype=f8, device=DEV) for _ in range(2))
        for b, n in enumerate(_lens(case)):
            if n == 0:
                continue
            for i in range(h):
                j = i * hk // h
                kj, vj = k[b, j, :n].to(f8), v[b, j, :n].to(f8)
                for r in range(0, Lq, 32768):  # bounded score blocks
                    qi = q[b, i, r:r + 32768].to(f8)
                    s = torch.einsum("nc,mc->nm", qi, kj) * scale
                    if op == "cross_fwd":
                        z = torch.logsumexp(s, dim=1)
                        o[b, i, r:r + 32768] = torch.einsum("nm,mc->nc", torch.exp(s - z[:, None]), vj)
                        lse[b, i, r:r + 32768] = z
                        continue
                    do, oi = (st[x][b, i, r:r + 32768].to(f8) for x in ("dout", "out"))
                    p = torch.exp(s - st["lse"][b, i, r:r + 32768].to(f8)[:, None])
                    ds = p * (torch.einsum("nc,mc->nm", do, vj) - torch.einsum("nc,nc->n", do, oi)[:, None])
                    o[b, i, r:r + 32768] = scale * torch.einsum("nm,mc->nc", ds, kj)
                    dk[b, j, :n] += scale * torch.einsum("nm,nc->mc", ds, qi)
                    dv[b, j, :n] += torch.einsum("nm,nc->mc", p, do)
        return (o, lse) if op == "cross_fwd" else (o, dk, dv)
    if op == "rope":
        T, H, W, d = (case[n] for n in ("T", "H", "W", "d"))
        # the rotation as a complex product, with the table's cos and sin as they are
        z, at = [], 0
        tab = torch.complex(st["table"][:, 0].to(f8), st["table"][:, 1].to(f8))
        idx = torch.meshgrid(*(torch.arange(n, device=DEV) for n in (T, H, W)), indexing="ij")
        for i, (n, da) in enumerate(zip((T, H, W), _axes(case))):
            z.append(tab[at:at + n * da // 2].view(n, da // 2)[idx[i]])
            at += n * da // 2
        z = torch.cat(z, dim=-1)
        if case["inverse"]:
            z = z.conj()
        r2 = z.shape[-1]
        outs = []
        for x in (st["q"], st["k"]):
            y = x.to(f8).contiguous()
            rot = y[..., :2 * r2]
            if case["pairs"] == "interleaved":
                c = torch.view_as_complex(rot.reshape(*rot.shape[:-1], r2, 2)) * z
                y[..., :2 * r2] = torch.view_as_real(c).flatten(-2)
            else:
                c = torch.complex(rot[..., :r2].contiguous(), rot[..., r2:].contiguous()) * z
                y[..., :2 * r2] = torch.cat((c.real, c.imag), dim=-1)
            outs.append(y)
        return tuple(outs)
    x, w, res = st["x"].to(f8), st["w"], st["res"]
    C = x.shape[1]
    if op == "norm":
        h = x if res is None else x + res.to(f8)
        y = h / torch.sqrt(torch.einsum("rc,rc->r", h, h) / C + EPS)[:, None]
        y = y if w is None else y * w.to(f8)
        if case["fp8"]:
            s = torch.stack([part.abs().amax(1) / 448.0 for part in y.split(128, dim=1)], dim=1)
            s = s.masked_fill(s == 0, 1.0)
            y = torch.cat([part / s[:, i:i + 1] for i, part in enumerate(y.split(128, dim=1))], dim=1)
            return (y, s) if res is None else (y, s, h)
        return y if res is None else (y, h)
    dy = st["dy"].to(f8)
    ms = torch.einsum("rc,rc->r", x, x) / C + EPS
    gw = dy if w is None else dy * w.to(f8)
    dx = gw / ms.sqrt()[:, None] - x * (torch.einsum("rc,rc->r", gw, x) / C / ms ** 1.5)[:, None]
    dx = dx if res is None else dx + res.to(f8)
    return dx if w is None else (dx, torch.einsum("rc,rc->c", dy, x / ms.sqrt()[:, None]))
