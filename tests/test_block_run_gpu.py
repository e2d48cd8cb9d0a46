"""A transformer block's attention half as a user runs it: norm with the residual, q and k norms and
rotary positions on the fused projection's views, 3D-DSA, cross attention to a padded batch of
prompts, norm, and the way back, each stage against its definition given that stage's own inputs."""
import numpy as np
import pytest
import torch

import oracle
import video_dit_sparse_dsa_b200 as dsa
from dsa_inputs import Workload, make_inputs
from tests import _block_ref as ref

pytestmark = pytest.mark.gpu
BF, EPS = torch.bfloat16, 1e-6
W = Workload("block", 2, 2, 128, (4, 16, 16), (2, 8, 8), (3, 3, 3), (-1, 1), "bf16", 5)
AXES, LK, LENS = (44, 42, 42), 77, (77, 20)


class Block:
    """Weights and inputs of one block; C = heads * 128 channels, N tokens."""

    def __init__(self, dev, seed):
        g = torch.Generator().manual_seed(seed)
        B, h, N = W.B, W.heads, W.n_tokens
        C = h * 128
        rn = lambda *s: torch.randn(*s, generator=g).to(BF).to(dev)  # noqa: E731
        self.x, self.r = rn(B, N, C), rn(B, N, C)
        self.w1, self.wq, self.wk, self.w2 = rn(C), rn(C), rn(C), (0.05 * rn(C).float()).to(BF)
        self.w_qkv, self.w_cross = (rn(C, 3 * C).float() / C ** 0.5).to(BF), (rn(C, C).float() / C ** 0.5).to(BF)
        self.text = rn(B, LK, 2, h, 128)
        self.lens = torch.tensor(LENS, dtype=torch.int32, device=dev)
        self.dy = rn(B, N, C)
        self.offsets = make_inputs(W).offsets.to(dev)
        self.table = dsa.rope_table(W.grid, AXES, device=dev)

    def heads_view(self, t):  # [B, N, C] (any row stride) -> [B, heads, N, 128]
        return t.unflatten(2, (W.heads, 128)).permute(0, 2, 1, 3)

    def run(self):
        """-> every stage's tensors by name."""
        s = {}
        B, h, N, C = W.B, W.heads, W.n_tokens, W.heads * 128
        s["y1"], s["h1"] = dsa.rms_norm(self.x, self.w1, EPS, residual=self.r)
        s["qkv"] = s["y1"] @ self.w_qkv
        q, k, v = s["qkv"].split(C, 2)
        s["qn"], _ = dsa.rms_norm(q, self.wq, EPS)
        s["kn"], _ = dsa.rms_norm(k, self.wk, EPS)
        grid = lambda t: self.heads_view(t).unflatten(2, tuple(W.grid))  # noqa: E731
        s["q"], s["k"] = dsa.rope(grid(s["qn"]), grid(s["kn"]), self.table, AXES)
        s["v"] = grid(v).contiguous()
        s["o"], s["lse"] = dsa.forward(s["q"], s["k"], s["v"], self.offsets, W.tile, W.window, W.scale)
        s["tokens"] = s["o"].flatten(2, 4).permute(0, 2, 1, 3).reshape(B, N, C)
        s["y2"], s["h2"] = dsa.rms_norm(s["tokens"], self.w2, EPS)
        s["cq"] = s["y2"] @ self.w_cross
        kv = self.text.permute(2, 0, 3, 1, 4)
        s["ck"], s["cv"] = kv[0], kv[1]
        s["co"], s["clse"] = dsa.forward_cross(self.heads_view(s["cq"]), kv[0], kv[1], self.lens)
        # back
        do = self.heads_view(self.dy)
        s["dcq"], s["dck"], s["dcv"] = dsa.backward_cross(self.heads_view(s["cq"]), kv[0], kv[1], s["co"], s["clse"], do,
                                                          self.lens)
        s["dy2"] = s["dcq"].permute(0, 2, 1, 3).reshape(B, N, C) @ self.w_cross.T
        s["dtokens"], s["dw2"] = dsa.rms_norm_backward(s["h2"], self.w2, s["dy2"], None, EPS)
        s["do"] = grid(s["dtokens"]).contiguous()
        s["dq"], s["dk"], s["dv"] = dsa.backward(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], self.offsets, W.tile,
                                                 W.window, W.scale)
        # the gradients of the q and k norms' rows, token-major again
        s["dqn"], s["dkn"] = (torch.empty_like(s["qn"]) for _ in range(2))
        dsa.rope(s["dq"], s["dk"], self.table, AXES, inverse=True, q_out=grid(s["dqn"]), k_out=grid(s["dkn"]))
        s["dqp"], s["dwq"] = dsa.rms_norm_backward(q, self.wq, s["dqn"], None, EPS)
        return s


def ok():
    st = dsa.device_status()
    assert st[0] == 0, f"device status {st}"


def test_block_stage_by_stage():
    b = Block("cuda", 31)
    s = b.run()
    ok()
    u = ref.U[BF]

    def norm(y, x, r, w, what, h=None):
        ry, rh = ref.norm(x, r, w, EPS)
        ref.close(y, ry, (u + ref.NORM_ERR) * ry.abs(), what)
        if h is not None:
            ref.close(h, rh, (u + 2.0 ** -24) * rh.abs(), what + " sum")

    def norm_bwd(dx, dw, h, w, dy, what):
        rx, rw, tx, tw = ref.norm_bwd(h, w, dy, None, EPS)
        ref.close(dx, rx, tx + u * rx.abs(), what + " dx")
        ref.close(dw, rw, tw + u * rw.abs(), what + " dw")

    C = W.heads * 128
    q, k, _ = s["qkv"].split(C, 2)
    norm(s["y1"], b.x, b.r, b.w1, "norm 1", s["h1"])
    norm(s["qn"], q, None, b.wq, "q norm")
    norm(s["kn"], k, None, b.wk, "k norm")
    norm(s["y2"], s["tokens"], None, b.w2, "norm 2")
    grid = lambda t: b.heads_view(t).unflatten(2, tuple(W.grid))  # noqa: E731
    for name, x, y, inverse in (("q", s["qn"], s["q"], False), ("k", s["kn"], s["k"], False)):
        want, tol = ref.rope(grid(x), W.grid, AXES, b.table, True, inverse)
        ref.close(y, want, tol + u * want.abs(), "rope " + name)
    for name, x, y in (("dq", s["dq"], s["dqn"]), ("dk", s["dk"], s["dkn"])):
        want, tol = ref.rope(x, W.grid, AXES, b.table, True, True)
        ref.close(grid(y), want, tol + u * want.abs(), "rope back " + name)
    geo = oracle.Geometry.of(W)
    cpu = {n: s[n].cpu() for n in ("q", "k", "v", "do")}
    o, lse = oracle.forward(geo, cpu["q"], cpu["k"], cpu["v"], b.offsets.cpu())
    assert float(np.abs(s["o"].float().cpu().numpy() - o).max()) <= 2e-2
    assert float(np.abs(s["lse"].cpu().numpy() - lse).max()) <= 2e-2
    for name, want in zip(("dq", "dk", "dv"), oracle.backward(geo, cpu["q"], cpu["k"], cpu["v"], cpu["do"], b.offsets.cpu())):
        assert float(np.abs(s[name].float().cpu().numpy() - want).max()) <= 2e-2, name
    cq = b.heads_view(s["cq"])
    ro, rl, tol = ref.cross(cq, s["ck"], s["cv"], LENS)
    ref.close(s["co"], ro, tol, "cross out")
    ref.close(s["clse"], rl, ref.LSE_TOL, "cross lse")
    rg, rt = ref.cross_bwd(cq, s["ck"], s["cv"], s["co"], s["clse"], b.heads_view(b.dy), LENS)
    for name, want, tol in zip(("dcq", "dck", "dcv"), rg, rt):
        ref.close(s[name], want, tol, name)
    norm_bwd(s["dtokens"], s["dw2"], s["h2"], b.w2, s["dy2"], "norm 2")
    norm_bwd(s["dqp"], s["dwq"], q, b.wq, s["dqn"], "q norm")


def test_block_graph_replays_with_new_inputs():
    b, other = Block("cuda", 32), Block("cuda", 33)
    want = [{n: t.clone() for n, t in x.run().items()} for x in (b, other)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        b.run()  # (the matrix library's workspace)
        with torch.cuda.graph(graph, stream=side):
            s = b.run()
    for x, expect in ((b, want[0]), (other, want[1])):
        with torch.cuda.stream(side):
            for n in ("x", "r", "w1", "wq", "wk", "w2", "w_qkv", "w_cross", "text", "dy"):
                getattr(b, n).copy_(getattr(x, n))
            graph.replay()
        torch.cuda.synchronize()
        ok()
        for n, t in expect.items():
            if n not in ("ck", "cv"):
                assert torch.equal(s[n], t), n


def test_offsets_past_32_bits():
    """Rows 2^24 elements apart in one buffer of 2.5e9 elements: the last rows lie past 2^31."""
    L, step = 150, 1 << 24
    buf = torch.zeros((L - 1) * step + 4096, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(34)
    at = iter(range(0, 4096, 128))

    def view(fill=True):
        t = buf.as_strided((1, 1, L, 128), (128, 128, step, 1), next(at))
        if fill:
            t.copy_(torch.randn(1, 1, L, 128, generator=g, device="cuda"))
        return t

    q, k, v, do = (view() for _ in range(4))
    out, dq, dk, dv = (view(False) for _ in range(4))
    _, lse = dsa.forward_cross(q, k, v, out=out)
    dsa.backward_cross(q, k, v, out, lse, do, dq=dq, dk=dk, dv=dv)
    ok()
    ro, rl, tol = ref.cross(q, k, v, None)
    ref.close(out, ro, tol, "out")
    ref.close(lse, rl, ref.LSE_TOL, "lse")
    rg, rt = ref.cross_bwd(q, k, v, out, lse, do, None)
    for name, a, want, t in zip(("dq", "dk", "dv"), (dq, dk, dv), rg, rt):
        ref.close(a, want, t, name)
    grid = (6, 5, 5)
    table = dsa.rope_table(grid, AXES, device="cuda")
    y = view(False)
    as_grid = lambda t: t.as_strided((1, 1, *grid, 128), (128, 128, 25 * step, 5 * step, step, 1), t.storage_offset())  # noqa: E731
    dsa.rope(as_grid(q), None, table, AXES, q_out=as_grid(y))
    ok()
    want, tol = ref.rope(as_grid(q), grid, AXES, table, True, False)
    ref.close(as_grid(y), want, tol + ref.U[BF] * want.abs(), "rope")
    x = q[0, 0]
    y, _ = dsa.rms_norm(x, None, EPS)
    dx, _ = dsa.rms_norm_backward(x, None, do[0, 0], None, EPS)
    ok()
    ry, _ = ref.norm(x, None, None, EPS)
    ref.close(y, ry, (ref.U[BF] + ref.NORM_ERR) * ry.abs(), "norm")
    rx, _, tx, _ = ref.norm_bwd(x, None, do[0, 0], None, EPS)
    ref.close(dx, rx, tx + ref.U[BF] * rx.abs(), "norm dx")
