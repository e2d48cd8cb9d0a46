"""The operators around the attention on another stream than the current one: what they allocate is
never memory that work queued on the current stream still uses."""
import os
import subprocess
import sys

import pytest
import torch

import video_dit_sparse_dsa_b200 as dsa

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
SLEEP = 300_000_000  # clocks, some 150 ms: the host queues everything else meanwhile


def rn(seed, *shape, dtype=BF):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(dtype)


def cross_args():
    q, k, v = rn(1, 2, 4, 5, 128), rn(2, 2, 2, 9000, 128), rn(3, 2, 2, 9000, 128)  # (keys in parts)
    p = dsa.Cross(B=2, heads=4, kv_heads=2, d=128, Lq=5, Lk=9000, scale=1.0, dtype=dsa.DSA_BF16)
    return q, k, v, rn(4, 2, 4, 5, 128), dsa.cross_workspace_size(p), dsa.cross_workspace_size(p, backward=True)


def _forward_cross():
    q, k, v, _, n, _ = cross_args()
    return lambda s: dsa.forward_cross(q, k, v, stream=s), n


def _backward_cross():
    q, k, v, do, _, n = cross_args()
    out, lse = dsa.forward_cross(q, k, v)
    return lambda s: dsa.backward_cross(q, k, v, out, lse, do, stream=s), n


def _rope_table():
    return lambda s: (dsa.rope_table((400, 500, 600), (44, 42, 42), stream=s),), 0


def _rope():
    q, k = rn(5, 1, 4, 4, 16, 16, 128), rn(6, 1, 4, 4, 16, 16, 128)
    t = dsa.rope_table((4, 16, 16), (44, 42, 42))
    return lambda s: dsa.rope(q, k, t, (44, 42, 42), stream=s), 0


def _rms_norm():
    x, r, w = rn(7, 3000, 520), rn(8, 3000, 520), rn(9, 520)
    return lambda s: dsa.rms_norm(x, w, residual=r, stream=s), 0


def _rms_norm_fp8():
    x, r, w = rn(7, 3000, 520), rn(8, 3000, 520), rn(9, 520)

    def call(s):
        y, scales, h = dsa.rms_norm_fp8(x, w, residual=r, stream=s)
        return y.view(torch.uint8), scales, h

    return call, 0


def _rms_norm_backward():
    x, dy, w = rn(7, 3000, 520), rn(8, 3000, 520), rn(9, 520)
    n = dsa.load_library().dsa_rmsnorm_bwd_workspace_size(dsa.Norm(3000, 520, 1e-6, dsa.DSA_BF16))
    return lambda s: dsa.rms_norm_backward(x, w, dy, stream=s), n


OPS = [_forward_cross, _backward_cross, _rope_table, _rope, _rms_norm, _rms_norm_fp8, _rms_norm_backward]


@pytest.mark.parametrize("queued", ["reads", "writes"])
@pytest.mark.parametrize("op", OPS, ids=lambda f: f.__name__[1:])
def test_memory_in_use_on_the_current_stream(op, queued):
    """Temporaries of the sizes that the call allocates, freed with their last use still queued: the
    call neither overwrites them before it nor is overwritten by it."""
    call, n_scratch = op()
    want = [t.clone() for t in call(None)]
    sizes = [t.numel() * t.element_size() for t in want] + ([n_scratch] if n_scratch else [])
    for other in (torch.cuda.Stream(), torch.cuda.default_stream()):
        current = torch.cuda.Stream()
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        with torch.cuda.stream(current):
            temps = [torch.full((n,), 5, dtype=torch.uint8, device=DEV) for n in sizes]
            kept = [torch.zeros_like(t) for t in temps]
            torch.cuda.synchronize()
            torch.cuda._sleep(SLEEP)
            for t, k in zip(temps, kept):
                k.copy_(t) if queued == "reads" else t.fill_(77)
            del temps, t
            got = call(other)
            assert not current.query(), "the current stream has run already: nothing was tested"
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        if queued == "reads":
            assert all(bool((k == 5).all()) for k in kept)
        del got
    assert dsa.device_status()[0] == 0


@pytest.mark.parametrize("op", OPS, ids=lambda f: f.__name__[1:])
def test_results_dropped_with_reads_queued(op):
    """Results of a call on another stream, dropped while the current one still has to read them:
    the next call there does not take their memory."""
    call, _ = op()
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    kept = [torch.zeros_like(t) for t in got]
    torch.cuda._sleep(SLEEP)
    for t, k in zip(got, kept):
        k.copy_(t)
    ptrs = {t.data_ptr() for t in got}
    del got, t
    again = call(side)
    assert ptrs.isdisjoint(t.data_ptr() for t in again)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want))


@pytest.mark.parametrize("op", OPS, ids=lambda f: f.__name__[1:])
def test_captured_on_a_given_stream(op):
    """Capture on a stream that is passed while it is the current one, and while it is not."""
    call, _ = op()
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = call(side.cuda_stream)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_refused_stream_leaves_the_device():
    x = rn(1, 4, 256)
    with pytest.raises((TypeError, ValueError)):
        dsa.rms_norm(x, stream="no stream")
    assert torch.cuda.current_device() == 0 and dsa.rms_norm(x)[0].shape == x.shape


@pytest.mark.parametrize("device", ["cuda", "cuda:0"])
def test_a_table_is_a_process_first_call(device):
    code = ("import video_dit_sparse_dsa_b200 as dsa; "
            f"t = dsa.rope_table((2, 3, 4), (4, 4, 4), device='{device}'); "
            "assert t.shape == (18, 2) and float(t[0, 0]) == 1.0")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root, timeout=300)
