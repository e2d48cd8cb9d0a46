"""The norm's backward over fp32's range of rows, and the 8-bit values' quotients."""
import pytest
import torch

from tests import _block_ref as ref
import video_dit_sparse_dsa_b200 as dsa

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("eps", [0.0, 1e-30])
@pytest.mark.parametrize("C", [7, 128, 1000, 5120, 16384])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_backward_of_small_and_large_rows(dtype, C, eps):
    """Rows of magnitude 1e-17 to 1e17 (their squares stay in range, rho^3 does not); a bound of the
    gradient is relative to it, so it holds at every magnitude."""
    g = torch.Generator().manual_seed(C)
    mag = torch.tensor([10.0 ** e for e in range(-17, 18)])[:, None]
    rows = mag.shape[0]
    h = (mag * torch.randn(rows, C, generator=g)).to(dtype)
    dy, w = torch.randn(rows, C, generator=g).to(dtype), (1 + 0.3 * torch.randn(C, generator=g)).to(dtype)
    rx, rw, tx, tw = ref.norm_bwd(h, w, dy, None, eps)
    assert torch.isfinite(rx).all() and float(rx.abs().max()) < 3e38
    dx, dw = dsa.rms_norm_backward(*(t.to(DEV) for t in (h, w, dy)), eps=eps)
    u = ref.U[dtype]
    # (a gradient near the type's least normal value, 2^-126, loses what its roundings leave below it)
    ref.close(dx, rx, tx + u * rx.abs() + 2.0 ** -126, "dx")
    ref.close(dw, rw, tw + u * rw.abs(), "dw")
    assert dsa.device_status()[0] == 0


@pytest.mark.parametrize("rows,C", [(4096, 5120), (8192, 1536), (200000, 128), (3000, 1537)])
def test_fp8_values_are_rounded_quotients(rows, C):
    """y8 = rn(y / s) bit for bit, with y as the fp32 norm gives it (the same sums) and s as returned."""
    x = torch.randn(rows, C, generator=torch.Generator(device=DEV).manual_seed(C), device=DEV)
    y, _ = dsa.rms_norm(x)
    y8, s, _ = dsa.rms_norm_fp8(x)
    y, s = y.cpu(), s.cpu()
    n = s.shape[1]
    amax = torch.nn.functional.pad(y.abs(), (0, n * 128 - C)).view(rows, n, 128).amax(-1)
    assert torch.equal(s, amax / 448)
    want = (y / s.repeat_interleave(128, 1)[:, :C]).to(torch.float8_e4m3fn)
    assert torch.equal(y8.cpu().view(torch.uint8), want.view(torch.uint8))


def test_fp8_of_an_infinite_channel():
    """A group with an infinite value: a scale of infinity, 0 for the finite ones, NaN for itself."""
    x = torch.randn(3, 256, generator=torch.Generator().manual_seed(1))
    w = torch.ones(256)
    w[5] = float("inf")
    y8, s, _ = dsa.rms_norm_fp8(x.to(DEV), w.to(DEV))
    y8, s = y8.float().cpu(), s.cpu()
    assert torch.isinf(s[:, 0]).all() and torch.isnan(y8[:, 5]).all()
    rest = [c for c in range(128) if c != 5]
    assert (y8[:, rest] == 0).all() and torch.isfinite(y8[:, 128:]).all()
