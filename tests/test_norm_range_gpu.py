"""The norm's backward over fp32's range of rows."""
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
