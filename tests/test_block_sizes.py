"""Sizes past the C structures' 32 bits are refused, not taken modulo 2^32 (CPU: shapes alone)."""
import pytest
import torch

import video_dit_sparse_dsa_b200 as dsa
from video_dit_sparse_dsa_b200 import build as dsa_build

BF = torch.bfloat16
BIG = 2 ** 32  # + a size that would be valid by itself


@pytest.fixture(scope="module", autouse=True)
def lib():
    dsa_build.build()


def meta(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype, device="meta")


def refused(f, *args, **kw):
    with pytest.raises(dsa.DsaError) as e:
        f(*args, **kw)
    assert e.value.status == 2


def test_what_ctypes_does():
    assert dsa.Norm(4, BIG + 256, 1e-6, dsa.DSA_BF16).C == 256


@pytest.mark.parametrize("q,k", [
    ((1, 2, BIG + 5, 128), (1, 2, 7, 128)), ((1, 2, 5, 128), (1, 2, BIG + 7, 128)), ((1, 2, 5, BIG + 128), (1, 2, 7, BIG + 128)),
    ((BIG + 1, 2, 5, 128), (BIG + 1, 2, 7, 128)), ((1, BIG + 2, 5, 128), (1, 2, 7, 128)), ((1, 2, 5, 128), (1, BIG + 2, 7, 128)),
])
def test_cross(q, k):
    q, k = meta(*q), meta(*k)
    refused(dsa.forward_cross, q, k, k)
    refused(dsa.backward_cross, q, k, k, q, meta(*q.shape[:3], dtype=torch.float32), q)


@pytest.mark.parametrize("axis", range(6))
def test_rope(axis):
    shape = [1, 2, 3, 4, 5, 64]
    shape[axis] += BIG
    x = meta(*shape)
    n = shape[2] * 8 + shape[3] * 12 + shape[4] * 12
    refused(dsa.rope, x, None, meta(n, 2, dtype=torch.float32), (16, 24, 24))


@pytest.mark.parametrize("grid,axes", [((BIG + 2, 3, 4), (16, 24, 24)), ((2, 3, 4), (16, BIG + 24, 24))])
def test_rope_table(grid, axes):
    refused(dsa.rope_table, grid, axes)


def test_norm():
    x = meta(4, BIG + 256)
    refused(dsa.rms_norm, x)
    refused(dsa.rms_norm, x, residual=x)
    refused(dsa.rms_norm_fp8, x)
    refused(dsa.rms_norm_backward, x, None, x)
