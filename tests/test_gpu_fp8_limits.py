"""The block-scaled FP8 operators at the limits of their kernels: shapes, strides, special
codes and scale bytes that test_gpu_fp8.py gives to some kernels, given to all of them. Bounds
as that file derives them, unless a test states its own."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from group_wise_bit_amd import binding as gwb      # must load: no fallback where a GPU is present
else:  # collected on CPU only to be skipped
    gwb = None

from test_gpu_fp8 import _check_gemm


@pytest.mark.parametrize("scale", ["f32", "e8m0"])
@pytest.mark.parametrize("M,N,K", [(65600, 200, 144), (131000, 250, 144)])
def test_gemm_more_tile_rows_than_units(M, N, K, scale):
    """One column of 256 x 256 tiles with more rows of them than compute units: no columns are
    left to split off."""
    _check_gemm(M, N, K, scale, (torch.bfloat16, torch.float16))
