"""The block-scaled FP8 operators at the limits of their kernels: shapes, strides, special
codes and scale bytes that test_gpu_fp8.py gives to some kernels, given to all of them. Bounds
as that file derives them, unless a test states its own."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.fp8 as o8
from _fp8_shapes import LONG, SHAPES

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from group_wise_bit_amd import binding as gwb      # must load: no fallback where a GPU is present
else:  # collected on CPU only to be skipped
    gwb = None

from test_gpu_fp8 import _check_gemm

DEV = "cuda"
U = 2.0 ** -24
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _quantized(v, rows, scale):
    return gwb.fp8_quantize(v, rows, scale)


def _operands(M, N, K, scale, seed, outlier=1.0):
    """Normal activations, 1 % of the channels `outlier` times larger; weights of unequal rows."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(M, K, generator=g, device=DEV)
    x *= torch.where(torch.rand(K, generator=g, device=DEV) < 0.01, outlier, 1.0)
    w = torch.randn(N, K, generator=g, device=DEV) * 0.015 * torch.exp(torch.randn(N, 1, generator=g, device=DEV) * 0.5)
    return _quantized(x, 1, scale), _quantized(w, 128, scale)


def _values64(q):
    """The exact values that codes and scales stand for."""
    R, K = q.codes.shape
    s = q.scales.double()
    s = s.t() if q.block_rows == 1 else s.repeat_interleave(128, 0)[:R]
    return q.codes.double() * s.repeat_interleave(128, 1)[:, :K]


def _byte_scales(b, scale):
    """E8M0 bytes as scales of either type (float32: byte 0 is 2^-127, 255 NaN)."""
    if scale == "e8m0":
        return b.to(torch.uint8).view(E8M0)
    s = torch.exp2(b.double() - 127).float()
    return torch.where(b == 255, torch.nan, s)


def _sorted(d):
    return [pytest.param(*v, id=k) for k, v in d.items()]


@pytest.mark.parametrize("scale", ["f32", "e8m0"])
@pytest.mark.parametrize("M,N,K", [(65600, 200, 144), (131000, 250, 144)])
def test_gemm_more_tile_rows_than_units(M, N, K, scale):
    """One column of 256 x 256 tiles with more rows of them than compute units: no columns are
    left to split off."""
    _check_gemm(M, N, K, scale, (torch.bfloat16, torch.float16))


# ------------------------------------------------------------------ surroundings
@pytest.mark.parametrize("scale", ["f32", "e8m0"])
@pytest.mark.parametrize("M,N,K", _sorted(SHAPES))
def test_gemm_strides_and_surroundings(M, N, K, scale):
    """Strided codes and scales with NaN all around them, and y strided, offset or unaligned: the
    results are those of the packed operands, bit for bit, and nothing beside y is written."""
    x, w = _operands(M, N, K, scale, 3 * M + N)

    def surround(q):
        R, Kq = q.codes.shape
        cb = torch.full((R + 2, Kq + 48), 0x7F, dtype=torch.uint8, device=DEV)
        cb[1:R + 1, 16:16 + Kq] = q.codes.view(torch.uint8)
        sr, sc = q.scales.shape
        raw = q.scales.view(torch.uint8) if scale == "e8m0" else q.scales
        sb = torch.full((sr + 2, sc + 3), 255 if scale == "e8m0" else float("nan"), dtype=raw.dtype, device=DEV)
        sb[1:sr + 1, 1:sc + 1] = raw
        sb = sb.view(E8M0) if scale == "e8m0" else sb
        return gwb.Fp8(cb[1:R + 1, 16:16 + Kq].view(E4M3), sb[1:sr + 1, 1:sc + 1], q.block_rows)

    xs, ws = surround(x), surround(w)
    for dt in DTYPES:
        want = gwb.fp8_gemm(x, w, dt)
        assert bool(torch.isfinite(want).all())
        for pad, off in ((0, 0), (4, 4), (3, 1)):
            buf = torch.full((M * (N + pad) + off + 8,), 9.0, dtype=dt, device=DEV)
            y = torch.as_strided(buf, (M, N), (N + pad, 1), off)
            gwb.fp8_gemm(xs, ws, out=y)
            assert torch.equal(y, want), (dt, pad, off)
            y.fill_(9.0)
            assert bool((buf == 9.0).all()), (dt, pad, off)
