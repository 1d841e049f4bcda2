"""What the Python binding of the FP8 operators refuses before it calls the library, on
stand-ins for GPU tensors: no GPU is touched, and a call that reached the library would fail."""
import ctypes

import pytest
import torch

gwb = pytest.importorskip("group_wise_bit_amd.binding", reason="libgwb.so not built")


class Tensor:
    """The part of a tensor that the binding looks at."""

    def __init__(self, shape, dtype=torch.bfloat16, dev=0, contiguous=True):
        self.shape, self.dtype, self.dev, self.contiguous = torch.Size(shape), dtype, dev, contiguous
        self.is_cuda, self.device = dev >= 0, torch.device("cuda", dev) if dev >= 0 else torch.device("cpu")

    def get_device(self):
        return self.dev

    def stride(self, d=None):
        s = [1]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        return tuple(s) if d is None else s[d]

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return self.contiguous

    def dim(self):
        return len(self.shape)


def fp8(R, K, rows=1, dev=0, sdev=None):
    kb = -(-K // 128)
    return gwb.Fp8(Tensor((R, K), torch.float8_e4m3fn, dev),
                   Tensor((kb, R) if rows == 1 else (-(-R // 128), kb), torch.float32, dev if sdev is None else sdev), rows)


class Lib:
    """The library, of which only the size queries may be called."""

    def __init__(self, real):
        self.real = real

    def __getattr__(self, name):
        if name.endswith("_workspace"):
            return getattr(self.real, name)

        def call(*args):
            raise AssertionError(f"{name} reached")
        return call


@pytest.fixture(autouse=True)
def no_gpu(monkeypatch):
    monkeypatch.setattr(gwb, "lib", Lib(gwb.lib))
    monkeypatch.setattr(gwb, "_device", lambda: 0)
    monkeypatch.setattr(gwb, "_stream", lambda: 0)


M, N, K = 64, 5120, 17408                   # splits K


def product(workspace, prepare):
    x, w, y = fp8(M, K), fp8(N, K, 128), Tensor((M, N))
    if prepare:
        return gwb.prepare_fp8_gemm(x, w, y, workspace)
    return gwb.fp8_gemm(x, w, out=y, workspace=workspace)


@pytest.mark.parametrize("prepare", [False, True])
@pytest.mark.parametrize("make", [lambda n: Tensor((n,), torch.uint8, dev=-1), lambda n: Tensor((n,), torch.uint8, dev=1),
                                  lambda n: Tensor((n,), torch.uint8, contiguous=False)],
                         ids=["cpu", "other device", "not contiguous"])
def test_gemm_workspace_is_device_memory(make, prepare):
    need = gwb.fp8_gemm_workspace_bytes(M, N, K)
    assert need > 0
    with pytest.raises(ValueError):
        product(make(need), prepare)


def test_gemm_workspace_is_counted_in_bytes():
    need = gwb.fp8_gemm_workspace_bytes(M, N, K)
    for dt in (torch.uint8, torch.float32, torch.float64):
        ws = Tensor((need // dt.itemsize,), dt)
        _, _, args = gwb._fp8_gemm_args(fp8(M, K), fp8(N, K, 128), None, Tensor((M, N)), ws)
        assert args[8] == ws.data_ptr() and args[9] == need


CALLS = {
    "quantize": lambda d: gwb.fp8_quantize(Tensor((8, 256), dev=d), out=fp8(8, 256, dev=d)),
    "prepare_quantize": lambda d: gwb.prepare_fp8_quantize(Tensor((8, 256), dev=d), fp8(8, 256, dev=d)),
    "rmsnorm": lambda d: gwb.rmsnorm_fp8(Tensor((8, 256), dev=d), out=fp8(8, 256, dev=d)),
    "prepare_rmsnorm": lambda d: gwb.prepare_rmsnorm_fp8(Tensor((8, 256), dev=d), None, 1e-6, None, fp8(8, 256, dev=d), None),
    "silu_mul": lambda d: gwb.silu_mul_fp8(Tensor((8, 512), dev=d), out=fp8(8, 256, dev=d)),
    "prepare_silu_mul": lambda d: gwb.prepare_silu_mul_fp8(Tensor((8, 512), dev=d), fp8(8, 256, dev=d)),
    "gemm": lambda d: gwb.fp8_gemm(fp8(8, 256, dev=d), fp8(16, 256, 128, dev=d), out=Tensor((8, 16), dev=d)),
    "prepare_gemm": lambda d: gwb.prepare_fp8_gemm(fp8(8, 256, dev=d), fp8(16, 256, 128, dev=d), Tensor((8, 16), dev=d)),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_tensors_of_another_device_are_refused(name):
    """Calls run on the current device and its stream: tensors of another one would be read
    there, in no order with what wrote them."""
    with pytest.raises(ValueError, match="current"):
        CALLS[name](1)
    if name.startswith("prepare"):
        CALLS[name](0)                                    # the same on the current device is accepted
    else:
        with pytest.raises(AssertionError, match="reached"):
            CALLS[name](0)


@pytest.mark.parametrize("M,N,K", [(64, 5120, 17408), (128, 5120, 5120), (40, 259, 2064)])
def test_a_product_that_splits_k_refuses_a_small_workspace(M, N, K):
    """In the library itself: these shapes do split, so the refusals are reached."""
    real, fake = gwb.lib.real, 1 << 20
    need = gwb.fp8_gemm_workspace_bytes(M, N, K)
    assert need > 0 and need % (4 * M * N) == 0
    x = gwb.Fp8Tensors(fake, fake, K, M, 1, 0)
    w = gwb.Fp8Tensors(fake, fake, K, -(-K // 128), 128, 0)

    def go(ws, nbytes):
        return real.gwb_fp8_gemm(ctypes.byref(x), M, ctypes.byref(w), N, K, fake, gwb.BF16, N, ws, nbytes, None)
    assert go(fake, need - 1) == gwb.E_SIZE
    assert go(None, need) == gwb.E_SIZE
    assert go(fake + 8, need) == gwb.E_UNSUPPORTED
