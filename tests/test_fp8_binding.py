"""What the Python binding of the FP8 operators refuses before it calls the library, on
stand-ins for GPU tensors: no GPU is touched, and a call that reached the library would fail."""
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
