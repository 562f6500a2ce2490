"""Matrices of the 8-bit path with 2^31 rows or columns and more: refused by the binding, and not
handed to the library as what is left of the number in 32 bits (no GPU: stand-ins for tensors, and
for the library)."""
import pytest
import torch

import invariant_bi_rmsnorm_gb300 as bi
from invariant_bi_rmsnorm_gb300 import _lib

BF, F8, U8 = torch.bfloat16, torch.float8_e4m3fn, torch.uint8
PAST = 2 ** 32 + 32  # 32 in 32 bits


class Tensor:
    """What the binding asks of a tensor on the current device."""
    is_cuda, device = True, "cuda:0"

    def __init__(self, shape, dtype):
        self.shape, self.dtype = tuple(shape), dtype

    def stride(self, i=None):
        st = [1]
        for n in reversed(self.shape[1:]):
            st.insert(0, st[0] * n)
        return tuple(st) if i is None else st[i]

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


def mat(rows, K):
    return Tensor((rows, K), F8), Tensor(bi.fp8_scales_shape(rows, K), U8)


def of(rows, K):
    return Tensor((rows, K), BF)


CALLS = {
    "quantize_fp8": lambda M, N, K: bi.quantize_fp8(of(M, K), *mat(M, K)),
    "fp8_read": lambda M, N, K: bi.fp8_read(*mat(M, K), out=of(M, K)),
    "rmsnorm_fp8": lambda M, N, K: bi.rmsnorm_fp8(of(M, K), Tensor((K,), BF), 1e-6, *mat(M, K)),
    "add_rmsnorm_fp8": lambda M, N, K: bi.add_rmsnorm_fp8(of(M, K), of(M, K), Tensor((K,), BF), 1e-6, None, *mat(M, K)),
    "gemm_fp8": lambda M, N, K: bi.gemm_fp8(*mat(M, K), *mat(N, K), out=of(M, N)),
    "gemm_fp8_swiglu": lambda M, N, K: bi.gemm_fp8_swiglu(*mat(M, K), *mat(N, K), *mat(M, N // 2)),
}


@pytest.fixture
def made(monkeypatch):
    """The calls that reach the library."""
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append((name, a)) or 0
    lib = Lib()
    monkeypatch.setattr(_lib, "load", lambda: lib)
    monkeypatch.setattr(_lib, "fp8_calls", None)
    monkeypatch.setattr(bi, "_device", lambda: 0)
    monkeypatch.setattr(bi, "_current_device", lambda: 0)
    monkeypatch.setattr(bi, "_raw_stream", lambda device: 0)
    return calls


@pytest.mark.parametrize("name", list(CALLS))
def test_the_largest_sizes_are_handed_over(name, made):
    CALLS[name](64, 64, 2 ** 31 - 16)
    assert len(made) == 1 and 2 ** 31 - 16 in made[0][1]


@pytest.mark.parametrize("name", list(CALLS))
def test_columns_past_32_bits_are_refused(name, made):
    with pytest.raises(ValueError, match="2\\^31"):
        CALLS[name](64, 64, PAST)
    assert not made


@pytest.mark.parametrize("M,N", [(PAST, 64), (64, PAST)])
@pytest.mark.parametrize("name", ["gemm_fp8", "gemm_fp8_swiglu"])
def test_rows_past_32_bits_are_refused(name, M, N, made):
    with pytest.raises(ValueError, match="2\\^31"):
        CALLS[name](M, N, 64)
    assert not made


@pytest.mark.parametrize("name", ["quantize_fp8", "fp8_read", "rmsnorm_fp8", "add_rmsnorm_fp8"])
def test_rows_are_64_bits_to_the_library(name, made):
    """Which refuses them itself."""
    CALLS[name](PAST, 64, 64)
    assert len(made) == 1 and PAST in made[0][1]
