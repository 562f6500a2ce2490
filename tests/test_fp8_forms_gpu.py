"""The 8-bit GEMM's forms at their borders, and calls that other tests do not make.

Which kernel a call runs on follows M, N and K; each of these sizes reaches another form or
lies at the border of one, and every row has to have the bits that a large batch gives it.
Operands are whole codes with scales over 2^+-8, so nothing but the order of the sums matters.
"""
import subprocess
import sys

import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_gb300 as bi
from invariant_bi_rmsnorm_gb300 import inputs
from tests._util import bits
from tests.test_fp8_gpu import check_gemm, random_matrix, rows_of

pytestmark = pytest.mark.gpu


# N: one CTA pair's tile of 128 and of 256 columns, about the pairs of a wave (76 x 128 and
# x 256), and where each CTA takes 256 rows of W; K: one, two, three and eight parts
@pytest.mark.parametrize("N,K", [(128, 1024), (256, 1040), (9728, 272), (9736, 272), (19456, 144), (19464, 144),
                                 (38912, 48), (38920, 48), (2048, 2064), (2304, 3088), (520, 8208)])
def test_rows_of_every_form(N, K):
    x, W = random_matrix(1100, K, N + 1, spread=8), random_matrix(N, K, N + 2, spread=8)
    full = bits(bi.gemm_fp8(*x, *W))
    for M in (1, 16, 17, 32, 33, 64, 65, 128, 129, 192, 193, 256, 257, 512, 513, 1024):
        assert np.array_equal(bits(bi.gemm_fp8(*rows_of(x, M), *W)), full[:M]), f"M = {M}"
    some = torch.arange(0, N, max(1, N // 97), device="cuda")
    check_gemm(bi.gemm_fp8(*rows_of(x, 40), *W)[:, some], rows_of(x, 40),
               bi.quantize_fp8(bi.fp8_read(*W)[some].contiguous()))
    bi.get_device_error()


@pytest.mark.parametrize("F,K", [(128, 1040), (4864, 144), (9728, 144), (9744, 144), (19472, 48), (1024, 3088), (2048, 4112)])
def test_swiglu_rows_of_every_form(F, K):
    x = random_matrix(600, K, F + 1, spread=2)
    W = bi.quantize_fp8(bi.interleave_gate_up(inputs.gemm_weight(2 * F, K, seed=F).cuda()))
    h, s = bi.gemm_fp8_swiglu(*x, *W)
    full = bi.fp8_read(h, s)
    assert torch.isfinite(full).all()
    for M in (1, 16, 17, 32, 33, 64, 65, 128, 129, 256, 257):
        a, b = bi.gemm_fp8_swiglu(*rows_of(x, M), *W)
        assert torch.equal(a.view(torch.uint8), h[:M].view(torch.uint8)), f"M = {M}"
        assert torch.equal(bi.fp8_read(a, b), full[:M]), f"M = {M}"
    bi.get_device_error()


@pytest.mark.parametrize("M", [1, 20, 100, 300, 1500])
def test_gemm_where_one_block_outweighs_the_rest(M):
    """The first block 2^30 times the others, and its products cancel in pairs to zero: what is
    left is the others' sum, which an accumulator that kept fewer than 24 bits of the largest
    term on its way, or an order that mixed blocks, would lose.  Whole numbers, so exact."""
    g = torch.Generator().manual_seed(M)
    K, N = 1152, 136
    a = torch.randint(-2, 3, (M, K), generator=g).float()
    b = torch.randint(-2, 3, (N, K), generator=g).float()
    a[:, :128] = torch.randint(1, 4, (M, 64), generator=g).float().repeat_interleave(2, 1) * 2.0 ** 20
    b[:, 0:128:2] = torch.randint(1, 4, (N, 64), generator=g).float()
    b[:, 1:128:2] = -b[:, 0:128:2]
    y = bi.gemm_fp8(*bi.quantize_fp8(a.to(torch.bfloat16).cuda()), *bi.quantize_fp8(b.to(torch.bfloat16).cuda()))
    assert torch.equal(y.cpu(), (a.double() @ b.double().T).to(torch.bfloat16))


FIRST_CALLS_CAPTURED = """
import torch, invariant_bi_rmsnorm_gb300 as bi
x = torch.ones(300, 528, dtype=torch.bfloat16, device="cuda")
w = torch.ones(528, dtype=torch.bfloat16, device="cuda")
bi.get_device_error()
for M in (2, 20, 50, 100, 300):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):  # nothing of this shape has run before
        n = bi.rmsnorm_fp8(x[:M], w)
        W = bi.quantize_fp8(torch.ones(64, 528, dtype=torch.bfloat16, device="cuda"))
        y = bi.gemm_fp8(*n, *W)
        h = bi.gemm_fp8_swiglu(*n, *W)
        z = bi.fp8_read(*h)
    g.replay()
    torch.cuda.synchronize()
    # g = u = 528, h = 528^2 = 278784 = 272.25 * 2^10, past the middle of 256 and 288
    assert (y == 528).all() and (z == 288 * 2.0 ** 10).all(), (M, y, z)
bi.get_device_error()
print("captured")
"""


def test_first_calls_inside_a_capture():
    """In a process of its own, where no kernel of the path has been loaded."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS_CAPTURED], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_the_same_matrix_on_both_sides_and_rows_given_twice():
    """x and W the same tensors (a Gram matrix, symmetric bit for bit where M and N are in one
    tile's reach), and a weight whose rows repeat."""
    x = random_matrix(200, 528, 3, spread=3)
    y = bi.gemm_fp8(*x, *x)
    check_gemm(y, x, x)
    assert torch.equal(y, y.t())
    W = bi.quantize_fp8(bi.fp8_read(*random_matrix(8, 528, 4, spread=3)).repeat(17, 1))
    y = bi.gemm_fp8(*x, *W)
    assert torch.equal(y.view(200, 17, 8), y[:, :8].unsqueeze(1).expand(-1, 17, -1))
    bi.get_device_error()


# where few rows take 128 W rows a CTA, 256, or every part in one CTA: by how many clusters of 4 and 8
# parts the SMs hold, which the buffers for the rows change
@pytest.mark.parametrize("N,K", [(14344, 4096), (16384, 4112), (24584, 2064), (2056, 8208), (8200, 8192), (10248, 8208)])
def test_few_rows_of_wide_weights(N, K):
    x, W = random_matrix(300, K, N + 3, spread=8), random_matrix(N, K, N + 4, spread=8)
    full = bits(bi.gemm_fp8(*x, *W))
    for M in (1, 2, 5, 8, 15, 16, 17, 24, 32, 33, 64):
        assert np.array_equal(bits(bi.gemm_fp8(*rows_of(x, M), *W)), full[:M]), f"M = {M}"
    some = torch.arange(0, N, max(1, N // 61), device="cuda")
    check_gemm(bi.gemm_fp8(*rows_of(x, 7), *W)[:, some], rows_of(x, 7),
               bi.quantize_fp8(bi.fp8_read(*W)[some].contiguous()))
    bi.get_device_error()


@pytest.mark.parametrize("F,K", [(2064, 8208), (4112, 8192), (7184, 4112), (12304, 2064)])
def test_few_rows_of_wide_gate_up_weights(F, K):
    x = random_matrix(300, K, F + 3, spread=2)
    W = bi.quantize_fp8(bi.interleave_gate_up(inputs.gemm_weight(2 * F, K, seed=F).cuda()))
    h, s = bi.gemm_fp8_swiglu(*x, *W)
    full = bi.fp8_read(h, s)
    for M in (1, 4, 5, 8, 16, 17, 32, 33, 48, 64, 65):
        a, b = bi.gemm_fp8_swiglu(*rows_of(x, M), *W)
        assert torch.equal(a.view(torch.uint8), h[:M].view(torch.uint8)), f"M = {M}"
        assert torch.equal(bi.fp8_read(a, b), full[:M]), f"M = {M}"
    bi.get_device_error()


FIRST_CALL_OF_SEVERAL_PARTS_CAPTURED = """
import torch, invariant_bi_rmsnorm_gb300 as bi
x = torch.ones(3, 4096, dtype=torch.bfloat16, device="cuda")
q, s = torch.zeros(3, 4096, dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros(bi.fp8_scales_shape(3, 4096), dtype=torch.uint8, device="cuda")
W, Ws = torch.zeros(136, 4096, dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros(bi.fp8_scales_shape(136, 4096), dtype=torch.uint8, device="cuda")
y = torch.zeros(3, 136, dtype=torch.bfloat16, device="cuda")
w = torch.ones(136, 4096, dtype=torch.bfloat16, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    bi.quantize_fp8(x, out=q, scales=s)
    bi.quantize_fp8(w, out=W, scales=Ws)
    bi.gemm_fp8(q, s, W, Ws, out=y)
g.replay()
torch.cuda.synchronize()
assert (y == 4096).all(), y
print("captured")
"""


def test_first_call_of_several_parts_inside_a_capture():
    """It asks the device how many clusters it holds."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_OF_SEVERAL_PARTS_CAPTURED], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
