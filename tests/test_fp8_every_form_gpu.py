"""Every kernel of the 8-bit products, each with several parts of K, against another one's bits and
against the oracle; and the pairs' kernel where a pair has several tiles of several parts, every row of it.

x and W are normal numbers whose blocks lie up to 2^+-6 apart, so that the order of the sums shows."""
import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_gb300 as bi
from tests._util import bits
from tests.test_fp8_form_names import FORMS, SWIGLU_FORMS
from tests.test_fp8_gpu import check_gemm, quantised

pytestmark = pytest.mark.gpu


def numbers(rows, K, seed, by):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(rows, K, generator=g, device="cuda")
    scale = torch.exp2(torch.randint(-by, by + 1, (rows, -(-K // 128)), generator=g, device="cuda").float())
    return (x * scale.repeat_interleave(128, 1)[:, :K]).to(torch.bfloat16)


def weight(N, K, swiglu):
    return bi.quantize_fp8(numbers(N, K, N + K, 1) * 0.02 if swiglu else numbers(N, K, N + K, 6))


def run(x, W, swiglu):
    """One call over bf16 rows x: its output's bits, for SwiGLU of codes and what they stand for."""
    q = bi.quantize_fp8(x.contiguous())
    if not swiglu:
        return bits(bi.gemm_fp8(*q, *W))
    h, s = bi.gemm_fp8_swiglu(*q, *W)
    return np.concatenate([h.view(torch.uint8).cpu().numpy().astype(np.uint16), bits(bi.fp8_read(h, s))], 1)


def check_oracle(x, W):
    """Rows of every tile of 128, about 60 columns."""
    M, N = x.shape[0], W[0].shape[0]
    y = bi.gemm_fp8(*bi.quantize_fp8(x), *W)
    rows = torch.tensor(sorted({r for t in range(0, M, 128) for r in (t, t + 31, t + 33, t + 95, t + 96, t + 127) if r < M} | {M - 1}))
    cols = torch.tensor(sorted(set(range(0, N, max(1, N // 61))) | {N - 1})).cuda()
    rows = rows.cuda()
    check_gemm(y[rows][:, cols], bi.quantize_fp8(x[rows].contiguous()), bi.quantize_fp8(bi.fp8_read(*W)[cols].contiguous()))


CASES = [(f, False, *s) for f, s in FORMS.items()] + [(f, True, *s) for f, s in SWIGLU_FORMS.items()]


@pytest.mark.parametrize("form,swiglu,M,N,K", CASES)
def test_every_form_against_another(form, swiglu, M, N, K):
    assert bi.gemm_fp8_form(M, N, K, swiglu) == form
    W = weight(N, K, swiglu)
    if form < 2000000:  # the pairs' kernel: its rows on few-row kernels, 32 at a time
        x = numbers(M, K, M, 2 if swiglu else 6)
        full = run(x, W, swiglu)
        for a in range(0, M, 32):
            assert bi.gemm_fp8_form(min(32, M - a), N, K, swiglu) >= 2000000
            assert np.array_equal(run(x[a:a + 32], W, swiglu), full[a:a + 32]), a
    else:
        R = next(R for R in (300, 600, 1200, 2500, 5000) if R > M and bi.gemm_fp8_form(R, N, K, swiglu) < 2000000)
        x = numbers(R, K, M, 2 if swiglu else 6)
        assert np.array_equal(run(x[:M], W, swiglu), run(x, W, swiglu)[:M])
        x = x[:M]
    if not swiglu:
        check_oracle(x, W)
    bi.get_device_error()


# several tiles a pair, their K in 3, 5 and 6 parts: accumulators in turn over tiles, and for SwiGLU
# the exchange of maxima in its two buffers
@pytest.mark.parametrize("form,swiglu,M,N,K", [(1128007, False, 1000, 6152, 4112), (1128007, False, 1000, 6152, 8208),
                                               (1256005, False, 600, 14344, 4112), (1256005, False, 900, 14344, 2064),
                                               (1256006, True, 600, 24608, 2064), (1256006, True, 900, 14368, 8208)])
def test_every_row_of_several_waves_of_several_parts(form, swiglu, M, N, K):
    assert bi.gemm_fp8_form(M, N, K, swiglu) == form
    tiles = -(-M // 256) * -(-N // (form // 1000 % 1000))
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    assert tiles > 2 * pairs
    x, W = numbers(M, K, M, 2 if swiglu else 6), weight(N, K, swiglu)
    full = run(x, W, swiglu)
    for a in range(0, M, 32):
        assert np.array_equal(run(x[a:a + 32], W, swiglu), full[a:a + 32]), a
    assert np.array_equal(run(x, W, swiglu), full)
    if not swiglu:
        check_oracle(x, W)
    bi.get_device_error()


def test_both_ctas_rows_past_2_to_the_31_bytes():
    """Tiles of either CTA of a pair, even and odd ones of 128 rows, from the first to the last."""
    rows, K = 540_000, 4096
    x = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(9))
    W = quantised(24, K, 11)
    y = bi.gemm_fp8(*bi.quantize_fp8(x), *W)
    for tile in (1, 2, 3, 2047, 2048, 2049, 4095, 4096, 4097, 4216, 4217, 4218):
        a, b = 128 * tile, min(128 * tile + 128, rows)
        assert np.array_equal(bits(y[a:b]), bits(bi.gemm_fp8(*bi.quantize_fp8(x[a:b]), *W))), tile
    bi.get_device_error()
