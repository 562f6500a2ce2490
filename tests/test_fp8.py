"""The 8-bit matrix format and the refusals of its entry points, without a GPU.

The oracle's quantiser is pinned by exact rational arithmetic; the library's entry
points are called with arguments that they have to refuse before any launch (pointers
are never dereferenced)."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from invariant_bi_rmsnorm_gb300 import _lib
from oracle import fp8

FAKE = 0x10000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return _lib.load()


def test_codes_are_the_format_s_numbers():
    v = fp8.code_values()
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(v), np.isnan(t)) and np.array_equal(v[~np.isnan(v)], t[~np.isnan(t)])
    assert np.nanmax(v) == 448 and sorted(set(np.abs(v[~np.isnan(v)])))[1] == 2.0 ** -9


def test_rounding_against_rationals():
    """Every pair of neighbouring codes: their middle goes to the even one, and what lies
    a little off it to the nearer."""
    pos = sorted(v for v in fp8.code_values() if v >= 0 and not np.isnan(v))
    pos = sorted(set(pos))
    for i, (a, b) in enumerate(zip(pos, pos[1:])):
        mid = (Fraction(a) + Fraction(b)) / 2
        even = a if i % 2 == 0 else b  # codes ascend with the values
        eps = (Fraction(b) - Fraction(a)) / 1024
        for x, want in ((mid, even), (mid - eps, a), (mid + eps, b)):
            assert Fraction(float(x)) == x
            for sign in (1, -1):
                assert fp8.round_e4m3(sign * float(x)) == sign * want


@pytest.mark.parametrize("e", [-133, -126, -119, -40, 0, 7, 100, 126, 127])
def test_scales_at_the_borders(e):
    """max|x| = 1.75 * 2^e fits 448 scales exactly; the next bf16 number up takes the next
    scale; the least scale is 2^-119."""
    for mant in (1.0, 1.5, 1.75, 1.7578125, 1.9921875):
        x = np.zeros((1, 128))
        x[0, 77] = -(mant * 2.0 ** e)
        b = int(fp8.scale_bytes(x)[0, 0])
        top = Fraction(mant) * Fraction(2) ** e
        assert b >= 8 and top <= 448 * Fraction(2) ** (b - 127)
        assert b == 8 or top > 448 * Fraction(2) ** (b - 128)
        q, _ = fp8.quantise(x)
        assert abs(q[0, 77]) <= 448 and (np.delete(q[0], 77) == 0).all()


def test_error_bound_and_special_blocks():
    g = np.random.default_rng(3)
    x = g.standard_normal((40, 400)) * np.exp2(g.integers(-20, 20, (40, 400)))
    x[5, 130], x[6, 399], x[7, 0] = np.nan, np.inf, -np.inf
    x[8, :128] = 0
    h, b = fp8.held(x), fp8.scale_bytes(x)
    assert b.shape == (40, 4)
    bad = np.zeros((40, 400), bool)
    bad[5, 128:256] = bad[6, 384:] = bad[7, :128] = True
    assert np.array_equal(np.isnan(h), bad)
    s = np.repeat(np.ldexp(1.0, b - 127), 128, axis=1)[:, :400]
    with np.errstate(invalid="ignore"):
        assert (np.abs(h - x) <= np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10))[~bad].all()
    assert b[8, 0] == 8 and (h[8, :128] == 0).all()


@pytest.mark.parametrize("rows,K", [(1, 16), (128, 512), (129, 528), (300, 1040)])
def test_tiles_hold_every_scale_once(lib, rows, K):
    spans = -(-K // 512)
    at = [fp8.place(r, c, spans) for r in range(rows) for c in range(-(-K // 128))]
    size = -(-rows // 128) * spans * 512
    assert len(set(at)) == len(at) and 0 <= min(at) and max(at) < size
    assert lib.bi_fp8_scales_size(rows, K) == size
    import invariant_bi_rmsnorm_gb300 as bi
    shape = bi.fp8_scales_shape(rows, K)
    assert shape[0] * shape[1] * shape[2] == size and shape[2] == _lib.FP8_TILE_BYTES


def test_scales_size_of_invalid_matrices(lib):
    for rows, K in ((-1, 16), (4, 0), (4, 8), (4, 24), (2 ** 31, 16)):
        assert lib.bi_fp8_scales_size(rows, K) == 0
    assert lib.bi_fp8_scales_size(0, 16) == 0


I, U, A = _lib.BI_ERR_INVALID_ARG, _lib.BI_ERR_UNSUPPORTED_SHAPE, _lib.BI_ERR_MISALIGNED


def _refuses(call, ok, cases):
    for want, change in cases:
        assert call(**{**ok, **change}) == want, change


def test_quantise_and_read_refusals(lib):
    ok = dict(x=FAKE, ld_x=64, rows=4, K=64, q=FAKE, ld_q=64, s=FAKE)
    bad = [(U, dict(K=8)), (U, dict(K=24, ld_x=64)), (U, dict(K=0)), (I, dict(rows=-1)), (I, dict(rows=2 ** 31)),
           (I, dict(ld_x=56)), (I, dict(ld_q=48)), (A, dict(ld_x=68)), (A, dict(ld_q=72)), (I, dict(x=None)),
           (I, dict(q=None)), (I, dict(s=None)), (A, dict(x=FAKE + 8)), (A, dict(q=FAKE + 8)), (A, dict(s=FAKE + 4)),
           (_lib.BI_OK, dict(rows=0, x=None, q=None, s=None))]
    _refuses(lambda x, ld_x, rows, K, q, ld_q, s: lib.bi_quantize_fp8(x, ld_x, rows, K, q, ld_q, s, None), ok, bad)
    _refuses(lambda x, ld_x, rows, K, q, ld_q, s: lib.bi_fp8_read(q, ld_q, s, rows, K, x, ld_x, None), ok, bad)


def test_norm_refusals(lib):
    ok = dict(x=FAKE, r=FAKE, ro=FAKE, w=FAKE, q=FAKE, s=FAKE, rows=4, H=64, ld_x=64, ld_r=64, ld_ro=64, ld_q=64, eps=1e-6)
    plain = [(U, dict(H=8)), (U, dict(H=24)), (U, dict(H=32784, ld_x=32784, ld_q=32784, ld_r=32784, ld_ro=32784)),
             (I, dict(rows=-1)), (I, dict(ld_x=56)), (I, dict(ld_q=48)), (A, dict(ld_x=68)), (A, dict(ld_q=72)),
             (I, dict(eps=-1.0)), (I, dict(eps=float("nan"))), (I, dict(x=None)), (I, dict(w=None)), (I, dict(q=None)),
             (I, dict(s=None)), (A, dict(x=FAKE + 2)), (A, dict(w=FAKE + 8)), (A, dict(q=FAKE + 8)), (A, dict(s=FAKE + 8)),
             (_lib.BI_OK, dict(rows=0, x=None, w=None, q=None, s=None))]
    _refuses(lambda x, r, ro, w, q, s, rows, H, ld_x, ld_r, ld_ro, ld_q, eps:
             lib.bi_rmsnorm_fp8(x, w, q, s, rows, H, ld_x, ld_q, eps, None), ok, plain)
    add = plain + [(I, dict(ld_r=56)), (I, dict(ld_ro=56)), (A, dict(ld_r=68)), (A, dict(ld_ro=68)), (I, dict(r=None)),
                   (I, dict(ro=None)), (A, dict(r=FAKE + 8)), (A, dict(ro=FAKE + 8))]
    _refuses(lambda x, r, ro, w, q, s, rows, H, ld_x, ld_r, ld_ro, ld_q, eps:
             lib.bi_add_rmsnorm_fp8(x, r, ro, w, q, s, rows, H, ld_x, ld_r, ld_ro, ld_q, eps, None), ok, add)


def test_gemm_refusals(lib):
    ok = dict(x=FAKE, xs=FAKE, W=FAKE, Ws=FAKE, y=FAKE, ys=FAKE, M=4, N=64, K=64, ld_x=64, ld_w=64, ld_y=64)
    both = [(I, dict(M=-1)), (U, dict(M=2 ** 31 - 1)), (U, dict(K=8)), (U, dict(K=72, ld_x=80, ld_w=80)),
            (I, dict(ld_x=48)), (I, dict(ld_w=48)), (I, dict(ld_y=48)), (A, dict(ld_x=72)), (A, dict(ld_w=72)),
            (I, dict(x=None)), (I, dict(xs=None)), (I, dict(W=None)), (I, dict(Ws=None)), (I, dict(y=None)),
            (A, dict(x=FAKE + 8)), (A, dict(xs=FAKE + 8)), (A, dict(W=FAKE + 8)), (A, dict(Ws=FAKE + 8)), (A, dict(y=FAKE + 8)),
            (_lib.BI_OK, dict(M=0, x=None, xs=None, W=None, Ws=None, y=None, ys=None))]
    _refuses(lambda x, xs, W, Ws, y, ys, M, N, K, ld_x, ld_w, ld_y:
             lib.bi_gemm_fp8(x, xs, W, Ws, y, M, N, K, ld_x, ld_w, ld_y, None), ok,
             both + [(U, dict(N=4)), (U, dict(N=12)), (A, dict(ld_y=68))])
    _refuses(lambda x, xs, W, Ws, y, ys, M, N, K, ld_x, ld_w, ld_y:  # N stands for F
             lib.bi_gemm_fp8_swiglu(x, xs, W, Ws, y, ys, M, N, K, ld_x, ld_w, ld_y, None), ok,
             both + [(U, dict(N=8)), (U, dict(N=24)), (U, dict(N=2 ** 30)), (A, dict(ld_y=72)), (I, dict(ys=None)), (A, dict(ys=FAKE + 8))])


def test_binding_refusals_on_the_cpu():
    """No CPU path: tensors of the right types and shapes are refused for where they are."""
    import invariant_bi_rmsnorm_gb300 as bi
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    q, s = x.to(torch.float8_e4m3fn), torch.zeros(bi.fp8_scales_shape(3, 64), dtype=torch.uint8)
    w = torch.ones(64, dtype=torch.bfloat16)
    for call in (lambda: bi.quantize_fp8(x), lambda: bi.fp8_read(q, s), lambda: bi.rmsnorm_fp8(x, w),
                 lambda: bi.add_rmsnorm_fp8(x, x, w), lambda: bi.gemm_fp8(q, s, q, s),
                 lambda: bi.gemm_fp8_swiglu(q, s, torch.zeros(32, 64).to(torch.float8_e4m3fn), s)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="2-D"):
        bi.quantize_fp8(x[0])
    with pytest.raises(ValueError, match="multiple of 16"):
        bi.gemm_fp8_swiglu(q, s, torch.zeros(48, 64).to(torch.float8_e4m3fn), s)
