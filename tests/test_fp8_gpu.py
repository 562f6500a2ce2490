"""The 8-bit linear path on the GPU, against the fp64 oracle of its format (oracle/fp8.py),
and the same bits whatever the batch.

Bounds, from the arithmetic:
  quantiser, read-back   none: bytes and bf16 values are exact.
  norms    the fp32 value in front of the one rounding is off by at most EPS_NORM of itself
           (a sum of up to 128 squares a thread, 13 more additions, half of that by the root;
           rsqrtf 2 ulp; two products), so what is held lies between what would be held of
           the exact value times 1 -+ EPS_NORM.
  GEMM     2^-8 |y| for the bf16 output, and K 2^-22 of the sum of magnitudes: each of the K
           exact products and K / 32 partial sums is kept to 2^-22 of that sum or better.
  SwiGLU   where g and u are exact in fp32, as the norms with EPS_SILU (exponential 2^-22 and
           the rounding of g log2 e, 2^-24 |g| 1.45; reciprocal, two products); elsewhere the
           GEMM's bounds on g and u carried through silu(g) u besides.
"""
import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_gb300 as bi
from invariant_bi_rmsnorm_gb300 import inputs
from oracle import fp8
from tests._util import bits

pytestmark = pytest.mark.gpu

EPS_NORM, EPS_SILU = 2.0 ** -17, 2.0 ** -18


def host(q, s):
    """Codes and scale tiles on the host."""
    return q.view(torch.uint8).cpu().numpy(), s.cpu().numpy()


def held_bounds(x, eps):
    """What 8 bits may hold of |x| (1 -+ eps): (least, most) magnitudes."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    lo, hi = np.full(a.shape, np.inf), np.zeros(a.shape)
    for bs in (fp8.scale_bytes(a * (1 - eps)), fp8.scale_bytes(a * (1 + eps))):
        s = np.repeat(np.ldexp(1.0, bs - 127), 128, axis=1)[:, :a.shape[1]]
        for f in (1 - eps, 1 + eps):
            v = fp8.round_e4m3(np.minimum(a * f / s, 448.0)) * s
            lo, hi = np.minimum(lo, v), np.maximum(hi, v)
    return lo, hi


def check_held(q, s, x, eps):
    got = fp8.read(*host(q, s))
    lo, hi = held_bounds(x, eps)
    assert ((lo <= np.abs(got)) & (np.abs(got) <= hi)).all()
    assert (np.sign(got) * np.sign(x) >= 0).all()


def random_matrix(rows, K, seed, spread=6):
    """An 8-bit matrix of any codes but NaN and scales over 2^(+-spread), with the bytes of its
    tiles that stand for nothing set to NaN."""
    g = np.random.default_rng(seed)
    codes = g.integers(0, 256, (rows, K)).astype(np.uint8)
    codes[(codes & 127) == 127] = 0
    tiles = np.full(bi.fp8_scales_shape(rows, K), 255, np.uint8)
    spans = tiles.shape[1]
    flat = tiles.reshape(-1)
    r, c = np.meshgrid(np.arange(rows), np.arange(-(-K // 128)), indexing="ij")
    at = ((r // 128) * spans + c // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + c % 4
    flat[at] = 127 + g.integers(-spread, spread + 1, at.shape)
    return (torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn), torch.from_numpy(tiles).cuda())


def quantised(rows, K, seed, std=1.0):
    return bi.quantize_fp8(inputs.normal_bf16((rows, K), seed, std=std).cuda())


def check_gemm(y, x, W):
    a, b = fp8.read(*host(*x)), fp8.read(*host(*W))
    ref, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    err = np.abs(y.cpu().double().numpy() - ref)
    bound = 2.0 ** -8 * np.abs(ref) + a.shape[1] * 2.0 ** -22 * mag
    assert (err <= bound).all(), f"{(err > bound).sum()} beyond the bound, first at {np.argwhere(err > bound)[0]}"


# ------------------------------------------------------ quantiser, read-back ----
@pytest.mark.parametrize("rows,K", [(1, 16), (3, 128), (33, 144), (129, 528), (257, 1040), (5, 4096), (40, 12288)])
def test_quantiser_bytes(rows, K):
    g = np.random.default_rng(rows * K)
    x = g.standard_normal((rows, K)) * np.exp2(g.integers(-12, 12, (rows, K)))
    x = torch.from_numpy(x).to(torch.bfloat16)
    q, s = bi.quantize_fp8(x.cuda())
    want, b = fp8.quantise(x.double().numpy())
    codes, tiles = host(q, s)
    assert np.array_equal(fp8.code_values()[codes], want)
    assert np.array_equal(fp8.read_scales(tiles, rows, K), b)
    assert np.array_equal(bi.fp8_read(q, s).cpu().double().numpy(), fp8.held(x.double().numpy()))
    bi.get_device_error()


def test_quantiser_on_every_bf16_number():
    """Every finite bf16 value as its block's largest, beside the halves of it that fall on
    ties, zeros of both signs and the smallest numbers; infinities and NaN in one block."""
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    every = every[torch.isfinite(every)]
    x = torch.zeros(len(every), 144, dtype=torch.bfloat16)
    x[:, 0] = every
    x[:, 1:20] = (every.double()[:, None] * torch.linspace(-1, 1, 19).double()).to(torch.bfloat16)
    x[:, 20], x[:, 21], x[:, 22] = -0.0, 2.0 ** -133, -2.0 ** -126
    x[:, 128] = every.flip(0)
    q, s = bi.quantize_fp8(x.cuda())
    want, b = fp8.quantise(x.double().numpy())
    codes, tiles = host(q, s)
    spans, r = 1, np.arange(len(every))
    got_b = np.stack([tiles.reshape(-1)[(r // 128) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + c] for c in range(2)], 1)
    assert np.array_equal(got_b, b)
    assert np.array_equal(fp8.code_values()[codes], want)
    x = inputs.normal_bf16((6, 400), 5)
    x[0, 5], x[1, 399], x[2, 130], x[3, 256:] = np.nan, np.inf, -np.inf, np.nan
    q, s = bi.quantize_fp8(x.cuda())
    want = fp8.held(x.double().numpy())
    assert np.array_equal(bi.fp8_read(q, s).cpu().double().numpy(), want, equal_nan=True)
    assert np.array_equal(np.isnan(want).sum(1), [128, 16, 128, 144, 0, 0])


def test_quantiser_strided_rows_and_untouched_bytes():
    x = inputs.normal_bf16((130, 600), 7).cuda()
    q = torch.full((130, 640), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.full(bi.fp8_scales_shape(130, 528), 0x55, dtype=torch.uint8, device="cuda")
    bi.quantize_fp8(x[:, 8:536], out=q[:, :528], scales=s)
    q1, s1 = bi.quantize_fp8(x[:, 8:536].contiguous())
    assert torch.equal(q[:, :528].view(torch.uint8), q1.view(torch.uint8))
    assert (q.view(torch.uint8)[:, 528:] == 0x55).all()
    assert np.array_equal(fp8.read_scales(s.cpu().numpy(), 130, 528), fp8.read_scales(s1.cpu().numpy(), 130, 528))
    assert (s.reshape(2, 2, 32, 4, 4)[1, :, 2:] == 0x55).all()  # rows past the last have no bytes of their own
    out = torch.full((130, 552), 7.0, dtype=torch.bfloat16, device="cuda")
    bi.fp8_read(q[:, :528], s, out=out[:, :528])
    assert torch.equal(out[:, :528], bi.fp8_read(q1, s1)) and (out[:, 528:] == 7).all()


# -------------------------------------------------------------------- norms ----
@pytest.mark.parametrize("rows,hidden", [(1, 16), (3, 144), (37, 4096), (130, 4112), (5, 5120), (9, 32768), (600, 256)])
def test_norms_hold_the_exact_norm(rows, hidden):
    x, w = inputs.rmsnorm_rows(rows, hidden, seed=hidden), inputs.rmsnorm_weight(hidden, seed=hidden + 1)
    xd = x.double().numpy()
    ref = xd / np.sqrt((xd ** 2).mean(1, keepdims=True) + 1e-6) * w.double().numpy()
    check_held(*bi.rmsnorm_fp8(x.cuda(), w.cuda(), 1e-6), ref, EPS_NORM)
    res = inputs.normal_bf16((rows, hidden), hidden + 2, std=4.0)
    total = (res.float() + x.float()).to(torch.bfloat16)
    td = total.double().numpy()
    ref = td / np.sqrt((td ** 2).mean(1, keepdims=True) + 1e-6) * w.double().numpy()
    kept, out = res.cuda(), torch.empty_like(res, device="cuda")
    q, s = bi.add_rmsnorm_fp8(x.cuda(), kept, w.cuda(), 1e-6, residual_out=out)
    check_held(q, s, ref, EPS_NORM)
    assert torch.equal(out.cpu(), total) and torch.equal(kept.cpu(), res)
    q2, s2 = bi.add_rmsnorm_fp8(x.cuda(), kept, w.cuda(), 1e-6)  # in place
    assert torch.equal(kept.cpu(), total) and torch.equal(q2.view(torch.uint8), q.view(torch.uint8))
    assert torch.equal(bi.fp8_read(q2, s2), bi.fp8_read(q, s))
    bi.get_device_error()


def test_norm_rows_alone_as_in_a_batch_and_special_rows():
    x, w = inputs.rmsnorm_rows(300, 1040, seed=3), inputs.rmsnorm_weight(1040, seed=4)
    x[7] = 0
    x[8, 9], x[9, 1000] = np.nan, np.inf
    x[10] = 1e15
    xd, wd = x.cuda(), w.cuda()
    full = bi.fp8_read(*bi.rmsnorm_fp8(xd, wd))
    for r in (0, 7, 10, 31, 32, 127, 128, 299):
        assert torch.equal(bi.fp8_read(*bi.rmsnorm_fp8(xd[r:r + 1], wd))[0], full[r])
    assert (full[7] == 0).all() and torch.isnan(full[8]).all() and torch.isfinite(full[10:]).all()
    # an infinity: its row's root mean square is one too, so finite values come out as x * 0,
    # the infinity as infinity * 0 = NaN, which is its block's
    assert torch.isnan(full[9, 896:1024]).all() and (full[9, :896] == 0).all() and (full[9, 1024:] == 0).all()
    view = torch.zeros(300, 1104, dtype=torch.bfloat16, device="cuda")
    view[:, 16:1056] = xd
    q = torch.full((300, 1088), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    q1, s1 = bi.rmsnorm_fp8(view[:, 16:1056], wd, out=q[:, :1040])
    assert np.array_equal(bits(bi.fp8_read(q1, s1)), bits(full))
    assert (q.view(torch.uint8)[:, 1040:] == 0x55).all()


def test_quantised_norm_of_bf16_exact_values_is_the_two_calls():
    """Where the bf16 norm rounds nothing (rows of +-1, weight 1, eps 0), norm and quantiser
    one after the other give the bytes of the fused call."""
    x = torch.where(torch.rand(70, 512, generator=torch.Generator().manual_seed(1)) < 0.5, -1.0, 1.0).to(torch.bfloat16).cuda()
    w = torch.exp2(torch.randint(-3, 4, (512,), generator=torch.Generator().manual_seed(2)).float()).to(torch.bfloat16).cuda()
    a, b = bi.rmsnorm_fp8(x, w, 0.0), bi.quantize_fp8(bi.rmsnorm(x, w, 0.0))
    assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8))
    assert torch.equal(bi.fp8_read(*a), bi.fp8_read(*b))


# --------------------------------------------------------------------- GEMM ----
# K: within a block, a block, short last blocks and spans, one to five parts, eight parts of 3
SIZES = [(1, 8, 16), (1, 136, 48), (2, 24, 128), (15, 256, 144), (16, 264, 512), (17, 1000, 528), (32, 8, 1024),
         (33, 120, 1040), (64, 264, 2064), (65, 256, 4096), (128, 136, 4112), (129, 512, 1552), (200, 264, 8208),
         (300, 1000, 528), (513, 2056, 272), (700, 520, 4112), (40, 264, 12288), (1030, 264, 12304)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_gemm_against_the_oracle(M, N, K):
    x, W = random_matrix(M, K, M + K), random_matrix(N, K, N + K)
    check_gemm(bi.gemm_fp8(*x, *W), x, W)
    bi.get_device_error()


def test_gemm_is_exact_where_fp32_is():
    """Small whole numbers: every sum is exact, so y is the bf16 rounding of the exact one."""
    g = torch.Generator().manual_seed(11)
    for M, N, K in ((5, 40, 400), (300, 2056, 1040)):
        a = torch.randint(-3, 4, (M, K), generator=g).to(torch.bfloat16)
        b = torch.randint(-3, 4, (N, K), generator=g).to(torch.bfloat16)
        y = bi.gemm_fp8(*bi.quantize_fp8(a.cuda()), *bi.quantize_fp8(b.cuda()))
        assert torch.equal(y.cpu(), (a.double() @ b.double().T).to(torch.bfloat16))


def rows_of(x, rows):
    """The first rows of an 8-bit matrix."""
    return x[0][:rows], x[1][:-(-rows // 128)]


@pytest.mark.parametrize("N,K", [(264, 4112), (4104, 528), (20000, 144), (136, 12288), (24, 48)])
def test_gemm_rows_keep_their_bits_in_any_batch(N, K):
    """Every form: 16, 32, 64 and 128 rows a CTA with one to eight parts in a cluster, and
    256 x 256 tiles; operands whose products cancel and spread over 2^+-40."""
    x, W = random_matrix(900, K, 5, spread=20), random_matrix(N, K, 6, spread=20)
    x[0][1::2] = x[0][::2]  # pairs of rows that cancel in part: the same, but for the signs of one half
    x[0].view(torch.uint8)[1::2, :K // 2] ^= 0x80
    full = bits(bi.gemm_fp8(*x, *W))
    for M in (1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 511, 513, 768):
        assert np.array_equal(bits(bi.gemm_fp8(*rows_of(x, M), *W)), full[:M]), f"M = {M}"
    perm = torch.randperm(900, generator=torch.Generator().manual_seed(9)).cuda()
    a = bi.quantize_fp8(bi.fp8_read(*quantised(900, K, 8)))
    one = bits(bi.gemm_fp8(*a, *W))
    b = bi.quantize_fp8(bi.fp8_read(*a)[perm].contiguous())
    assert np.array_equal(bits(bi.gemm_fp8(*b, *W)), one[perm.cpu().numpy()])
    assert np.array_equal(bits(bi.gemm_fp8(*b, *W)), bits(bi.gemm_fp8(*b, *W)))
    bi.get_device_error()


@pytest.mark.parametrize("M", [3, 40, 100, 600])
def test_gemm_of_extreme_numbers(M):
    """Products of 0 and subnormal codes, scales to either end, sums that leave fp32 or cancel
    to zero; NaN and infinities of one row or one weight row stay in that row or column."""
    K, N = 1040, 264
    x, W = random_matrix(M, K, 21, spread=3), random_matrix(N, K, 22, spread=3)
    x[0].view(torch.uint8)[0] = 0
    x[0].view(torch.uint8)[1] = 0x81  # the least subnormal, negative
    x[1].reshape(-1)[[fp8.place(2, c, 3) for c in range(9)]] = 247  # as large as the quantiser makes them
    W[1].reshape(-1)[[fp8.place(5, c, 3) for c in range(9)]] = 8    # and as small
    y = bi.gemm_fp8(*x, *W)
    assert (y[0] == 0).all() and torch.isfinite(y[1]).all()
    rest = [r for r in range(M) if r != 2]
    cols = [n for n in range(N) if n != 5]
    a, b = fp8.read(*host(*x)), fp8.read(*host(*W))
    ref, mag = (a @ b.T)[rest][:, cols], (np.abs(a) @ np.abs(b).T)[rest][:, cols]
    err = np.abs(y.cpu().double().numpy()[rest][:, cols] - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) + K * 2.0 ** -22 * mag).all()
    before = bits(y)
    xb, wb = inputs.normal_bf16((M, K), 31), inputs.normal_bf16((N, K), 32)
    clean = bits(bi.gemm_fp8(*bi.quantize_fp8(xb.cuda()), *bi.quantize_fp8(wb.cuda())))
    xb[1, 700], wb[7, 3] = np.inf, np.nan
    y = bi.gemm_fp8(*bi.quantize_fp8(xb.cuda()), *bi.quantize_fp8(wb.cuda()))
    nan = torch.isnan(y).cpu().numpy()
    want = np.zeros_like(nan)
    want[1], want[:, 7] = True, True
    assert np.array_equal(nan, want) and np.array_equal(bits(y)[~want], clean[~want])
    assert np.array_equal(before, bits(bi.gemm_fp8(*x, *W)))
    bi.get_device_error()


@pytest.mark.parametrize("M", [5, 150, 600])
def test_gemm_strided_operands_and_untouched_columns(M):
    xf = torch.zeros(M, 1104, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    Wf = torch.zeros(200, 1168, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    x, W = random_matrix(M, 1040, 41), random_matrix(200, 1040, 42)
    xf[:, 16:1056] = x[0]
    Wf[:, 64:1104] = W[0]
    out = torch.full((M, 240), 3.0, dtype=torch.bfloat16, device="cuda")
    bi.gemm_fp8(xf[:, 16:1056], x[1], Wf[:, 64:1104], W[1], out=out[:, 8:208])
    assert torch.equal(out[:, 8:208], bi.gemm_fp8(*x, *W))
    assert (out[:, :8] == 3).all() and (out[:, 208:] == 3).all()


def test_empty_calls():
    W = quantised(64, 64, 1)
    x = bi.quantize_fp8(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert x[0].shape == (0, 64) and x[1].shape == (0, 1, 512)
    assert bi.gemm_fp8(*x, *W).shape == (0, 64)
    h, hs = bi.gemm_fp8_swiglu(*x, *W)
    assert h.shape == (0, 32) and hs.shape == (0, 1, 512)
    assert bi.fp8_read(*x).shape == (0, 64)
    bi.get_device_error()


# ------------------------------------------------------------------- SwiGLU ----
@pytest.mark.parametrize("M,F,K", [(1, 16, 128), (7, 144, 256), (33, 128, 400), (100, 272, 256), (130, 128, 144), (600, 400, 272)])
def test_swiglu_of_exact_sums(M, F, K):
    """Whole codes and W scales of 2^-5: g and u are exact, so the held h has EPS_SILU only."""
    g = torch.Generator().manual_seed(M + F)
    x = torch.randint(-3, 4, (M, K), generator=g).to(torch.bfloat16)
    W = (torch.randint(-3, 4, (2 * F, K), generator=g).float() * 2.0 ** -5).to(torch.bfloat16)
    Wi = bi.interleave_gate_up(W.cuda())
    h, s = bi.gemm_fp8_swiglu(*bi.quantize_fp8(x.cuda()), *bi.quantize_fp8(Wi))
    gu = x.double().numpy() @ W.double().numpy().T
    check_held(h, s, fp8.swiglu(gu[:, :F], gu[:, F:]), EPS_SILU)
    bi.get_device_error()


@pytest.mark.parametrize("M,F,K", [(1, 12288, 4096), (20, 144, 4112), (50, 400, 2064), (129, 1024, 1040), (520, 528, 4096)])
def test_swiglu_against_the_oracle(M, F, K):
    x, W = quantised(M, K, 51), inputs.gemm_weight(2 * F, K, seed=52)
    Wq = bi.quantize_fp8(bi.interleave_gate_up(W.cuda()))
    h, s = bi.gemm_fp8_swiglu(*x, *Wq)
    a, b = fp8.read(*host(*x)), fp8.read(*host(*Wq))
    gate = np.arange(2 * F) % 16 < 8
    bg, bu = b[gate], b[~gate]
    g, u = a @ bg.T, a @ bu.T
    dg, du = (K * 2.0 ** -22 * (np.abs(a) @ np.abs(w).T) for w in (bg, bu))
    sig = 1 / (1 + np.exp(-g))
    ref = g * sig * u
    off = (np.abs(sig * (1 + g * (1 - sig))) + dg) * (np.abs(u) + du) * dg + np.abs(g * sig) * du + EPS_SILU * np.abs(ref)
    got, scale = fp8.read(*host(h, s)), fp8.read_scales(s.cpu().numpy(), M, F)
    step = np.repeat(np.ldexp(1.0, scale - 127), 128, axis=1)[:, :F]
    bound = off + np.maximum((np.abs(ref) + off) * 2.0 ** -4, step * 2.0 ** -10)
    assert (np.abs(got - ref) <= bound).all()
    want = fp8.scale_bytes(ref)
    assert (np.abs(scale - want) <= 1).all() and (scale != want).mean() <= 0.01
    bi.get_device_error()


@pytest.mark.parametrize("F,K", [(272, 4112), (12288, 272), (16, 48), (128, 12288)])
def test_swiglu_rows_keep_their_bits_in_any_batch(F, K):
    x, W = quantised(600, K, 61), bi.quantize_fp8(bi.interleave_gate_up(inputs.gemm_weight(2 * F, K, seed=62).cuda()))
    h, s = bi.gemm_fp8_swiglu(*x, *W)
    full = fp8.read(*host(h, s))
    for M in (1, 16, 17, 32, 33, 64, 65, 128, 129, 256, 257, 400):
        a, b = bi.gemm_fp8_swiglu(*rows_of(x, M), *W)
        assert torch.equal(a.view(torch.uint8), h[:M].view(torch.uint8)), f"M = {M}"
        assert np.array_equal(fp8.read_scales(b.cpu().numpy(), M, F), fp8.read_scales(s.cpu().numpy(), 600, F)[:M])
    assert np.isfinite(full).all()


@pytest.mark.parametrize("M", [4, 40, 100, 300])
def test_swiglu_nan_stays_in_its_block_and_unused_bytes_do_not_matter(M):
    F, K = 272, 528
    xb, Wb = inputs.normal_bf16((M, K), 71), bi.interleave_gate_up(inputs.gemm_weight(2 * F, K, seed=72).cuda())
    x, W = bi.quantize_fp8(xb.cuda()), bi.quantize_fp8(Wb)
    clean = bi.fp8_read(*bi.gemm_fp8_swiglu(*x, *W))
    # every byte that stands for nothing says NaN
    for (q, s), rows in ((x, M), (W, 2 * F)):
        used = torch.zeros(s.numel(), dtype=torch.bool, device="cuda")
        at = [fp8.place(r, c, s.shape[1]) for r in range(rows) for c in range(-(-K // 128))]
        used[torch.tensor(at, device="cuda")] = True
        s.view(-1)[~used] = 255
    h = torch.full((M, 320), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    hs = torch.full(bi.fp8_scales_shape(M, F), 0x55, dtype=torch.uint8, device="cuda")
    bi.gemm_fp8_swiglu(*x, *W, out=h[:, :F], scales=hs)
    assert torch.equal(bi.fp8_read(h[:, :F], hs), clean) and (h.view(torch.uint8)[:, F:] == 0x55).all()
    xb[1, 3] = np.nan
    y = bi.fp8_read(*bi.gemm_fp8_swiglu(*bi.quantize_fp8(xb.cuda()), *W))
    assert torch.isnan(y[1]).all() and torch.equal(y[2:], clean[2:]) and torch.equal(y[0], clean[0])
    q, s = W[0].clone(), W[1].clone()
    q.view(torch.uint8)[16 * 16 + 8] = 0x7F  # up row 128: one NaN output, so its whole block
    y = bi.fp8_read(*bi.gemm_fp8_swiglu(*x, q, s))
    assert torch.isnan(y[:, 128:256]).all()
    assert torch.equal(y[:, :128], clean[:, :128]) and torch.equal(y[:, 256:], clean[:, 256:])
    bi.get_device_error()


# ------------------------------------------------- together, streams, graphs ----
def mlp(x, res, w, Wgu, Wd, out=None, **kw):
    q, s = bi.add_rmsnorm_fp8(x, res, w, 1e-6, residual_out=out, **kw)
    h, hs = bi.gemm_fp8_swiglu(q, s, *Wgu, **kw)
    return (q, s), (h, hs), bi.gemm_fp8(h, hs, *Wd, **kw)


def mlp_weights(H, F, seed):
    return (inputs.rmsnorm_weight(H, seed=seed).cuda(),
            bi.quantize_fp8(bi.interleave_gate_up(inputs.gemm_weight(2 * F, H, seed=seed + 1).cuda())),
            quantised(H, F, seed + 2, std=0.02))


@pytest.mark.parametrize("M", [1, 24, 300])
def test_a_feed_forward_block_stage_by_stage(M):
    """Each call's output within its bound of the oracle's on what it was given."""
    H, F = 1040, 2064
    w, Wgu, Wd = mlp_weights(H, F, 81)
    x, res = inputs.rmsnorm_rows(M, H, seed=84), inputs.normal_bf16((M, H), 85, std=4.0)
    total = (x.float() + res.float()).to(torch.bfloat16).double().numpy()
    n, h, y = mlp(x.cuda(), res.cuda(), w, Wgu, Wd)
    check_held(*n, total / np.sqrt((total ** 2).mean(1, keepdims=True) + 1e-6) * w.cpu().double().numpy(), EPS_NORM)
    check_gemm(y, h, Wd)
    a, b = fp8.read(*host(*n)), fp8.read(*host(*Wgu))
    gate = np.arange(2 * F) % 16 < 8
    ref = fp8.swiglu(a @ b[gate].T, a @ b[~gate].T)
    got = fp8.read(*host(*h))
    assert np.linalg.norm(got - ref) <= 0.05 * np.linalg.norm(ref)  # 2^-4 at most of each value
    rows = [0, M - 1]
    for r in rows:
        one = mlp(x[r:r + 1].cuda(), res[r:r + 1].cuda(), w, Wgu, Wd)[2]
        assert np.array_equal(bits(one[0]), bits(y[r]))
    bi.get_device_error()


def test_other_streams_and_two_at_once():
    H, F = 1040, 2064
    w, Wgu, Wd = mlp_weights(H, F, 91)
    xs = [inputs.rmsnorm_rows(M, H, seed=94 + M).cuda() for M in (3, 200, 600)]
    res = [torch.zeros_like(x) for x in xs]
    want = [mlp(x, r.clone(), w, Wgu, Wd)[2] for x, r in zip(xs, res)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        got = []
        for x, r, st in zip(xs, res, streams):
            got.append(mlp(x, r, w, Wgu, Wd, out=torch.empty_like(r), stream=st)[2])
        torch.cuda.synchronize()
        assert all(np.array_equal(bits(a), bits(b)) for a, b in zip(got, want))
    # a stream given by its handle
    y = bi.gemm_fp8(*quantised(5, H, 3), *quantised(40, H, 4), stream=streams[0].cuda_stream)
    torch.cuda.synchronize()
    assert np.array_equal(bits(y), bits(bi.gemm_fp8(*quantised(5, H, 3), *quantised(40, H, 4))))
    bi.get_device_error()


def test_captured_and_replayed():
    """Two graphs of the block over buffers of their own, replayed in turn and over new inputs."""
    H, F = 1040, 2064
    w, Wgu, Wd = mlp_weights(H, F, 101)
    runs = []
    for M in (2, 300):
        x, res = (torch.zeros(M, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        mlp(x, res, w, Wgu, Wd, out=torch.empty_like(res))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = mlp(x, res, w, Wgu, Wd, out=torch.empty_like(res))[2]
        runs.append((g, x, res, y))
    for k in range(3):
        for g, x, res, y in runs:
            x.copy_(inputs.rmsnorm_rows(x.shape[0], H, seed=110 + k))
            res.copy_(inputs.normal_bf16(tuple(res.shape), 120 + k))
        for g, *_ in runs:
            g.replay()
        torch.cuda.synchronize()
        for g, x, res, y in runs:
            assert np.array_equal(bits(y), bits(mlp(x, res.clone(), w, Wgu, Wd)[2]))
    bi.get_device_error()


def test_past_2_to_the_31_bytes():
    """Rows whose codes and bf16 values lie past 2^31 bytes."""
    rows, K = 540_000, 4096
    x = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator("cuda").manual_seed(5))
    q, s = bi.quantize_fp8(x)
    W = quantised(24, K, 7)
    y = bi.gemm_fp8(q, s, *W)
    n, ns = bi.rmsnorm_fp8(x, torch.ones(K, dtype=torch.bfloat16, device="cuda"))
    back = bi.fp8_read(q, s)
    for a, b in ((0, 128), (262_144, 262_272), (524_288, 524_416), (539_904, 540_000)):
        part = bi.quantize_fp8(x[a:b])
        assert torch.equal(q[a:b].view(torch.uint8), part[0].view(torch.uint8))
        assert torch.equal(back[a:b], bi.fp8_read(*part))
        assert np.array_equal(bits(y[a:b]), bits(bi.gemm_fp8(*part, *W)))
        m = bi.rmsnorm_fp8(x[a:b], torch.ones(K, dtype=torch.bfloat16, device="cuda"))
        assert torch.equal(n[a:b].view(torch.uint8), m[0].view(torch.uint8))
    bi.get_device_error()


# ----------------------------------------------------------------- refusals ----
def test_binding_refusals():
    x = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    q, s = bi.quantize_fp8(x)
    W, Ws = quantised(32, 64, 1)
    for call, why in (
            (lambda: bi.quantize_fp8(x.float()), "bfloat16"), (lambda: bi.quantize_fp8(x.t()), "unit stride"),
            (lambda: bi.quantize_fp8(x, scales=s[:, :, :256]), "shape"), (lambda: bi.quantize_fp8(x, out=x), "float8"),
            (lambda: bi.quantize_fp8(x, out=q[:2]), "shape"), (lambda: bi.fp8_read(x, s), "float8"),
            (lambda: bi.fp8_read(q, s.float()), "uint8"), (lambda: bi.fp8_read(q, s, out=x[:2]), "shape"),
            (lambda: bi.rmsnorm_fp8(x, w[:32]), "shape"), (lambda: bi.rmsnorm_fp8(x, w.cpu()), "CUDA"),
            (lambda: bi.add_rmsnorm_fp8(x, x[:2], w), "shape"), (lambda: bi.add_rmsnorm_fp8(x, x, w, residual_out=x.float()), "bfloat16"),
            (lambda: bi.gemm_fp8(q, s, W[:, :32], Ws), "shape"), (lambda: bi.gemm_fp8(q, s, W, s.expand(2, 1, 512)), "contiguous"),
            (lambda: bi.gemm_fp8(q, s, W, s.repeat(2, 1, 1)), "shape"),
            (lambda: bi.gemm_fp8(q, s, W, Ws, out=x), "shape"), (lambda: bi.gemm_fp8(q, s.cpu(), W, Ws), "CUDA"),
            (lambda: bi.gemm_fp8(x, s, W, Ws), "float8"), (lambda: bi.gemm_fp8_swiglu(q, s, W[:24], Ws), "multiple of 16"),
            (lambda: bi.gemm_fp8_swiglu(q, s, W, Ws, out=q), "shape")):
        with pytest.raises(ValueError, match=why):
            call()
    for call in (lambda: bi.quantize_fp8(x[:, :24]), lambda: bi.quantize_fp8(x[:, 4:36]), lambda: bi.gemm_fp8(q, s, W[:12], Ws)):
        with pytest.raises(bi.BiError):
            call()
    bi.get_device_error()


@pytest.mark.parametrize("hidden,rows", [(16, 9), (128, 8200), (144, 100), (256, 33), (272, 2100), (512, 2500), (528, 2500),
                                         (768, 2048), (1024, 2051), (1040, 8192), (2048, 8195), (2064, 8192)])
def test_norms_of_short_rows_one_by_one_and_all_at_once(hidden, rows):
    """A warp or a CTA a row, by length and number of rows: the same bytes, and the sum in place."""
    x = inputs.rmsnorm_rows(rows, hidden, seed=hidden).cuda()
    w, res = inputs.rmsnorm_weight(hidden, seed=hidden + 1).cuda(), inputs.normal_bf16((rows, hidden), hidden + 2, std=4.0).cuda()
    x[3, 5], x[4, hidden - 1], x[5] = float("nan"), float("inf"), 0
    some = [0, 3, 4, 5, 7, 8, rows - 1]
    q, s = bi.rmsnorm_fp8(x, w)
    full = bi.fp8_read(q, s)
    total = torch.empty_like(res)
    q2, s2 = bi.add_rmsnorm_fp8(x, res, w, residual_out=total)
    full2 = bi.fp8_read(q2, s2)
    assert np.array_equal(bits(total), bits((res.float() + x.float()).to(torch.bfloat16)))
    for r in some:
        a, b = bi.rmsnorm_fp8(x[r:r + 1], w)
        assert torch.equal(a.view(torch.uint8)[0], q.view(torch.uint8)[r]), r
        assert np.array_equal(bits(bi.fp8_read(a, b))[0], bits(full[r:r + 1])[0]), r
        kept = res[r:r + 1].clone()
        a, b = bi.add_rmsnorm_fp8(x[r:r + 1], kept, w)
        assert torch.equal(a.view(torch.uint8)[0], q2.view(torch.uint8)[r]), r
        assert np.array_equal(bits(bi.fp8_read(a, b))[0], bits(full2[r:r + 1])[0]), r
        assert np.array_equal(bits(kept), bits(total[r:r + 1]))
    fine = [r for r in range(0, rows, max(1, rows // 50)) if r not in (3, 4)]
    xd = x[fine].double().cpu().numpy()
    ref = xd / np.sqrt((xd ** 2).mean(1, keepdims=True) + 1e-6) * w.double().cpu().numpy()
    check_held(*bi.rmsnorm_fp8(x[fine].contiguous(), w), ref, EPS_NORM)
    # rows lie apart, the sum in place, bytes between the rows as they were
    wide = torch.zeros(rows, hidden + 32, dtype=torch.bfloat16, device="cuda")
    wide[:, 16:16 + hidden] = res
    codes = torch.full((rows, hidden + 16), 0x55, dtype=torch.uint8, device="cuda")
    bi.add_rmsnorm_fp8(x, wide[:, 16:16 + hidden], w, out=codes.view(torch.float8_e4m3fn)[:, :hidden])
    assert np.array_equal(bits(wide[:, 16:16 + hidden].contiguous()), bits(total)) and (wide[:, :16] == 0).all()
    assert torch.equal(codes[:, :hidden], q2.view(torch.uint8)) and (codes[:, hidden:] == 0x55).all()
    bi.get_device_error()
