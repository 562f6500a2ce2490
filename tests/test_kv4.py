"""The 4-bit cache's format and the new entry points' refusals, without a GPU.

The oracle's quantiser is pinned by exact rational arithmetic; the library's
entry points are called with arguments that they have to refuse before any
launch (pointers are never dereferenced)."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from invariant_bi_rmsnorm_gb300 import _lib
from oracle import kv4

FAKE = 0x10000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return _lib.load()


def _bf16(x) -> np.ndarray:
    return torch.tensor(np.asarray(x), dtype=torch.float64).to(torch.bfloat16).double().numpy()


def _sig4(q: Fraction) -> Fraction:
    """q > 0 rounded to 4 significant bits, nearest even, by rational arithmetic."""
    e = 0
    while q >= 16:
        q, e = q / 2, e + 1
    while q < 8:
        q, e = q * 2, e - 1
    return Fraction(round(q)) * Fraction(2) ** e  # Fraction.__round__ is half to even


@pytest.mark.parametrize("mantissa", range(128, 256))
def test_scale_and_codes_against_rationals(mantissa):
    """Every bf16 mantissa of the largest magnitude, with the other 31 values
    spread over it, exact ties (n + 1/2) s among them where bf16 has them."""
    amax = Fraction(mantissa, 64)
    s = _sig4(amax / 7)
    ties = [float((Fraction(2 * k + 1) * s) / 2) for k in range(-7, 7)]
    rest = np.linspace(-1, 1, 17) * float(amax)
    row = np.zeros(128)
    row[:32] = np.clip(_bf16(np.concatenate([[float(amax)], ties, rest])), -float(amax), float(amax))
    n, sc = kv4.quantise(row)
    assert Fraction(sc[0]) == s and (sc[1:] == 0).all() and (n[32:] == 0).all()
    for x, got in zip(row[:32], n[:32]):
        want = max(-7, min(7, round(Fraction(x) / s)))
        assert got == want
        assert abs(Fraction(x) - want * s) <= s / 2
    v = kv4.values(n, sc)
    assert np.array_equal(_bf16(v), v)  # exact in bf16


def test_special_groups():
    row = np.zeros(128)
    row[5], row[40], row[70] = np.nan, np.inf, 2.0 ** 123
    row[100] = -(2.0 ** 123) * (1 - 2.0 ** -8)
    n, s = kv4.quantise(row)
    assert np.isnan(s[:3]).all() and np.isfinite(s[3]) and n[100] == -7


@pytest.mark.parametrize("is_v", [False, True])
def test_pack_and_unpack(is_v):
    rng = np.random.default_rng(3)
    x = _bf16(rng.standard_normal((2, 16, 128)) * np.exp(rng.standard_normal((2, 16, 1))))
    b = np.full((2, kv4.BLOCK), 0xA5, dtype=np.uint8)
    order = rng.permutation(16)
    for i, r in enumerate(order):
        before = b.copy()
        kv4.write(b, is_v, r, x[:, r])
        assert (before != b).sum() <= 2 * (64 + 8)  # one token's own bytes
    assert np.array_equal(kv4.unpack(b, is_v), kv4.values(*kv4.quantise(x)))
    # every code of the block has a place of its own
    byte, shift = kv4._positions(is_v)
    assert len({(int(a), int(c)) for a, c in zip(byte.ravel(), shift.ravel())}) == 2048 and byte.max() < 1024


def test_kv4_append_refusals(lib):
    ok = dict(k=FAKE, ldk=1024, v=FAKE, ldv=1024, T=4, Hkv=8, D=128, slots=FAKE, kc=FAKE, vc=FAKE,
              np_=16, page=16)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.bi_kv4_append(a["k"], a["ldk"], a["v"], a["ldv"], a["T"], a["Hkv"], a["D"],
                                 a["slots"], a["kc"], a["vc"], a["np_"], a["page"], None)
    assert call(T=-1) == _lib.BI_ERR_INVALID_ARG
    assert call(Hkv=0) == _lib.BI_ERR_INVALID_ARG
    assert call(np_=0) == _lib.BI_ERR_INVALID_ARG
    assert call(ldk=1016) == _lib.BI_ERR_INVALID_ARG
    assert call(ldv=1028) == _lib.BI_ERR_MISALIGNED
    assert call(D=64) == _lib.BI_ERR_UNSUPPORTED_SHAPE
    assert call(page=32) == _lib.BI_ERR_UNSUPPORTED_SHAPE
    assert call(np_=2 ** 24) == _lib.BI_ERR_UNSUPPORTED_SHAPE
    assert call(k=None) == _lib.BI_ERR_INVALID_ARG
    assert call(slots=None) == _lib.BI_ERR_INVALID_ARG
    assert call(kc=FAKE + 8) == _lib.BI_ERR_MISALIGNED
    assert call(slots=FAKE + 2) == _lib.BI_ERR_MISALIGNED
    assert call(T=0, k=None, v=None) == _lib.BI_OK


def test_qk_norm_rope_append_kv4_refusals(lib):
    ok = dict(qkv=FAKE, ld=6144, T=4, Hq=32, Hkv=8, D=128, pos=FAKE, slots=FAKE, rope=FAKE, mp=64,
              qw=FAKE, kw=None, eps=1e-6, q=FAKE, kc=FAKE, vc=FAKE, np_=16, page=16)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.bi_qk_norm_rope_append_kv4(
            a["qkv"], a["ld"], a["T"], a["Hq"], a["Hkv"], a["D"], a["pos"], a["slots"], a["rope"],
            a["mp"], a["qw"], a["kw"], a["eps"], a["q"], a["kc"], a["vc"], a["np_"], a["page"], None)
    assert call(ld=6136) == _lib.BI_ERR_INVALID_ARG
    assert call(ld=6148) == _lib.BI_ERR_MISALIGNED
    assert call(D=64) == _lib.BI_ERR_UNSUPPORTED_SHAPE
    assert call(np_=2 ** 24) == _lib.BI_ERR_UNSUPPORTED_SHAPE
    assert call(eps=float("nan")) == _lib.BI_ERR_INVALID_ARG
    assert call(vc=FAKE + 4) == _lib.BI_ERR_MISALIGNED
    assert call(T=0) == _lib.BI_OK


def test_kv4_read_refusals(lib):
    ok = dict(kc=FAKE, vc=FAKE, bt=FAKE, mp=8, lens=FAKE, S=3, Hkv=8, D=128, page=16, np_=16, msl=128,
              ko=FAKE, vo=FAKE)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.bi_kv4_read(a["kc"], a["vc"], a["bt"], a["mp"], a["lens"], a["S"], a["Hkv"],
                               a["D"], a["page"], a["np_"], a["msl"], a["ko"], a["vo"], None)
    assert call(S=-1) == _lib.BI_ERR_INVALID_ARG
    assert call(msl=129) == _lib.BI_ERR_INVALID_ARG  # beyond the block table
    assert call(msl=0) == _lib.BI_ERR_INVALID_ARG
    assert call(S=65536) == _lib.BI_ERR_UNSUPPORTED_SHAPE
    assert call(D=96) == _lib.BI_ERR_UNSUPPORTED_SHAPE
    assert call(ko=FAKE + 2) == _lib.BI_ERR_MISALIGNED
    assert call(lens=FAKE + 1) == _lib.BI_ERR_MISALIGNED
    assert call(bt=None) == _lib.BI_ERR_INVALID_ARG
    assert call(S=0) == _lib.BI_OK


def test_decode_attention_kv4_refusals(lib):
    ok = dict(q=FAKE, k=FAKE, v=FAKE, bt=FAKE, mp=64, lens=FAKE, B=4, Hq=32, Hkv=8, D=128,
              page=16, np_=256, msl=1000, scale=0.088, out=FAKE, ws=FAKE, wsb=10 ** 9, s=None)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.bi_decode_attention_kv4(
            a["q"], a["k"], a["v"], a["bt"], a["mp"], a["lens"], a["B"], a["Hq"], a["Hkv"], a["D"],
            a["page"], a["np_"], a["msl"], a["scale"], a["out"], a["ws"], a["wsb"], a["s"])
    assert call(D=64) == _lib.BI_ERR_UNSUPPORTED_SHAPE
    assert call(page=32) == _lib.BI_ERR_UNSUPPORTED_SHAPE
    assert call(Hq=30) == _lib.BI_ERR_UNSUPPORTED_SHAPE
    assert call(Hq=80, Hkv=8) == _lib.BI_ERR_UNSUPPORTED_SHAPE  # group 10 > 8
    assert call(B=65536) == _lib.BI_ERR_UNSUPPORTED_SHAPE
    assert call(np_=2 ** 27) == _lib.BI_ERR_UNSUPPORTED_SHAPE
    assert call(msl=64 * 16 + 1) == _lib.BI_ERR_INVALID_ARG
    assert call(scale=0.0) == _lib.BI_ERR_INVALID_ARG
    assert call(scale=float("inf")) == _lib.BI_ERR_INVALID_ARG
    assert call(wsb=100) == _lib.BI_ERR_WORKSPACE_TOO_SMALL
    assert call(ws=None) == _lib.BI_ERR_WORKSPACE_TOO_SMALL
    assert call(ws=FAKE + 8) == _lib.BI_ERR_MISALIGNED
    assert call(k=FAKE + 8) == _lib.BI_ERR_MISALIGNED
    assert call(lens=None) == _lib.BI_ERR_INVALID_ARG
    assert call(B=0) == _lib.BI_OK


def test_logprobs_top_refusals(lib):
    ok = dict(x=FAKE, rows=4, vocab=1024, ld=1024, t=FAKE, lp=FAKE, lse=FAKE, h=FAKE, k=20, ids=FAKE,
              top=FAKE)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.bi_logprobs_top(a["x"], a["rows"], a["vocab"], a["ld"], a["t"], a["lp"], a["lse"],
                                   a["h"], a["k"], a["ids"], a["top"], None)
    assert call(rows=-1) == _lib.BI_ERR_INVALID_ARG
    assert call(k=0) == _lib.BI_ERR_INVALID_ARG
    assert call(k=33) == _lib.BI_ERR_UNSUPPORTED_SHAPE
    assert call(vocab=16, ld=16, k=17) == _lib.BI_ERR_UNSUPPORTED_SHAPE
    assert call(vocab=1020) == _lib.BI_ERR_UNSUPPORTED_SHAPE
    assert call(ld=1016) == _lib.BI_ERR_INVALID_ARG
    assert call(ld=1028) == _lib.BI_ERR_MISALIGNED
    assert call(x=FAKE + 8) == _lib.BI_ERR_MISALIGNED
    assert call(t=None) == _lib.BI_ERR_INVALID_ARG   # logprob_out without targets
    assert call(lp=None) == _lib.BI_ERR_INVALID_ARG  # targets without logprob_out
    assert call(ids=None) == _lib.BI_ERR_INVALID_ARG
    assert call(rows=0, x=None) == _lib.BI_OK


def test_binding_refuses_cpu_tensors():
    import invariant_bi_rmsnorm_gb300 as bi
    kc, vc = bi.kv4_cache(4, 2, device="cpu")
    assert kc.shape == (4, 2, bi.KV4_BLOCK_BYTES) and kc.dtype == torch.uint8
    rows = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    idx = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        bi.kv4_append(rows, rows, idx, kc, vc)
    with pytest.raises(ValueError, match="CUDA"):
        bi.kv4_read(kc, vc, idx[None], idx[:1], 16, rows, rows)
    with pytest.raises(ValueError, match="CUDA"):
        bi.decode_attention_kv4(rows, kc, vc, idx[None], idx, 16)
    with pytest.raises(ValueError, match="CUDA"):
        bi.logprobs_top(rows[0], None, 1)
