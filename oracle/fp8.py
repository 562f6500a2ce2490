"""fp64 oracle of the 8-bit matrix format and of the products over it (include/bi.h,
"8-bit matrices").

TEST INFRASTRUCTURE; shares no code with the CUDA library.  Plain definitions: 128
consecutive values of a row (the last block may be shorter) are held as e4m3 codes and
one scale 2^(b - 127),

    b = the least number from 8 up with max|x| <= 448 * 2^(b - 127);  255 where the
        block holds a NaN or an infinity
    code = x / 2^(b - 127) rounded to nearest even (NaN throughout for b = 255)

and stand for code * 2^(b - 127).  Pins (tests/test_fp8.py): every code against
rational arithmetic, scales at the borders, tiles against a byte-by-byte loop.
"""
from __future__ import annotations

import numpy as np

BLOCK, TILE = 128, 512


def scale_bytes(x) -> np.ndarray:
    """b of every block of x [rows, K] -> int [rows, ceil(K / 128)]."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    out = []
    for at in range(0, x.shape[1], BLOCK):
        top = x[:, at:at + BLOCK].max(axis=1)
        ok = np.isfinite(top)
        m, e = np.frexp(np.where(ok, top, 1.0))  # top = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
        e = np.where(m > 0.875, e - 8, e - 9)
        b = np.where(np.where(ok, top, 1.0) > 0, np.maximum(e + 127, 8), 8)
        out.append(np.where(ok, b, 255))
    return np.stack(out, axis=1)


def round_e4m3(v) -> np.ndarray:
    """v with |v| <= 448 rounded to the nearest e4m3 number, ties to even (fp64)."""
    v = np.asarray(v, dtype=np.float64)
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)  # 4 significant bits; subnormals below 2^-6
    return np.rint(v / step) * step


def quantise(x):
    """x [rows, K] (fp64) -> (values q of the codes [rows, K], b [rows, blocks])."""
    x = np.asarray(x, dtype=np.float64)
    b = scale_bytes(x)
    s = np.repeat(np.where(b == 255, np.nan, np.ldexp(1.0, b - 127)), BLOCK, axis=1)[:, :x.shape[1]]
    with np.errstate(invalid="ignore"):
        return np.where(np.isnan(s), np.nan, round_e4m3(np.where(np.isnan(s), 0.0, x / s))), b


def held(x) -> np.ndarray:
    """What 8 bits hold of x [rows, K] (fp64)."""
    q, b = quantise(x)
    with np.errstate(invalid="ignore"):
        return q * np.repeat(np.ldexp(1.0, b - 127), BLOCK, axis=1)[:, :q.shape[1]]


def code_values() -> np.ndarray:
    """The number that each of the 256 codes is: sign, 4 bits of exponent (bias 7), 3 of
    mantissa; exponent and mantissa all ones is NaN."""
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = np.nan if (e, m) == (15, 7) else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = -v if c & 128 else v
    return out


def place(row: int, block: int, spans: int) -> int:
    """Byte offset of a block's scale."""
    return ((row // 128) * spans + block // 4) * TILE + 16 * (row % 32) + 4 * (row % 128 // 32) + block % 4


def read_scales(tiles, rows: int, K: int) -> np.ndarray:
    """Scale bytes [rows, blocks] out of tiles [ceil(rows / 128), ceil(K / 512), 512]."""
    flat = np.asarray(tiles, dtype=np.uint8).reshape(-1)
    blocks, spans = -(-K // BLOCK), -(-K // TILE)
    return np.array([[flat[place(r, c, spans)] for c in range(blocks)] for r in range(rows)],
                    dtype=np.int64).reshape(rows, blocks)


def read(codes, tiles) -> np.ndarray:
    """What an 8-bit matrix (codes uint8 [rows, K], scale tiles) stands for (fp64)."""
    codes = np.asarray(codes, dtype=np.uint8)
    b = read_scales(tiles, *codes.shape)
    with np.errstate(invalid="ignore"):
        return code_values()[codes] * np.repeat(np.ldexp(1.0, b - 127), BLOCK, axis=1)[:, :codes.shape[1]]


def swiglu(g, u) -> np.ndarray:
    g = np.asarray(g, dtype=np.float64)
    return g / (1.0 + np.exp(-g)) * u
