"""fp64 oracle of the 4-bit KV-cache format (include/bi.h, "The 4-bit cache").

TEST INFRASTRUCTURE; shares no code with the CUDA library.  Plain definitions:
a group of 32 consecutive dims is held as codes n + 8 and a scale s,

    s = max|x| / 7 rounded to 4 significant bits (nearest even);  NaN if the
        group holds a NaN, an infinity or a magnitude of 2^123 or more, 0 if
        every magnitude is below 2^-120
    n = x / s rounded to nearest even, clamped to -7 .. 7 (0 where s is 0 or NaN)

and stands for n * s.  Pins (tests/test_kv4.py): the error bound s / 2, exact
ties by rational arithmetic, every scale mantissa, packing against a
dim-by-dim loop over the documented bit positions.
"""
from __future__ import annotations

import numpy as np

BLOCK = 1152


def _round_sig4(x: np.ndarray) -> np.ndarray:
    """x >= 0 rounded to 4 significant bits, nearest even (fp64, exact)."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 16.0), e - 4)


def quantise(x) -> tuple[np.ndarray, np.ndarray]:
    """bf16-exact rows x [..., 128] -> (n [..., 128], s [..., 4]) in fp64."""
    g = np.asarray(x, dtype=np.float64)
    g = g.reshape(*g.shape[:-1], 4, 32)
    amax = np.abs(g).max(-1)  # a NaN comes through
    ok = amax < 2.0 ** 123
    s = np.where(ok, _round_sig4(np.where(ok, amax, 0.0) / 7.0), np.nan)
    s = np.where(amax < 2.0 ** -120, 0.0, s)
    live = (s > 0)[..., None]
    with np.errstate(invalid="ignore"):
        n = np.where(live, np.clip(np.rint(g / np.where(live, s[..., None], 1.0)), -7, 7), 0.0)
    return n.reshape(*n.shape[:-2], 128), s


def values(n, s) -> np.ndarray:
    n = np.asarray(n, dtype=np.float64)
    return (n.reshape(*n.shape[:-1], 4, 32) * np.asarray(s)[..., None]).reshape(n.shape)


def _position(is_v: bool, token: int, dim: int) -> tuple[int, int]:
    """(byte, shift within it) of the code of one token's dim in a block."""
    if is_v:
        w, h, p, g = dim // 64, dim % 64 // 32, dim % 32 // 8, dim % 8
        word = 128 * (token // 8) + 16 * g + 4 * (token % 8 // 2) + 2 * (token % 2) + w
        code = 4 * h + p
    else:
        j, p, t, e = dim // 32, dim % 32 // 8, dim % 8 // 2, dim % 2
        word, code = 16 * token + 4 * t + j, p + 4 * e
    return 4 * word + code // 2, 4 * (code % 2)


def _positions(is_v: bool):
    at = np.array([[_position(is_v, r, d) for d in range(128)] for r in range(16)])
    return at[..., 0], at[..., 1]


def unpack(blocks, is_v: bool) -> np.ndarray:
    """Block bytes [..., 1152] -> values [..., 16, 128] in fp64."""
    b = np.asarray(blocks, dtype=np.uint8)
    byte, shift = _positions(is_v)
    n = ((b[..., byte] >> shift) & 15).astype(np.int64) - 8
    bits = b[..., 1024::2].astype(np.uint32) | (b[..., 1025::2].astype(np.uint32) << 8)
    s = (bits << 16).view(np.float32).astype(np.float64).reshape(*b.shape[:-1], 16, 4)
    return values(n, s)


def write(blocks: np.ndarray, is_v: bool, token: int, x) -> None:
    """Quantise row x [..., 128] into token `token` of blocks [..., 1152], in place."""
    n, s = quantise(x)
    byte, shift = _positions(is_v)
    code = (n + 8).astype(np.uint8)
    for d in range(128):
        at, sh = byte[token, d], shift[token, d]
        blocks[..., at] = (blocks[..., at] & (0xF0 if sh == 0 else 0x0F)) | (code[..., d] << sh)
    with np.errstate(invalid="ignore"):
        bits = s.astype(np.float32).view(np.uint32) >> 16
    for g in range(4):
        blocks[..., 1024 + 8 * token + 2 * g] = bits[..., g] & 0xFF
        blocks[..., 1025 + 8 * token + 2 * g] = bits[..., g] >> 8
