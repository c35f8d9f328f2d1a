"""ORACLE -- test infrastructure only (tests).

Reference for 4-bit caches, in numpy fp64 (the pages have no counterpart): OCP E2M1 codes with
an E4M3 scale for every 16 elements of a row and one scale per KV head.

  encode   the definition of the quantiser, and how far each input lies from a border between
           two codes or two scales (a result in fp32 may round to either side there);
  pack     rows into pages, the layout that the library reads;
  values   what a page stands for.
"""
from __future__ import annotations

import numpy as np

from .feeder import encode_e4m3_value

PAGE, D, BLOCK = 64, 128, 16
CODES, UNIT = PAGE * D // 2, PAGE * D // 2 + PAGE * D // BLOCK
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def encode_e2m1(x):
    """Code 0..15 nearest to x, ties to the even code, saturated at +-6; the sign of zero kept."""
    a = np.abs(np.asarray(x, np.float64))
    mid = (GRID[1:] + GRID[:-1]) / 2
    code = np.zeros(a.shape, np.int64)
    for i, m in enumerate(mid):            # between codes i and i + 1: the even one on a tie
        code = np.where((a > m) | ((a == m) & ((i + 1) % 2 == 0)), i + 1, code)
    return (code + 8 * np.signbit(x)).astype(np.uint8)


def decode_e2m1(code):
    code = np.asarray(code)
    return np.where(code & 8, -1.0, 1.0) * GRID[code & 7]


def e4m3_byte(x):
    """The byte of a non-negative E4M3 value."""
    import torch
    return torch.from_numpy(np.asarray(x, np.float64)).to(torch.float8_e4m3fn).view(
        torch.uint8).numpy()


def e4m3_value(byte):
    import torch
    b = torch.from_numpy(np.ascontiguousarray(byte, np.uint8))
    return b.view(torch.float8_e4m3fn).double().numpy()


def encode(y):
    """y [..][128] in units of the head's scale: (codes [..][128], scales [..][8] as values)."""
    y = np.asarray(y, np.float64)
    blocks = y.reshape(*y.shape[:-1], -1, BLOCK)
    s = encode_e4m3_value(np.abs(blocks).max(-1) / 6.0)
    with np.errstate(divide="ignore", invalid="ignore"):
        z = np.where(s[..., None] > 0, blocks / s[..., None], 0.0)
    return encode_e2m1(z).reshape(y.shape), s


def row_bytes(codes, scales):
    """(64 bytes of codes, 8 of scales) for rows of codes [..][128], scale values [..][8]."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4), e4m3_byte(scales)


def pack(y):
    """Rows y [P][Hkv][64][128] as pages [P][Hkv][UNIT]."""
    c, s = row_bytes(*encode(y))
    return np.concatenate([c.reshape(*c.shape[:2], CODES), s.reshape(*s.shape[:2], UNIT - CODES)],
                          -1)


def unpack(pool):
    """(codes [P][Hkv][64][128], scale bytes [P][Hkv][64][8]) of pages [P][Hkv][UNIT]."""
    pool = np.asarray(pool)
    b = pool[..., :CODES].reshape(*pool.shape[:2], PAGE, D // 2)
    codes = np.stack([b & 15, b >> 4], -1).reshape(*pool.shape[:2], PAGE, D)
    return codes, pool[..., CODES:].reshape(*pool.shape[:2], PAGE, D // BLOCK)


def values(pool, scale=None):
    """fp64 values [P][Hkv][64][128] of pages (NaN where a block's scale is)."""
    codes, s = unpack(pool)
    x = decode_e2m1(codes) * np.repeat(e4m3_value(s), BLOCK, -1)
    return x if scale is None else x * np.asarray(scale, np.float64)[None, :, None, None]
