"""The format of include/bi_fp4.h in numpy, written from its definition: codes by search among the sixteen
values, scales bit by bit, tiles by their byte formula.  Test infrastructure."""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"mxfp4": 32, "nvfp4": 16}


def bf16_values(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32)


def e4m3_value(byte: np.ndarray) -> np.ndarray:
    b = byte.astype(np.int64)
    e, m = b // 8 % 16, b % 8
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
    return np.where(b == 0x7F, np.nan, v)


E4M3 = e4m3_value(np.arange(127))                     # ascending


def e4m3_nearest(v: np.ndarray) -> np.ndarray:
    """Byte of the nearest E4M3 value to v >= 0, ties to even, at most 448."""
    v = np.minimum(v.astype(np.float64), 448.0)
    i = np.clip(np.searchsorted(E4M3, v, side="right") - 1, 0, 125)
    mid = (E4M3[i] + E4M3[i + 1]) / 2                 # (exact in 64 bits)
    return np.where((v > mid) | ((v == mid) & (i % 2 == 1)), i + 1, i).astype(np.uint8)


def e2m1_nearest(y: np.ndarray) -> np.ndarray:
    """Code of the nearest E2M1 value, ties to even, at most 6, signs kept."""
    a = np.minimum(np.abs(y.astype(np.float64)), 6.0)
    i = np.clip(np.searchsorted(GRID, a, side="right") - 1, 0, 6)
    mid = (GRID[i] + GRID[i + 1]) / 2
    code = np.where((a > mid) | ((a == mid) & (i % 2 == 1)), i + 1, i).astype(np.uint8)
    return code | (np.signbit(y).astype(np.uint8) << 3)


def quantise(x: np.ndarray, kind: str, g: float = 1.0):
    """x float32 [R, K] (bf16 values) -> codes [R, K] uint8 (one an element), scale bytes [R, K / block]."""
    R, K = x.shape
    x = x.reshape(R, -1, BLOCK[kind]).astype(np.float32)
    bad = ~np.isfinite(x).all(-1)
    top = np.where(bad, np.float32(0), np.abs(np.where(np.isfinite(x), x, 0)).max(-1)).astype(np.float32)
    with np.errstate(all="ignore"):
        if kind == "mxfp4":
            e = np.where(top > 0, np.floor(np.log2(np.maximum(top.astype(np.float64), 1e-300))) - 2, -127)
            e = np.maximum(e, -127).astype(np.int64)
            byte = (e + 127).astype(np.uint8)
            codes = e2m1_nearest(x.astype(np.float64) * 2.0 ** -e[..., None].astype(np.float64))
            nan = 255
        else:
            six = np.float32(6) * np.float32(g)
            byte = e4m3_nearest(top / six)
            unit = (e4m3_value(byte).astype(np.float32) * np.float32(g))[..., None]
            y = np.where(unit > 0, x / np.where(unit > 0, unit, np.float32(1)), np.copysign(np.float32(0), x))
            codes = e2m1_nearest(y)
            nan = 0x7F
    codes = np.where(bad[..., None], 0, codes).astype(np.uint8).reshape(R, K)
    return codes, np.where(bad, nan, byte).astype(np.uint8)


def pack(codes: np.ndarray) -> np.ndarray:
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(packed: np.ndarray) -> np.ndarray:
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)


def values(packed: np.ndarray, scales: np.ndarray, kind: str, g: float = 1.0) -> np.ndarray:
    """64-bit values of packed codes [..., K / 2] and scale bytes [..., K / block]."""
    v = np.concatenate([GRID, -GRID])[unpack(packed)]
    s = 2.0 ** (scales.astype(np.float64) - 127) if kind == "mxfp4" else e4m3_value(scales) * np.float64(np.float32(g))
    if kind == "mxfp4":
        s = np.where(scales == 255, np.nan, s)
    return v * np.repeat(s, BLOCK[kind], -1)


def tile_offsets(R: int, C: int) -> np.ndarray:
    r, c = np.arange(R)[:, None], np.arange(C)[None]
    return ((r // 128) * (C // 4) + c // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + c % 4


def to_tiles(s: np.ndarray, fill: int = 0) -> np.ndarray:
    R, C = s.shape
    out = np.full(-(-R // 128) * (C // 4) * 512, fill, np.uint8)
    out[tile_offsets(R, C)] = s
    return out.reshape(-(-R // 128), C // 4, 32, 4, 4)


def from_tiles(t: np.ndarray, R: int) -> np.ndarray:
    return t.reshape(-1)[tile_offsets(R, 4 * t.shape[1])]
