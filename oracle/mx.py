"""Plain forms of the 4-bit microscaled (MX) operators in numpy and 64 bits:
test infrastructure, sharing no code with the library.

Codes and scales are laid out as include/gemm_mx.h says: value k of a row in
byte k // 2 (lower four bits for even k), 32 values to a scale byte.
"""
from __future__ import annotations

import numpy as np

# The E2M1 elements by code: sign, two exponent bits (bias 1), one mantissa bit.
ELEMENTS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def code_bytes(K: int) -> int:
    return -(-K // 32) * 16


def scale_bytes(K: int) -> int:
    return -(-K // 512) * 16


def quantize(x: np.ndarray):
    """(codes, scales) of the rows of x (any float type; taken as float64)."""
    x = np.asarray(x, dtype=np.float64)
    rows, K = x.shape
    codes = np.zeros((rows, code_bytes(K)), np.uint8)
    scales = np.zeros((rows, scale_bytes(K)), np.uint8)
    for b in range(-(-K // 32)):
        blk = np.zeros((rows, 32))
        part = x[:, 32 * b:32 * b + 32]
        blk[:, :part.shape[1]] = part
        bad = ~np.isfinite(blk).all(axis=1)
        blk[bad] = 0.0
        m = np.abs(blk).max(axis=1)
        # frexp: m = f 2^e with f in [1/2, 1), so floor(log2 m) = e - 1
        e = np.where(m > 0, np.frexp(m)[1] - 1 - 2, -127)
        e = np.clip(e, -127, 127)
        z = np.ldexp(np.abs(blk), -e[:, None])  # exact in float64
        # Nearest element; on a tie the one whose code is even.  The elements'
        # midpoints, and whether the lower neighbour's code is even there.
        code = np.zeros(z.shape, np.uint8)
        for c in range(7):
            mid = (ELEMENTS[c] + ELEMENTS[c + 1]) / 2
            code += (z > mid) if c % 2 == 0 else (z >= mid)
        code |= np.where(np.signbit(blk) & (z >= 0), 8, 0).astype(np.uint8)
        code[bad] = 0
        codes[:, 16 * b:16 * b + 16] = code[:, 0::2] | (code[:, 1::2] << 4)
        scales[:, b] = np.where(bad, 255, e + 127)
    return codes, scales


def values(codes: np.ndarray, scales: np.ndarray, K: int) -> np.ndarray:
    """The float64 values of MX rows (last axis bytes; leading axes kept)."""
    nb = -(-K // 32)
    c = np.asarray(codes)[..., :16 * nb]
    nib = np.stack([c & 15, c >> 4], axis=-1).reshape(*c.shape[:-1], 32 * nb)
    v = ELEMENTS[nib & 7] * np.where(nib & 8, -1.0, 1.0)
    s = np.asarray(scales)[..., :nb].astype(np.int64)
    unit = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    v = v * np.repeat(unit, 32, axis=-1)
    return v[..., :K]


def random_rows(rng, rows: int, K: int, low: int = 120, high: int = 130, pad: int = 0):
    """Random codes (zero past K) and scale bytes in [low, high); the bytes past
    the last block hold `pad`."""
    nb = -(-K // 32)
    nib = rng.integers(0, 16, (rows, 32 * nb), dtype=np.uint8)
    nib[:, K:] = 0
    codes = nib[:, 0::2] | (nib[:, 1::2] << 4)
    scales = np.full((rows, scale_bytes(K)), pad, np.uint8)
    scales[:, :nb] = rng.integers(low, high, (rows, nb), dtype=np.uint8)
    return codes, scales


def round_to(x: np.ndarray, fmt: str) -> np.ndarray:
    """float64 values rounded once to bf16, f16 or f32, as float64."""
    if fmt == "f32":
        return x.astype(np.float32).astype(np.float64)
    if fmt == "f16":
        return x.astype(np.float16).astype(np.float64)
    # bf16: 8 significant bits, exponents of fp32 (subnormals below 2^-126)
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.frexp(np.where(np.isfinite(x) & (x != 0), x, 1.0))[1]
        step = np.ldexp(1.0, np.maximum(e - 8, -133))
        y = np.where(np.isfinite(x), np.rint(x / step) * step, x)
        return np.where(np.abs(y) > 3.3895313892515355e38, np.copysign(np.inf, y), y)
