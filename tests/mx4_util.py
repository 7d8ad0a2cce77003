"""Plain 64-bit forms of the MXFP4 format and of the layer's gradients, for the tests of the kernels.
numpy only; written from the format's definition (OCP Microscaling v1.0) and the formulas."""
from __future__ import annotations

import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
U32 = 2.0 ** -24      # half a step of fp32, relative
UB16 = 2.0 ** -8      # half a step of bf16, relative


def quantize(x: np.ndarray):
    """x [rows, cols] (any float) -> (code magnitudes and signs as bytes [rows, cols], scale bytes [rows, cols/32])."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[0], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    v = np.where(bad[..., None], 0.0, b)
    m = np.abs(v).max(-1)
    e = np.where(m > 0, np.maximum(np.frexp(np.where(m > 0, m, 1.0))[1] - 3, -127), 0)
    a = np.minimum(np.abs(np.ldexp(v, -e[..., None])), 6.0)
    # nearest grid point; among two equally near ones the even code
    d = np.abs(a[..., None] - GRID)
    near = d == d.min(-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(-1, keepdims=True), even, near)
    code = pick.argmax(-1).astype(np.uint8)
    code = code | (np.signbit(v).astype(np.uint8) << 3)
    code = np.where(bad[..., None], 0, code).astype(np.uint8)
    scale = np.where(bad, 255, e + 127).astype(np.uint8)
    return code.reshape(x.shape), scale


def pack(code: np.ndarray) -> np.ndarray:
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed: np.ndarray) -> np.ndarray:
    return np.stack([packed & 15, packed >> 4], -1).reshape(packed.shape[:-1] + (-1,))


def values(code: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """Unpacked codes [..., cols] and scale bytes [..., cols/32] -> fp64 values (NaN where the scale byte is 0xFF)."""
    v = np.where(code & 8, -1.0, 1.0) * GRID[code & 7]
    s = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
    return (v.reshape(scale.shape + (32,)) * s[..., None]).reshape(code.shape)


def dequantize(packed, scale):
    return values(unpack(packed), scale)


def random_weights(g: np.random.Generator, *shape, lo=119, hi=124):
    packed = g.integers(0, 256, size=shape[:-1] + (shape[-1] // 2,), dtype=np.uint8)
    scale = g.integers(lo, hi, size=shape[:-1] + (shape[-1] // 32,), dtype=np.uint8)
    return packed, scale


def sum_bound(k: int) -> float:
    """Relative (to the sum of absolute products) bound on the tensor core's fp32 accumulation over k
    products: the products are exact, the accumulator is rounded or truncated once per 32-deep step
    (2^-23 each), and aligning a step's up to 64 products costs at most 64 such units more."""
    return (k / 32 + 64) * 2.0 ** -23


def random_offsets(g: np.random.Generator, groups: int, rows: int, skew: float = 0.0) -> np.ndarray:
    p = np.exp(-skew * np.log1p(g.permutation(groups)))
    n = g.multinomial(rows, p / p.sum())
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def silu(x):
    return x / (1.0 + np.exp(-x))
