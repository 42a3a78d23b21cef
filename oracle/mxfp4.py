"""Oracle: MXFP4 quantisation, the tiled layout, and the products on it.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

MXFP4 is the OCP microscaling format with E2M1 elements: blocks of 32
consecutive values of a row share X = 2^(byte - 127).  For a block with
a = max |x| the scale is byte = max(floor(log2 a) - 2 + 127, 0) (2 being the
exponent of E2M1's largest value, 6), 0 for a == 0; a value's code is x / X
to the nearest of +-{0, .5, 1, 1.5, 2, 3, 4, 6}, ties to the even code,
saturating, sign kept.  A block with a NaN or an infinity has byte 255 (NaN)
and zero codes.

Everything is computed in float64, where dividing by X, E2M1 products and
their scaling are exact.  Sums of a product are float64 sums of exact terms;
they are exact for the blocks' usual scale ranges, and their rounding is
counted in the bounds.
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
U = 2.0 ** -24


def pad_rows(rows: int) -> int:
    return -(-rows // 32) * 32


def quant(x: np.ndarray):
    """(codes uint8 [..., k] one nibble a value, bytes uint8 [..., k/32])."""
    b = np.asarray(x, dtype=np.float32).reshape(*x.shape[:-1], -1, 32).astype(np.float64)
    a = np.max(np.abs(b), axis=-1)  # NaN wins
    bad = ~np.isfinite(a)
    _, e = np.frexp(np.where(bad, 1.0, a))  # a = f 2^e, f in [.5, 1)
    byte = np.where(a > 0, np.maximum(e - 1 - 2 + 127, 0), 0)
    with np.errstate(invalid="ignore"):
        v = np.where(bad[..., None], 0.0, b) / np.exp2(byte - 127.0)[..., None]
    mag = np.abs(v)
    hi = np.clip(np.searchsorted(GRID, mag), 1, 7)
    up, down = GRID[hi] - mag, mag - GRID[hi - 1]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)
    code = code + 8 * (np.signbit(v) & ~bad[..., None])
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 255, byte).astype(np.uint8)


def dequant(codes: np.ndarray, byte: np.ndarray) -> np.ndarray:
    """float64 values; NaN for byte 255."""
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    x = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127.0))
    return v * np.repeat(x, 32, axis=-1)


def tile(codes: np.ndarray, byte: np.ndarray):
    """The tiled layout of [rows][k] codes and [rows][k/32] bytes, one value
    at a time from its place in the formula of include/rz_fp8.h."""
    rows, k = codes.shape
    p = pad_rows(rows)
    tc = np.zeros(p * k // 2, dtype=np.uint8)
    ts = np.zeros(p * k // 32, dtype=np.uint8)
    r, c = np.meshgrid(np.arange(rows), np.arange(k), indexing="ij")
    at = (((r // 32) * (k // 64) + c // 64) * 2 + c // 32 % 2) * 512 + r % 32 * 16 + c % 32 // 2
    for odd in (0, 1):
        sel = c % 2 == odd
        tc[at[sel]] |= codes[sel] << (4 * odd)
    r, c = np.meshgrid(np.arange(rows), np.arange(0, k, 32), indexing="ij")
    ts[(((r // 32) * (k // 256) + c // 256) * 2 + c // 32 % 2) * 128 + r % 32 * 4 + c // 64 % 4] = byte
    return tc.reshape(p // 32, k // 64, 1024), ts.reshape(p // 32, k // 256, 256)


def quant_tiled(x: np.ndarray):
    return tile(*quant(x))


def gemm(a: np.ndarray, w: np.ndarray):
    """(a w^T, its error bound) for float64 values of MXFP4 tensors.

    Products of E2M1 values are exact.  Each fp32 addition, inside the matrix
    core or outside, errs by at most 2u relative (truncation; u to nearest),
    and there are fewer than K on the way of any term, so the error is at most
    gamma_K(2u) sum |a w|, plus the float64 sum's own gamma_K(2^-53).  Results
    under 2^-126, which the matrix core may flush, are not counted."""
    k = a.shape[1]
    g = 2 * k * U / (1 - 2 * k * U) + k * 2.0 ** -53
    return a @ w.T, g * (np.abs(a) @ np.abs(w).T)


def gemv(x: np.ndarray, w: np.ndarray):
    """(x w^T, bound) for fp32 x.

    One token: fp32 multiply-adds, one rounding (u) each, at most k + k/32 on
    the way of a term.  More: x is the exact sum of three parts of its sign,
    the products of the parts are exact, and a product passes fewer than k
    additions in the matrix core (2u each, truncation) and k/256 + 2 outside
    it.  Both are within gamma_{2 (k + k/32)} sum |x w|."""
    k = x.shape[1]
    t = 2 * (k + k // 32) * U
    g = t / (1 - t) + k * 2.0 ** -53
    x = x.astype(np.float64)
    return x @ w.T, g * (np.abs(x) @ np.abs(w).T)


def gated(gate, up):
    """(silu(g) u, bound) from two products (value, bound).

    silu's kernel: e = exp2(RN(-g log2 e)): the argument errs by 2u relative
    (constant and product), so e by 2 u |g| relative, the exponential, the
    addition, the reciprocal and the two products by 1, 1/2, 1, 1/2 and 1/2 ulp
    (an ulp is at most 2u): together under (2 |g| + 9) u relative.  The errors of g and u come
    on top (|silu'| < 1.1).  Where e^-g overflows the kernel gives -0 for a
    value below 1e-34."""
    (g, bg), (u, bu) = gate, up
    with np.errstate(over="ignore"):
        s = g / (1 + np.exp(-g))
    h = s * u
    return h, np.abs(h) * (2 * np.abs(g) + 9) * U + 1.1 * bg * (np.abs(u) + bu) + np.abs(s) * bu + 1e-34 * np.abs(u)
