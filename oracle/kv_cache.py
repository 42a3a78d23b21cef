"""Oracle: the quantised key/value cache, written and read back.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

A row (one token, one head) is quantised by itself: E4M3 as the activation
conversion does with the row's own absmax (``fp8_path``, ``e4m3``), or MXFP4
(``mxfp4``).
"""
from __future__ import annotations

import numpy as np

from . import e4m3, fp8_path, mxfp4

E4M3, MXFP4 = 0, 1


def empty(fmt: int, slots: int, heads: int, dim: int, fill=0):
    """(codes, scales) of a cache with every byte `fill`."""
    codes = np.full((slots, heads, dim if fmt == E4M3 else dim // 2), fill, dtype=np.uint8)
    if fmt == E4M3:
        return codes, np.full((slots, heads, 4), fill, dtype=np.uint8).view(np.float32)[..., 0]
    return codes, np.full((slots, heads, dim // 32), fill, dtype=np.uint8)


def quant_row(fmt: int, x: np.ndarray):
    if fmt == MXFP4:
        c, b = mxfp4.quant(x)
        return c[0::2] | (c[1::2] << 4), b
    q, dq = fp8_path.scales_from_absmax(fp8_path.absmax(x))
    return e4m3.encode_scaled(x, q), dq


def write(fmt: int, x: np.ndarray, slots: np.ndarray, codes: np.ndarray, scales: np.ndarray) -> None:
    """x fp32 [tokens][heads][dim] into the rows `slots`, in place."""
    for t, s in enumerate(slots):
        if not 0 <= s < codes.shape[0]:
            continue
        for h in range(x.shape[1]):
            codes[s, h], scales[s, h] = quant_row(fmt, x[t, h])


def read_row(fmt: int, codes: np.ndarray, scales) -> np.ndarray:
    """fp32 values of one row."""
    if fmt == MXFP4:
        c = np.empty(codes.size * 2, dtype=np.uint8)
        c[0::2], c[1::2] = codes & 15, codes >> 4
        return mxfp4.dequant(c, scales).astype(np.float32)
    with np.errstate(all="ignore"):
        return (e4m3.decode(codes).astype(np.float32) * np.float32(scales)).astype(np.float32)


def read(fmt: int, codes, scales, page_len: int, table, offsets, out: np.ndarray) -> None:
    """Sequences into out fp32 [rows][heads][dim], in place."""
    for b in range(len(offsets) - 1):
        for row in range(offsets[b], min(offsets[b + 1], out.shape[0])):
            page, at = divmod(int(row) - int(offsets[b]), page_len)
            s = int(table[b, page]) * page_len + at if page < table.shape[1] and table[b, page] >= 0 else -1
            for h in range(out.shape[1]):
                out[row, h] = read_row(fmt, codes[s, h], scales[s, h]) if 0 <= s < codes.shape[0] else 0.0
