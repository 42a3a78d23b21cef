"""Oracle: pages and slots of a step, attention of one token over the cache,
page bounds and the choice of pages by them.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Pages, slots and choices are Python and numpy integers, one sequence and page
at a time.  Attention is float64 over the values that ``kv_cache.read_row``
gives, one sequence and head at a time, with the error bound of the kernels.
"""
from __future__ import annotations

import numpy as np

from . import e4m3, kv_cache, mxfp4

U = 2.0 ** -24
TINY = np.float32(2.0 ** -100)


def plan(lens, keep, offsets, tokens, page_len, table, free, count):
    """(slots, lens_out, count_out); table and free are updated in place."""
    seqs, width = table.shape
    stack, falls = [int(x) for x in free[:count]], any(offsets[b + 1] < offsets[b] for b in range(seqs))
    rows = []
    for b in range(seqs):
        new = int(offsets[b + 1]) - int(offsets[b])
        held, need = -(-int(lens[b]) // page_len), -(-(int(keep[b]) + new) // page_len)
        ok = 0 <= keep[b] <= lens[b] and not falls and held <= width and need <= width and int(keep[b]) + new < 2 ** 31
        rows.append((ok, held, need, new))
        if ok:
            stack += [int(x) for x in table[b, need:held]]
    free[:len(stack)] = stack
    lens_out, slots, short = np.array(lens, dtype=np.int32), np.full(tokens, -1, dtype=np.int64), False
    for b, (ok, held, need, new) in enumerate(rows):
        if ok and need > held:
            short = short or need - held > len(stack)
            ok = not short
        if not ok:
            continue
        for j in range(held, need):
            table[b, j] = stack.pop()
        lens_out[b] = keep[b] + new
        for t in range(max(int(offsets[b]), 0), min(int(offsets[b + 1]), tokens)):
            page, at = divmod(int(keep[b]) + t - int(offsets[b]), page_len)
            slots[t] = int(table[b, page]) * page_len + at
    return slots, lens_out, np.array([len(stack)], dtype=np.int32)


def values(fmt: int, codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """Every row of a cache as kv_cache.read_row gives it, fp32 [slots][heads][dim]."""
    with np.errstate(all="ignore"):
        if fmt == kv_cache.E4M3:
            return (e4m3.decode(codes).astype(np.float32) * scales[..., None]).astype(np.float32)
        c = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)
        return mxfp4.dequant(c, scales).astype(np.float32)


def slots_of(b, h, n, page_len, table, num_slots, pages=None):
    """The slots that (sequence b of n tokens, key head h) attends."""
    cols = range(-(-max(n, 0) // page_len)) if pages is None else pages[b, h]
    out = []
    for p in cols:
        if not 0 <= p < table.shape[1] or table[b, p] < 0:
            continue
        for at in range(page_len):
            s = int(table[b, p]) * page_len + at
            if int(p) * page_len + at < n and s < num_slots:
                out.append(s)
    return out


def attention(k, v, q, page_len, table, lens, scale, pages=None, blocks=False):
    """(out [seqs][q_heads][dim], lse [seqs][q_heads], bound of out, bound of
    lse) in float64, for the caches' values k and v (values()).

    The kernels' errors, u = 2^-24.  q and the weights are held as two fp16
    parts, the second the first's rounding, rounded: 2^-11 of 2^-11, 4 u in all,
    where neither is subnormal.  Subnormal parts err by 2^-25 at most: q is
    scaled so that its largest magnitude is at least 2^14, hence 2^-39 of it;
    a weight w <= 1 is taken times 2^14 times its row's scale over a power of
    two at most twice the largest scale that it is summed with, hence 2^-38 of
    the largest value (in a row as it is written the largest code is the
    format's; one of zeros has E4M3's scale of 1 or MXFP4's least one, and the
    first counts as none).  That power stays outside the exponential.  A score is a sum
    of 2 dim exact products and as many additions of 2 u each (truncation),
    with a row's scale (2 u: as read, and as multiplied) and q's product with
    the rounded scale log2(e) (3 u): it errs by at most gamma_{4 dim + 10}, and
    so gamma_{8 dim}, times sum |scale q k|.  Its way back from powers of two is
    exact; the exponential's argument, its difference to the largest one so
    far, is rounded, and so is every later difference of maxima up to the last
    join's, together at most 2 max |s| (u |s|, with log2(e) twice more; 4 |s|
    bounds it).  The exponential errs by 1 ulp, and a weight's scale and parts by
    6 u: e covers them as a weight's relative error.  Weights and their sum
    pass at most 3 additions and 1 rescaling (2 u each) a position and 64 in
    the joins: gamma_{8 n + 64}.  Numerator and denominator each err by
    (e^e - 1) <= 1.25 e.

    `blocks` (MXFP4): a row is held relative to its largest block's scale X, as
    fp16 whose least step is 2^-24.  A block 2^-23 X or more is exact, a smaller
    one's values err by half a step, 2^-25 X.  The row's largest magnitude is at
    least 4 X (a written block's largest lies in [4, 8) of its scale): 2^-27 of
    it, for a key times every |scale q|, for a value its weight."""
    seqs, heads_q, dim = q.shape
    heads = k.shape[1]
    group = heads_q // heads
    out, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    tol, ltol = np.zeros(q.shape), np.zeros(q.shape[:2])
    gamma = lambda t: t * U / (1 - t * U)  # noqa: E731
    for b in range(seqs):
        for h in range(heads):
            at = slots_of(b, h, int(lens[b]), page_len, table, k.shape[0], pages)
            if not at:
                continue
            kk, vv = k[at, h].astype(np.float64), v[at, h].astype(np.float64)
            for g in range(h * group, (h + 1) * group):
                x = q[b, g].astype(np.float64) * scale
                with np.errstate(all="ignore"):
                    s = kk @ x
                    top = s.max()
                    if top == -np.inf:
                        continue
                    w = np.exp(s - top)
                    lse[b, g] = top + np.log(w.sum())
                    w /= w.sum()
                    out[b, g] = w @ vv
                    far = np.max(np.abs(s)[np.isfinite(s)], initial=0.0)
                    e = gamma(8 * dim) * (np.abs(kk) @ np.abs(x)).max() + 2.0 ** -39 * np.abs(x).max() * np.abs(kk).sum(1).max() + (4 * far + 12) * U
                    if blocks:
                        e += 2.0 ** -27 * np.abs(kk).max() * np.abs(x).sum()
                        tol[b, g] += 2.0 ** -27 * (w @ np.abs(vv).max(1))
                    tol[b, g] += (2.5 * e + gamma(8 * len(at) + 64)) * (w @ np.abs(vv)) + len(at) * 2.0 ** -38 * np.abs(vv).max()
                    ltol[b, g] = 1.25 * e + gamma(8 * len(at) + 64) + 4 * U * abs(lse[b, g])
    return out, lse, tol, ltol


def sized(a) -> np.float32:
    return np.float32(a) if a >= TINY else np.float32(1)


def bounds(k, slots, page_len, codes, scales):
    """Update codes [pages][heads][2][dim] and scales [pages][heads] for the pages of `slots` (k: values())."""
    last = {}
    for s in slots:
        if 0 <= s < k.shape[0]:
            last[int(s) // page_len] = max(last.get(int(s) // page_len, 0), int(s) % page_len)
    for p, n in last.items():
        if p >= codes.shape[0]:
            continue
        for h in range(k.shape[1]):
            x = k[p * page_len:p * page_len + n + 1, h]
            if not np.isfinite(x).all():
                codes[p, h, 0], codes[p, h, 1], scales[p, h] = 127, -127, np.inf
                continue
            a = sized(np.abs(x).max())
            inv = np.float32(127) / a
            codes[p, h, 0] = np.clip(np.ceil(x.max(0) * inv), -127, 127)
            codes[p, h, 1] = np.clip(np.floor(x.min(0) * inv), -127, 127)
            scales[p, h] = a / np.float32(127)


def scores(q, codes, scales):
    """fp32 [n] scores of pages with bounds codes [n][2][dim] and scales [n] for the group's queries [group][dim]."""
    best = np.full(len(scales), -np.inf, dtype=np.float32)
    c = codes.astype(np.int64)
    with np.errstate(all="ignore"):
        for row in q.astype(np.float32):
            a = sized(np.max(np.abs(row)[~np.isnan(row)], initial=0.0))
            x = row * (np.float32(127) / a)
            n = np.clip(np.rint(np.where(np.isnan(x), 0, x)), -127, 127).astype(np.int64)
            dots = np.maximum(n * c[:, 0], n * c[:, 1]).sum(1)
            s = dots.astype(np.float32) * scales * (a / np.float32(127))
            best = np.maximum(best, np.where(np.isnan(s), np.float32(np.inf), s))
    return best


def select(q, codes, scales, page_len, table, lens, budget):
    """int32 [seqs][heads][budget]."""
    seqs, width = table.shape
    heads = codes.shape[1]
    group = q.shape[1] // heads
    out = np.full((seqs, heads, budget), -1, dtype=np.int32)
    for b in range(seqs):
        n = min(-(-max(int(lens[b]), 0) // page_len), width)
        cols = np.array([p for p in range(n) if 0 <= table[b, p] < codes.shape[0]], dtype=np.int64)
        for h in range(heads if len(cols) else 0):
            at = table[b, cols]
            s = scores(q[b, h * group:(h + 1) * group], codes[at, h], scales[at, h])
            ends = (cols == 0) | (cols == n - 1)
            take = sorted(cols[np.lexsort((cols, np.where(ends, 0, -s), ~ends))[:budget]])
            out[b, h, :len(take)] = take
    return out
