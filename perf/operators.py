"""Measured cases of the MXFP4 operators and of the quantised key/value cache.

MXFP4 (the OCP microscaling format): a row's values in blocks of 32, each
block a shared power of two X = 2^(byte - 127) and 32 E2M1 codes.

    a = max |x| of the block, byte = max(floor(log2 a) - 2 + 127, 0),
    code = x / X to the nearest of +-{0, .5, 1, 1.5, 2, 3, 4, 6}, ties to the
    even code, saturating at 6.

A tensor [rows][k] is kept in tiles, rows padded to a multiple of 32 with zero
codes and scales: codes [rows/32][k/64][2][32][16 bytes] (64-column slab, its
half of 32 columns, row, that row's block with the even element in the low
nibble), scales [rows/32][k/256][2][32][4] (256-column slab, half, row, the
four 64-column slabs).

The sizes are those of the repository's workloads: K = 3584, N = 18944 (gate
and up), 3584 (down, K = 18944), 512 (keys and values: 4 heads of 128),
4608 (small batches), at 1 to 4096 tokens.
"""
import math

import numpy as np
import torch

own = False  # False: the plain forms; True: the library's entry points

Q4_K, Q6_K = 12, 14
E4M3, MXFP4 = 0, 1
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the attention input of a small odd batch, quantised for one layer's products
        {"name": "quant_tokens", "op": "quant", "m": 37, "k": 3584},
        # the down projection's input at prefill
        {"name": "quant_prefill", "op": "quant", "m": 2048, "k": 18944},
        # a gate weight converted once when a model is loaded
        {"name": "pack_gate", "op": "pack", "qtype": Q4_K, "n": 18944, "k": 3584},
        # a small serving batch through a fused projection
        {"name": "gemm_batch", "op": "gemm", "m": 37, "n": 4608, "k": 3584},
        # the key projection of a prompt of odd length
        {"name": "gemm_keys", "op": "gemm", "m": 509, "n": 512, "k": 3584},
        # the down projection at prefill
        {"name": "gemm_down", "op": "gemm", "m": 2048, "n": 3584, "k": 18944},
        # one token through the same projection as gemm_batch, its input not quantised
        {"name": "gemv_token", "op": "gemv", "m": 1, "n": 4608, "k": 3584},
        # the gate and up projections with the activation between them, one token and prefill
        {"name": "gated_token", "op": "gated_gemv", "m": 1, "n": 18944, "k": 3584},
        {"name": "gated_prefill", "op": "gated", "m": 2048, "n": 18944, "k": 3584},
        # one decoding step of 64 sequences: a row each into the paged cache
        {"name": "cache_step", "op": "kv_write", "fmt": E4M3, "tokens": 64, "heads": 4, "dim": 128, "page": 16},
        # a prompt written to the cache in 4 bits and read back for its attention
        {"name": "cache_prompt", "op": "kv_both", "fmt": MXFP4, "tokens": 4096, "heads": 4, "dim": 128, "page": 64},
        # a ragged batch with long contexts read back
        {"name": "cache_context", "op": "kv_read", "fmt": E4M3, "tokens": 131072, "seqs": 24, "heads": 4, "dim": 128,
         "page": 16},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "pack", "gemm", "gemm", "gemv", "gated", "gated_gemv", "kv_write", "kv_both", "kv_read"])
    k = 256 * _log(rng, 1, 74)
    if op == "quant":
        return {"op": op, "m": _log(rng, 1, 2048), "k": k}
    if op == "pack":
        n = min(_log(rng, 16, 18944), 18944 * 3584 // k)
        return {"op": op, "qtype": rng.choice([Q4_K, Q6_K]), "n": n, "k": k}
    if op in ("gemm", "gated"):
        m, n = _log(rng, 1, 4096), _log(rng, 16, 18944)
        while m * n * k > 2048 * 18944 * 3584:
            m = (m + 1) // 2
        return {"op": op, "m": m, "n": n, "k": k}
    if op in ("gemv", "gated_gemv"):
        n = min(_log(rng, 16, 18944), 18944 * 3584 // k)
        return {"op": op, "m": rng.randint(1, 8), "n": n, "k": k}
    case = {"op": op, "fmt": rng.choice([E4M3, MXFP4]) if op != "kv_write" else E4M3,
            "heads": rng.randint(1, 8), "dim": rng.choice([64, 96, 128, 160, 192, 256]), "page": rng.choice([1, 7, 16, 48, 64, 128])}
    row = case["heads"] * case["dim"]
    if op == "kv_read":
        case["tokens"] = min(_log(rng, 1, 131072), 131072 * 512 // row)
        case["seqs"] = rng.randint(1, 32)
    else:
        case["tokens"] = min(_log(rng, 1, 4096), 4096 * 512 // row)
    return case


# ---------------------------------------------------------------- codecs

def _device():
    return torch.device("cuda")


def _pad32(rows):
    return (rows + 31) // 32 * 32


def _mx_values(x):
    """(codes' values as x / X rounded, X's byte) of the blocks of 32 along the last axis."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    a = b.abs().amax(-1)
    byte = (torch.frexp(a)[1] - 1 - 2 + 127).clamp(0, 254)
    byte = torch.where(a > 0, byte, torch.zeros_like(byte))
    v = torch.ldexp(b.double(), (127 - byte).unsqueeze(-1))  # exact: a power of two
    mag = v.abs()
    step = torch.where(mag < 2, 0.5, torch.where(mag < 4, 1.0, 2.0)).to(mag)
    mag = (torch.round(mag / step) * step).clamp(max=6.0)
    return torch.copysign(mag, v).float(), byte


def _mx_decode(vals, byte):
    return torch.ldexp(vals, byte.unsqueeze(-1) - 127).reshape(*byte.shape[:-1], byte.shape[-1] * 32)


def _mx_nibbles(vals):
    mag = vals.abs()
    idx = torch.where(mag < 2, mag * 2, torch.where(mag < 4, mag + 2, mag / 2 + 4)).to(torch.uint8)
    idx = torch.where(torch.signbit(vals), idx + 8, idx)
    return idx[..., 0::2] | (idx[..., 1::2] << 4)


def _mx_table():
    g = torch.tensor(GRID, device=_device())
    return torch.cat([g, -g])


def _nibble_values(by):
    t = _mx_table()
    i = by.to(torch.int64)
    return torch.stack([t[i & 15], t[i >> 4]], -1).flatten(-2)


def _tile(x):
    """An fp32 [rows][k] as tiled MXFP4 (codes, scales)."""
    rows, k = x.shape
    p = _pad32(rows)
    vals, byte = _mx_values(x)
    nib = torch.zeros(p, k // 32, 16, dtype=torch.uint8, device=x.device)
    nib[:rows] = _mx_nibbles(vals)
    sc = torch.zeros(p, k // 32, dtype=torch.uint8, device=x.device)
    sc[:rows] = byte.to(torch.uint8)
    codes = nib.view(p // 32, 32, k // 64, 2, 16).permute(0, 2, 3, 1, 4).contiguous().view(p // 32, k // 64, 1024)
    scales = sc.view(p // 32, 32, k // 256, 4, 2).permute(0, 2, 4, 1, 3).contiguous().view(p // 32, k // 256, 256)
    return codes, scales


def _untile(codes, scales, rows):
    """Tiled MXFP4 as its fp32 values [rows][k]."""
    g, slabs, _ = codes.shape
    k = slabs * 64
    nib = codes.view(g, slabs, 2, 32, 16).permute(0, 3, 1, 2, 4).reshape(g * 32, k // 32, 16)[:rows]
    sc = scales.view(g, k // 256, 2, 32, 4).permute(0, 3, 1, 4, 2).reshape(g * 32, k // 32)[:rows]
    return _mx_decode(_nibble_values(nib), sc.to(torch.int32))


def _e4m3(x):
    """The library's E4M3 conversion of rows: (float8 codes, fp32 scale a'/448) with q = 448/a',
    |x q| < 2^-6 to zero, nearest even, at most 448."""
    a = x.abs().amax(-1)
    a = torch.where(a == 0, torch.ones_like(a), a)
    y = x * (448.0 / a).unsqueeze(-1)
    e = torch.frexp(y.abs())[1] - 1
    r = torch.ldexp(torch.round(torch.ldexp(y, 3 - e)), e - 3).clamp(-448.0, 448.0)
    r = torch.where(y.abs() < 2.0 ** -6, torch.zeros_like(r), r)
    return r.to(torch.float8_e4m3fn), a / 448.0


def _q4k(b):
    """fp32 values [blocks][256] of Q4_K super-blocks [blocks][144]."""
    d = b[:, 0:2].contiguous().view(torch.float16).double()
    dmin = b[:, 2:4].contiguous().view(torch.float16).double()
    s = b[:, 4:16].to(torch.int32)
    lo, mid, hi = s[:, 0:4], s[:, 4:8], s[:, 8:12]
    sc = torch.cat([lo & 63, (hi & 15) | (lo >> 6 << 4)], 1).double()
    mn = torch.cat([mid & 63, (hi >> 4) | (mid >> 6 << 4)], 1).double()
    qs = b[:, 16:144].view(-1, 4, 32)
    q = torch.stack([qs & 15, qs >> 4], 2).view(-1, 8, 32).double()
    return ((d * sc).unsqueeze(-1) * q - (dmin * mn).unsqueeze(-1)).float().view(-1, 256)


def _q6k(b):
    """fp32 values [blocks][256] of Q6_K super-blocks [blocks][210]."""
    d = b[:, 208:210].contiguous().view(torch.float16).double()
    ql = b[:, 0:128].reshape(-1, 2, 2, 32).to(torch.int32)
    qh = b[:, 128:192].reshape(-1, 2, 1, 32).to(torch.int32)
    low = torch.cat([ql & 15, ql >> 4], 2)  # [blocks][half][part][32]
    shift = torch.tensor([0, 2, 4, 6], device=b.device, dtype=torch.int32).view(1, 1, 4, 1)
    q = (low | ((qh >> shift & 3) << 4)) - 32
    sc = b[:, 192:208].contiguous().view(torch.int8).double().view(-1, 2, 4, 2, 1)
    return (d.view(-1, 1, 1, 1, 1) * sc * q.view(-1, 2, 4, 2, 16).double()).float().view(-1, 256)


# ---------------------------------------------------------------- inputs

def _blocks(g, qtype, nb):
    """Random K-quant super-blocks: f16 scales uniform in [1e-3, 2e-2], uniform bytes elsewhere."""
    size, at = (144, (0, 2)) if qtype == Q4_K else (210, (208,))
    b = torch.randint(0, 256, (nb, size), dtype=torch.uint8, device=_device(), generator=g)
    for o in at:
        d = torch.rand(nb, 1, device=_device(), generator=g) * 0.019 + 0.001
        b[:, o:o + 2] = d.half().view(torch.uint8)
    return b


def _normal(g, *shape):
    return torch.randn(*shape, device=_device(), generator=g)


def _activation(g, m, k):
    """N(0, 1) tokens with a few strong channels, as activations have."""
    x = _normal(g, m, k)
    hot = torch.randperm(k, device=_device(), generator=g)[:8]
    x[:, hot] *= 20.0
    return x


def prepare(case, seed):
    g = torch.Generator(device=_device())
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "quant":
        m, k = case["m"], case["k"]
        s["x"] = _activation(g, m, k)
        if k == 18944:  # a down projection's input
            s["x"] = torch.nn.functional.silu(_normal(g, m, k)) * _normal(g, m, k)
    elif op == "pack":
        s["blocks"] = _blocks(g, case["qtype"], case["n"] * (case["k"] // 256))
    elif op in ("gemm", "gated"):
        m, n, k = case["m"], case["n"], case["k"]
        s["a"] = _tile(_activation(g, m, k))
        s["w"] = _tile(_normal(g, n, k) * 0.02)
        if op == "gated":
            s["u"] = _tile(_normal(g, n, k) * 0.02)
    elif op in ("gemv", "gated_gemv"):
        m, n, k = case["m"], case["n"], case["k"]
        s["x"] = _activation(g, m, k)
        s["w"] = _tile(_normal(g, n, k) * 0.02)
        if op == "gated_gemv":
            s["u"] = _tile(_normal(g, n, k) * 0.02)
    else:
        _prepare_cache(case, g, seed, s)
    return s


def _prepare_cache(case, g, seed, s):
    """A paged cache in use and, for writes, new rows: k and v as column ranges of one fused
    projection's output, so their rows are strided."""
    dev = _device()
    t, h, d, page = case["tokens"], case["heads"], case["dim"], case["page"]
    r = np.random.RandomState(seed % (1 << 31))
    seqs = min(case.get("seqs", 1), t)
    if case["op"] == "kv_write":  # a row for each sequence, anywhere in its last page
        seqs, ends = t, np.arange(t + 1)
        pages = t + 8
    else:
        cuts = np.sort(r.choice(np.arange(1, t), seqs - 1, replace=False)) if seqs > 1 else np.zeros(0, np.int64)
        ends = np.concatenate([[0], cuts, [t]])
        pages = int(np.sum(-(-np.diff(ends) // page))) + 8
    order = r.permutation(pages)
    s["pages"] = pages
    if case["op"] == "kv_write":
        s["slots"] = torch.from_numpy(order[:t].astype(np.int64) * page + r.randint(0, page, t)).to(dev)
    else:
        lens = np.diff(ends)
        need = -(-lens // page)
        table = np.zeros((seqs, int(need.max())), np.int32)
        at = np.concatenate([[0], np.cumsum(need)])
        for b in range(seqs):
            table[b, :need[b]] = order[at[b]:at[b + 1]]
        s["table"] = torch.from_numpy(table).to(dev)
        s["offsets"] = torch.from_numpy(ends.astype(np.int32)).to(dev)
        if case["op"] == "kv_both":
            pos = np.arange(t)
            s["slots"] = torch.from_numpy(table[0, pos // page].astype(np.int64) * page + pos % page).to(dev)
    n = pages * page
    for c in ("k", "v"):
        if case["fmt"] == E4M3:
            old = (_normal(g, n, h, d) * 100).clamp(-440, 440)
            s[c + "_codes"] = torch.where(old.abs() < 2.0 ** -6, torch.zeros_like(old), old).to(torch.float8_e4m3fn).view(torch.uint8)
            s[c + "_scales"] = torch.rand(n, h, device=dev, generator=g) * 0.01 + 0.005
        else:
            vals, byte = _mx_values(_normal(g, n, h, d))
            s[c + "_codes"] = _mx_nibbles(vals).reshape(n, h, d // 2)
            s[c + "_scales"] = byte.to(torch.uint8)
    if case["op"] != "kv_read":
        qkv = _normal(g, t, 3 * h * d)
        s["k"] = qkv[:, h * d:2 * h * d].view(t, h, d)
        s["v"] = qkv[:, 2 * h * d:].view(t, h, d)


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    return (_run_own if own else _run_plain)(case, s)


def _run_plain(case, s):
    op = case["op"]
    if op == "quant":
        return _mx_decode(*_mx_values(s["x"])).to(torch.bfloat16)
    if op == "pack":
        w = (_q4k if case["qtype"] == Q4_K else _q6k)(s["blocks"]).view(case["n"], case["k"])
        return _mx_decode(*_mx_values(w)).to(torch.bfloat16)
    if op in ("gemm", "gated", "gemv", "gated_gemv"):
        x = _untile(*s["a"], case["m"]) if "a" in s else s["x"]
        y = x @ _untile(*s["w"], case["n"]).t()
        if "u" in s:
            y = y / (1 + torch.exp(-y)) * (x @ _untile(*s["u"], case["n"]).t())
        return y
    out = {}
    if "slots" in s:
        for c in ("k", "v"):
            if case["fmt"] == E4M3:
                codes, scale = _e4m3(s[c])
                s[c + "_codes"][s["slots"]] = codes.view(torch.uint8)
                s[c + "_scales"][s["slots"]] = scale
            else:
                vals, byte = _mx_values(s[c])
                s[c + "_codes"][s["slots"]] = _mx_nibbles(vals).reshape(case["tokens"], case["heads"], case["dim"] // 2)
                s[c + "_scales"][s["slots"]] = byte.to(torch.uint8)
    if op == "kv_write":
        return _cache_state(s)
    row = torch.arange(case["tokens"], device=_device())
    seq = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    pos = row - s["offsets"].long()[seq]
    slot = s["table"][seq, pos // case["page"]].long() * case["page"] + pos % case["page"]
    for c in ("k", "v"):
        codes, scale = s[c + "_codes"][slot], s[c + "_scales"][slot]
        if case["fmt"] == E4M3:
            x = codes.view(torch.float8_e4m3fn).float() * scale.unsqueeze(-1)
        else:
            x = _mx_decode(_nibble_values(codes).view(case["tokens"], case["heads"], -1, 32), scale.to(torch.int32))
        out[c] = x.to(torch.bfloat16)
    return out


def _cache_state(s):
    """The cache after a write, as the values it holds."""
    return {"k": s["k_codes"].view(torch.float8_e4m3fn), "ks": s["k_scales"],
            "v": s["v_codes"].view(torch.float8_e4m3fn), "vs": s["v_scales"]}


def _run_own(case, s):
    import fp8_prefill_gemm_amd as rz
    op = case["op"]
    if op == "quant":
        codes, scales = rz.rz_mxfp4_quant(s["x"])
        return rz.rz_mxfp4_dequant(codes, scales, case["m"], dtype=torch.bfloat16)
    if op == "pack":
        codes, scales = rz.rz_mxfp4_pack_weight(case["qtype"], s["blocks"], case["n"], case["k"])
        return rz.rz_mxfp4_dequant(codes, scales, case["n"], dtype=torch.bfloat16)
    if op == "gemm":
        return rz.rz_mxfp4_gemm(*s["a"], case["m"], *s["w"], case["n"])
    if op == "gated":
        return rz.rz_mxfp4_gated(*s["a"], case["m"], s["w"], s["u"], case["n"])
    if op == "gemv":
        return rz.rz_mxfp4_gemv(*s["w"], case["n"], s["x"])
    if op == "gated_gemv":
        return rz.rz_mxfp4_gated_gemv(s["w"], s["u"], case["n"], s["x"])
    fmt = rz.KV_E4M3 if case["fmt"] == E4M3 else rz.KV_MXFP4
    cache = (s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
    if "slots" in s:
        rz.rz_kv_cache_write(fmt, s["k"], s["v"], s["slots"], *cache)
    if op == "kv_write":
        return _cache_state(s)
    k, v = rz.rz_kv_cache_read(fmt, *cache, case["page"], s["table"], s["offsets"], case["tokens"], dtype=torch.bfloat16)
    return {"k": k, "v": v}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    mx = 17 / 32  # bytes a value
    if op == "quant":
        return {"bytes": case["m"] * case["k"] * (4 + 2), "flops": 0}
    if op == "pack":
        n = case["n"] * case["k"]
        return {"bytes": n * ((144 if case["qtype"] == Q4_K else 210) / 256 + 2), "flops": 0}
    if op in ("gemm", "gated", "gemv", "gated_gemv"):
        m, n, k = case["m"], case["n"], case["k"]
        w = 2 if op.startswith("gated") else 1
        return {"bytes": w * n * k * mx + m * k * (4 if op.endswith("gemv") else mx) + 4 * m * n, "flops": 2.0 * w * m * n * k}
    t, h, d = case["tokens"], case["heads"], case["dim"]
    held = 2 * t * h * (d + 4 if case["fmt"] == E4M3 else d * mx)
    if op == "kv_write":
        return {"bytes": 2 * t * h * d * 4 + held, "flops": 0}
    if op == "kv_read":
        return {"bytes": held + 2 * t * h * d * 2, "flops": 0}
    return {"bytes": 2 * t * h * d * (4 + 2) + held, "flops": 0}


# ---------------------------------------------------------------- from the definitions, in 64 bits

def _nearest(x, grid):
    """x to the nearest of the ascending non-negative grid (ties to the even index), signs kept; in 64 bits."""
    mag = x.abs()
    hi = torch.searchsorted(grid, mag).clamp(1, len(grid) - 1)
    up, down = grid[hi], grid[hi - 1]
    take = (mag - down > up - mag) | ((mag - down == up - mag) & (hi % 2 == 0))
    return torch.where(take, up, down) * torch.sign(x)


def _exact_mx(x):
    b = x.double().reshape(-1, 32)
    a = b.abs().amax(1, keepdim=True)
    scale = torch.exp2(torch.floor(torch.log2(a.clamp(min=1e-45))) - 2)
    # log2 may be off by one next to a power of two
    scale = torch.where(scale * 8 <= a, scale * 2, torch.where(scale * 4 > a, scale / 2, scale))
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    return (_nearest(b / scale, grid) * scale).reshape(x.shape)


def _exact_weight(codes, scales, rows):
    """Tiled MXFP4 as 64-bit values, element by element from its place."""
    k = codes.shape[1] * 64
    grid = torch.tensor(GRID, dtype=torch.float64, device=codes.device)
    col = torch.arange(k, device=codes.device)
    sub = (col // 64) * 1024 + (col // 32 % 2) * 512 + col % 32 // 2
    at = (col // 256) * 256 + (col // 32 % 2) * 128 + col // 64 % 4
    out = torch.empty(rows, k, dtype=torch.float64, device=codes.device)
    for r0 in range(0, rows, 1024):
        r = torch.arange(r0, min(r0 + 1024, rows), device=codes.device).unsqueeze(1)
        byte = codes.view(-1)[(r // 32) * (k * 16) + sub + (r % 32) * 16].to(torch.int64)
        nib = byte >> (4 * (col % 2)) & 15
        e = scales.view(-1)[(r // 32) * k + at + (r % 32) * 4].double() - 127
        out[r0:r0 + 1024] = grid[nib & 7] * torch.where(nib > 7, -1.0, 1.0) * torch.exp2(e)
    return out


def _exact_kquant(qtype, blocks):
    """Super-blocks' values, a column at a time from the format's fields, rounded to fp32."""
    b = blocks.to(torch.int64)
    f16 = lambda o: blocks[:, o:o + 2].contiguous().view(torch.float16)[:, 0].double()  # noqa: E731
    out = torch.empty(b.shape[0], 256, dtype=torch.float32, device=b.device)
    for i in range(256):
        if qtype == Q4_K:
            j = i // 32
            q = b[:, 16 + 32 * (i // 64) + i % 32] >> (4 * (j % 2)) & 15
            if j < 4:
                sc, mn = b[:, 4 + j] & 63, b[:, 8 + j] & 63
            else:
                sc = b[:, 8 + j] & 15 | b[:, j] >> 6 << 4
                mn = b[:, 8 + j] >> 4 | b[:, 4 + j] >> 6 << 4
            out[:, i] = (f16(0) * (sc * q) - f16(2) * mn).float()
        else:
            half, p, l = i // 128, i % 128 // 32, i % 32
            low = b[:, 64 * half + l + 32 * (p & 1)] >> (4 * (p >> 1)) & 15
            q = (low | (b[:, 128 + 32 * half + l] >> (2 * p) & 3) << 4) - 32
            sc = b[:, 192 + 8 * half + l // 16 + 2 * p]
            sc = torch.where(sc > 127, sc - 256, sc)
            out[:, i] = (f16(208) * (sc * q)).float()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        return _exact_mx(s["x"])
    if op == "pack":
        return _exact_mx(_exact_kquant(case["qtype"], s["blocks"]).view(case["n"], case["k"]))
    if op in ("gemm", "gated", "gemv", "gated_gemv"):
        x = _exact_weight(*s["a"], case["m"]) if "a" in s else s["x"].double()
        y = x @ _exact_weight(*s["w"], case["n"]).t()
        if "u" in s:
            y = y * torch.sigmoid(y) * (x @ _exact_weight(*s["u"], case["n"]).t())
        return y
    grid8 = torch.tensor([0.0] + [2.0 ** e * (1 + f / 8) for e in range(-6, 9) for f in range(8) if not (e == 8 and f == 7)],
                         dtype=torch.float64, device=_device())

    def held(c, at):
        """What cache c holds in the slots `at`, rows of 64-bit values."""
        codes, scale = s[c + "_codes"][at], s[c + "_scales"][at]
        if case["fmt"] == E4M3:
            v = codes.to(torch.int64)
            e, f = (v >> 3 & 15).double(), (v & 7).double()
            mag = torch.where(e > 0, torch.exp2(e - 7) * (1 + f / 8), torch.exp2(torch.tensor(-9.0, dtype=torch.float64, device=v.device)) * f)
            return torch.where(v > 127, -mag, mag), scale.double()
        grid = torch.tensor(GRID, dtype=torch.float64, device=codes.device)
        both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int64)
        x = grid[both & 7] * torch.where(both > 7, -1.0, 1.0)
        return x * torch.exp2(scale.double() - 127).repeat_interleave(32, -1), None

    def fresh(c):
        """Rows of c as E4M3 holds them; scale and product rounded to fp32 as the format says."""
        a = s[c].abs().amax(-1)
        a = torch.where(a == 0, torch.ones_like(a), a).double()
        y = (s[c].double() * (448 / a).float().double().unsqueeze(-1)).float().double()
        # the grid's index of 2^-6 is 1 and its codes' lowest bits are those of index - 1
        v = torch.where(y.abs() < 2.0 ** -6, torch.zeros_like(y), _nearest_from(y, grid8))
        return v, (a / 448).float().double()

    def _nearest_from(y, grid):
        mag = y.abs()
        hi = torch.searchsorted(grid, mag).clamp(1, len(grid) - 1)
        up, down = grid[hi], grid[hi - 1]
        take = (mag - down > up - mag) | ((mag - down == up - mag) & ((hi - 1) % 2 == 0))
        return torch.where(take, up, down) * torch.sign(y)

    if op == "kv_write":
        out = {}
        every = torch.arange(s["pages"] * case["page"], device=_device())
        for c in ("k", "v"):
            v, scale = held(c, every)
            v[s["slots"]], scale[s["slots"]] = fresh(c)
            out[c], out[c + "s"] = v, scale
        return out
    if op == "kv_both":
        if case["fmt"] == MXFP4:
            return {c: _exact_mx(s[c].contiguous()) for c in ("k", "v")}
        return {c: v * scale.unsqueeze(-1) for c in ("k", "v") for v, scale in [fresh(c)]}
    off, table, page = s["offsets"].tolist(), s["table"].long(), case["page"]
    slots = []
    for b in range(len(off) - 1):
        p = torch.arange(off[b + 1] - off[b], device=_device())
        slots.append(table[b, p // page] * page + p % page)
    slots = torch.cat(slots)
    out = {}
    for c in ("k", "v"):
        v, scale = held(c, slots)
        out[c] = v if scale is None else v * scale.unsqueeze(-1)
    return out
