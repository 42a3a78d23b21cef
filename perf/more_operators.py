"""Measured cases of serving from the quantised, paged key/value cache.

A cache row is one head of one token. E4M3: codes [slot][head][dim] and an
fp32 scale a row, a value is code * scale. MXFP4: E2M1 codes
[slot][head][dim/2] (even element in the low nibble) and a scale byte for each
32 values, 2^(byte - 127). Position p of sequence b is slot
table[b][p / page] * page + p % page.

plan     pages and slots of a step. Sequence b holds lens[b] tokens, keeps
         keep[b] of them and adds offsets[b+1] - offsets[b]. Pages that it no
         longer needs go onto the stack free[0 .. count), in order of sequence
         and page; then pages that it lacks come from the stack's top, in the
         same order. A sequence is refused (left as it was, its tokens without
         a slot) where keep is not in [0, lens], where it needs more pages than
         the table has columns, and from the first one on that the stack cannot
         serve, if it lacks pages itself.
attend   out[b][h] = sum_p w_p v_p, w = softmax(scale q[b][h] . k_p) over the
         positions p < lens[b], or over those of them that lie in the pages
         chosen for (b, key head); query head h reads key head h / group. lse =
         log sum exp of the scores. An empty sequence gives zeros and -inf.
bounds   of each page that `slots` names and each head: the largest and the
         smallest value of each column over the page's filled rows (those up
         to the last slot named), as whole numbers of scale = a / 127, a the
         largest magnitude (1 where it is under 2^-100): ceil(hi * (127 / a))
         and floor(lo * (127 / a)), at most 127 in size.
select   the `budget` pages of the highest score for each sequence and key
         head, ascending, -1 behind the last. With the query as whole numbers
         n_d = rint(q_d * (127 / a)) of qs = a / 127, a page's score is the
         largest over the group's queries of (sum_d max(n_d hi_d, n_d lo_d)) *
         scale * qs; the first and the last page are always taken, ties go to
         the lower page.

Sizes: 28 query heads over 4 key/value heads of 128 (projections of 3584 and
512), as in the repository's workloads, and other layouts around them.
"""
import math

import numpy as np
import torch

own = False  # False: the plain forms; True: the library's entry points

E4M3, MXFP4 = 0, 1
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TINY = 2.0 ** -100


def listed():
    return [
        # one decoding step of 64 sequences: a token each, some at a page's border, some just ended or started
        {"name": "plan_step", "op": "plan", "seqs": 64, "new": 64, "context": 65536, "page": 16},
        # prompts of a ragged batch admitted while others go on
        {"name": "plan_prompts", "op": "plan", "seqs": 96, "new": 131072, "context": 131072, "page": 16},
        # the first tokens of one short chat
        {"name": "attend_one", "op": "attend", "fmt": E4M3, "seqs": 1, "tokens": 37, "heads": 4, "group": 7, "dim": 128, "page": 16,
         "type": "f32", "lse": False},
        # a serving batch of 64 ragged sequences
        {"name": "attend_batch", "op": "attend", "fmt": E4M3, "seqs": 64, "tokens": 65536, "heads": 4, "group": 7, "dim": 128,
         "page": 16, "type": "bf16", "lse": False},
        # one long document
        {"name": "attend_long", "op": "attend", "fmt": E4M3, "seqs": 1, "tokens": 131072, "heads": 4, "group": 7, "dim": 128,
         "page": 64, "type": "f32", "lse": True},
        # a 4-bit cache of long contexts, one key head in eight
        {"name": "attend_mx", "op": "attend", "fmt": MXFP4, "seqs": 24, "tokens": 131072, "heads": 4, "group": 8, "dim": 128,
         "page": 64, "type": "f32", "lse": False},
        # a head for each query, odd sizes throughout
        {"name": "attend_heads", "op": "attend", "fmt": MXFP4, "seqs": 13, "tokens": 5003, "heads": 5, "group": 1, "dim": 96,
         "page": 7, "type": "f16", "lse": True},
        # the pages' bounds after a decoding step, and after a prompt
        {"name": "bounds_step", "op": "bounds", "fmt": E4M3, "seqs": 64, "new": 64, "heads": 4, "dim": 128, "page": 64},
        {"name": "bounds_prompt", "op": "bounds", "fmt": MXFP4, "seqs": 3, "new": 32768, "heads": 4, "dim": 128, "page": 32},
        # which pages of a batch a step reads
        {"name": "select_batch", "op": "select", "seqs": 32, "tokens": 262144, "heads": 4, "group": 7, "dim": 128, "page": 32,
         "budget": 64},
        # a long document read by its best pages, alone and in a batch
        {"name": "sparse_long", "op": "sparse", "fmt": E4M3, "seqs": 1, "tokens": 131072, "heads": 4, "group": 7, "dim": 128,
         "page": 16, "budget": 128, "type": "f32"},
        {"name": "sparse_batch", "op": "sparse", "fmt": MXFP4, "seqs": 24, "tokens": 131072, "heads": 4, "group": 7, "dim": 128,
         "page": 64, "budget": 32, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "attend", "attend", "attend", "bounds", "select", "sparse", "sparse"])
    if op == "plan":
        seqs = _log(rng, 1, 1024)
        return {"op": op, "seqs": seqs, "new": _log(rng, 1, 131072), "context": _log(rng, seqs, 131072), "page": rng.choice([1, 7, 16, 48, 64, 128])}
    case = {"op": op, "heads": rng.randint(1, 8), "dim": rng.choice([64, 96, 128, 160, 192, 256])}
    most = 131072 * 512 // (case["heads"] * case["dim"])
    if op != "select":
        case["fmt"] = rng.choice([E4M3, MXFP4])
    if op == "bounds":
        case["page"] = rng.choice([8, 16, 24, 32, 64, 128])
        case["new"] = min(_log(rng, 1, 32768), most // 4)
        case["seqs"] = min(rng.randint(1, 64), case["new"])
        return case
    case["group"] = rng.randint(1, 16)
    case["tokens"] = min(_log(rng, 1, 131072), most)
    case["seqs"] = rng.randint(1, 64)
    case["page"] = rng.choice([1, 7, 16, 48, 64, 128]) if op == "attend" else rng.choice([16, 24, 32, 64, 128])
    if op != "attend":
        case["budget"] = min(_log(rng, 2, 256), max(2, -(-_longest(case["seqs"], case["tokens"]) // case["page"])))
    if op != "select":
        case["type"] = rng.choice(["f32", "f16", "bf16"])
    if op == "attend":
        case["lse"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------- inputs

def _device():
    return torch.device("cuda")


def _normal(g, *shape):
    return torch.randn(*shape, device=_device(), generator=g)


def _longest(seqs, tokens):
    """The most that one of `seqs` sequences of `tokens` in all holds: a table's width goes by it."""
    return min(tokens, 3 * -(-tokens // seqs) + 64)


def _lengths(r, seqs, tokens, least=0, idle=0.0):
    """Ragged lengths that sum to `tokens`, up to _longest() each, at least `least`; a share `idle` of them is nearly empty."""
    w = r.uniform(0.05, 1.0, seqs) ** 2 * np.where(r.rand(seqs) < idle, 1e-9, 1.0)
    n = np.floor(w / w.sum() * (tokens - least * seqs)).astype(np.int64) + least
    n = np.minimum(n, _longest(seqs, tokens))
    short = tokens - n.sum()
    for b in r.permutation(seqs):
        n[b] += min(short, _longest(seqs, tokens) - n[b])
        short = tokens - n.sum()
    return n


def _fill_cache(s, g, fmt, slots, heads, dim):
    """Rows as the cache's write leaves them, N(0, 1) with columns of their own sizes."""
    size = torch.exp(_normal(g, heads, dim) * 0.3)
    edges = torch.tensor([(a + b) / 2 for a, b in zip(GRID[:-1], GRID[1:])], device=_device())
    for c in ("k", "v"):
        x = _normal(g, slots, heads, dim) * size
        if fmt == E4M3:
            a = x.abs().amax(-1).clamp(min=1e-6)
            y = x * (448.0 / a).unsqueeze(-1)
            y = torch.where(y.abs() < 2.0 ** -6, torch.zeros_like(y), y)
            s[c + "_codes"], s[c + "_scales"] = y.to(torch.float8_e4m3fn).view(torch.uint8), a / 448.0
        else:
            b = x.view(slots, heads, dim // 32, 32)
            byte = (torch.frexp(b.abs().amax(-1))[1] - 3 + 127).clamp(0, 254)
            code = torch.bucketize(torch.ldexp(b.abs(), (127 - byte).unsqueeze(-1)), edges).to(torch.uint8)
            code = torch.where(b < 0, code + 8, code).view(slots, heads, dim)
            s[c + "_codes"], s[c + "_scales"] = code[..., 0::2] | (code[..., 1::2] << 4), byte.to(torch.uint8)


def _pages(s, r, lens, page, width, pages):
    """A page table of sequences of these lengths in a cache of `pages`, in any order; entries behind a sequence's pages name none."""
    need = -(-lens // page)
    order = r.permutation(pages).astype(np.int32)
    table = np.full((len(lens), width), -1, np.int32)
    at = np.concatenate([[0], np.cumsum(need)])
    for b in range(len(lens)):
        table[b, :need[b]] = order[at[b]:at[b + 1]]
    s["table"] = torch.from_numpy(table).to(_device())
    s["lens"] = torch.from_numpy(lens.astype(np.int32)).to(_device())
    return order[at[-1]:]


def _prepare_plan(case, r, s):
    dev, seqs, page = _device(), case["seqs"], case["page"]
    lens = _lengths(r, seqs, case["context"])
    keep = lens.copy()
    ended = r.rand(seqs) < 0.1
    keep[ended] = 0
    back = ~ended & (r.rand(seqs) < 0.1)  # the last tokens of a guess taken back
    keep[back] = np.maximum(keep[back] - r.randint(1, 8, int(back.sum())), 0)
    # a decoding step: a token each; or prompts
    new = np.ones(seqs, np.int64) if case["new"] == seqs else _lengths(r, seqs, case["new"], idle=0.2)
    lack = int(np.maximum(-(-(keep + new) // page) - -(-lens // page), 0).sum())
    width = -(-(_longest(seqs, case["context"]) + _longest(seqs, case["new"])) // page) + 1
    pages = (case["context"] + case["new"]) // page + 2 * seqs + 16
    rest = _pages(s, r, lens, page, width, pages)
    if r.rand() < 0.25:  # too few for all of them
        rest = rest[:max(1, lack * 3 // 4)]
    free = np.full(pages, -1, np.int32)
    free[:len(rest)] = rest
    for name, x in (("keep", keep), ("offsets", np.concatenate([[0], np.cumsum(new)])), ("free", free), ("count", np.array([len(rest)]))):
        s[name] = torch.from_numpy(x.astype(np.int32)).to(dev)


def _prepare_bounds(case, r, s):
    """Slots just written: the last tokens of sequences, and the cache that holds them."""
    new = _lengths(r, case["seqs"], case["new"], 1)
    if case["new"] == case["seqs"]:
        before = r.randint(0, 4 * case["page"], case["seqs"])
    else:
        before = np.where(r.rand(case["seqs"]) < 0.5, 0, r.randint(0, 2 * case["page"], case["seqs"]))
    width = -(-_longest(case["seqs"], case["new"]) // case["page"]) + 5
    pages = case["new"] // case["page"] + 6 * case["seqs"] + 8
    _pages(s, r, before + new, case["page"], width, pages)
    table, slots = s["table"].cpu().numpy(), []
    for b in range(case["seqs"]):
        p = np.arange(before[b], before[b] + new[b])
        slots.append(table[b, p // case["page"]].astype(np.int64) * case["page"] + p % case["page"])
    s["slots"] = torch.from_numpy(np.concatenate(slots)).to(_device())
    return pages


def prepare(case, seed):
    g = torch.Generator(device=_device())
    g.manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 31))
    op, s = case["op"], {"case": case}
    if op == "plan":
        _prepare_plan(case, r, s)
        return s
    page, heads, dim = case["page"], case["heads"], case["dim"]
    if op == "bounds":
        pages = _prepare_bounds(case, r, s)
    else:
        pages = case["tokens"] // page + case["seqs"] + 8
        _pages(s, r, _lengths(r, case["seqs"], case["tokens"]), page, -(-_longest(case["seqs"], case["tokens"]) // page), pages)
        qkv = _normal(g, case["seqs"], heads * (case["group"] + 2) * dim) * 1.5  # a fused projection's output
        s["q"] = qkv[:, :heads * case["group"] * dim].view(case["seqs"], heads * case["group"], dim)
        s["scale"] = dim ** -0.5
        if case.get("lse"):
            s["lse"] = torch.empty(case["seqs"], heads * case["group"], device=_device())
    if op != "select":
        _fill_cache(s, g, case["fmt"], pages * page, heads, dim)
    if op == "bounds":
        s["bounds"] = torch.randint(-127, 128, (pages, heads, 2, dim), dtype=torch.int8, device=_device(), generator=g)
        s["bound_scales"] = torch.rand(pages, heads, device=_device(), generator=g)
    elif op == "select":
        x = _normal(g, pages, heads, 2, dim) * 40
        hi, lo = (x.amax(2) + 60).clamp(-127, 127), (x.amin(2) - 60).clamp(-127, 127)
        s["bounds"] = torch.stack([hi, lo], 2).to(torch.int8)
        s["bound_scales"] = torch.exp(_normal(g, pages, heads) * 0.2) * 0.02
    elif op == "sparse":
        rows = _values(s, torch.arange(pages * page, device=_device()), "k", case["fmt"]).view(pages, page, heads, dim)
        s["bounds"], s["bound_scales"] = _whole_bounds(rows.amax(1), rows.amin(1))
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    return (_run_own if own else _run_plain)(case, s)


def _values(s, slot, c, fmt, head=None):
    """fp32 rows of cache c in these slots (of all heads, or of the heads `head`)."""
    at = slot if head is None else (slot, head)
    codes, scale = s[c + "_codes"][at], s[c + "_scales"][at]
    if fmt == E4M3:
        return codes.view(torch.float8_e4m3fn).float() * scale.unsqueeze(-1)
    g = torch.tensor(GRID, device=codes.device)
    i = codes.to(torch.int64)
    v = torch.stack([torch.cat([g, -g])[i & 15], torch.cat([g, -g])[i >> 4]], -1)
    return torch.ldexp(v.view(*scale.shape, 32), scale.to(torch.int32).unsqueeze(-1) - 127).view(*codes.shape[:-1], -1)


def _whole_bounds(hi, lo):
    """Column maxima and minima [..., dim] as whole numbers [..., 2, dim] of a scale; largest and infinite where a value is none."""
    a = torch.maximum(hi.abs(), lo.abs()).amax(-1)
    fine = torch.isfinite(a)
    a = torch.where(fine & (a >= TINY), a, torch.ones_like(a))
    most = torch.full_like(a, 127.0)  # a tensor: a division by a number is not rounded once
    inv = (most / a).unsqueeze(-1)
    hi, lo = torch.ceil(hi * inv).clamp(-127, 127), torch.floor(lo * inv).clamp(-127, 127)
    f = fine.unsqueeze(-1)
    both = torch.stack([torch.where(f, hi, torch.full_like(hi, 127.0)), torch.where(f, lo, torch.full_like(lo, -127.0))], -2)
    return both.to(torch.int8), torch.where(fine, a / most, torch.full_like(a, math.inf))


def _run_plain(case, s):
    op = case["op"]
    if op == "plan":
        return _plan(case, s)
    if op == "bounds":
        return _bounds(case, s)
    if op == "select":
        return _select(case, s)
    if op == "sparse":
        pages = _select(case, s)
        return {"out": _attend(case, s, pages)[0], "pages": pages}
    out, lse = _attend(case, s, None)
    if not case["lse"]:
        return out
    s["lse"].copy_(lse)
    return {"out": out, "lse": s["lse"]}


def _plan(case, s):
    page, table, free = case["page"], s["table"], s["free"]
    seqs, width = table.shape
    lens, keep, off = s["lens"].long(), s["keep"].long(), s["offsets"].long()
    new = off[1:] - off[:-1]
    held, need = (lens + page - 1) // page, (keep + new + page - 1) // page
    ok = (keep >= 0) & (keep <= lens) & (new >= 0) & (need <= width) & (held <= width)
    give, take = torch.where(ok, (held - need).clamp(min=0), 0), torch.where(ok, (need - held).clamp(min=0), 0)
    have = s["count"].long() + give.sum()
    before_give, before_take = give.cumsum(0) - give, take.cumsum(0) - take
    fits = ok & ((take == 0) | (before_take + take <= have))
    col = torch.arange(width, device=table.device)
    giving = (col >= need.unsqueeze(1)) & (col < held.unsqueeze(1)) & ok.unsqueeze(1)
    to = s["count"].long() + before_give.unsqueeze(1) + col - need.unsqueeze(1)
    stack = torch.cat([free, free[:1]])  # the last place: what is not given
    stack[torch.where(giving & (to < len(free)), to, len(free))] = table
    free.copy_(stack[:-1])
    taking = (col >= held.unsqueeze(1)) & (col < need.unsqueeze(1)) & fits.unsqueeze(1)
    of = have - 1 - before_take.unsqueeze(1) - (col - held.unsqueeze(1))
    table.copy_(torch.where(taking, free[of.clamp(0, len(free) - 1)], table))
    t = torch.arange(case["new"], device=table.device)
    row = torch.searchsorted(off[1:].contiguous(), t, right=True).clamp(max=seqs - 1)
    pos = keep[row] + t - off[row]
    slot = table[row, (pos // page).clamp(0, width - 1)].long() * page + pos % page
    return {"slots": torch.where(fits[row], slot, -1), "lens": torch.where(fits, keep + new, lens).int(),
            "count": (have - torch.where(fits, take, 0).sum()).int(), "table": table, "free": free}


def _bounds(case, s):
    page, slots = case["page"], s["slots"]
    p, at = slots // page, slots % page
    pages = s["bounds"].shape[0]
    last = torch.full((pages,), -1, dtype=torch.int64, device=slots.device).scatter_reduce(0, p, at, "amax")
    if slots.numel() * page < pages * page:  # a row of each page's values for each slot
        every = p.unsqueeze(1) * page + torch.arange(page, device=slots.device)
        n = last[p]
    else:
        every = torch.arange(pages * page, device=slots.device).view(pages, page)
        n = last
    x = _values(s, every, "k", case["fmt"])  # [.., page, heads, dim]
    live = (torch.arange(page, device=slots.device) <= n.unsqueeze(1)).view(-1, page, 1, 1)
    hi, lo = torch.where(live, x, -math.inf).amax(1), torch.where(live, x, math.inf).amin(1)
    codes, scales = _whole_bounds(hi, lo)
    if every.shape[0] == pages and slots.numel() * page >= pages * page:
        named = (last >= 0).view(-1, 1)
        s["bounds"].copy_(torch.where(named.view(-1, 1, 1, 1), codes, s["bounds"]))
        s["bound_scales"].copy_(torch.where(named, scales, s["bound_scales"]))
    else:
        s["bounds"][p] = codes
        s["bound_scales"][p] = scales
    return {"bounds": s["bounds"], "scales": s["bound_scales"]}


def _select(case, s):
    page, heads, budget, table = case["page"], case["heads"], case["budget"], s["table"]
    seqs, width = table.shape
    q = s["q"].reshape(seqs, heads, -1, case["dim"])
    a = q.abs().amax(-1)
    a = torch.where(a >= TINY, a, torch.ones_like(a))
    most = torch.full_like(a, 127.0)
    n = torch.round(q * (most / a).unsqueeze(-1)).clamp(-127, 127)
    at = table.clamp(min=0).long()
    b = s["bounds"][at].float().permute(0, 2, 3, 4, 1).reshape(seqs, heads, -1, width)  # [seqs, heads, 2 dim, width]
    dots = torch.matmul(torch.cat([n.clamp(min=0), n.clamp(max=0)], -1), b)  # sums of whole numbers below 2^24: exact
    score = (dots * s["bound_scales"][at].permute(0, 2, 1).unsqueeze(2) * (a / most).unsqueeze(-1)).amax(2)
    col = torch.arange(width, device=table.device)
    used = ((s["lens"] + page - 1) // page).clamp(max=width).view(-1, 1, 1)
    score = torch.where((col == 0) | (col == used - 1), math.inf, score)
    score = torch.where((col < used) & (table >= 0).unsqueeze(1), score, -math.inf)
    best, order = torch.sort(score, dim=-1, descending=True, stable=True)
    order = torch.where(best > -math.inf, order, width)[..., :budget]
    order = torch.cat([order, order.new_full((seqs, heads, max(0, budget - width)), width)], -1).sort(-1)[0]
    return torch.where(order < width, order, -1).int()


def _attend(case, s, pages):
    page, heads, fmt, table = case["page"], case["heads"], case["fmt"], s["table"]
    seqs, width = table.shape
    q = s["q"].reshape(seqs, heads, -1, case["dim"])
    if pages is None:
        pos = torch.arange(width * page, device=q.device).expand(seqs, 1, -1)
        named = torch.ones_like(pos, dtype=torch.bool)
    else:
        pos = (pages.long().unsqueeze(-1) * page + torch.arange(page, device=q.device)).flatten(2)
        named = (pages >= 0).repeat_interleave(page, -1)
    ids = torch.gather(table.long().unsqueeze(1).expand(-1, pos.shape[1], -1), 2, (pos // page).clamp(0, width - 1))
    slot = ids * page + pos % page
    live = named & (pos < s["lens"].view(-1, 1, 1)) & (ids >= 0)
    slot = torch.where(live, slot, 0)
    if pages is None:
        k, v = (_values(s, slot.squeeze(1), c, fmt).permute(0, 2, 1, 3) for c in ("k", "v"))
    else:
        head = torch.arange(heads, device=q.device).view(1, -1, 1).expand_as(slot)
        k, v = (_values(s, slot, c, fmt, head) for c in ("k", "v"))
    score = torch.matmul(q, k.transpose(-1, -2).contiguous()) * s["scale"]
    score = torch.where(live.unsqueeze(2), score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    w = torch.exp(score - top)
    total = w.sum(-1, keepdim=True)
    out = torch.matmul(w, torch.where(live.unsqueeze(-1), v, 0.0)) / torch.where(total == 0, torch.ones_like(total), total)
    return out.reshape(seqs, -1, case["dim"]).to(TYPES[case["type"]]), (top + torch.log(total)).reshape(seqs, -1)


def _run_own(case, s):
    import fp8_prefill_gemm_amd as rz
    op = case["op"]
    if op == "plan":
        slots, lens, count = rz.rz_kv_plan(s["lens"], s["offsets"], case["new"], case["page"], s["table"], s["free"], s["count"],
                                           keep=s["keep"])
        return {"slots": slots, "lens": lens, "count": count, "table": s["table"], "free": s["free"]}
    cache = tuple(s.get(n) for n in ("k_codes", "k_scales", "v_codes", "v_scales"))
    if op == "bounds":
        rz.rz_kv_bounds(rz.KV_E4M3 if case["fmt"] == E4M3 else rz.KV_MXFP4, *cache[:2], s["slots"], case["page"], s["bounds"], s["bound_scales"])
        return {"bounds": s["bounds"], "scales": s["bound_scales"]}
    pages = None
    if op != "attend":
        pages = rz.rz_kv_select(s["q"], s["bounds"], s["bound_scales"], case["page"], s["table"], s["lens"], case["budget"])
        if op == "select":
            return pages
    fmt = rz.KV_E4M3 if case["fmt"] == E4M3 else rz.KV_MXFP4
    out = rz.rz_kv_attention(fmt, s["q"], *cache, case["page"], s["table"], s["lens"], s["scale"], pages=pages, lse=s.get("lse"),
                             dtype=TYPES[case["type"]])
    if op == "sparse":
        return {"out": out, "pages": pages}
    return {"out": out, "lse": s["lse"]} if case["lse"] else out


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, page = case["op"], case["page"]
    if op == "plan":
        pages = case["new"] / page + case["seqs"]
        return {"bytes": case["new"] * 8 + pages * 8 + case["seqs"] * 20, "flops": 0}
    heads, dim = case["heads"], case["dim"]
    row = heads * (dim + 4) if case.get("fmt") == E4M3 else heads * dim * 17 / 32
    if op == "bounds":
        pages = case["new"] / page + case["seqs"]
        rows = case["new"] if case["new"] > case["seqs"] else case["seqs"] * (page + 1) / 2
        return {"bytes": rows * row + pages * heads * (2 * dim + 4) + 8 * case["new"], "flops": 0}
    group, seqs, tokens = case["group"], case["seqs"], case["tokens"]
    q = seqs * heads * group * dim * 4
    size = 4 if case.get("type") == "f32" else 2
    rows = tokens
    bytes_, flops = q, 0.0
    if op != "attend":
        pages = tokens / page
        rows = min(tokens, seqs * case["budget"] * page)
        bytes_ += pages * heads * (2 * dim + 4) + seqs * heads * case["budget"] * 4
        flops += 2.0 * pages * heads * group * 2 * dim
    if op != "select":
        bytes_ += 2 * rows * row + seqs * heads * group * dim * size + tokens / page * 4
        flops += 4.0 * rows * heads * group * dim
    return {"bytes": bytes_, "flops": flops}


# ---------------------------------------------------------------- from the definitions, in 64 bits

def _held(s, c, slots, head, fmt):
    """64-bit values [n, dim] of one head's rows in these slots."""
    codes, scale = s[c + "_codes"][slots, head].to(torch.int64), s[c + "_scales"][slots, head].double()
    if fmt == E4M3:
        e, f = codes >> 3 & 15, (codes & 7).double()
        mag = torch.where(e > 0, torch.exp2((e - 7).double()) * (1 + f / 8), f * 2.0 ** -9)
        return torch.where(codes > 127, -mag, mag) * scale.unsqueeze(1)
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(1)
    mag = torch.tensor(GRID, dtype=torch.float64, device=codes.device)[nib & 7]
    return torch.where(nib > 7, -mag, mag) * torch.exp2(scale - 127).repeat_interleave(32, 1)


def _chosen(case, s, b, h, n):
    """The pages that select takes for sequence b of n pages and key head h, from the definition in whole numbers."""
    if n <= case["budget"]:
        return list(range(n))
    q = s["q"][b, h * case["group"]:(h + 1) * case["group"]].cpu().numpy()
    at = s["table"][b, :n].long()
    bounds, scale = s["bounds"][at, h].cpu().numpy().astype(np.int64), s["bound_scales"][at, h].cpu().numpy()
    best = np.full(n, -np.inf, np.float32)
    for row in q:
        a = np.float32(np.abs(row).max())
        a = a if a >= np.float32(TINY) else np.float32(1)
        w = np.clip(np.rint(row * (np.float32(127) / a)), -127, 127).astype(np.int64)
        dots = np.maximum(bounds[:, 0] * w, bounds[:, 1] * w).sum(1)
        best = np.maximum(best, dots.astype(np.float32) * scale * (a / np.float32(127)))
    best[[0, n - 1]] = np.inf
    return sorted(np.argsort(-best, kind="stable")[:case["budget"]].tolist())


def exact(case, seed):
    op = case["op"]
    if op in ("plan", "select"):
        return None  # whole numbers
    s = prepare(case, seed)
    page, dim, dev = case["page"], case["dim"], _device()
    if op == "bounds":  # the scales; what they count is whole
        scales, last = s["bound_scales"].double(), {}
        for x in s["slots"].tolist():
            last[x // page] = max(last.get(x // page, 0), x % page)
        for p, n in last.items():
            rows = torch.arange(p * page, p * page + n + 1, device=dev)
            for h in range(case["heads"]):
                a = _held(s, "k", rows, h, case["fmt"]).abs().max()
                scales[p, h] = torch.where(a < TINY, torch.ones_like(a), a) / 127
        return {"bounds": None, "scales": scales}
    group = case["group"]
    lens = s["lens"].tolist()
    out = torch.zeros(case["seqs"], case["heads"] * group, dim, dtype=torch.float64, device=dev)
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device=dev)
    for b, n in enumerate(lens):
        for h in range(case["heads"] if n else 0):
            pos = torch.arange(n, device=dev)
            if op == "sparse":
                keep = torch.zeros(-(-n // page), dtype=torch.bool, device=dev)
                keep[torch.tensor(_chosen(case, s, b, h, len(keep)), device=dev)] = True
                pos = pos[keep[pos // page]]
            slots = s["table"][b, pos // page].long() * page + pos % page
            rows = slice(h * group, (h + 1) * group)
            x = (s["q"][b, rows].double() @ _held(s, "k", slots, h, case["fmt"]).t()) * s["scale"]
            lse[b, rows] = torch.logsumexp(x, 1)
            out[b, rows] = torch.softmax(x, 1) @ _held(s, "v", slots, h, case["fmt"])
    if op == "sparse":
        return {"out": out, "pages": None}
    return {"out": out, "lse": lse} if case["lse"] else out
