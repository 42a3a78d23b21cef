"""GPU parity of page planning, page bounds and page selection against the CPU
oracle (needs an MI355X): everything equal; and a serving loop that runs them
with the cache's write and the attention that reads it."""
import numpy as np
import pytest

import workloads as W
from oracle import kv_cache, kv_serve
from test_gpu_kv_attention import FORMATS, check, dev, fill, host, paged, raw_cache

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def rz():
    import fp8_prefill_gemm_amd as rz
    rz.lib()  # loud failure if the HIP library is missing
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return rz


# ---------------------------------------------------------------- plan

def i32(x):
    return np.asarray(x, dtype=np.int32)


def planned(seqs, page, longest, new, seed, short=0, bad=False):
    """A step's inputs: sequences with pages of their own, some ended, some taken back, and the pages that are left."""
    g = W.rng(seed)
    lens = g.integers(0, longest + 1, seqs)
    keep = lens.copy()
    keep[g.random(seqs) < 0.2] = 0
    keep = np.maximum(keep - (g.random(seqs) < 0.2) * g.integers(0, 5, seqs), 0)
    add = g.integers(0, new + 1, seqs) * (g.random(seqs) < 0.8)
    need = -(-lens // page)
    pages = int(need.sum()) + int(-(-add // page).sum()) + seqs + 4
    order = g.permutation(pages)
    width = -(-(longest + new) // page) + 1
    table = np.full((seqs, width), -1, dtype=np.int32)
    at = 0
    for b in range(seqs):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    free = np.full(pages, -1, dtype=np.int32)
    count = max(0, pages - at - short)
    free[:count] = order[at:at + count]
    if bad:
        keep[g.random(seqs) < 0.2] = longest + 9
        keep[g.random(seqs) < 0.1] = -1
    offsets = np.concatenate([[0], np.cumsum(add)])
    return i32(lens), i32(keep), i32(offsets), int(offsets[-1]), table, free, count


def check_plan(rz, page, lens, keep, offsets, tokens, table, free, count):
    t, f = dev(table), dev(free)
    want_t, want_f = table.copy(), free.copy()
    want = kv_serve.plan(lens, lens if keep is None else keep, offsets, tokens, page, want_t, want_f, count)
    args = (dev(lens), dev(offsets), tokens, page, t, f, dev(i32([count])))
    for _ in range(2):  # outputs of its own: the same again
        got = rz.rz_kv_plan(*args, keep=None if keep is None else dev(keep))
        for a, b in zip(got, want):
            assert np.array_equal(host(a), b)
        assert np.array_equal(host(t), want_t) and np.array_equal(host(f), want_f)


@pytest.mark.parametrize("seqs,page,longest,new,short", [(1, 16, 40, 1, 0), (1, 1, 0, 300, 0), (64, 16, 300, 1, 0), (64, 16, 300, 1, 1000), (3, 7, 2000, 9000, 0),
                                                         (130, 64, 500, 200, 40), (1024, 3, 20, 4, 900), (1025, 16, 60, 40, 0), (2500, 5, 9, 9, 3000)])
def test_plan(rz, seqs, page, longest, new, short):
    """Steps and prompts, with pages enough and too few, of one sequence and of more than a workgroup has threads."""
    for seed in range(3):
        print(f"plan seqs={seqs} page={page} longest={longest} new={new} short={short} seed={seed}", flush=True)
        check_plan(rz, page, *planned(seqs, page, longest, new, seed, short))


def test_plan_refuses_what_does_not_fit(rz):
    for seed in range(4):
        check_plan(rz, 4, *planned(90, 4, 30, 8, seed, bad=True))
    lens, keep, offsets, tokens, table, free, count = planned(40, 4, 30, 12, 9)
    check_plan(rz, 4, lens, None, offsets, tokens, table, free, count)  # keep: all
    check_plan(rz, 4, lens, keep, offsets, tokens, np.ascontiguousarray(table[:, :5]), free, count)  # too narrow a table
    check_plan(rz, 4, lens, keep, offsets, tokens, table, free, 0)
    check_plan(rz, 2 ** 31 - 1, i32([5, 0]), i32([5, 0]), i32([0, 3, 4]), 4, i32([[1], [-1]]), i32([0, 2]), 1)  # positions times pages past 2^32
    check_plan(rz, 16, i32([2 ** 31 - 2]), i32([2 ** 31 - 2]), i32([0, 9]), 9, np.zeros((1, 3), dtype=np.int32), free, 3)


@pytest.mark.parametrize("tokens", [20, 5000])
def test_plan_tokens_left_out(rz, tokens):
    """New tokens before the first and behind the last that slots are asked for: they have pages all the same."""
    lens, table = i32([3, 0, 9]), np.full((3, 2000), -1, dtype=np.int32)
    table[0, 0], table[2, :3] = 1999, [1990, 1991, 1992]
    free = np.arange(1980, dtype=np.int32)
    check_plan(rz, 4, lens, lens, i32([-9, 6, 11, tokens + 30]), tokens, table, free, 1980)


@pytest.mark.parametrize("seqs,new", [(3, 9), (90, 8), (1024, 40), (1025, 3), (2500, 9)])
def test_plan_of_decreasing_offsets(rz, seqs, new):
    """Offsets that decrease once, anywhere, and by as little as one: every sequence stays as it is."""
    for seed, at in enumerate((0, seqs // 2, seqs - 1)):
        lens, keep, offsets, tokens, table, free, count = planned(seqs, 4, 30, new, seed)
        offsets = offsets.copy()
        offsets[at + 1:] += offsets[at] - 1 - offsets[at + 1]
        for n in (max(0, int(offsets.max())), tokens):  # all of the tokens, and more than the offsets name
            check_plan(rz, 4, lens, keep, offsets, n, table, free, count)
        slots, then, left = rz.rz_kv_plan(dev(lens), dev(offsets), tokens, 4, dev(table), dev(free), dev(i32([count])), keep=dev(keep))
        assert (host(slots) == -1).all() and np.array_equal(host(then), lens) and host(left).tolist() == [count]


def test_plan_tokens_of_no_sequence(rz):
    """Tokens before the first and behind the last sequence, more tokens than the offsets name, no sequence at all."""
    lens, table, free = i32([3, 0]), i32([[2, -1], [-1, -1]]), i32([5, 4, 1])
    slots, then, left = rz.rz_kv_plan(dev(lens), dev(i32([2, 4, 5])), 8, 4, dev(table), dev(free), dev(i32([3])))
    assert host(slots).tolist() == [-1, -1, 11, 4, 16, -1, -1, -1] and host(then).tolist() == [5, 1] and host(left).tolist() == [1]
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    slots, then, left = rz.rz_kv_plan(none, dev(i32([0])), 5000, 4, torch.zeros((0, 2), dtype=torch.int32, device="cuda"), dev(free), dev(i32([2])))
    assert (host(slots) == -1).all() and then.numel() == 0 and host(left).tolist() == [2]


@pytest.mark.parametrize("new", [1, 300])
def test_plan_in_place(rz, new):
    """Lengths and count updated where they are, as a captured step does it."""
    lens, keep, offsets, tokens, table, free, count = planned(50, 16, 200, new, 30)
    a = [dev(x) for x in (lens, offsets, table, free, i32([count]), keep)]
    want_t, want_f = table.copy(), free.copy()
    want = kv_serve.plan(lens, keep, offsets, tokens, 16, want_t, want_f, count)
    slots, then, left = rz.rz_kv_plan(a[0], a[1], tokens, 16, a[2], a[3], a[4], keep=a[5], lens_out=a[0], count_out=a[4])
    for got, ref in zip((slots, a[0], a[4], a[2], a[3]), (*want, want_t, want_f)):
        assert np.array_equal(host(got), ref)
    b = [dev(x) for x in (lens, offsets, table, free, i32([count]), keep)]
    rz.rz_kv_plan(b[0], b[1], tokens, 16, b[2], b[3], b[4], keep=b[5], lens_out=b[5], count_out=b[4])
    assert np.array_equal(host(b[5]), want[1]) and np.array_equal(host(b[2]), want_t)


def test_plan_stack_that_overflows(rz):
    """Counts outside the stack, and pages given back to a full one, write nothing outside it."""
    lens, table = i32([40, 40]), np.arange(20, dtype=np.int32).reshape(2, 10)
    for count in (-5, 3, 99):
        free = torch.full((8,), 50, dtype=torch.int32, device="cuda")
        whole = free[2:5]  # a stack of three inside
        _, then, left = rz.rz_kv_plan(dev(lens), dev(i32([0, 0, 0])), 0, 4, dev(table), whole, dev(i32([count])), keep=dev(i32([0, 0])))
        got = host(free)
        assert (got[:2] == 50).all() and (got[5:] == 50).all() and host(left).tolist() == [3] and host(then).tolist() == [0, 0]


# ---------------------------------------------------------------- bounds

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page,lens,before,heads,dim", [(16, [37], [0], 4, 128), (16, [1, 17, 40, 33], [0, 16, 39, 3], 1, 32), (7, [20, 70], [13, 0], 3, 96), (1, [5], [2], 2, 64),
                                                        (64, [700, 130], [0, 65], 2, 256), (5, [9, 41], [8, 40], 1, 512), (24, [200], [199], 5, 160), (128, [2000], [0], 1, 64)])
def test_bounds(rz, fmt, page, lens, before, heads, dim):
    """New tokens of sequences that begin inside a page; rows behind the last hold NaN; other pages stay."""
    print(f"bounds fmt={fmt} page={page} lens={lens} before={before} heads={heads} dim={dim}", flush=True)
    table, used, slots = paged(page, lens, 40)
    cache = raw_cache(fmt, slots, heads, dim, 41)
    fill(fmt, cache, used, 42)
    named = np.concatenate([[int(table[b, p // page]) * page + p % page for p in range(before[b], lens[b])] for b in range(len(lens))]).astype(np.int64)
    g = W.rng(43)
    pages = slots // page
    codes, scales = g.integers(-128, 128, (pages, heads, 2, dim)).astype(np.int8), g.random((pages, heads)).astype(np.float32)
    dc, ds = dev(codes), dev(scales)
    rz.rz_kv_bounds(fmt, dev(cache[0]), dev(cache[1]), dev(named), page, dc, ds)
    kv_serve.bounds(kv_serve.values(fmt, *cache[:2]), named, page, codes, scales)
    assert np.array_equal(host(dc), codes) and np.array_equal(host(ds), scales)


@pytest.mark.parametrize("fmt", FORMATS)
def test_bounds_of_many_pages(rz, fmt):
    """A prompt's pages by more tokens than a workgroup looks over, the same slot named twice, each page's last filled in part."""
    page, heads, dim, lens = 3, 5, 32, [4001, 2, 5003]
    table, used, slots = paged(page, lens, 46)
    cache = raw_cache(fmt, slots, heads, dim, 47)
    fill(fmt, cache, used, 48)
    named = np.repeat(used, 2)
    codes, scales = np.zeros((slots // page, heads, 2, dim), dtype=np.int8), np.zeros((slots // page, heads), dtype=np.float32)
    dc, ds = dev(codes), dev(scales)
    rz.rz_kv_bounds(fmt, dev(cache[0]), dev(cache[1]), dev(named), page, dc, ds)
    kv_serve.bounds(kv_serve.values(fmt, *cache[:2]), named, page, codes, scales)
    assert np.array_equal(host(dc), codes) and np.array_equal(host(ds), scales)


@pytest.mark.parametrize("fmt", FORMATS)
def test_bounds_of_special_rows(rz, fmt):
    """NaN and infinite rows, zeros, tiny and huge ones; slots that are none; a cache that ends inside a page."""
    page, heads, dim, slots = 4, 2, 64, 30
    cache = raw_cache(fmt, slots, heads, dim, 44)
    fill(fmt, cache, np.arange(slots), 45)
    codes, sc = cache[0], cache[1]
    codes[4:8] = 0
    if fmt == kv_cache.E4M3:
        codes[9, 0, 3] = 0x7F
        sc[13, 1] = np.inf
        sc[16:20], sc[20:24] = 2.0 ** -140, 3e35
        codes[24:28, 0, 5:] = 0  # one column alone
    else:
        sc[9, 0, 1] = 255
        sc[16:20], sc[20:24] = 0, 250
        sc[13, 1] = 254  # past the fp32 range: infinite
    named = np.array([0, 3, -1, 4, 5, 6, 7, 99, 8, 11, 12, 13, 14, 19, 20, 23, 25, 28, 29, 1 << 40], dtype=np.int64)
    got_c, got_s = torch.zeros((7, heads, 2, dim), dtype=torch.int8, device="cuda"), torch.zeros((7, heads), device="cuda")
    rz.rz_kv_bounds(fmt, dev(codes), dev(sc), dev(named), page, got_c, got_s)
    want_c, want_s = np.zeros((7, heads, 2, dim), dtype=np.int8), np.zeros((7, heads), dtype=np.float32)
    kv_serve.bounds(kv_serve.values(fmt, codes, sc), named, page, want_c, want_s)
    assert np.array_equal(host(got_s), want_s) and np.array_equal(host(got_c), want_c)
    assert np.isinf(want_s).sum() >= 2


# ---------------------------------------------------------------- select

def ranked(pages, heads, dim, seed, kinds=0):
    g = W.rng(seed)
    x = g.integers(-127, 128, (pages, heads, 2, dim))
    codes = np.sort(x, axis=2)[:, :, ::-1].astype(np.int8)
    scales = (0.01 + 0.02 * g.random((pages, heads))).astype(np.float32)
    if kinds:  # few different pages: many ties
        which = g.integers(0, kinds, pages)
        codes, scales = codes[which], scales[which]
    return np.ascontiguousarray(codes), np.ascontiguousarray(scales)


@pytest.mark.parametrize("page,lens,heads,group,dim,budget,kinds", [
    (16, [37], 4, 7, 128, 2, 0), (16, [1, 0, 160, 161], 1, 1, 32, 4, 0), (64, [64 * 300, 64 * 299 + 1, 5], 2, 16, 64, 20, 0), (1, [1500, 1024, 1025], 3, 2, 96, 256, 0),
    (16, [16 * 700, 999], 2, 3, 256, 1, 0), (16, [16 * 900], 2, 17, 160, 300, 5), (32, [32 * 64] * 9, 2, 5, 512, 63, 3), (128, [50000, 130, 128], 1, 40, 192, 64, 0),
    (1, [9000], 1, 2, 64, 4000, 7), (16, [300, 300], 8, 1, 128, 1000, 0), (1, [30000, 7], 1, 3, 32, 900, 0), (1, [40000], 2, 1, 32, 37, 0), (1, [4096] * 9, 16, 1, 32, 129, 50),
    (1, [512, 511, 1], 2, 2, 64, 60, 0), (1, [513, 512, 3], 2, 2, 64, 60, 0), (2, [16384, 7], 1, 2, 96, 500, 9), (2, [16386], 1, 2, 96, 500, 0), (1, [32768], 1, 1, 32, 4097, 3)])
def test_select(rz, page, lens, heads, group, dim, budget, kinds):
    """One page to thousands, budgets below and above them, many equal scores, more queries than a tile holds."""
    print(f"select page={page} lens={lens} heads={heads} group={group} dim={dim} budget={budget}", flush=True)
    table, _, slots = paged(page, lens, 50)
    codes, scales = ranked(slots // page, heads, dim, 51, kinds)
    row = heads * group * dim
    fused = W.act_normal(52, len(lens), row + 32)
    q = fused[:, 32:].reshape(len(lens), heads * group, dim)
    got = rz.rz_kv_select(dev(fused)[:, 32:].view(len(lens), heads * group, dim), dev(codes), dev(scales), page, dev(table), dev(i32(lens)), budget)
    assert np.array_equal(host(got), kv_serve.select(q, codes, scales, page, table, lens, budget))


def test_select_special(rz):
    """Pages outside the cache, lengths past the table, infinite scales, queries of zeros, NaN and infinities, equal pages throughout."""
    page, heads, group, dim = 8, 2, 3, 64
    codes, scales = ranked(12, heads, dim, 53)
    scales[3], scales[5, 1] = np.inf, 0.0
    table = np.array([[0, -1, 3, 12, 4, 5, 6, 7, 2 ** 31 - 1, 9], [9, 8, 7, 6, 5, 4, 3, 2, 1, 0], [2] * 10, [1, 2, 3, 4, 5, -2 ** 31, 7, 8, 9, 10]], dtype=np.int32)
    lens = [80, 1000, 75, 44]
    q = W.act_normal(54, 4, heads * group * dim).reshape(4, heads * group, dim)
    q[0, :3], q[1, 1], q[1, 4, 7], q[1, 5, 8], q[3, 3:] = 0, np.nan, np.nan, np.inf, 2.0 ** -120
    q[3, 0], q[3, 1, 3] = 3e38, -np.inf
    for budget in (1, 2, 3, 5, 11):
        got = rz.rz_kv_select(dev(q), dev(codes), dev(scales), page, dev(table), dev(i32(lens)), budget)
        assert np.array_equal(host(got), kv_serve.select(q, codes, scales, page, table, lens, budget)), budget
    got = rz.rz_kv_select(dev(q), dev(codes), dev(scales), page, torch.zeros((4, 0), dtype=torch.int32, device="cuda"), dev(i32(lens)), 3)
    assert (host(got) == -1).all()


@pytest.mark.parametrize("page,lens", [(4, [64, 61, 4, 5, 0, 33]), (1, [700, 512, 2]), (2, [9000, 1])])
@pytest.mark.parametrize("budget", [1, 2, 3, 7, 40])
def test_select_keeps_the_newest_page(rz, page, lens, budget):
    """A sequence's first and last page among pages whose keys hold a NaN, as many as the budget and more."""
    heads, group, dim = 2, 3, 64
    table, _, slots = paged(page, lens, 55)
    codes, scales = ranked(slots // page, heads, dim, 56)
    scales[W.rng(57).random(scales.shape) < 0.6] = np.inf
    q = W.act_normal(58, len(lens), heads * group * dim).reshape(len(lens), heads * group, dim)
    got = host(rz.rz_kv_select(dev(q), dev(codes), dev(scales), page, dev(table), dev(i32(lens)), budget))
    assert np.array_equal(got, kv_serve.select(q, codes, scales, page, table, lens, budget))
    for b, n in enumerate(lens):
        used = -(-n // page)
        for row in got[b]:
            taken = set(row[row >= 0].tolist())
            assert len(taken) == min(used, budget)
            assert ({0, used - 1} if budget > 1 else {0}) <= taken if used else not taken


@pytest.mark.parametrize("fmt", FORMATS)
def test_caches_of_nothing(rz, fmt):
    """A cache without slots, bounds of no pages, steps of no tokens, batches of no sequences."""
    heads, dim, seqs = 2, 64, 3
    none = [dev(x) for c in range(2) for x in kv_cache.empty(fmt, 0, heads, dim)]
    codes, scales = torch.zeros((0, heads, 2, dim), dtype=torch.int8, device="cuda"), torch.zeros((0, heads), device="cuda")
    q, table, lens = torch.ones((seqs, 4, dim), device="cuda"), torch.zeros((seqs, 700), dtype=torch.int32, device="cuda"), dev(i32([9, 0, 5000]))
    lse = torch.zeros((seqs, 4), device="cuda")
    assert not rz.rz_kv_attention(fmt, q, *none, 8, table, lens, 1.0, lse=lse).any() and (lse == -np.inf).all()
    assert (rz.rz_kv_select(q, codes, scales, 8, table, lens, 5) == -1).all()
    assert (rz.rz_kv_select(q, codes, scales, 8, table[:, :9].contiguous(), lens, 5) == -1).all()
    slots = torch.zeros(4, dtype=torch.int64, device="cuda")
    rz.rz_kv_bounds(fmt, *none[:2], slots, 8, codes, scales)
    rz.rz_kv_bounds(fmt, *none[:2], slots[:0], 8, codes, scales)
    assert rz.rz_kv_select(q[:0], codes, scales, 8, table[:0], lens[:0], 5).shape == (0, heads, 5)
    torch.cuda.synchronize()


def test_choices_on_two_streams_and_in_a_graph(rz):
    """Scores and choices of two batches at once, each with a workspace of its own, and replayed over new queries and lengths."""
    sets = []
    for i, (page, lens) in enumerate(((4, [9000, 30]), (8, [700, 6000, 1]))):
        table, _, slots = paged(page, lens, 80 + i)
        codes, scales = ranked(slots // page, 2, 64, 82 + i)
        q = W.act_normal(84 + i, len(lens), 6 * 64).reshape(len(lens), 6, 64)
        sets.append(((dev(q), dev(codes), dev(scales), page, dev(table), dev(i32(lens)), 40), kv_serve.select(q, codes, scales, page, table, lens, 40)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [rz.rz_kv_select(*sets[i % 2][0], stream=streams[i % 2]) for i in range(20)]
    torch.cuda.synchronize()
    assert all(np.array_equal(host(x), sets[i % 2][1]) for i, x in enumerate(got))
    graphs = []
    for args, _ in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = rz.rz_kv_select(*args)
        graphs.append((g, out))
    for seed in range(3):
        for (args, _), (g, out) in zip(sets, graphs):
            args[0].copy_(dev(W.act_normal(90 + seed, args[0].shape[0], 6 * 64).reshape(args[0].shape)))
            args[5].copy_(args[5] - 1)
        for g, out in graphs:
            g.replay()
        eager = [rz.rz_kv_select(*args) for args, _ in sets]
        assert all(np.array_equal(host(out), host(e)) for (_, out), e in zip(graphs, eager))
        assert not np.array_equal(host(eager[0]), sets[0][1])


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("fmt", FORMATS)
def test_serving_loop(rz, fmt):
    """Prompts, steps, an end and a new start, guesses taken back: plan, write, bounds, select and attention in place and, for
    the steps, as one captured graph; every output against the oracle's run of the same steps."""
    seqs, width, page, heads, group, dim, budget = 4, 12, 8, 2, 3, 64, 3
    pages = 30
    g = W.rng(60)
    lens, table, free, count = np.zeros(seqs, dtype=np.int32), np.full((seqs, width), -1, dtype=np.int32), g.permutation(pages).astype(np.int32), pages
    pair = [kv_cache.empty(fmt, pages * page, heads, dim) for _ in range(2)]
    bounds, bscales = np.zeros((pages, heads, 2, dim), dtype=np.int8), np.zeros((pages, heads), dtype=np.float32)
    d_lens, d_table, d_free, d_count = dev(lens), dev(table), dev(free), dev(i32([count]))
    cache, d_b, d_s = [dev(x) for c in pair for x in c], dev(bounds), dev(bscales)
    row = heads * dim

    def step(qkv, keep, offsets, tokens):
        slots, _, _ = rz.rz_kv_plan(d_lens, offsets, tokens, page, d_table, d_free, d_count, keep=keep, lens_out=d_lens, count_out=d_count)
        k, v = (qkv[:, (group + i) * row:(group + i + 1) * row].view(tokens, heads, dim) for i in range(2))
        rz.rz_kv_cache_write(fmt, k, v, slots, *cache)
        rz.rz_kv_bounds(fmt, *cache[:2], slots, page, d_b, d_s)
        return slots

    def attend(q):
        chosen = rz.rz_kv_select(q, d_b, d_s, page, d_table, d_lens, budget)
        return (rz.rz_kv_attention(fmt, q, *cache, page, d_table, d_lens, 0.2), chosen,
                rz.rz_kv_attention(fmt, q, *cache, page, d_table, d_lens, 0.2, pages=chosen))

    d_keep, d_off = torch.zeros(seqs, dtype=torch.int32, device="cuda"), dev(i32(range(seqs + 1)))
    d_qkv = torch.zeros((seqs, (group + 2) * row), device="cuda")
    d_q = torch.zeros((seqs, heads * group, dim), device="cuda")
    graph = None
    keeps = [[0, 0, 0, 0]] + [None] * 9
    news = [[40, 3, 17, 0], [1] * 4, [1] * 4, [1, 1, 60, 8], [1] * 4, [30, 1, 1, 1], [1] * 4, [1] * 4, [1] * 4, [1] * 4]
    for i, new in enumerate(news):
        keep = lens.copy() if keeps[i] is None else i32(keeps[i])
        if i == 3:
            keep[2] = 0  # ended; another starts in its place
        if i == 6:
            keep[0] -= 5  # a guess taken back
        if i == 7:
            keep[1] = 0
        offsets = i32(np.concatenate([[0], np.cumsum(new)]))
        tokens = int(offsets[-1])
        qkv = W.act_normal(70 + i, tokens, (group + 2) * row)
        q = W.act_normal(90 + i, seqs, heads * group * dim).reshape(seqs, heads * group, dim)
        if new == [1] * 4:
            if graph is None:  # recorded once, replayed for every such step
                saved = [x.clone() for x in (d_lens, d_table, d_free, d_count, *cache, d_b, d_s)]
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    g_slots = step(d_qkv, d_keep, d_off, seqs)
                    g_out = attend(d_q)
                for x, y in zip((d_lens, d_table, d_free, d_count, *cache, d_b, d_s), saved):
                    assert torch.equal(x, y)  # recording runs nothing
            d_keep.copy_(dev(keep)), d_qkv.copy_(dev(qkv)), d_q.copy_(dev(q))
            graph.replay()
            slots, out = g_slots, g_out
        else:
            slots = step(dev(qkv), dev(keep), dev(offsets), tokens)
            out = attend(dev(q))
        want_slots, lens, left = kv_serve.plan(lens, keep, offsets, tokens, page, table, free, count)
        count = int(left[0])
        for c, (codes, sc) in enumerate(pair):
            kv_cache.write(fmt, qkv[:, (group + c) * row:(group + c + 1) * row].reshape(tokens, heads, dim), want_slots, codes, sc)
        k, v = (kv_serve.values(fmt, *c) for c in pair)
        kv_serve.bounds(k, want_slots, page, bounds, bscales)
        for a, b in ((slots, want_slots), (d_lens, lens), (d_table, table), (d_b, bounds), (d_s, bscales), (d_count, left)):
            assert np.array_equal(host(a), b), i
        assert np.array_equal(host(d_free)[:count], free[:count])
        chosen = kv_serve.select(q, bounds, bscales, page, table, lens, budget)
        assert np.array_equal(host(out[1]), chosen), i
        check(out[0], None, kv_serve.attention(k, v, q, page, table, lens, 0.2), "f32")
        check(out[2], None, kv_serve.attention(k, v, q, page, table, lens, 0.2, chosen), "f32")
    assert (lens > 0).all()
