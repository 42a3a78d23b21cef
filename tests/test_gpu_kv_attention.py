"""GPU parity of single-token attention over the paged cache against the CPU
oracle (needs an MI355X), within the bound that the oracle derives."""
import ctypes

import numpy as np
import pytest

import workloads as W
from oracle import kv_cache, kv_serve

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FORMATS = [kv_cache.E4M3, kv_cache.MXFP4]
TYPES = {"f32": (torch.float32, 2.0 ** -24), "f16": (torch.float16, 2.0 ** -11), "bf16": (torch.bfloat16, 2.0 ** -8)}


@pytest.fixture(scope="module")
def rz():
    import fp8_prefill_gemm_amd as rz
    rz.lib()  # loud failure if the HIP library is missing
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return rz


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def raw_cache(fmt, slots, heads, dim, seed, poison=True):
    """[k_codes, k_scales, v_codes, v_scales] of random rows; where `poison`, every row reads as NaN or infinite until
    `keep` rows are put in place by fill()."""
    g = W.rng(seed)
    out = []
    for _ in range(2):
        if fmt == kv_cache.E4M3:
            out += [np.full((slots, heads, dim), 0x7F, np.uint8), np.full((slots, heads), np.nan, np.float32)]
        else:
            out += [g.integers(0, 256, (slots, heads, dim // 2)).astype(np.uint8), np.full((slots, heads, dim // 32), 255, np.uint8)]
    return out


def fill(fmt, cache, at, seed, spread=1.0):
    """Rows `at` of the cache as values of size about `spread`."""
    g = W.rng(seed)
    n, heads = len(at), cache[0].shape[1]
    for c, s in ((0, 1), (2, 3)):
        w = cache[c].shape[2]
        if fmt == kv_cache.E4M3:
            codes = g.integers(0, 256, (n, heads, w)).astype(np.uint8)
            codes[(codes & 127) < 48] ^= 64  # magnitudes of 0.5 to 448
            codes[(codes & 127) == 127] = 0
            cache[c][at], cache[s][at] = codes, (spread * 0.01 * np.exp(0.3 * g.standard_normal((n, heads)))).astype(np.float32)
        else:
            cache[c][at] = g.integers(0, 256, (n, heads, w)).astype(np.uint8)
            cache[s][at] = (g.integers(124, 127, (n, heads, w // 16)) + round(np.log2(spread))).astype(np.uint8)


def paged(page, lens, seed, spare=3, width=None):
    """(table, slots in use): pages in any order; entries behind a sequence's pages are -1."""
    need = [-(-max(n, 0) // page) for n in lens]
    pages = sum(need) + spare
    order = W.rng(seed).permutation(pages)
    table = np.full((len(lens), width or max(1, max(need))), -1, dtype=np.int32)
    used, at = [], 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n][:table.shape[1]]
        used += [int(order[at + p // page]) * page + p % page for p in range(max(lens[b], 0))]
        at += n
    return table, np.array(used, dtype=np.int64), pages * page


def check(got, lse, want, kind, whole=2.0 ** -19):
    """Every value within the oracle's bound and half a step of its type; the whole within `whole`, what independent errors
    of that size make: the bound's sums taken as square roots of their lengths, at least 2^-19."""
    out, lref, tol, ltol = want
    unit = TYPES[kind][1]
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - out) <= tol * (1 + unit) + np.abs(out) * unit + (2.0 ** -25 if kind == "f16" else 0)).all()
    norm = np.linalg.norm(out)
    if norm:
        assert np.linalg.norm(got - out) <= norm * (whole + unit * 1.01)
    if lse is not None:
        lse = host(lse).astype(np.float64)
        empty = np.isneginf(lref)
        assert np.array_equal(np.isneginf(lse), empty)
        assert (np.abs(lse[~empty] - lref[~empty]) <= ltol[~empty]).all()


def run(rz, fmt, cache, q, page, table, lens, scale, kind="f32", pages=None, **kw):
    lse = torch.full(q.shape[:2], 3.0, device="cuda")
    out = rz.rz_kv_attention(fmt, q, *[dev(c) for c in cache], page, dev(table), dev(np.array(lens, dtype=np.int32)), scale,
                             pages=None if pages is None else dev(pages), dtype=TYPES[kind][0], lse=lse, **kw)
    return out, lse


def case(rz, fmt, page, lens, heads, group, dim, kind="f32", seed=0):
    print(f"attention fmt={fmt} page={page} lens={lens} heads={heads} group={group} dim={dim} {kind}", flush=True)
    table, used, slots = paged(page, lens, seed)
    cache = raw_cache(fmt, slots, heads, dim, seed)
    fill(fmt, cache, used, seed + 1)
    row = heads * group * dim
    fused = W.act_normal(seed + 2, len(lens), row + 64)  # a fused projection's output: strided sequences
    q = dev(fused)[:, 64:].view(len(lens), heads * group, dim)
    k, v = (kv_serve.values(fmt, *c) for c in (cache[:2], cache[2:]))
    want = kv_serve.attention(k, v, fused[:, 64:].reshape(len(lens), heads * group, dim), page, table, lens, dim ** -0.5)
    out, lse = run(rz, fmt, cache, q, page, table, lens, dim ** -0.5, kind)
    check(out, lse, want, kind)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page,lens,heads,group,dim,kind", [
    (16, [37], 4, 7, 128, "f32"), (1, [1, 0, 5], 1, 1, 32, "f32"), (7, [20, 5, 0, 70, 33], 3, 2, 96, "bf16"),
    (64, [300, 64, 65], 2, 16, 64, "f16"), (5, [129, 128, 127, 31, 32, 33, 1], 1, 17, 160, "f32"), (48, [1000], 2, 40, 192, "f32"),
    (128, [5, 700], 8, 3, 256, "bf16"), (16, [0, 0], 2, 5, 128, "f32"), (3, [2] * 70, 2, 4, 64, "f32"),
])
def test_attention(rz, fmt, page, lens, heads, group, dim, kind):
    """Empty and one-token sequences, pages that end inside a tile, odd groups and more queries than a tile holds; rows that
    are not attended hold NaN."""
    case(rz, fmt, page, lens, heads, group, dim, kind)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", range(32, 513, 32))
def test_every_dim(rz, fmt, dim):
    case(rz, fmt, 16, [70, 3], 2, 5, dim, "f32", dim)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page,lens,heads,group,dim", [(16, [9000], 1, 7, 128), (64, [1, 6000, 40, 2500], 2, 4, 64), (16, [3000] * 5, 1, 1, 256)])
def test_long_sequences(rz, fmt, page, lens, heads, group, dim):
    """Sequences that are split over workgroups and joined."""
    case(rz, fmt, page, lens, heads, group, dim)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("seqs,heads,group,dim,page,longest", [(200, 8, 1, 64, 16, 5000), (700, 1, 3, 32, 5, 2000), (1300, 2, 9, 32, 16, 1500), (65, 4, 2, 96, 32, 3000)])
def test_ragged_batches(rz, fmt, seqs, heads, group, dim, page, longest):
    """More sequences than a wave looks at at once and than there are workers; many of none or a few positions, the last long."""
    g = W.rng(seqs)
    lens = [int(n) for n in g.integers(0, 40, seqs) * (g.random(seqs) < 0.7)]
    lens[seqs // 3], lens[-1] = longest // 2, longest
    case(rz, fmt, page, lens, heads, group, dim, seed=seqs)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("growth", [1, -1])
def test_values_that_grow(rz, fmt, growth):
    """One workgroup's run of thousands of positions whose values grow, and shrink, by powers of two along it: 500 positions
    make the result, so its 8 n + 64 roundings of 2^-24 are 4064, sqrt(4064) 2^-24 = 2^-18.0 if they are independent."""
    n, page, heads, group, dim = 5000, 16, 1, 3, 64
    table, used, slots = paged(page, [n], 70)
    cache = raw_cache(fmt, slots, heads, dim, 70)
    fill(fmt, cache, used, 71)
    up = np.arange(n) // 500 * 12 * growth
    if fmt == kv_cache.E4M3:
        cache[3][used] *= np.exp2(up)[:, None].astype(np.float32)
    else:
        cache[3][used] = (cache[3][used].astype(np.int64) + (up - (108 if growth > 0 else 0))[:, None, None]).clip(0, 254).astype(np.uint8)
    q = W.act_normal(72, 1, heads * group * dim).reshape(1, heads * group, dim)
    k, v = (kv_serve.values(fmt, *c) for c in (cache[:2], cache[2:]))
    d = [dev(c) for c in cache] + [dev(table), dev(np.array([n], dtype=np.int32)), dev(q)]
    p = [ctypes.c_void_p(t.data_ptr()) for t in d]
    for lens in ([n], [1025], [1024], [2049]):
        want = kv_serve.attention(k, v, q, page, table, lens, 0.1)
        d[5].copy_(torch.tensor(lens, dtype=torch.int32))
        out = torch.empty((1, heads * group, dim), device="cuda")
        torch.cuda.synchronize()
        assert rz.lib().rz_kv_attention(fmt, p[6], heads * group, heads * group * dim, *p[:4], slots, heads, dim, page, p[4], 1,
                                        table.shape[1], p[5], None, 0, 0.1, 0, ctypes.c_void_p(out.data_ptr()), None, None, None) == 0
        check(out, None, want, "f32", 2.0 ** -18)
        check(run(rz, fmt, cache, d[6], page, table, lens, 0.1)[0], None, want, "f32", 2.0 ** -18)


@pytest.mark.parametrize("fmt", FORMATS)
def test_two_calls_at_once(rz, fmt):
    """Two batches on two streams, many times over, each with a workspace of its own: the bits of one after the other."""
    page, heads, group, dim = 16, 2, 4, 64
    sets = []
    for i, lens in enumerate(([3000, 5, 0, 700], [1500] * 3)):
        table, used, slots = paged(page, lens, 73 + i)
        cache = raw_cache(fmt, slots, heads, dim, 73 + i)
        fill(fmt, cache, used, 75 + i)
        q = dev(W.act_normal(77 + i, len(lens), heads * group * dim).reshape(len(lens), heads * group, dim))
        sets.append((q, *[dev(c) for c in cache], page, dev(table), dev(np.array(lens, dtype=np.int32)), 0.1))
    want = [rz.rz_kv_attention(fmt, *a) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [rz.rz_kv_attention(fmt, *sets[i % 2], stream=streams[i % 2]) for i in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i % 2]) for i, x in enumerate(got))


@pytest.mark.parametrize("fmt", FORMATS)
def test_without_workspace(rz, fmt):
    """The C call without a workspace: no split, the same values within the bound; with one, the same bits on every call."""
    lens, page, heads, group, dim = [2000, 10, 513], 16, 2, 3, 128
    table, used, slots = paged(page, lens, 5)
    cache = raw_cache(fmt, slots, heads, dim, 5)
    fill(fmt, cache, used, 6)
    q = W.act_normal(7, 3, heads * group * dim).reshape(3, heads * group, dim)
    k, v = (kv_serve.values(fmt, *c) for c in (cache[:2], cache[2:]))
    want = kv_serve.attention(k, v, q, page, table, lens, 0.1)
    d = [dev(c) for c in cache] + [dev(table), dev(np.array(lens, dtype=np.int32)), dev(q)]
    p = [ctypes.c_void_p(t.data_ptr()) for t in d]
    out = torch.empty((3, heads * group, dim), device="cuda")
    torch.cuda.synchronize()
    assert rz.lib().rz_kv_attention(fmt, p[6], heads * group, heads * group * dim, *p[:4], slots, heads, dim, page, p[4], 3,
                                    table.shape[1], p[5], None, 0, 0.1, 0, ctypes.c_void_p(out.data_ptr()), None, None, None) == 0
    check(out, None, want, "f32")
    outs = [run(rz, fmt, cache, d[6], page, table, lens, 0.1)[0] for _ in range(3)]
    check(outs[0], None, want, "f32")
    assert all(torch.equal(outs[0], o) for o in outs)


@pytest.mark.parametrize("fmt", FORMATS)
def test_tables_that_name_nothing(rz, fmt):
    """Pages outside the cache, lengths past the table, negative lengths: such positions do not count."""
    page, heads, group, dim = 8, 2, 3, 64
    table = np.array([[3, -5, 8, 2 ** 31 - 1], [7, 0, -2 ** 31, 1], [2, 4, 5, 6], [-1, -1, -1, -1], [1, 2, 3, 4]], dtype=np.int32)
    lens = [30, 27, 1000, 20, -3]
    cache = raw_cache(fmt, 8 * page, heads, dim, 8)
    fill(fmt, cache, np.arange(8 * page), 9)
    q = W.act_normal(10, 5, heads * group * dim).reshape(5, heads * group, dim)
    k, v = (kv_serve.values(fmt, *c) for c in (cache[:2], cache[2:]))
    out, lse = run(rz, fmt, cache, dev(q), page, table, lens, 0.2)
    check(out, lse, kv_serve.attention(k, v, q, page, table, lens, 0.2), "f32")
    assert not out[3:].any()
    out, lse = run(rz, fmt, cache, dev(q), page, np.zeros((5, 0), dtype=np.int32), lens, 0.2)  # a table without columns
    assert not out.any() and (lse == -np.inf).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_chosen_pages(rz, fmt):
    """Pages named in any order, twice, beyond the sequence or the table, and none at all."""
    page, heads, group, dim, lens = 8, 2, 5, 128, [61, 40, 5, 0]
    table, used, slots = paged(page, lens, 11)
    cache = raw_cache(fmt, slots, heads, dim, 11)
    fill(fmt, cache, used, 12)
    g = W.rng(13)
    pages = np.full((4, heads, 6), -1, dtype=np.int32)
    pages[0, 0], pages[0, 1] = [0, 2, 3, 5, 7, -1], [7, 1, 1, 99, -7, 8]
    pages[1, 0, :3], pages[1, 1, 5] = [4, 5, 2 ** 31 - 1], 0
    pages[2], pages[3] = g.integers(-2, 9, (heads, 6)), 0
    q = W.act_normal(14, 4, heads * group * dim).reshape(4, heads * group, dim)
    k, v = (kv_serve.values(fmt, *c) for c in (cache[:2], cache[2:]))
    for chosen in (pages, np.full((4, heads, 6), -1, dtype=np.int32), np.zeros((4, heads, 0), dtype=np.int32)):
        out, lse = run(rz, fmt, cache, dev(q), page, table, lens, 0.1, pages=chosen)
        check(out, lse, kv_serve.attention(k, v, q, page, table, lens, 0.1, chosen), "f32")
    every = np.tile(np.arange(8, dtype=np.int32), (4, heads, 1))
    out, lse = run(rz, fmt, cache, dev(q), page, table, lens, 0.1, pages=every)
    check(out, lse, kv_serve.attention(k, v, q, page, table, lens, 0.1), "f32")


@pytest.mark.parametrize("fmt", FORMATS)
def test_chosen_pages_of_long_sequences(rz, fmt):
    """A choice long enough to be split."""
    page, heads, group, dim, lens = 16, 2, 4, 64, [5000, 3001]
    table, used, slots = paged(page, lens, 15)
    cache = raw_cache(fmt, slots, heads, dim, 15)
    fill(fmt, cache, used, 16)
    g = W.rng(17)
    pages = np.full((2, heads, 150), -1, dtype=np.int32)
    for b in range(2):
        for h in range(heads):
            n = -(-lens[b] // page)
            pages[b, h, :149 - b] = np.sort(g.permutation(n)[:149 - b])
    q = W.act_normal(18, 2, heads * group * dim).reshape(2, heads * group, dim)
    k, v = (kv_serve.values(fmt, *c) for c in (cache[:2], cache[2:]))
    out, lse = run(rz, fmt, cache, dev(q), page, table, lens, 0.1, pages=pages)
    check(out, lse, kv_serve.attention(k, v, q, page, table, lens, 0.1, pages), "f32")


@pytest.mark.parametrize("fmt", FORMATS)
def test_sharp_scores(rz, fmt):
    """Scores of thousands: the largest takes all, wherever it lies; scores far below zero; a scale of zero and a negative one."""
    page, heads, group, dim, lens = 16, 2, 3, 64, [700, 45]
    table, used, slots = paged(page, lens, 19)
    cache = raw_cache(fmt, slots, heads, dim, 19)
    fill(fmt, cache, used, 20, 8.0)
    k, v = (kv_serve.values(fmt, *c) for c in (cache[:2], cache[2:]))
    q = W.act_normal(21, 2, heads * group * dim).reshape(2, heads * group, dim)
    for scale in (3.0, -3.0, 0.0):
        out, lse = run(rz, fmt, cache, dev(q), page, table, lens, scale)
        want = kv_serve.attention(k, v, q, page, table, lens, scale)
        out64 = out.double().cpu().numpy()
        assert (np.abs(out64 - want[0]) <= want[2] + np.abs(want[0]) * 2.0 ** -24).all()
        assert (np.abs(host(lse) - want[1]) <= want[3]).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_values_that_are_none(rz, fmt):
    """A NaN in a key or value reaches the queries of its own sequence and head alone; a NaN query its own row."""
    page, heads, group, dim, lens = 16, 2, 3, 64, [50, 33, 20]
    table, used, slots = paged(page, lens, 22)
    cache = raw_cache(fmt, slots, heads, dim, 22)
    fill(fmt, cache, used, 23)
    q = W.act_normal(24, 3, heads * group * dim).reshape(3, heads * group, dim)
    want, _ = run(rz, fmt, cache, dev(q), page, table, lens, 0.1)
    s0, s1 = int(used[41]), int(used[50 + 7])
    for c, at in ((0, (s0, 1)), (2, (s1, 0))):
        if fmt == kv_cache.E4M3:
            cache[c][at][5] = 0xFF
        else:
            cache[c + 1][at][0] = 255
    q[2, 4, 9] = np.nan
    got, lse = run(rz, fmt, cache, dev(q), page, table, lens, 0.1)
    bad = torch.zeros((3, heads * group), dtype=torch.bool)
    bad[0, group:] = True  # the key
    bad[2, 4] = True
    assert torch.equal(lse.isnan().cpu(), bad)
    ok = ~bad
    ok[1, :group] = False  # the value: some of the columns
    assert got[bad.cuda()].isnan().all() and torch.equal(got[ok.cuda()], want[ok.cuda()])
    cols = got[1, :group].isnan()
    assert cols.any() and not cols.all() and torch.equal(got[1, :group][~cols], want[1, :group][~cols])
    if fmt == kv_cache.E4M3:
        assert (cols.sum(1) == 1).all() and cols[:, 5].all()


@pytest.mark.parametrize("dim", [64, 96, 128, 512])
def test_blocks_far_apart(rz, dim):
    """MXFP4 rows whose blocks' scales differ by up to 2^45, against the bound for those; queries that meet small blocks alone."""
    page, heads, group, lens = 16, 2, 3, [300, 33, 1]
    table, used, slots = paged(page, lens, 90)
    cache = raw_cache(1, slots, heads, dim, 90)
    g = W.rng(91)
    for c in (0, 2):
        x = g.standard_normal((len(used), heads, dim // 32, 32)) * np.exp2(-45 * g.random((len(used), heads, dim // 32, 1)))
        kv_cache.write(1, x.reshape(len(used), heads, dim).astype(np.float32), used, cache[c], cache[c + 1])
    q = W.act_normal(92, 3, heads * group * dim).reshape(3, heads * group, dim)
    q[:, 1, 32:] = 0
    q[:, 2, :32] = 0
    k, v = (kv_serve.values(1, *c) for c in (cache[:2], cache[2:]))
    out, lse = run(rz, 1, cache, dev(q), page, table, lens, 0.3)
    check(out, lse, kv_serve.attention(k, v, q, page, table, lens, 0.3, blocks=True), "f32")


def test_small_and_large_rows(rz):
    """E4M3 rows with scales of 2^-90 to 2^90, queries to match."""
    page, heads, dim, lens = 16, 1, 64, [40, 40]
    table, used, slots = paged(page, lens, 25)
    for up, down in ((90, -90), (-90, 90)):
        cache = raw_cache(0, slots, heads, dim, 25)
        fill(0, cache, used, 26)
        cache[1] *= np.float32(2.0 ** up)
        cache[3] *= np.float32(2.0 ** down)
        q = W.act_normal(27, 2, dim).reshape(2, 1, dim) * np.float32(2.0 ** -up)
        k, v = (kv_serve.values(0, *c) for c in (cache[:2], cache[2:]))
        out, lse = run(rz, 0, cache, dev(q), page, table, lens, 0.1)
        check(out, lse, kv_serve.attention(k, v, q, page, table, lens, 0.1), "f32")


@pytest.mark.parametrize("fmt", FORMATS)
def test_long_context(rz, fmt):
    """131072 positions in 64 bits on the device, every value."""
    n, page, heads, group, dim = 131072, 64, 2, 7, 128
    table, used, slots = paged(page, [n], 28, 0)
    cache = raw_cache(fmt, slots, heads, dim, 28)
    fill(fmt, cache, used, 29)
    q = W.act_normal(30, 1, heads * group * dim).reshape(1, heads * group, dim)
    out, lse = run(rz, fmt, cache, dev(q), page, table, [n], 0.09)
    k, v = (dev(kv_serve.values(fmt, *c)).double() for c in (cache[:2], cache[2:]))
    for h in range(heads):
        s = dev(q).double()[0, h * group:(h + 1) * group] @ k[:, h].t().contiguous() * 0.09
        ref = torch.softmax(s, 1) @ v[:, h]
        assert (out[0, h * group:(h + 1) * group] - ref).norm() <= ref.norm() * 2.0 ** -18  # chains of thousands of additions
        assert (lse[0, h * group:(h + 1) * group] - torch.logsumexp(s, 1)).abs().max() <= 2.0 ** -18 * 12


def test_on_streams_and_in_a_graph(rz):
    """A side stream gives the current one's bits; a captured call follows its inputs, lengths among them."""
    page, heads, group, dim = 16, 2, 7, 128
    table, used, slots = paged(page, [900, 300], 31)
    cache = raw_cache(0, slots, heads, dim, 31)
    fill(0, cache, used, 32)
    d = [dev(c) for c in cache]
    t, lens = dev(table), dev(np.array([900, 300], dtype=np.int32))
    q = dev(W.act_normal(33, 2, heads * group * dim).reshape(2, heads * group, dim))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    call = lambda **kw: rz.rz_kv_attention(0, q, *d, page, t, lens, 0.1, **kw)  # noqa: E731
    want, got = call(), call(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(want, got)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        graphs.append((g, out))
    for i, n in enumerate(([900, 300], [1, 299], [0, 0], [899, 17])):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        q.copy_(dev(W.act_normal(34 + i, 2, heads * group * dim).reshape(2, heads * group, dim)))
        for g, out in graphs:
            g.replay()
        eager = call()
        torch.cuda.synchronize()
        for g, out in graphs:
            assert torch.equal(out, eager)


def test_offsets_past_32_bits(rz):
    """Slots whose bytes lie past 2^32."""
    heads, group, dim, slots = 8, 2, 512, (1 << 20) + 64
    d = [torch.zeros(s, dtype=t, device="cuda") for _ in range(2) for s, t in (((slots, heads, dim), torch.uint8), ((slots, heads), torch.float32))]
    small = raw_cache(0, 48, heads, dim, 35)
    fill(0, small, np.arange(48), 36)
    at = [slots // 16 - 1, 0, slots // 16 - 3]
    for i, p in enumerate(at):
        for x, y in zip(d, small):
            x[p * 16:p * 16 + 16] = dev(y[i * 16:i * 16 + 16])
    q = W.act_normal(37, 1, heads * group * dim).reshape(1, heads * group, dim)
    k, v = (kv_serve.values(0, *c) for c in (small[:2], small[2:]))
    out = rz.rz_kv_attention(0, dev(q), *d, 16, dev(np.array([at], dtype=np.int32)), dev(np.array([45], dtype=np.int32)), 0.05)
    check(out, None, kv_serve.attention(k, v, q, 16, np.array([[0, 1, 2]]), [45], 0.05), "f32")


def test_refused_call_leaves_its_output(rz):
    q = torch.zeros((1, 3, 64), device="cuda")
    cache = [torch.zeros((16, 2, 64), dtype=torch.uint8, device="cuda"), torch.zeros((16, 2), device="cuda")] * 2
    t, n = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    out = torch.full((1, 3, 64), 5.0, device="cuda")
    with pytest.raises(rz.RzError, match="multiple of heads") as e:
        rz.rz_kv_attention(0, q, *cache, 16, t, n, 1.0, out=out)
    assert e.value.status == -3 and (out == 5).all()
    with pytest.raises(rz.RzError, match="finite"):
        rz.rz_kv_attention(0, q[:, :2], *cache, 16, t, n, float("inf"))
    assert rz.rz_kv_attention(0, q[:0, :2], *cache, 16, t[:0], n[:0], 1.0).shape == (0, 2, 64)
