"""GPU parity of the quantised key/value cache against the CPU oracle (needs
an MI355X): codes, scales and read-back values equal."""
import numpy as np
import pytest

import workloads as W
from oracle import kv_cache

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FORMATS = [kv_cache.E4M3, kv_cache.MXFP4]


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


def bits(a):
    return np.ascontiguousarray(a).view(np.uint8)


def caches(fmt, slots, heads, dim, fill=0x35):
    """(oracle k and v caches, device copies in call order)."""
    pair = [kv_cache.empty(fmt, slots, heads, dim, fill) for _ in range(2)]
    return pair, [dev(x) for c in pair for x in c]


def check_cache(pair, device):
    for want, got in zip([x for c in pair for x in c], device):
        assert np.array_equal(bits(host(got)), bits(want))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens,heads,dim", [(1, 1, 32), (3, 4, 128), (65, 3, 96), (17, 1, 512), (40, 5, 64), (9, 2, 288), (33, 8, 256)])
def test_write(rz, fmt, tokens, heads, dim):
    """Strided tokens (columns of one fused projection), slots in any order, some dropped."""
    g = W.rng(tokens + dim)
    slots = g.permutation(tokens + 9)[:tokens].astype(np.int64)
    if tokens > 2:
        slots[1], slots[2] = -1, tokens + 9
    row = heads * dim
    qkv = W.act_normal(dim + heads, tokens, 3 * row)
    qkv[0, row:row + 32] = 0
    pair, d = caches(fmt, tokens + 9, heads, dim)
    k, v = (qkv[:, i * row:(i + 1) * row].reshape(tokens, heads, dim) for i in (1, 2))
    for x, c in zip((k, v), pair):
        kv_cache.write(fmt, x, slots, *c)
    dq = dev(qkv)
    rz.rz_kv_cache_write(fmt, dq[:, row:2 * row].view(tokens, heads, dim), dq[:, 2 * row:].view(tokens, heads, dim), dev(slots), *d)
    check_cache(pair, d)


@pytest.mark.parametrize("fmt", FORMATS)
def test_write_special_rows(rz, fmt):
    """All-zero, NaN, infinite, subnormal and largest values, one row each."""
    f = np.finfo(np.float32)
    x = W.act_normal(7, 8, 64).reshape(8, 1, 64)
    x[0] = 0
    x[1, 0, 5] = np.nan
    x[2, 0, 6] = np.inf
    x[3, 0, 7] = -np.inf
    x[4] = 2.0 ** -140
    x[5, 0, 40] = f.max
    x[6] = np.nan
    pair, d = caches(fmt, 8, 1, 64)
    slots = np.arange(8, dtype=np.int64)[::-1].copy()
    for c in pair:
        with np.errstate(all="ignore"):
            kv_cache.write(fmt, x, slots, *c)
    rz.rz_kv_cache_write(fmt, dev(x), dev(x), dev(slots), *d)
    check_cache(pair, d)


def filled(fmt, slots, heads, dim, seed):
    """A cache of random rows, as the oracle writes them."""
    pair, _ = caches(fmt, slots, heads, dim)
    for i, c in enumerate(pair):
        kv_cache.write(fmt, W.act_normal(seed + i, slots, heads * dim).reshape(slots, heads, dim), np.arange(slots), *c)
    return pair, [dev(x) for c in pair for x in c]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page,lens,heads,dim", [(1, [3], 1, 32), (16, [1, 0, 33, 16], 4, 128), (7, [20, 5, 7], 3, 96), (64, [100], 2, 256), (5, [9, 40], 1, 512),
                                                  (16, [700, 1, 5000, 3000], 1, 64), (3, [9], 70, 32)])
def test_read(rz, fmt, page, lens, heads, dim):
    """Pages that end inside the batch, empty sequences, a row before and rows behind the sequences left as they were."""
    need = [max(1, -(-n // page)) for n in lens]
    pages = sum(need) + 2
    g = W.rng(page)
    order = g.permutation(pages)
    table = np.full((len(lens), max(need) + 1), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    offsets = np.concatenate([[1], 1 + np.cumsum(lens)]).astype(np.int32)
    rows = int(offsets[-1]) + 3
    pair, d = filled(fmt, pages * page, heads, dim, 20)
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        outs = [torch.full((rows, heads, dim), 7.0, device="cuda", dtype=dtype) for _ in range(2)]
        rz.rz_kv_cache_read(fmt, *d, page, dev(table), dev(offsets), rows, *outs)
        for c, got in zip(pair, outs):
            want = np.full((rows, heads, dim), 7.0, dtype=np.float32)
            kv_cache.read(fmt, *c, page, table, offsets, want)
            assert torch.equal(got.cpu(), torch.from_numpy(want).to(dtype)), dtype


@pytest.mark.parametrize("fmt", FORMATS)
def test_read_bad_pages(rz, fmt):
    """Page numbers outside the cache, a table too short for its sequence, fewer rows than the offsets name."""
    pair, d = filled(fmt, 8 * 4, 2, 64, 30)
    table = np.array([[3, -5, 8, 2 ** 31 - 1], [7, 0, -2 ** 31, 1]], dtype=np.int32)
    offsets = np.array([0, 19, 40], dtype=np.int32)  # 19 positions: past the 4 pages of 4
    rows = 33
    outs = rz.rz_kv_cache_read(fmt, *d, 4, dev(table), dev(offsets), rows)
    for c, got in zip(pair, outs):
        want = np.zeros((rows, 2, 64), dtype=np.float32)
        kv_cache.read(fmt, *c, 4, table, offsets, want)
        assert np.array_equal(host(got), want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_write_then_read_prompt_and_steps(rz, fmt):
    """A prompt and then single tokens, as they are served: pages filled in turn, read back whole."""
    heads, dim, page, total, prompt = 4, 128, 16, 50, 43
    x = [W.act_normal(40 + i, total, heads * dim).reshape(total, heads, dim) for i in range(2)]
    table = np.array([[5, 2, 7, 0]], dtype=np.int32)
    pos = np.arange(total)
    slots = (table[0, pos // page] * page + pos % page).astype(np.int64)
    pair, d = caches(fmt, 8 * page, heads, dim)
    for lo, hi in [(0, prompt)] + [(t, t + 1) for t in range(prompt, total)]:
        rz.rz_kv_cache_write(fmt, dev(x[0][lo:hi]), dev(x[1][lo:hi]), dev(slots[lo:hi]), *d)
    for i in range(2):
        kv_cache.write(fmt, x[i], slots, *pair[i])
    check_cache(pair, d)
    outs = rz.rz_kv_cache_read(fmt, *d, page, dev(table), dev(np.array([0, total], dtype=np.int32)), total, dtype=torch.bfloat16)
    for i in range(2):
        want = np.empty((total, heads, dim), dtype=np.float32)
        kv_cache.read(fmt, *pair[i], page, table, [0, total], want)
        assert torch.equal(outs[i].cpu(), torch.from_numpy(want).to(torch.bfloat16))


def test_on_a_stream_and_refusals(rz):
    """A write and a read on a side stream, as on the current one; a refused call leaves the cache as it was."""
    heads, dim, n = 2, 64, 9
    x = dev(W.act_normal(70, n, heads * dim).reshape(n, heads, dim))
    slots = dev(W.rng(71).permutation(12)[:n].astype(np.int64))
    table, offsets = slots.to(torch.int32).view(1, n), dev(np.array([0, n], dtype=np.int32))
    got = []
    for stream in (None, torch.cuda.Stream()):
        _, cache = caches(kv_cache.MXFP4, 12, heads, dim)
        torch.cuda.synchronize()
        rz.rz_kv_cache_write(kv_cache.MXFP4, x, x, slots, *cache, stream=stream)
        got.append(rz.rz_kv_cache_read(kv_cache.MXFP4, *cache, 1, table, offsets, n, dtype=torch.float16, stream=stream))
        torch.cuda.synchronize()
    for a, b in zip(*got):
        assert torch.equal(a, b)
    _, cache = caches(kv_cache.E4M3, 4, 1, 48)
    before = [host(c) for c in cache]
    with pytest.raises(rz.RzError, match="multiple of 32") as e:
        rz.rz_kv_cache_write(kv_cache.E4M3, torch.zeros((1, 1, 48), device="cuda"), torch.zeros((1, 1, 48), device="cuda"),
                             torch.zeros(1, dtype=torch.int64, device="cuda"), *cache)
    assert e.value.status == -3 and all(np.array_equal(host(c), b) for c, b in zip(cache, before))


def test_projection_to_cache(rz):
    """One layer's step: activation -> MXFP4 product -> cache -> read back, captured and replayed."""
    m, d, heads, dim = 37, 512, 2, 64
    row = heads * dim
    w = rz.rz_mxfp4_pack_weight(W.Q4_K, dev(W.weight_blocks(W.Q4_K, 50, 2 * row, d)), 2 * row, d)
    x = torch.zeros((m, d), device="cuda")
    slots = dev(W.rng(51).permutation(48)[:m].astype(np.int64))
    table = slots.to(torch.int32).view(1, m)
    offsets = dev(np.array([0, m], dtype=np.int32))
    _, cache = caches(kv_cache.E4M3, 48, heads, dim)

    def step():
        kv = rz.rz_mxfp4_gemm(*rz.rz_mxfp4_quant(x), m, *w, 2 * row)
        rz.rz_kv_cache_write(kv_cache.E4M3, kv[:, :row].view(m, heads, dim), kv[:, row:].view(m, heads, dim), slots, *cache)
        return (kv, *rz.rz_kv_cache_read(kv_cache.E4M3, *cache, 1, table, offsets, m))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        x.copy_(dev(W.act_normal(52 + i, m, d)))
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, step()):
            assert torch.equal(got, want)
        kv = out[0].view(m, 2, heads, dim)
        for c in range(2):  # half a step of E4M3 (2^-4 relative, 2^-6/448 of the row's largest below it), scale and product rounded
            ref = kv[:, c]
            top = ref.abs().amax(-1, keepdim=True)
            assert ((out[1 + c] - ref).abs() <= ref.abs() * (2.0 ** -4 + 2.0 ** -21) + top * (2.0 ** -6 / 448 * 1.001)).all()


def test_large_offsets(rz):
    """Slots whose bytes lie past 2^32."""
    heads, dim, slots = 8, 512, (1 << 20) + 40
    d = [torch.zeros(s, dtype=t, device="cuda") for _ in range(2) for s, t in (((slots, heads, dim), torch.uint8), ((slots, heads), torch.float32))]
    x = W.act_normal(60, 3, heads * dim).reshape(3, heads, dim)
    at = np.array([slots - 1, 5, (1 << 20) + 1], dtype=np.int64)
    rz.rz_kv_cache_write(kv_cache.E4M3, dev(x), dev(-x), dev(at), *d)
    small = kv_cache.empty(kv_cache.E4M3, 3, heads, dim)
    kv_cache.write(kv_cache.E4M3, x, np.arange(3), *small)
    for i, s in enumerate(at):
        assert np.array_equal(host(d[0][int(s)]), small[0][i]) and np.array_equal(host(d[1][int(s)]), small[1][i])
    out, _ = rz.rz_kv_cache_read(kv_cache.E4M3, *d, 1, dev(at.astype(np.int32).reshape(1, 3)), dev(np.array([0, 3], dtype=np.int32)), 3)
    want = np.empty((3, heads, dim), dtype=np.float32)
    kv_cache.read(kv_cache.E4M3, *small, 1, np.arange(3).reshape(1, 3), [0, 3], want)
    assert np.array_equal(host(out), want)
