"""GPU parity of attention over the paged cache at the ends of what its bound
holds for (needs an MI355X): rows of nothing beside small ones, scales and
queries from one end of the range to the other, scores past 2^24."""
import ctypes

import numpy as np
import pytest

import workloads as W
from oracle import kv_cache, kv_serve
from test_gpu_kv_attention import FORMATS, check, dev, fill, host, paged, raw_cache, run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def rz():
    import fp8_prefill_gemm_amd as rz
    rz.lib()  # loud failure if the HIP library is missing
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return rz


def whole(rz, fmt, cache, q, page, table, lens, scale):
    """The C call without a workspace: one workgroup a sequence and key head."""
    d = [dev(c) for c in cache] + [dev(table), dev(np.array(lens, dtype=np.int32)), dev(q)]
    p = [ctypes.c_void_p(t.data_ptr()) for t in d]
    out = torch.empty(q.shape, device="cuda")
    slots, heads = cache[1].shape[:2]
    torch.cuda.synchronize()
    assert rz.lib().rz_kv_attention(fmt, p[6], q.shape[1], q.shape[1] * q.shape[2], *p[:4], slots, heads, q.shape[2], page, p[4], len(lens),
                                    table.shape[1], p[5], None, 0, scale, 0, ctypes.c_void_p(out.data_ptr()), None, None, None) == 0
    return out


def both(rz, fmt, cache, q, page, table, lens, scale, exact=2.0 ** -19):
    """Whole and split, every value within the oracle's bound."""
    k, v = (kv_serve.values(fmt, *c) for c in (cache[:2], cache[2:]))
    want = kv_serve.attention(k, v, q, page, table, lens, scale)
    check(whole(rz, fmt, cache, q, page, table, lens, scale), None, want, "f32", exact)
    out, lse = run(rz, fmt, cache, dev(q), page, table, lens, scale)
    check(out, lse, want, "f32", exact)


@pytest.mark.parametrize("down", [-100, -97, -93])
def test_smallest_value_scales(rz, down):
    """E4M3 rows of the smallest scales, one position taking nearly all the weight with a value of one column: in the other
    columns the result is of the weights that are left."""
    page, heads, dim, n = 16, 1, 64, 40
    table, used, slots = paged(page, [n], 7)
    cache = raw_cache(0, slots, heads, dim, 7)
    fill(0, cache, used, 8)
    g = W.rng(9)
    k = (0.1 * g.standard_normal((n, heads, dim))).astype(np.float32)
    k[5] = 1
    kv_cache.write(0, k, used, *cache[:2])
    cache[2][used[5], 0, 1:] = 0
    cache[2][used[5], 0, 0] = 0x7E
    cache[3][used] = (2.0 ** down * (1 + g.random((n, heads)))).astype(np.float32)
    q = np.abs(W.act_normal(10, 1, dim)).reshape(1, 1, dim)
    both(rz, 0, cache, q, page, table, [n], 18.0 / float(q.sum()))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("first,then", [(-100, 89), (89, -100), (-100, -20)])
def test_values_from_end_to_end(rz, fmt, first, then):
    """One workgroup's run of positions whose values' scales are of one end of the range, then of the other: the sum of the
    weights is of all of them."""
    page, heads, group, dim, n = 16, 1, 3, 64, 2100
    table, used, slots = paged(page, [n], 11)
    cache = raw_cache(fmt, slots, heads, dim, 11)
    fill(fmt, cache, used, 12)
    for at, e in ((used[:1024], first), (used[1024:], then)):
        if fmt == kv_cache.E4M3:
            cache[3][at] = (2.0 ** e * (1 + W.rng(13).random((len(at), heads)))).astype(np.float32)
        else:
            cache[3][at] = 127 + e
    q = W.act_normal(14, 1, group * dim).reshape(1, group, dim)
    # 1076 positions and more make the result: sqrt(8 * 1076 + 64) roundings of 2^-24 are 2^-17.4 if they are independent
    both(rz, fmt, cache, q, page, table, [n], 0.05, 2.0 ** -17.4)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [32, 128, 512])
@pytest.mark.parametrize("n,at", [(8, 3), (40, 39), (2500, 0), (2500, 1100)])
@pytest.mark.parametrize("size", [1e-5, 2.0 ** -40])
def test_value_rows_of_zeros(rz, fmt, dim, n, at, size):
    """A row of zeros among values of `size`, as an ordinary position and as the one that takes most of the weight: the others
    count as they do without it."""
    page, heads, group = 16, 2, 3
    table, used, slots = paged(page, [n], 1)
    cache = [x for _ in range(2) for x in kv_cache.empty(fmt, slots, heads, dim, 255)]
    g = W.rng(2)
    k, v = (g.standard_normal((n, heads, dim)).astype(np.float32) for _ in range(2))
    v *= np.float32(size)
    v[at, 0] = 0
    for sink in (False, True):
        if sink:
            k[at] = 6.0 * np.abs(k).max()
        kv_cache.write(fmt, k, used, *cache[:2])
        kv_cache.write(fmt, v, used, *cache[2:])
        assert not kv_serve.values(fmt, *cache[2:])[used[at], 0].any()
        q = np.abs(W.act_normal(3, 1, heads * group * dim)).reshape(1, heads * group, dim)
        both(rz, fmt, cache, q, page, table, [n], 0.5 / dim)


@pytest.mark.parametrize("negative", [False, True])
def test_value_rows_of_the_scale_of_zeros(rz, negative):
    """E4M3 rows whose largest magnitude is 1 have the scale that rows of zeros have, and count; a zero's sign does not."""
    page, heads, group, dim, n = 16, 1, 2, 64, 50
    table, used, slots = paged(page, [n], 4)
    cache = [x for _ in range(2) for x in kv_cache.empty(0, slots, heads, dim, 255)]
    g = W.rng(5)
    v = 1e-6 * g.standard_normal((n, heads, dim))
    v[7], v[9], v[11] = 0, 0, 0
    v[7, 0, 63], v[9, 0, 0] = 1, -1
    kv_cache.write(0, g.standard_normal((n, heads, dim)).astype(np.float32), used, *cache[:2])
    kv_cache.write(0, v.astype(np.float32), used, *cache[2:])
    assert (cache[3][used[[7, 9, 11]]] == np.float32(1) / np.float32(448)).all()
    if negative:
        cache[2][used[11], 0, ::2] = 0x80
    q = W.act_normal(6, 1, group * dim).reshape(1, group, dim)
    both(rz, 0, cache, q, page, table, [n], 0.2)
    # the rows of 1 out of the way: the row of zeros alone must not set the unit
    cache[2][used[[7, 9]]], cache[3][used[[7, 9]]] = cache[2][used[8]], cache[3][used[8]]
    both(rz, 0, cache, q, page, table, [n], 0.2)


@pytest.mark.parametrize("scale,down,up", [(2.0 ** -16, -100, 88), (2.0 ** -30, -95, 88), (-2.0 ** -14, -99, 85), (1e-30, 0, 88), (2.0 ** 30, -100, 60), (1e-42, 0, 0)])
def test_small_and_large_scales(rz, scale, down, up):
    """Queries of 2^down with keys of scales of 2^up: what their products lose to scale they do not get back."""
    page, heads, group, dim, n = 16, 1, 2, 64, 40
    table, used, slots = paged(page, [n], 15)
    cache = raw_cache(0, slots, heads, dim, 15)
    fill(0, cache, used, 16)
    cache[1][used] *= np.float32(2.0 ** up * 64)
    q = (W.act_normal(17, 1, group * dim) * 2.0 ** down).astype(np.float32).reshape(1, group, dim)
    both(rz, 0, cache, q, page, table, [n], float(np.float32(scale)))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [30, 700, 5000])
@pytest.mark.parametrize("size", [20, 25, 33, 50, 80])
@pytest.mark.parametrize("scale", [1.0, -0.37])
def test_scores_past_2_to_the_24(rz, fmt, n, size, scale):
    """Queries of one column, so that scores have their keys' order to the last bit: where they are 2^20 and more the largest
    takes all.  Its weight is 1 and their sum is 1, so what is left, in roundings of 2^-24, are the weight's parts (4), the
    value's as it is read (1) and four additions of 2 at most: 16 bounds it.  A score has q's product with scale log2(e) (3),
    its parts (4), two additions (4) and the row's scale (2), and lse 2 for its way back from powers of two: 15."""
    page, heads, group, dim = 16, 1, 3, 64
    table, used, slots = paged(page, [n], 18)
    cache = raw_cache(fmt, slots, heads, dim, 18)
    g = W.rng(19 + n)
    kv_cache.write(fmt, g.standard_normal((n, heads, dim)).astype(np.float32), used, *cache[:2])
    kv_cache.write(fmt, g.standard_normal((n, heads, dim)).astype(np.float32), used, *cache[2:])
    if fmt == kv_cache.MXFP4:  # few different values: one position ahead of the others
        cache[0][used] &= 0xBB
        cache[0][used[n // 2]] = np.where(scale > 0, 0x77, 0xFF)
        cache[1][used] = 127
    q = np.zeros((1, group, dim), dtype=np.float32)
    for i in range(group):
        q[0, i, 21 * i] = 1.25 * 2.0 ** size * (1 + i)
    k, v = (kv_serve.values(fmt, *c)[used, 0].astype(np.float64) for c in (cache[:2], cache[2:]))
    s = q[0].astype(np.float64) @ k.T * np.float32(scale)
    top = s.argmax(1)
    gap = np.sort(s, 1)[:, -1] - np.sort(s, 1)[:, -2]
    assert (gap > 2.0 ** -18 * np.abs(s).max(1)).all() and (gap > 40).all()
    outs = [whole(rz, fmt, cache, q, page, table, [n], scale)]
    out, lse = run(rz, fmt, cache, dev(q), page, table, [n], scale)
    assert (np.abs(host(lse)[0] - s.max(1)) <= 15 * 2.0 ** -24 * s.max(1)).all()
    for x in (*outs, out):
        x = host(x)[0].astype(np.float64)
        assert np.isfinite(x).all()
        assert (np.abs(x - v[top]) <= 16 * 2.0 ** -24 * np.abs(v[top]) + n * 2.0 ** -38 * np.abs(v).max()).all()
