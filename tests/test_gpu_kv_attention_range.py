"""GPU parity of attention over the paged cache at the ends of what its bound
holds for (needs an MI355X)."""
import ctypes

import numpy as np
import pytest

import workloads as W
from oracle import kv_cache, kv_serve
from test_gpu_kv_attention import FORMATS, check, dev, fill, paged, raw_cache, run

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
