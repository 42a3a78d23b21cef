"""The serving oracle against cases worked out by hand."""
import numpy as np
import pytest

from oracle import kv_cache, kv_serve


def test_plan_by_hand():
    """Pages of 4: one sequence grows past its page, one ends, one starts, one stays inside its page."""
    table = np.array([[7, -1, -1], [3, 5, -1], [-1, -1, -1], [2, -1, -1]], dtype=np.int32)
    free = np.array([1, 6, 0, 9, 9, 9, 9, 9], dtype=np.int32)
    slots, lens, count = kv_serve.plan([4, 6, 0, 1], [4, 0, 0, 1], [0, 1, 1, 6, 7], 8, 4, table, free, 3)
    # 3 and 5 come back on top of 1 6 0; sequence 0 takes 5, sequence 2 takes 3 and 0
    assert lens.tolist() == [5, 0, 5, 2] and count.tolist() == [2]
    assert slots.tolist() == [20, 12, 13, 14, 15, 0, 9, -1]
    assert table.tolist() == [[7, 5, -1], [3, 5, -1], [3, 0, -1], [2, -1, -1]]
    assert free.tolist() == [1, 6, 0, 3, 5, 9, 9, 9]


def test_plan_refusals_by_hand():
    """A sequence that the stack cannot serve stops those behind it that lack pages, and only those."""
    table = np.full((5, 4), -1, dtype=np.int32)
    table[3, 0], table[4, 0] = 8, 9
    free = np.arange(4, dtype=np.int32)
    #                                lens               keep              new: 2, 12, 1, 1, 1
    slots, lens, count = kv_serve.plan([0, 0, 0, 1, 1], [0, 0, 0, 1, 2], [0, 2, 14, 15, 16, 17], 17, 4, table, free, 3)
    assert lens.tolist() == [2, 0, 0, 2, 1]  # the last one keeps more than it has
    assert count.tolist() == [2] and slots[:2].tolist() == [8, 9] and (slots[2:15] == -1).all()
    assert slots[15:].tolist() == [33, -1]
    slots, lens, _ = kv_serve.plan([0], [0], [0, 17], 17, 4, np.full((1, 4), -1, dtype=np.int32), np.arange(9, dtype=np.int32), 9)
    assert lens.tolist() == [0] and (slots == -1).all()  # five pages, four columns


def test_plan_of_decreasing_offsets_by_hand():
    """Which tokens are whose is not known: no sequence gets any, and no page moves."""
    table = np.array([[7, 2, -1], [3, -1, -1], [-1, -1, -1]], dtype=np.int32)
    free, before = np.array([1, 6, 0, 9], dtype=np.int32), table.copy()
    slots, lens, count = kv_serve.plan([5, 4, 0], [1, 4, 0], [0, 4, 3, 8], 8, 4, table, free, 3)
    assert (slots == -1).all() and lens.tolist() == [5, 4, 0] and count.tolist() == [3]
    assert np.array_equal(table, before) and free.tolist() == [1, 6, 0, 9]


def test_slots_of_by_hand():
    table = np.array([[2, -1, 9, 0]], dtype=np.int32)
    assert kv_serve.slots_of(0, 0, 7, 2, table, 8) == [4, 5, 0]  # page 1 names nothing, page 2 lies outside
    pages = np.array([[[3, 0, -1, 4]]], dtype=np.int32)
    assert kv_serve.slots_of(0, 0, 7, 2, table, 8, pages) == [0, 4, 5]
    assert kv_serve.slots_of(0, 0, 0, 2, table, 8) == []


@pytest.mark.parametrize("fmt", [kv_cache.E4M3, kv_cache.MXFP4])
def test_values_are_the_caches(fmt):
    r = np.random.default_rng(1)
    codes = r.integers(0, 256, (5, 2, 64 if fmt == kv_cache.E4M3 else 32)).astype(np.uint8)
    scales = r.random((5, 2)).astype(np.float32) if fmt == kv_cache.E4M3 else r.integers(100, 140, (5, 2, 2)).astype(np.uint8)
    got = kv_serve.values(fmt, codes, scales)
    for s in range(5):
        for h in range(2):
            assert np.array_equal(got[s, h], kv_cache.read_row(fmt, codes[s, h], scales[s, h]), equal_nan=True)


def test_attention_by_hand():
    """Two positions with scores 0 and log 3, one query head of two on each key head; an empty sequence."""
    k, v = np.zeros((4, 2, 32), dtype=np.float32), np.zeros((4, 2, 32), dtype=np.float32)
    k[1, :, 0], v[0, :, 1], v[1, :, 1], v[:, 1] = 1, 4, 8, 1
    q = np.zeros((2, 4, 32), dtype=np.float32)
    q[:, :, 0] = 2 * np.log(3)
    out, lse, tol, ltol = kv_serve.attention(k, v, q, 2, np.array([[0], [0]]), [2, 0], 0.5)
    assert np.allclose(lse[0], np.log(4)) and np.allclose(out[0, :2, 1], 7) and np.allclose(out[0, 2:], 1)
    assert not out[1].any() and (lse[1] == -np.inf).all() and (tol >= 0).all() and tol[0].max() < 1e-3 and ltol.max() < 1e-3


def test_bounds_by_hand():
    k = np.zeros((6, 1, 32), dtype=np.float32)
    k[:, 0, 0], k[:, 0, 1], k[5, 0, 2] = [1, 2, -3, 9, 0, 0], [0.01, 0.02, 0.03, 0, 0, 0], np.nan
    codes, scales = np.full((3, 1, 2, 32), 5, dtype=np.int8), np.full((3, 1), 7, dtype=np.float32)
    kv_serve.bounds(k, [2, 5, -1, 9], 2, codes, scales)
    assert (codes[0] == 5).all() and scales[0, 0] == 7  # not named
    # page 1: filled up to slot 2 alone
    assert codes[1, 0, :, 0].tolist() == [-127, -127] and codes[1, 0, :, 1].tolist() == [2, 1] and scales[1, 0] == np.float32(3) / np.float32(127)
    assert (codes[2, 0, 0] == 127).all() and (codes[2, 0, 1] == -127).all() and scales[2, 0] == np.inf
    z = np.zeros((2, 1, 32), dtype=np.float32)
    kv_serve.bounds(z, [0, 1], 2, codes, scales)
    assert not codes[0].any() and scales[0, 0] == np.float32(1) / np.float32(127)


def test_select_keeps_the_newest_page():
    """Pages of infinite bounds come behind the first and the last page, whatever their number."""
    codes, scales = np.ones((6, 1, 2, 32), dtype=np.int8), np.ones((6, 1), dtype=np.float32)
    scales[1:5] = np.inf
    q, table = np.ones((1, 1, 32), dtype=np.float32), np.array([[0, 1, 2, 3, 4, 5]], dtype=np.int32)
    pick = lambda n, budget: kv_serve.select(q, codes, scales, 4, table, [n], budget)[0, 0].tolist()  # noqa: E731
    assert pick(24, 2) == [0, 5] and pick(24, 3) == [0, 1, 5] and pick(24, 5) == [0, 1, 2, 3, 5] and pick(24, 1) == [0]
    assert pick(13, 2) == [0, 3]
    scales[5] = 2.0
    assert pick(24, 1) == [0]  # of the two the lower, whatever they score


def test_bounds_hold():
    """hi * scale and lo * scale enclose the values to the scale's rounding, and a score is at least every n . k."""
    r = np.random.default_rng(2)
    k = (r.standard_normal((64, 2, 96)) * np.exp(r.standard_normal((1, 2, 96)))).astype(np.float32)
    codes, scales = np.zeros((8, 2, 2, 96), dtype=np.int8), np.zeros((8, 2), dtype=np.float32)
    kv_serve.bounds(k, range(64), 8, codes, scales)
    x = k.reshape(8, 8, 2, 96)
    s = scales[:, None, :, None].astype(np.float64)
    assert (x <= codes[:, None, :, 0] * s * (1 + 1e-6)).all() and (x >= codes[:, None, :, 1] * s - np.abs(x).max() * 1e-6).all()
    q = r.standard_normal((1, 96)).astype(np.float32)
    got = kv_serve.scores(q, codes[:, 0], scales[:, 0])
    a = np.abs(q).max()
    n = np.rint(q[0].astype(np.float64) * 127 / a) * a / 127
    assert (got >= (x[:, :, 0] @ n).max(1) - 1e-3).all()


def test_select_by_hand():
    """Ties to the lower page, the first and last page always, a page outside the cache never, -1 behind the last."""
    codes = np.zeros((6, 1, 2, 32), dtype=np.int8)
    codes[:, 0, 0, 0] = [1, 5, 3, 5, 2, 1]
    scales = np.ones((6, 1), dtype=np.float32)
    q = np.zeros((1, 1, 32), dtype=np.float32)
    q[0, 0, 0] = 2
    table = np.array([[0, 1, 2, 3, 4, 5]], dtype=np.int32)
    pick = lambda n, budget, t=table: kv_serve.select(q, codes, scales, 4, t, [n], budget)[0, 0].tolist()  # noqa: E731
    assert pick(24, 3) == [0, 1, 5] and pick(24, 4) == [0, 1, 3, 5] and pick(17, 4) == [0, 1, 3, 4]
    assert pick(24, 1) == [0] and pick(5, 4) == [0, 1, -1, -1] and pick(0, 2) == [-1, -1] and pick(99, 2) == [0, 5]
    assert pick(24, 3, np.array([[0, -1, 2, 6, 4, 5]], dtype=np.int32)) == [0, 2, 5]
    q[0, 0, 0] = -1  # the lower bounds count
    codes[2, 0, 1, 0] = -9
    assert pick(24, 3) == [0, 2, 5]
