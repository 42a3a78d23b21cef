"""Pins of the MXFP4 and cache oracles that do not re-derive them: fixed
points of the format, ties, closed forms and the layout's corner bytes."""
import numpy as np
import pytest

from oracle import kv_cache, mxfp4

VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def block(*head, fill=0.0):
    x = np.full(32, fill, dtype=np.float32)
    x[:len(head)] = head
    return x


def test_grid_values_are_fixed_points():
    """A block that holds the grid itself (absmax 6, X = 1) keeps it, at every scale."""
    both = np.array(VALUES + [-v for v in VALUES], dtype=np.float64)
    x = np.concatenate([both, both])
    for e in (-126, -20, 0, 1, 100, 125):
        c, b = mxfp4.quant(np.ldexp(x, e).astype(np.float32))
        assert b.tolist() == [127 + e]
        assert c[:16].tolist() == list(range(16))
        assert np.array_equal(mxfp4.dequant(c, b), np.ldexp(x, e))


@pytest.mark.parametrize("x,code", [
    (0.25, 0), (0.2500001, 1), (0.75, 2), (0.7499999, 1), (1.25, 2), (1.75, 4), (2.5, 4), (2.5000002, 5),
    (3.5, 6), (5.0, 6), (5.000001, 7), (6.5, 7), (7.9999, 7), (-0.25, 8), (-0.75, 10), (-7.5, 15), (-0.0, 8)])
def test_ties_and_saturation(x, code):
    """Next to a 4.0 (X = 1): ties to the even code, past 6 saturates."""
    c, b = mxfp4.quant(block(x, 4.0))
    assert b.tolist() == [127] and c[0] == code and c[1] == 6


@pytest.mark.parametrize("a,byte", [
    (0.0, 0), (1.0, 125), (1.9999999, 125), (2.0, 126), (4.0, 127), (7.9999995, 127), (8.0, 128), (3.4e38, 252),
    (2.0 ** -125, 0), (2.0 ** -124, 1), (2.0 ** -126, 0), (2.0 ** -149, 0), (np.inf, 255), (-np.inf, 255), (np.nan, 255)])
def test_scale_byte(a, byte):
    c, b = mxfp4.quant(block(0.0, a))
    assert b.tolist() == [byte]
    if byte == 255:
        assert not c.any() and np.isnan(mxfp4.dequant(c, b)).all()


def test_one_bad_block_leaves_the_next():
    x = np.concatenate([block(1.0, np.nan), block(1.0, fill=2.0)])
    v = mxfp4.dequant(*mxfp4.quant(x))
    assert np.isnan(v[:32]).all() and v[32] == 1.0 and (v[33:] == 2.0).all()


def test_layout_corners():
    """Bytes of single values: (r, c) -> offset, written out by hand for k = 512."""
    k = 512
    for (r, c), code_at, scale_at in [((0, 0), 0, 0), ((0, 1), 0, 0), ((0, 32), 512, 128), ((1, 0), 16, 4), ((0, 64), 1024, 1),
                                      ((0, 256), 4096, 256), ((32, 0), 8192, 512), ((33, 511), 8192 + 7 * 1024 + 512 + 16 + 15, 512 + 256 + 128 + 4 + 3)]:
        x = np.zeros((40, k), dtype=np.float32)
        x[r, c] = 4.0
        tc, ts = mxfp4.quant_tiled(x)
        assert tc.shape == (2, 8, 1024) and ts.shape == (2, 2, 256)
        assert np.flatnonzero(tc).tolist() == [code_at] and tc.reshape(-1)[code_at] == (6 << 4 if c % 2 else 6)
        assert np.flatnonzero(ts).tolist() == [scale_at] and ts.reshape(-1)[scale_at] == 127


def test_products_closed_form():
    a = np.full((2, 64), 0.5)
    w = np.full((3, 64), -3.0)
    y, b = mxfp4.gemm(a, w)
    assert (y == -96.0).all() and (b > 0).all() and (b < 96 * 64 * 2.0 ** -22).all()
    h, _ = mxfp4.gated((np.array([[0.0, 2.0]]), 0.0), (np.array([[5.0, 3.0]]), 0.0))
    assert h[0, 0] == 0 and abs(h[0, 1] - 6 / (1 + np.exp(-2.0))) < 1e-15


@pytest.mark.parametrize("fmt", [kv_cache.E4M3, kv_cache.MXFP4])
def test_cache_round_trip_and_bounds(fmt):
    """Powers of two survive; dropped tokens, short tables and foreign slots read as they should."""
    x = np.ones((3, 2, 64), dtype=np.float32)
    x[1] = -4.0
    codes, scales = kv_cache.empty(fmt, 8, 2, 64)
    kv_cache.write(fmt, x, np.array([6, 3, -1]), codes, scales)
    assert not codes[[0, 1, 2, 4, 5, 7]].any()
    out = np.full((6, 2, 64), 9.0, dtype=np.float32)
    kv_cache.read(fmt, codes, scales, 2, np.array([[3, 7], [1, -1]]), [1, 2, 5], out)
    rel = 0 if fmt == kv_cache.MXFP4 else 2.0 ** -22  # RN(1/448) * 448 is within an ulp of 1
    assert (out[[0, 5]] == 9).all()
    assert np.abs(out[1] - 1).max() <= rel            # page 3, position 0: slot 6
    assert (out[2] == 0).all() and np.abs(out[3] + 4).max() <= 4 * rel  # page 1: slots 2 and 3
    assert (out[4] == 0).all()                        # page -1
