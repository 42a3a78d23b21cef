"""What the small-batch products state of weights at the top of the scale range
(needs an MI355X)."""
import numpy as np
import pytest

import workloads as W
from oracle import mxfp4
from test_gpu_mxfp4 import dev, host, random_tensor, tiled

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def rz():
    import fp8_prefill_gemm_amd as rz
    rz.lib()  # loud failure if the HIP library is missing
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return rz


@pytest.mark.parametrize("m", [1, 2, 3, 8])
def test_weights_past_fp32(rz, m):
    """One weight a row, every code at scale bytes 250 to 254, times 2^-20: exact where the weight fits fp32
    (parts of x with at most 8 bits leave one rounding-free term), an infinity or a NaN where not."""
    k, rows = 512, [(b, c) for b in range(250, 255) for c in range(16)]
    codes, byte = np.zeros((len(rows), k), dtype=np.uint8), np.zeros((len(rows), k // 32), dtype=np.uint8)
    for r, (b, c) in enumerate(rows):
        col = (37 * r) % k
        codes[r, col], byte[r, col // 32] = c, b
    w = mxfp4.dequant(codes, byte)
    x = np.full((m, k), 2.0 ** -20, dtype=np.float32)
    y = host(rz.rz_mxfp4_gemv(*tiled((codes, byte)), len(rows), dev(x))).astype(np.float64)
    fits = (np.abs(w) < 2.0 ** 128).all(1)
    assert fits.any() and not fits.all()
    assert np.array_equal(y[:, fits], (x.astype(np.float64) @ w.T)[:, fits])
    assert not np.isfinite(y[:, ~fits]).any()


@pytest.mark.parametrize("m,n,k", [(40, 70, 512), (1700, 4000, 512)])
def test_gemm_stated_bound_down_to_zero(rz, m, n, k):
    """Products from 2^-152 to 2^-87: within the stated bound, flushed ones counted."""
    a, w = random_tensor(301, m, k), random_tensor(302, n, k)
    g = W.rng(303)
    a[1][:] = g.integers(52, 82, a[1].shape)
    w[1][:] = g.integers(52, 82, w[1].shape)
    ref, bound = mxfp4.gemm(mxfp4.dequant(*a), mxfp4.dequant(*w))
    y = host(rz.rz_mxfp4_gemm(*tiled(a), m, *tiled(w), n)).astype(np.float64)
    assert (np.abs(y - ref) <= bound + 2 * k * 2.0 ** -126).all()


@pytest.mark.parametrize("m", [1, 2, 8])
def test_gemv_stated_bound_down_to_zero(rz, m):
    """Products from 2^-238 to 2^-90 and inputs from 2^-110 on: within the stated bound, underflow counted."""
    n, k = 70, 512
    w = random_tensor(304, n, k)
    g = W.rng(305)
    w[1][:] = g.integers(0, 30, w[1].shape)
    x = np.ldexp(np.where(g.integers(0, 2, (m, k)), 1.0, -1.0) * (1 + g.random((m, k))), g.integers(-110, 5, (m, k))).astype(np.float32)
    ref, bound = mxfp4.gemv(x, mxfp4.dequant(*w))
    y = host(rz.rz_mxfp4_gemv(*tiled(w), n, dev(x))).astype(np.float64)
    assert (np.abs(y - ref) <= bound + 2 * k * 2.0 ** -126).all()
