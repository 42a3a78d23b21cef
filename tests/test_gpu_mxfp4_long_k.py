"""MXFP4 products whose waves take more than two turns of K, one shape or more
for every kernel (needs an MI355X): a wrong stage, prefetch or scale register
shows from the second or third turn on only."""
import numpy as np
import pytest

import workloads as W
from oracle import mxfp4
from test_gpu_mxfp4 import host, random_tensor, same, small_scale, tiled, within
from test_mxfp4_plans import CASES

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def rz():
    import fp8_prefill_gemm_amd as rz
    rz.lib()  # loud failure if the HIP library is missing
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return rz


def some_rows(m):
    """At most 128 tokens: the first, the last 40, others anywhere."""
    if m <= 128:
        return np.arange(m)
    return np.unique(np.concatenate([np.arange(8), W.rng(m).integers(8, m - 40, 80), np.arange(m - 40, m)]))


@pytest.mark.parametrize("gated,plan,shape", CASES)
def test_every_kernel_with_a_long_k(rz, gated, plan, shape):
    m, n, k = shape
    print(f"mxfp4 long K m={m} n={n} k={k} gated={gated}", flush=True)
    assert rz.rz_mxfp4_gemm_plan(m, n, k, gated)[:3] == plan
    a, w = random_tensor(500 + m, m, k, 3), random_tensor(501 + n, n, k, 3)
    sel = some_rows(m)
    av = mxfp4.dequant(a[0][sel], a[1][sel])
    if not gated:
        y = rz.rz_mxfp4_gemm(*tiled(a), m, *tiled(w), n)
        return within(y[torch.from_numpy(sel).cuda()], *mxfp4.gemm(av, mxfp4.dequant(*w)))
    g, u = small_scale(w, 8), small_scale(random_tensor(502 + n, n, k, 3), 8)
    ta, tg, tu = tiled(a), tiled(g), tiled(u)
    h = rz.rz_mxfp4_gated(*ta, m, tg, tu, n)
    within(h[torch.from_numpy(sel).cuda()], *mxfp4.gated(mxfp4.gemm(av, mxfp4.dequant(*g)), mxfp4.gemm(av, mxfp4.dequant(*u))))
    hc, hs = rz.rz_mxfp4_gated_quant(*ta, m, tg, tu, n)
    tc, ts = mxfp4.quant_tiled(host(h))
    same(hs, ts)
    same(hc, tc)
