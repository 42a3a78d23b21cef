"""Which kernel an MXFP4 product launches, and that every one is tested with K
long enough for each of its stages (no GPU needed)."""
import ctypes
import os

import pytest

import fp8_prefill_gemm_amd as rz

# (tokens, weight rows, ways) of a workgroup, and shapes that launch it with K past two full turns of its
# waves: an odd and an even number of 256-column steps where the stages alternate.
PLAIN = {
    (32, 32, 8): [(31, 70, 4864)],
    (64, 32, 8): [(37, 4608, 4864), (37, 4608, 4352)],
    (64, 64, 4): [(250, 3500, 4864), (300, 3300, 2816)],
    (64, 256, 1): [(520, 4500, 2304), (640, 3584, 3584)],
    (96, 256, 1): [(2048, 4608, 2304), (1500, 3584, 4608)],
    (128, 256, 1): [(1541, 4001, 2304), (1990, 7100, 2560)],
    (160, 256, 1): [(4135, 2300, 4352), (4135, 2300, 4608)],
    (192, 256, 1): [(4135, 2500, 4352), (4135, 2500, 4608)],
}
# gated: rows of each weight; widths are multiples of 256 for the MXFP4 output
GATED = {
    (32, 32, 8): [(37, 256, 4864)],
    (64, 32, 4): [(128, 4608, 2304), (100, 4608, 2816)],
    (64, 128, 1): [(160, 9472, 2304), (160, 9472, 2560)],
    (96, 128, 1): [(2048, 2304, 2304), (1500, 1792, 4608)],
    (128, 128, 1): [(1990, 1792, 2304), (1990, 3584, 2560)],
    (160, 128, 1): [(4135, 1024, 4352), (4135, 1024, 4608)],
    (192, 128, 1): [(4135, 1280, 4352), (4135, 1280, 4608)],
}
CASES = [(g, plan, s) for g, kernels in ((False, PLAIN), (True, GATED)) for plan, shapes in kernels.items() for s in shapes]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(rz.lib_path()):
        pytest.skip("librz_fp8.so not built")


@pytest.mark.parametrize("gated,plan,shape", CASES)
def test_long_k_shapes_reach_their_kernel(gated, plan, shape):
    m, n, k = shape
    rows, cols, ways, groups = rz.rz_mxfp4_gemm_plan(m, n, k, gated)
    assert (rows, cols, ways) == plan
    assert groups == -(-m // rows) * -(-n // cols)
    assert k // 256 > 2 * ways, "a wave takes a third turn"
    if gated:
        assert n % 256 == 0


def test_plan_arguments():
    out = (ctypes.c_int32 * 4)()
    p = ctypes.cast(out, ctypes.c_void_p)
    L = rz.lib()
    assert L.rz_mxfp4_gemm_plan(4, 8, 256, 0, None) == -1
    for m, n, k in ((4, 8, 0), (4, 8, 300), (4, 8, 1 << 24), (4, 1 << 24, 256), (0x80000000, 1, 256)):
        assert L.rz_mxfp4_gemm_plan(m, n, k, 0, p) == -3
    for m, n in ((0, 8), (8, 0), (0, 0)):
        assert rz.rz_mxfp4_gemm_plan(m, n, 256) == (0, 0, 0, 0)


def test_plans_cover_the_output():
    """The grid holds every tile, and every plan is one of the kernels above."""
    for gated, kernels in ((False, PLAIN), (True, GATED)):
        for m in (1, 31, 32, 33, 64, 97, 250, 511, 1025, 2048, 4135, 1 << 20):
            for n in (1, 33, 512, 2300, 4608, 9000, 18944, 40000):
                for k in (256, 2048, 2304, 4096, 4352, 18944):
                    rows, cols, ways, groups = rz.rz_mxfp4_gemm_plan(m, n, k, gated)
                    assert (rows, cols, ways) in kernels
                    assert groups == -(-m // rows) * -(-n // cols)
