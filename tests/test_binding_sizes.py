"""Sizes beyond 32 bits reach no entry point: the C functions count rows,
columns, heads, sequences and pages in uint32, so the binding refuses what
would wrap.  Zero-size and one-element tensors stand in for the large ones; the
checks come before any other, so no GPU is needed."""
import os

import pytest

import fp8_prefill_gemm_amd as rz

torch = pytest.importorskip("torch")

F32, U8, I32, I64 = torch.float32, torch.uint8, torch.int32, torch.int64
BIG = 1 << 32  # wraps to 0, BIG + 256 to 256


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(rz.lib_path()):
        pytest.skip("librz_fp8.so not built")


def none(*shape, dtype=U8):
    """A contiguous tensor of `shape` with a zero among its sizes: no memory."""
    return torch.empty(shape, dtype=dtype)


def mx0(k):
    """An MXFP4 tensor of no rows and k columns."""
    return none(0, k // 64, 1024), none(0, k // 256, 256)


WIDE = mx0(BIG + 256)
CACHE = [none(0, 2, 64), none(0, 2, dtype=F32)] * 2
MANY_HEADS = [none(0, BIG + 2, 64), none(0, BIG + 2, dtype=F32)] * 2
WIDE_ROWS = [none(0, 2, BIG + 64), none(0, 2, dtype=F32)] * 2
HALF_ROWS = [none(0, 2, BIG // 2 + 32), none(0, 2, BIG // 32 + 2)] * 2  # dim = 2^32 + 64
SLOTS, TAB, OFF = none(0, dtype=I64), torch.zeros(2, 4, dtype=I32), torch.zeros(3, dtype=I32)
X = none(0, 2, 64, dtype=F32)

CALLS = {
    "quant columns": lambda: rz.rz_mxfp4_quant(none(0, BIG + 256, dtype=F32)),
    "quant rows": lambda: rz.rz_mxfp4_quant(none(BIG + 32, 0, dtype=F32)),
    "dequant columns": lambda: rz.rz_mxfp4_dequant(*WIDE, 0),
    "gemm columns": lambda: rz.rz_mxfp4_gemm(*WIDE, 0, *WIDE, 0),
    "gated columns": lambda: rz.rz_mxfp4_gated(*WIDE, 0, WIDE, WIDE, 0),
    "gated_quant columns": lambda: rz.rz_mxfp4_gated_quant(*WIDE, 0, WIDE, WIDE, 0),
    "gemv columns": lambda: rz.rz_mxfp4_gemv(*WIDE, 0, none(0, BIG + 256, dtype=F32)),
    "gated_gemv columns": lambda: rz.rz_mxfp4_gated_gemv(WIDE, WIDE, 0, none(0, BIG + 256, dtype=F32)),
    "gemv rows": lambda: rz.rz_mxfp4_gemv(none(0, 0, 1024), none(0, 0, 256), 0, none(BIG + 1, 0, dtype=F32)),
    "write tokens": lambda: rz.rz_kv_cache_write(0, none(BIG + 1, 2, 0, dtype=F32), none(BIG + 1, 2, 0, dtype=F32), SLOTS,
                                                 *[none(4, 2, 0), torch.zeros(4, 2)] * 2),
    "write heads": lambda: rz.rz_kv_cache_write(0, none(0, BIG + 2, 64, dtype=F32), none(0, BIG + 2, 64, dtype=F32), SLOTS, *MANY_HEADS),
    "write dim": lambda: rz.rz_kv_cache_write(0, none(0, 2, BIG + 64, dtype=F32), none(0, 2, BIG + 64, dtype=F32), SLOTS, *WIDE_ROWS),
    "write dim of nibbles": lambda: rz.rz_kv_cache_write(1, none(0, 2, BIG + 64, dtype=F32), none(0, 2, BIG + 64, dtype=F32), SLOTS, *HALF_ROWS),
    "read heads": lambda: rz.rz_kv_cache_read(0, *MANY_HEADS, 16, TAB, OFF, 0),
    "read dim": lambda: rz.rz_kv_cache_read(0, *WIDE_ROWS, 16, TAB, OFF, 0),
    "read pages": lambda: rz.rz_kv_cache_read(0, *CACHE, 16, none(0, BIG + 4, dtype=I32), torch.zeros(1, dtype=I32), 0),
    "read sequences": lambda: rz.rz_kv_cache_read(0, *CACHE, 16, none(BIG + 2, 0, dtype=I32), OFF, 0),
}


@pytest.mark.parametrize("what", CALLS)
def test_sizes_past_32_bits_are_refused(what):
    with pytest.raises(ValueError, match="=42949.* to 4294967295"):
        CALLS[what]()


def test_packed_weight_sizes():
    """n and k are plain numbers, checked as such."""
    for n, k in ((BIG, 256), (1, BIG + 256)):
        with pytest.raises(ValueError, match="to 4294967295"):
            rz.rz_mxfp4_pack_weight(12, torch.zeros(144, dtype=U8), n, k)
