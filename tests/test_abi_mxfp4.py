"""Refusals of the MXFP4 and cache entry points, checked without a GPU: bad
arguments return their status before any HIP call, and the binding raises
before it calls.  The pointers are fake addresses, never dereferenced."""
import os

import pytest

import fp8_prefill_gemm_amd as rz

torch = pytest.importorskip("torch")

OK, NULL, QTYPE, SHAPE, ALIGN, HIP, VALUE = 0, -1, -2, -3, -4, -5, -6
P = 0x7F0000001000
BAD = 0x7F0000001008
BIG_K = (1 << 24) - 256


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(rz.lib_path()):
        pytest.skip("librz_fp8.so not built")
    return rz.lib()


def refuses_each(f, args, pointers, status=NULL, value=None):
    """f refuses `args` with each of the pointer positions replaced in turn."""
    for i in pointers:
        a = list(args)
        a[i] = value
        assert f(*a) == status, i


def test_sizes(L):
    assert [L.rz_mxfp4_pad_rows(r) for r in (0, 1, 32, 33, 2048)] == [0, 32, 32, 64, 2048] == [rz.rz_mxfp4_pad_rows(r) for r in (0, 1, 32, 33, 2048)]
    assert L.rz_mxfp4_code_bytes(33, 512) == 64 * 256 and L.rz_mxfp4_scale_bytes(33, 512) == 64 * 16
    assert L.rz_mxfp4_code_bytes(33, 300) == 0 == L.rz_mxfp4_scale_bytes(33, 0)


def test_quant(L):
    good = (P, 4, 256, P, P, None)
    refuses_each(L.rz_mxfp4_quant, good, (0, 3, 4))
    refuses_each(L.rz_mxfp4_quant, good, (0, 3, 4), ALIGN, BAD)
    for k in (0, 100, 257, BIG_K + 256):
        assert L.rz_mxfp4_quant(P, 4, k, P, P, None) == SHAPE
    assert L.rz_mxfp4_quant(P, 1 << 20, 1 << 20, P, P, None) == SHAPE
    assert L.rz_mxfp4_quant(P, 0xFFFFFFFF, 256, P, P, None) == SHAPE
    assert L.rz_mxfp4_quant(None, 0, 256, None, None, None) == OK


def test_pack_weight(L):
    good = (12, P, 4, 256, P, P, None)
    refuses_each(L.rz_mxfp4_pack_weight, good, (1, 4, 5))
    refuses_each(L.rz_mxfp4_pack_weight, good, (1, 4, 5), ALIGN, BAD)
    assert L.rz_mxfp4_pack_weight(2, P, 4, 256, P, P, None) == QTYPE
    assert L.rz_mxfp4_pack_weight(12, P, 0, 256, P, P, None) == SHAPE
    assert L.rz_mxfp4_pack_weight(12, P, 4, 128, P, P, None) == SHAPE
    assert L.rz_mxfp4_pack_weight(14, P, 1 << 23, 1 << 15, P, P, None) == SHAPE


def test_dequant(L):
    good = (P, P, 4, 256, 0, P, None)
    refuses_each(L.rz_mxfp4_dequant, good, (0, 1, 5))
    refuses_each(L.rz_mxfp4_dequant, good, (0, 1, 5), ALIGN, BAD)
    assert L.rz_mxfp4_dequant(P, P, 4, 256, 3, P, None) == VALUE
    assert L.rz_mxfp4_dequant(P, P, 4, 64, 0, P, None) == SHAPE
    assert L.rz_mxfp4_dequant(None, None, 0, 256, 2, None, None) == OK


def test_gemm(L):
    good = (P, P, 4, P, P, 8, 256, P, None)
    refuses_each(L.rz_mxfp4_gemm, good, (0, 1, 3, 4, 7))
    refuses_each(L.rz_mxfp4_gemm, good, (0, 1, 3, 4, 7), ALIGN, BAD)
    for m, n, k in ((4, 8, 0), (4, 8, 300), (4, 8, BIG_K + 256), (4, 1 << 24, 256), (1 << 30, 1 << 10, 256), (0x80000000, 1, 256)):
        assert L.rz_mxfp4_gemm(P, P, m, P, P, n, k, P, None) == SHAPE
    assert L.rz_mxfp4_gemm(None, None, 0, None, None, 8, 256, None, None) == OK
    assert L.rz_mxfp4_gemm(None, None, 4, None, None, 0, 256, None, None) == OK


def test_gated(L):
    good = (P, P, 4, P, P, P, P, 256, 256, P, None)
    refuses_each(L.rz_mxfp4_gated, good, (0, 1, 3, 4, 5, 6, 9))
    refuses_each(L.rz_mxfp4_gated, good, (0, 1, 3, 4, 5, 6, 9), ALIGN, BAD)
    assert L.rz_mxfp4_gated(P, P, 4, P, P, P, P, 256, 100, P, None) == SHAPE
    good = (P, P, 4, P, P, P, P, 256, 256, P, P, None)
    refuses_each(L.rz_mxfp4_gated_quant, good, (0, 1, 3, 4, 5, 6, 9, 10))
    refuses_each(L.rz_mxfp4_gated_quant, good, (0, 1, 3, 4, 5, 6, 9, 10), ALIGN, BAD)
    assert L.rz_mxfp4_gated_quant(P, P, 4, P, P, P, P, 288, 256, P, P, None) == SHAPE
    assert L.rz_mxfp4_gated_quant(None, None, 0, None, None, None, None, 256, 256, None, None, None) == OK


def test_gemv(L):
    good = (P, P, 8, 256, P, 4, P, None)
    refuses_each(L.rz_mxfp4_gemv, good, (0, 1, 4, 6))
    refuses_each(L.rz_mxfp4_gemv, good, (0, 1, 4, 6), ALIGN, BAD)
    assert L.rz_mxfp4_gemv(P, P, 8, 256, P, 9, P, None) == SHAPE
    assert L.rz_mxfp4_gemv(P, P, 8, 250, P, 1, P, None) == SHAPE
    good = (P, P, P, P, 8, 256, P, 4, P, None)
    refuses_each(L.rz_mxfp4_gated_gemv, good, (0, 1, 2, 3, 6, 8))
    refuses_each(L.rz_mxfp4_gated_gemv, good, (0, 1, 2, 3, 6, 8), ALIGN, BAD)
    assert L.rz_mxfp4_gated_gemv(P, P, P, P, 8, 256, P, 9, P, None) == SHAPE


def test_kv_write(L):
    good = [0, P, P, 4, 2, 64, 128, 128, P, 10, P, P, P, P, None]
    refuses_each(L.rz_kv_cache_write, good, (1, 2, 8, 10, 11, 12, 13))
    refuses_each(L.rz_kv_cache_write, good, (1, 2, 10, 11, 12, 13), ALIGN, BAD)
    refuses_each(L.rz_kv_cache_write, good, (8,), ALIGN, P + 4)
    for at, v, status in ((0, 2, VALUE), (4, 0, SHAPE), (5, 0, SHAPE), (5, 48, SHAPE), (5, 544, SHAPE), (6, 124, SHAPE), (7, 130, SHAPE),
                          (9, 1 << 40, SHAPE), (4, 1 << 22, SHAPE)):
        assert L.rz_kv_cache_write(*(good[:at] + [v] + good[at + 1:])) == status, (at, v)
    assert L.rz_kv_cache_write(1, None, None, 0, 2, 64, 0, 0, None, 10, None, None, None, None, None) == OK


def test_kv_call_too_large(L):
    """Grids count lanes in 32 bits: more than 2^33 values in one call are refused, as are 2^31 sequences."""
    for tokens, heads, dim, status in (((1 << 28) + 1, 1, 32, SHAPE), ((1 << 20) + 1, 64, 128, SHAPE), (1 << 31, 1, 32, SHAPE)):
        assert L.rz_kv_cache_write(0, P, P, tokens, heads, dim, heads * dim, heads * dim, P, 10, P, P, P, P, None) == status
        assert L.rz_kv_cache_read(1, P, P, P, P, 64, heads, dim, 16, P, 3, 4, P, tokens, 2, P, P, None) == status
    assert L.rz_kv_cache_read(1, P, P, P, P, 64, 1, 32, 16, P, 0xFFFFFFFF, 4, P, 1, 2, P, P, None) == SHAPE


def test_kv_read(L):
    good = [1, P, P, P, P, 64, 2, 64, 16, P, 3, 4, P, 20, 2, P, P, None]
    refuses_each(L.rz_kv_cache_read, good, (1, 2, 3, 4, 9, 12, 15, 16))
    refuses_each(L.rz_kv_cache_read, good, (1, 2, 3, 4, 15, 16), ALIGN, BAD)
    refuses_each(L.rz_kv_cache_read, good, (9, 12), ALIGN, P + 2)
    for at, v, status in ((0, -1, VALUE), (14, 3, VALUE), (8, 0, SHAPE), (6, 0, SHAPE), (7, 40, SHAPE), (13, 0x80000000, SHAPE)):
        assert L.rz_kv_cache_read(*(good[:at] + [v] + good[at + 1:])) == status, (at, v)
    assert L.rz_kv_cache_read(*(good[:13] + [0] + good[14:])) == OK


# The binding's checks of a CPU tensor end with the one for a device, so what
# they say before it can be tested here: every call below names its own fault.
F32, U8, I32, I64 = torch.float32, torch.uint8, torch.int32, torch.int64


def mx(rows, k):
    g = (rows + 31) // 32
    return torch.zeros(g, k // 64, 1024, dtype=U8), torch.zeros(g, k // 256, 256, dtype=U8)


def f32(*shape):
    return torch.zeros(*shape)


A, X = mx(37, 512), f32(37, 512)
Wt = mx(70, 512)

ACCEPTED = [
    lambda: rz.rz_mxfp4_quant(X),
    lambda: rz.rz_mxfp4_quant(X, *A),
    lambda: rz.rz_mxfp4_pack_weight(12, torch.zeros(2 * 2, 144, dtype=U8), 2, 512),
    lambda: rz.rz_mxfp4_dequant(*A, 37, dtype=torch.bfloat16),
    lambda: rz.rz_mxfp4_gemm(*A, 37, *Wt, 70),
    lambda: rz.rz_mxfp4_gated(*A, 37, Wt, Wt, 70),
    lambda: rz.rz_mxfp4_gated_quant(*A, 37, mx(256, 512), mx(256, 512), 256),
    lambda: rz.rz_mxfp4_gemv(*Wt, 70, f32(2, 512)),
    lambda: rz.rz_mxfp4_gated_gemv(Wt, Wt, 70, f32(2, 512)),
]

REFUSED = [
    ("x: expected a contiguous Float", lambda: rz.rz_mxfp4_quant(torch.zeros(2, 256, dtype=torch.bfloat16))),
    ("x: expected a contiguous Float", lambda: rz.rz_mxfp4_quant(f32(2, 512)[:, :256])),
    ("x: expected 2 dimensions", lambda: rz.rz_mxfp4_quant(f32(2, 2, 256))),
    ("blocks: 143 bytes, 144 needed", lambda: rz.rz_mxfp4_pack_weight(12, torch.zeros(143, dtype=U8), 1, 256)),
    ("n=-1", lambda: rz.rz_mxfp4_pack_weight(12, torch.zeros(144, dtype=U8), -1, 256)),
    ("blocks: expected a contiguous Byte", lambda: rz.rz_mxfp4_pack_weight(12, torch.zeros(144), 1, 256)),
    ("input: expected a contiguous Byte", lambda: rz.rz_mxfp4_dequant(*A, 65)),
    ("dtype: expected float32, float16 or bfloat16", lambda: rz.rz_mxfp4_dequant(*A, 37, dtype=torch.float64)),
    ("a: expected a contiguous Byte", lambda: rz.rz_mxfp4_gemm(*A, 70, *Wt, 70)),
    ("w: expected a contiguous Byte", lambda: rz.rz_mxfp4_gemm(*A, 37, *Wt, 37)),
    ("w: expected a contiguous Byte", lambda: rz.rz_mxfp4_gemm(*A, 37, Wt[0].view(-1), Wt[1], 70)),
    ("operands have k=512 and k=768", lambda: rz.rz_mxfp4_gemm(*A, 37, *mx(70, 768), 70)),
    ("a: expected a contiguous Byte", lambda: rz.rz_mxfp4_gemm(A[0], mx(37, 768)[1], 37, *Wt, 70)),
    ("m=-1", lambda: rz.rz_mxfp4_gemm(*A, -1, *Wt, 70)),
    ("m=4294967296", lambda: rz.rz_mxfp4_gemm(*A, 1 << 32, *Wt, 70)),
    ("operands have k=512 and k=256", lambda: rz.rz_mxfp4_gated(*A, 37, Wt, mx(70, 256), 70)),
    ("a: expected a contiguous Byte", lambda: rz.rz_mxfp4_gated_quant(*mx(65, 512), 37, mx(256, 512), mx(256, 512), 256)),
    ("x: expected a contiguous Float", lambda: rz.rz_mxfp4_gemv(*Wt, 70, f32(2, 256))),
    ("x: expected a contiguous Float", lambda: rz.rz_mxfp4_gemv(*Wt, 70, f32(512))),
    ("operands have k=512 and k=768", lambda: rz.rz_mxfp4_gated_gemv(Wt, mx(70, 768), 70, f32(2, 512))),
]

C = [torch.zeros(10, 2, 64, dtype=U8), f32(10, 2)] * 2
K, SL = f32(3, 2, 64), torch.zeros(3, dtype=I64)
TAB, OFF = torch.zeros(2, 4, dtype=I32), torch.zeros(3, dtype=I32)

ACCEPTED += [
    lambda: rz.rz_kv_cache_write(0, K, f32(3, 256)[:, 128:].view(3, 2, 64), SL, *C),
    lambda: rz.rz_kv_cache_read(0, *C, 16, TAB, OFF, 5, dtype=torch.float16),
]
REFUSED += [
    ("fmt=2", lambda: rz.rz_kv_cache_write(2, K, K, SL, *C)),
    ("k_scales: expected a contiguous Byte", lambda: rz.rz_kv_cache_write(1, K, K, SL, *C)),
    ("k_scales: expected a contiguous Float", lambda: rz.rz_kv_cache_write(0, K, K, SL, C[0], f32(10, 2, 1), *C[2:])),
    ("v_codes: expected a contiguous Byte", lambda: rz.rz_kv_cache_write(0, K, K, SL, *C[:2], C[0][:9], C[1])),
    ("v: expected a contiguous Float", lambda: rz.rz_kv_cache_write(0, K, f32(4, 2, 64), SL, *C)),
    ("k: expected a contiguous Float", lambda: rz.rz_kv_cache_write(0, f32(3, 64, 2).transpose(1, 2), K, SL, *C)),
    ("k: expected a contiguous Float", lambda: rz.rz_kv_cache_write(0, f32(1, 2, 64).expand(3, 2, 64), K, SL, *C)),
    ("k: expected a contiguous Float", lambda: rz.rz_kv_cache_write(0, K.half(), K, SL, *C)),
    ("slots: expected a contiguous Long", lambda: rz.rz_kv_cache_write(0, K, K, SL.int(), *C)),
    ("slots: expected a contiguous Long", lambda: rz.rz_kv_cache_write(0, K, K, SL[:2], *C)),
    ("offsets: expected a contiguous Int", lambda: rz.rz_kv_cache_read(0, *C, 16, TAB, OFF[:2], 5)),
    ("page_table: expected a contiguous Int", lambda: rz.rz_kv_cache_read(0, *C, 16, TAB.long(), OFF, 5)),
    ("page_table: expected 2 dimensions", lambda: rz.rz_kv_cache_read(0, *C, 16, TAB[0], OFF, 5)),
    ("page_len=0", lambda: rz.rz_kv_cache_read(0, *C, 0, TAB, OFF, 5)),
    ("rows=-1", lambda: rz.rz_kv_cache_read(0, *C, 16, TAB, OFF, -1)),
    ("dtype: expected", lambda: rz.rz_kv_cache_read(0, *C, 16, TAB, OFF, 5, dtype=torch.float64)),
]


@pytest.mark.parametrize("i", range(len(ACCEPTED)))
def test_binding_wants_a_device(L, i):
    with pytest.raises(ValueError, match="works on device"):
        ACCEPTED[i]()


@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_binding_refuses(L, i):
    with pytest.raises(ValueError) as e:
        REFUSED[i][1]()
    assert str(e.value).startswith(REFUSED[i][0]) or REFUSED[i][0] in str(e.value)


def test_binding_wants_tensors(L):
    with pytest.raises(TypeError, match="x: expected a tensor, got list"):
        rz.rz_mxfp4_quant([1.0])
    with pytest.raises(TypeError):
        rz.rz_mxfp4_gemm(*A, 37.0, *Wt, 70)
