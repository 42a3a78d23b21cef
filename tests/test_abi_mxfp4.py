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


def test_kv_read(L):
    good = [1, P, P, P, P, 64, 2, 64, 16, P, 3, 4, P, 20, 2, P, P, None]
    refuses_each(L.rz_kv_cache_read, good, (1, 2, 3, 4, 9, 12, 15, 16))
    refuses_each(L.rz_kv_cache_read, good, (1, 2, 3, 4, 15, 16), ALIGN, BAD)
    refuses_each(L.rz_kv_cache_read, good, (9, 12), ALIGN, P + 2)
    for at, v, status in ((0, -1, VALUE), (14, 3, VALUE), (8, 0, SHAPE), (6, 0, SHAPE), (7, 40, SHAPE), (13, 0x80000000, SHAPE)):
        assert L.rz_kv_cache_read(*(good[:at] + [v] + good[at + 1:])) == status, (at, v)
    assert L.rz_kv_cache_read(*(good[:13] + [0] + good[14:])) == OK


class Fake:
    """Enough of a device tensor for the binding's checks."""

    def __init__(self, dtype, *shape, strides=None, device="cuda:0"):
        self.dtype, self.shape, self.device, self.is_cuda = dtype, torch.Size(shape), torch.device(device), True
        self._strides = strides or torch.empty(shape, device="meta").stride()

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self, i=None):
        return tuple(self._strides) if i is None else self._strides[i]

    def get_device(self):
        return self.device.index

    def is_contiguous(self):
        return tuple(self._strides) == torch.empty(self.shape, device="meta").stride()

    def data_ptr(self):
        return P


F32, U8, I32, I64 = torch.float32, torch.uint8, torch.int32, torch.int64


def mx(rows, k, **kw):
    g = (rows + 31) // 32
    return Fake(U8, g, k // 64, 1024, **kw), Fake(U8, g, k // 256, 256, **kw)


def test_binding_refuses(L):
    a, w, o = mx(37, 512), mx(70, 512), Fake(F32, 37, 70)
    bad = [
        lambda: rz.rz_mxfp4_quant(torch.zeros(2, 256)),
        lambda: rz.rz_mxfp4_quant(Fake(torch.bfloat16, 2, 256), *mx(2, 256)),
        lambda: rz.rz_mxfp4_quant(Fake(F32, 2, 256, strides=(512, 1)), *mx(2, 256)),
        lambda: rz.rz_mxfp4_quant(Fake(F32, 33, 256), *mx(2, 256)),
        lambda: rz.rz_mxfp4_pack_weight(12, Fake(U8, 143), 1, 256, *mx(1, 256)),
        lambda: rz.rz_mxfp4_dequant(*a, 65, out=Fake(F32, 65, 512)),
        lambda: rz.rz_mxfp4_dequant(*a, 37, dtype=torch.float64),
        lambda: rz.rz_mxfp4_dequant(*a, 37, out=Fake(F32, 36, 512)),
        lambda: rz.rz_mxfp4_gemm(*a, 70, *w, 70, y=o),
        lambda: rz.rz_mxfp4_gemm(*a, 37, *w, 37, y=Fake(F32, 37, 37)),
        lambda: rz.rz_mxfp4_gemm(*a, 37, *mx(70, 768), 70, y=o),
        lambda: rz.rz_mxfp4_gemm(a[0], mx(37, 768)[1], 37, *w, 70, y=o),
        lambda: rz.rz_mxfp4_gemm(*a, 37, *w, 70, y=Fake(F32, 70, 37)),
        lambda: rz.rz_mxfp4_gemm(*a, 37, *mx(70, 512, device="cuda:1"), 70, y=o),
        lambda: rz.rz_mxfp4_gated(*a, 37, w, mx(70, 256), 70, h=o),
        lambda: rz.rz_mxfp4_gated(*a, -1, w, w, 70, h=o),
        lambda: rz.rz_mxfp4_gated_quant(*a, 37, mx(256, 512), mx(256, 512), 256, *mx(65, 256)),
        lambda: rz.rz_mxfp4_gemv(*w, 70, Fake(F32, 2, 256), y=Fake(F32, 2, 70)),
        lambda: rz.rz_mxfp4_gated_gemv(w, mx(70, 768), 70, Fake(F32, 2, 512), h=Fake(F32, 2, 70)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"case {i} was not refused")


def test_binding_refuses_cache(L):
    c = [Fake(U8, 10, 2, 64), Fake(F32, 10, 2)] * 2
    k, slots = Fake(F32, 3, 2, 64), Fake(I64, 3)
    t, off = Fake(I32, 2, 4), Fake(I32, 3)
    bad = [
        lambda: rz.rz_kv_cache_write(2, k, k, slots, *c),
        lambda: rz.rz_kv_cache_write(1, k, k, slots, *c),
        lambda: rz.rz_kv_cache_write(0, k, Fake(F32, 4, 2, 64), slots, *c),
        lambda: rz.rz_kv_cache_write(0, k, k, Fake(I32, 3), *c),
        lambda: rz.rz_kv_cache_write(0, k, k, Fake(I64, 2), *c),
        lambda: rz.rz_kv_cache_write(0, k, Fake(F32, 3, 2, 64, strides=(128, 1, 2)), slots, *c),
        lambda: rz.rz_kv_cache_write(0, Fake(torch.float16, 3, 2, 64), k, slots, *c),
        lambda: rz.rz_kv_cache_write(0, k, k, slots, c[0], Fake(F32, 10, 2, 1), c[2], c[3]),
        lambda: rz.rz_kv_cache_read(0, *c, 16, t, Fake(I32, 2), 5),
        lambda: rz.rz_kv_cache_read(0, *c, 16, Fake(I64, 2, 4), off, 5),
        lambda: rz.rz_kv_cache_read(0, *c, 0, t, off, 5),
        lambda: rz.rz_kv_cache_read(0, *c, 16, t, off, -1),
        lambda: rz.rz_kv_cache_read(0, *c, 16, t, off, 5, Fake(F32, 5, 2, 32), Fake(F32, 5, 2, 32)),
        lambda: rz.rz_kv_cache_read(0, *c, 16, t, off, 5, Fake(F32, 5, 2, 64), Fake(torch.float16, 5, 2, 64)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"case {i} was not refused")
