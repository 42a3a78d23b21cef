"""Refusals of the serving entry points, checked without a GPU: bad arguments
return their status before any HIP call, and the binding raises before it
calls.  The pointers are fake addresses, never dereferenced."""
import os

import pytest

import fp8_prefill_gemm_amd as rz
from test_abi_mxfp4 import ALIGN, BAD, F32, I32, I64, NULL, OK, P, SHAPE, U8, VALUE, f32, refuses_each

torch = pytest.importorskip("torch")
ODD = P + 2


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(rz.lib_path()):
        pytest.skip("librz_fp8.so not built")
    return rz.lib()


def changed(good, at, v):
    return [*good[:at], v, *good[at + 1:]]


def test_plan(L):
    #       lens keep off seqs tokens page table width free pages count lens_out count_out slots ws stream
    good = [P, P, P, 4, 9, 16, P, 8, P, 50, P, P, P, P, P, None]
    refuses_each(L.rz_kv_plan, good, (0, 2, 6, 8, 10, 11, 12, 13))
    if L.rz_kv_plan_workspace_bytes(4, 9):
        refuses_each(L.rz_kv_plan, good, (14,))
    refuses_each(L.rz_kv_plan, good, (0, 1, 2, 6, 8, 10, 11, 12), ALIGN, ODD)
    refuses_each(L.rz_kv_plan, good, (13,), ALIGN, P + 4)
    refuses_each(L.rz_kv_plan, good, (14,), ALIGN, BAD)
    for at, v in ((5, 0), (3, 0x7FFFFFFF), (4, 0x80000000), (9, 0x80000000)):
        assert L.rz_kv_plan(*changed(good, at, v)) == SHAPE, (at, v)
    assert L.rz_kv_plan(*changed(changed(good, 3, 1 << 20), 7, 1 << 20)) == SHAPE


#            fmt q q_heads stride kc ks vc vs slots heads dim page table seqs width lens pages budget scale dtype out lse ws stream
ATTENTION = [0, P, 6, 6 * 64, P, P, P, P, 64, 2, 64, 16, P, 3, 4, P, None, 0, 0.5, 0, P, None, P, None]


def test_attention(L):
    f = L.rz_kv_attention
    refuses_each(f, ATTENTION, (1, 4, 5, 6, 7, 12, 15, 20))
    refuses_each(f, ATTENTION, (1, 4, 5, 6, 7, 20, 22), ALIGN, BAD)
    refuses_each(f, ATTENTION, (12, 15, 21), ALIGN, ODD)
    chosen = changed(changed(ATTENTION, 17, 5), 16, P)
    refuses_each(f, chosen, (16,), ALIGN, ODD)
    for at, v, status in ((0, 2, VALUE), (19, 3, VALUE), (18, float("inf"), VALUE), (18, float("nan"), VALUE), (2, 0, SHAPE), (2, 5, SHAPE), (2, 1 << 21, SHAPE), (3, 380, SHAPE),
                          (3, 386, SHAPE), (9, 0, SHAPE), (10, 0, SHAPE), (10, 40, SHAPE), (10, 544, SHAPE), (11, 0, SHAPE), (8, 1 << 40, SHAPE), (13, 1 << 30, SHAPE)):
        assert f(*changed(ATTENTION, at, v)) == status, (at, v)
    assert f(*changed(chosen, 17, 1 << 27)) == SHAPE
    assert f(0, None, 6, 0, None, None, None, None, 64, 2, 64, 16, None, 0, 4, None, None, 0, 0.5, 0, None, None, None, None) == OK
    assert L.rz_kv_attention_workspace_bytes(0, 6, 2, 64) == 0 == L.rz_kv_attention_workspace_bytes(3, 5, 2, 64)


def test_bounds(L):
    good = [0, P, P, 64, 2, 64, 16, P, 9, P, P, None]
    refuses_each(L.rz_kv_bounds, good, (1, 2, 7, 9, 10))
    refuses_each(L.rz_kv_bounds, good, (1, 2, 9, 10), ALIGN, BAD)
    refuses_each(L.rz_kv_bounds, good, (7,), ALIGN, P + 4)
    for at, v, status in ((0, 2, VALUE), (3, 1 << 40, SHAPE), (4, 0, SHAPE), (5, 40, SHAPE), (6, 0, SHAPE), (8, 0xFFFFFFFF, SHAPE)):
        assert L.rz_kv_bounds(*changed(good, at, v)) == status, (at, v)
    assert L.rz_kv_bounds(0, None, None, 64, 2, 64, 16, None, 0, None, None, None) == OK
    assert L.rz_kv_bounds(0, None, None, 15, 2, 64, 16, None, 9, None, None, None) == OK  # no whole page


def test_select(L):
    #       q q_heads stride bounds scales pages heads dim page table seqs width lens budget out ws stream
    good = [P, 6, 6 * 64, P, P, 20, 2, 64, 16, P, 3, 4, P, 2, P, P, None]
    refuses_each(L.rz_kv_select, good, (0, 3, 4, 9, 12, 14))
    long = changed(changed(good, 11, 100000), 15, None)  # too many pages for one launch
    assert L.rz_kv_select_workspace_bytes(3, 2, 100000) == 3 * 2 * 100000 * 4 and L.rz_kv_select(*long) == NULL
    refuses_each(L.rz_kv_select, good, (0, 3, 4, 15), ALIGN, BAD)
    refuses_each(L.rz_kv_select, good, (9, 12, 14), ALIGN, ODD)
    for at, v in ((1, 0), (1, 5), (2, 380), (2, 386), (6, 0), (7, 48), (8, 0), (13, 0), (11, 1 << 25), (10, 1 << 21)):
        assert L.rz_kv_select(*changed(good, at, v)) == SHAPE, (at, v)
    assert L.rz_kv_select(None, 6, 0, None, None, 20, 2, 64, 16, None, 0, 4, None, 2, None, None, None) == OK


def test_select_budget_past_31_bits(L):
    """A choice is filled up with -1 by 32-bit places a workgroup's width apart, which would wrap for budgets near 2^32."""
    good = [P, 6, 6 * 64, P, P, 20, 2, 64, 16, P, 1, 4, P, 2, P, P, None]
    for budget in (0x80000000, 0xFFFFFC01, 0xFFFFFFFF):
        assert L.rz_kv_select(*changed(good, 13, budget)) == SHAPE, budget
        assert L.rz_kv_select(None, 6, 0, None, None, 20, 2, 64, 16, None, 0, 4, None, budget, None, None, None) == SHAPE, budget


# The binding's checks of a CPU tensor end with the one for a device.
C = [torch.zeros(32, 2, 64, dtype=U8), f32(32, 2)] * 2
MX = [torch.zeros(32, 2, 32, dtype=U8), torch.zeros(32, 2, 2, dtype=U8)] * 2
Q, TAB, LENS, OFF = f32(3, 6, 64), torch.zeros(3, 4, dtype=I32), torch.zeros(3, dtype=I32), torch.zeros(4, dtype=I32)
FREE, ONE, SL = torch.zeros(9, dtype=I32), torch.zeros(1, dtype=I32), torch.zeros(5, dtype=I64)
B, BS = torch.zeros(2, 2, 2, 64, dtype=torch.int8), f32(2, 2)

ACCEPTED = [
    lambda **k: rz.rz_kv_plan(LENS, OFF, 5, 16, TAB, FREE, ONE, **k),
    lambda **k: rz.rz_kv_plan(LENS, OFF, 5, 16, TAB, FREE, ONE, keep=LENS, **k),
    lambda **k: rz.rz_kv_attention(0, Q, *C, 16, TAB, LENS, 0.1, **k),
    lambda **k: rz.rz_kv_attention(1, f32(3, 400)[:, 16:].view(3, 6, 64), *MX, 16, TAB, LENS, 1, pages=torch.zeros(3, 2, 0, dtype=I32), dtype=torch.float16, **k),
    lambda **k: rz.rz_kv_bounds(0, *C[:2], SL, 16, B, BS, **k),
    lambda **k: rz.rz_kv_bounds(1, *MX[:2], SL, 16, B, BS, **k),
    lambda **k: rz.rz_kv_select(Q, B, BS, 16, TAB, LENS, 2, **k),
]

REFUSED = [
    ("lens: expected a contiguous Int", lambda **k: rz.rz_kv_plan(LENS.long(), OFF, 5, 16, TAB, FREE, ONE, **k)),
    ("offsets: expected a contiguous Int", lambda **k: rz.rz_kv_plan(LENS, OFF[:3], 5, 16, TAB, FREE, ONE, **k)),
    ("page_table: expected a contiguous Int", lambda **k: rz.rz_kv_plan(LENS, OFF, 5, 16, torch.zeros(4, 3, dtype=I32).t(), FREE, ONE, **k)),
    ("page_table: expected 2 dimensions", lambda **k: rz.rz_kv_plan(LENS, OFF, 5, 16, TAB[0], FREE, ONE, **k)),
    ("free_pages: expected 1 dimension", lambda **k: rz.rz_kv_plan(LENS, OFF, 5, 16, TAB, TAB, ONE, **k)),
    ("free_count: expected a contiguous Int", lambda **k: rz.rz_kv_plan(LENS, OFF, 5, 16, TAB, FREE, FREE, **k)),
    ("keep: expected a contiguous Int", lambda **k: rz.rz_kv_plan(LENS, OFF, 5, 16, TAB, FREE, ONE, keep=OFF, **k)),
    ("page_len=0", lambda **k: rz.rz_kv_plan(LENS, OFF, 5, 0, TAB, FREE, ONE, **k)),
    ("tokens=-1", lambda **k: rz.rz_kv_plan(LENS, OFF, -1, 16, TAB, FREE, ONE, **k)),
    ("tokens=4294967296", lambda **k: rz.rz_kv_plan(LENS, OFF, 1 << 32, 16, TAB, FREE, ONE, **k)),
    ("fmt=2", lambda **k: rz.rz_kv_attention(2, Q, *C, 16, TAB, LENS, 0.1, **k)),
    ("q: expected a contiguous Float", lambda **k: rz.rz_kv_attention(0, Q.half(), *C, 16, TAB, LENS, 0.1, **k)),
    ("q: expected a contiguous Float", lambda **k: rz.rz_kv_attention(0, Q[:2], *C, 16, TAB, LENS, 0.1, **k)),
    ("q: expected a contiguous Float", lambda **k: rz.rz_kv_attention(0, f32(3, 64, 6).transpose(1, 2), *C, 16, TAB, LENS, 0.1, **k)),
    ("q: expected a contiguous Float", lambda **k: rz.rz_kv_attention(0, f32(3, 384), *C, 16, TAB, LENS, 0.1, **k)),
    ("k_scales: expected a contiguous Byte", lambda **k: rz.rz_kv_attention(1, Q, *C, 16, TAB, LENS, 0.1, **k)),
    ("v_codes: expected a contiguous Byte", lambda **k: rz.rz_kv_attention(0, Q, *C[:2], C[0][:9], C[1], 16, TAB, LENS, 0.1, **k)),
    ("page_table: expected a contiguous Int", lambda **k: rz.rz_kv_attention(0, Q, *C, 16, TAB.long(), LENS, 0.1, **k)),
    ("lens: expected a contiguous Int", lambda **k: rz.rz_kv_attention(0, Q, *C, 16, TAB, OFF, 0.1, **k)),
    ("pages: expected a contiguous Int", lambda **k: rz.rz_kv_attention(0, Q, *C, 16, TAB, LENS, 0.1, pages=torch.zeros(3, 6, 2, dtype=I32), **k)),
    ("pages: expected 3 dimensions", lambda **k: rz.rz_kv_attention(0, Q, *C, 16, TAB, LENS, 0.1, pages=TAB, **k)),
    ("lse: expected a contiguous Float", lambda **k: rz.rz_kv_attention(0, Q, *C, 16, TAB, LENS, 0.1, lse=f32(3, 2), **k)),
    ("dtype: expected", lambda **k: rz.rz_kv_attention(0, Q, *C, 16, TAB, LENS, 0.1, dtype=torch.float64, **k)),
    ("page_len=0", lambda **k: rz.rz_kv_attention(0, Q, *C, 0, TAB, LENS, 0.1, **k)),
    ("k_scales: expected a contiguous Float", lambda **k: rz.rz_kv_bounds(0, C[0], MX[1], SL, 16, B, BS, **k)),
    ("slots: expected a contiguous Long", lambda **k: rz.rz_kv_bounds(0, *C[:2], SL.int(), 16, B, BS, **k)),
    ("bounds: expected a contiguous Char", lambda **k: rz.rz_kv_bounds(0, *C[:2], SL, 8, B, BS, **k)),
    ("bounds: expected a contiguous Char", lambda **k: rz.rz_kv_bounds(0, *C[:2], SL, 16, B.to(U8), BS, **k)),
    ("bounds: expected 4 dimensions", lambda **k: rz.rz_kv_bounds(0, *C[:2], SL, 16, B[0], BS, **k)),
    ("bound_scales: expected a contiguous Float", lambda **k: rz.rz_kv_bounds(0, *C[:2], SL, 16, B, f32(2), **k)),
    ("q: expected a contiguous Float", lambda **k: rz.rz_kv_select(f32(3, 6, 32), B, BS, 16, TAB, LENS, 2, **k)),
    ("budget=0", lambda **k: rz.rz_kv_select(Q, B, BS, 16, TAB, LENS, 0, **k)),
    ("pages: expected a contiguous Int", lambda **k: rz.rz_kv_select(Q, B, BS, 16, TAB, LENS, 2, pages=torch.zeros(3, 2, 3, dtype=I32), **k)),
]
#: Outputs are checked behind the device: these end there on a CPU.
ACCEPTED.append(REFUSED.pop())


class Stream:
    """Stands in for a torch stream: the calls below end before it is used."""
    cuda_stream = 0


@pytest.mark.parametrize("kw", [{}, {"stream": Stream()}])
@pytest.mark.parametrize("i", range(len(ACCEPTED)))
def test_binding_wants_a_device(L, i, kw):
    f = ACCEPTED[i] if callable(ACCEPTED[i]) else ACCEPTED[i][1]
    with pytest.raises(ValueError, match="works on device"):
        f(**kw)


@pytest.mark.parametrize("kw", [{}, {"stream": Stream()}])
@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_binding_refuses(L, i, kw):
    with pytest.raises(ValueError) as e:
        REFUSED[i][1](**kw)
    assert REFUSED[i][0] in str(e.value)


def test_binding_wants_tensors_and_numbers(L):
    with pytest.raises(TypeError, match="lens: expected a tensor, got list"):
        rz.rz_kv_plan([1], OFF, 5, 16, TAB, FREE, ONE)
    with pytest.raises(TypeError):
        rz.rz_kv_attention(0, Q, *C, 16, TAB, LENS, "1")
    with pytest.raises(TypeError):
        rz.rz_kv_select(Q, B, BS, 16.0, TAB, LENS, 2)
    with pytest.raises(TypeError, match="q: expected a tensor, got NoneType"):
        rz.rz_kv_select(None, B, BS, 16, TAB, LENS, 2)


def test_sizes_past_32_bits(L):
    big = 1 << 32
    none = lambda *s, dtype=U8: torch.empty(s, dtype=dtype)  # noqa: E731
    for call in (lambda: rz.rz_kv_plan(LENS, OFF, 5, 16, none(0, big + 4, dtype=I32), FREE, ONE),
                 lambda: rz.rz_kv_plan(LENS, OFF, 5, big + 16, TAB, FREE, ONE),
                 lambda: rz.rz_kv_attention(0, none(0, big + 2, 0, dtype=F32), *C, 16, TAB[:0], LENS[:0], 1.0),
                 lambda: rz.rz_kv_attention(0, Q, *C, 16, TAB, LENS, 1.0, pages=none(0, 2, big + 2, dtype=I32)),
                 lambda: rz.rz_kv_select(Q, none(0, big + 2, 2, 64, dtype=torch.int8), none(0, big + 2, dtype=F32), 16, TAB, LENS, 2),
                 lambda: rz.rz_kv_select(Q, B, BS, 16, TAB, LENS, big + 2)):
        with pytest.raises(ValueError, match="=42949.* to 4294967295"):
            call()
