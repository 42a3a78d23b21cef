"""What a call says of wrong arguments does not depend on `stream`: the same
errors with a stream as without one (no GPU: every check comes before the
stream is used)."""
import os

import pytest

import fp8_prefill_gemm_amd as rz
from test_abi_mxfp4 import ACCEPTED, REFUSED

torch = pytest.importorskip("torch")

NAMES = ["rz_mxfp4_quant", "rz_mxfp4_pack_weight", "rz_mxfp4_dequant", "rz_mxfp4_gemm", "rz_mxfp4_gated", "rz_mxfp4_gated_quant",
         "rz_mxfp4_gemv", "rz_mxfp4_gated_gemv", "rz_kv_cache_write", "rz_kv_cache_read"]


class Stream:
    """Stands in for a torch stream: the calls below end before it is used."""
    cuda_stream = 0


@pytest.fixture
def on_a_stream(monkeypatch):
    """Every call of the module takes `stream`."""
    if not os.path.exists(rz.lib_path()):
        pytest.skip("librz_fp8.so not built")
    for name in NAMES:
        f = getattr(rz, name)
        monkeypatch.setattr(rz, name, lambda *a, _f=f, **kw: _f(*a, stream=Stream(), **kw))


@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_refusals(on_a_stream, i):
    with pytest.raises(ValueError) as e:
        REFUSED[i][1]()
    assert REFUSED[i][0] in str(e.value)


@pytest.mark.parametrize("i", range(len(ACCEPTED)))
def test_wants_a_device(on_a_stream, i):
    with pytest.raises(ValueError, match="works on device"):
        ACCEPTED[i]()


def test_wants_tensors(on_a_stream):
    with pytest.raises(TypeError, match="x: expected a tensor, got list"):
        rz.rz_mxfp4_quant([1.0])
    with pytest.raises(TypeError, match="w: expected a tensor, got NoneType"):
        rz.rz_mxfp4_gemv(None, None, 70, torch.zeros(2, 512))


def test_outputs_that_are_no_tensors(on_a_stream):
    """The element type is taken from the outputs only where they are tensors."""
    codes, scales = torch.zeros(2, 8, 1024, dtype=torch.uint8), torch.zeros(2, 2, 256, dtype=torch.uint8)
    cache = [torch.zeros(10, 2, 64, dtype=torch.uint8), torch.zeros(10, 2)] * 2
    table, offsets = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for bad in ([1.0], 7):
        for call in (lambda: rz.rz_mxfp4_dequant(codes, scales, 37, out=bad),
                     lambda: rz.rz_kv_cache_read(0, *cache, 16, table, offsets, 5, k_out=bad),
                     lambda: rz.rz_kv_cache_read(0, *cache, 16, table, offsets, 5, v_out=bad)):
            with pytest.raises((TypeError, ValueError), match="expected a tensor|works on device"):
                call()
