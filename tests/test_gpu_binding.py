"""The binding's outputs and streams on the GPU (needs an MI355X)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def rz():
    import fp8_prefill_gemm_amd as rz
    rz.lib()  # loud failure if the HIP library is missing
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return rz


def test_outputs_are_the_streams_blocks(rz):
    """A freed output goes back to the stream it was made on, not to the current one; the current stream stays."""
    x = torch.randn((2048, 16384), device="cuda")  # 16 MB of codes: a segment of its own
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.current_stream()
    codes, scales = rz.rz_mxfp4_quant(x, stream=side)
    assert torch.cuda.current_stream() == before
    with pytest.raises(rz.RzError, match="exceeds 8"):  # a refusal restores it too
        rz.rz_mxfp4_gemv(codes, scales, 2048, x[:9], stream=side)
    assert torch.cuda.current_stream() == before
    torch.cuda.synchronize()
    at, shape = codes.data_ptr(), codes.shape
    del codes
    assert torch.empty(shape, dtype=torch.uint8, device="cuda").data_ptr() != at
    with torch.cuda.stream(side):
        assert torch.empty(shape, dtype=torch.uint8, device="cuda").data_ptr() == at


def test_default_stream_from_another(rz):
    """The default stream as an argument while another is current: the same bits, made on the default stream."""
    x = torch.randn((2048, 16384), device="cuda")
    want = rz.rz_mxfp4_quant(x)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = rz.rz_mxfp4_quant(x, stream=torch.cuda.default_stream())
        assert torch.cuda.current_stream() == side
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        at, shape = got[0].data_ptr(), got[0].shape
        del got, a, b
        assert torch.empty(shape, dtype=torch.uint8, device="cuda").data_ptr() != at
    assert torch.empty(shape, dtype=torch.uint8, device="cuda").data_ptr() == at
