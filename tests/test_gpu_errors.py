"""A failed call is reported once (run on a B200): the next one answers for itself alone."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from two_sided_adaptive_bakron_b200 import build
    build.build()
    from two_sided_adaptive_bakron_b200 import bakron
    return bakron


def _refused_by_cuda(bk):
    """Reads a status word on a stream that is being captured: the runtime refuses to wait there."""
    driver = ctypes.CDLL("libcuda.so.1")
    stream, graph = torch.cuda.Stream(), ctypes.c_void_p()
    handle = ctypes.c_void_p(stream.cuda_stream)
    st = bk.new_status("cuda")
    torch.cuda.synchronize()
    assert driver.cuStreamBeginCapture_v2(handle, 2) == 0          # 2: this stream only
    code = bk.bakron_read_status(st, stream)
    driver.cuStreamEndCapture(handle, ctypes.byref(graph))
    assert not graph.value                                         # the capture is void
    return code


@pytest.mark.parametrize("call", ["pack4", "matvec4", "rms_norm_q8", "distill", "row_scales"])
def test_an_error_is_not_kept_for_the_next_call(bk, call):
    x = torch.randn(4, 64, device="cuda")
    codes = torch.zeros(32, 64, dtype=torch.int8, device="cuda")
    layer = bk.PackedLayer(codes, torch.ones(32, device="cuda"))
    idx, top = torch.zeros(4, 1, dtype=torch.int32, device="cuda"), torch.zeros(4, 1, device="cuda")
    calls = {"pack4": lambda: bk.PackedLayer(codes, torch.ones(32, device="cuda")),
             "matvec4": lambda: layer.matvec(x), "rms_norm_q8": lambda: bk.rms_norm_q8(x),
             "distill": lambda: bk.distill(x, idx, top), "row_scales": lambda: bk.row_scales(x, 64, 7.5)}
    calls[call]()
    assert _refused_by_cuda(bk) == bk.BAKRON_ERR_CUDA
    calls[call]()
    torch.cuda.synchronize()
