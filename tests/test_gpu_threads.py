"""Calls from several host threads at once (run on a B200): every entry point may be called from any
thread, so a call's launch does not depend on what another thread's call set up in between."""
import threading

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


def _at_once(calls, times=400):
    """Each call ``times`` over in a thread of its own, on a stream of its own; what they raised."""
    torch.cuda.synchronize()
    errors, start = [], threading.Barrier(len(calls))

    def work(call):
        stream = torch.cuda.Stream()
        start.wait()
        try:
            with torch.cuda.stream(stream):
                for _ in range(times):
                    call()
            stream.synchronize()
        except Exception as e:      # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return errors


def test_products_of_layers_of_different_sizes(bk):
    """Blocks of the same kernel with different amounts of shared memory."""
    import ctypes
    book = (ctypes.c_float * 16)(*range(16))
    calls, checks = [], []
    for m, n, cb in [(64, 4096, None), (96, 1024, None), (64, 8192, None), (48, 4096, book),
                     (80, 1024, book), (16, 8192, book)]:
        codes = torch.randint(0, 8, (m, n), device="cuda", dtype=torch.int8)
        layer = bk.PackedLayer(codes, torch.rand(m, -(-n // 128), device="cuda"), 128, cb)
        x = torch.randn(4, n, device="cuda").bfloat16()
        y = torch.empty(4, m, device="cuda", dtype=torch.bfloat16)
        checks.append((layer.matvec(x), y))

        def call(m=m, n=n, cb=cb, packed=layer.packed, x=x, y=y, fn=bk.lib().bakron_matvec4):
            code = fn(packed.data_ptr(), m, n, 128, cb, 4, x.data_ptr(), 2, n, None, 0, 4,
                      y.data_ptr(), 2, m, torch.cuda.current_stream().cuda_stream)
            assert code == 0, bk.status_string(code)
        calls.append(call)
    assert _at_once(calls, 4000) == []
    assert all(torch.equal(a, b) for a, b in checks)
