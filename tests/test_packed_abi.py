"""CPU checks of the entry points around a packed layer: what they refuse, before any device work."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from two_sided_adaptive_bakron_b200 import build as B

INVALID = -1


@pytest.fixture(scope="module")
def bk():
    B.build()
    from two_sided_adaptive_bakron_b200 import bakron
    return bakron


@pytest.fixture(scope="module")
def L(bk):
    return bk.lib()


P = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1002)


def test_layout_bytes(bk):
    assert bk.bakron_pack4_bytes(16, 64, 64) == 512 + 64
    assert bk.bakron_pack4_bytes(17, 65, 32) == 4 * 512 + 2 * 3 * 64
    assert bk.bakron_pack4_bytes(1, 1, 1) == 512 + 64
    for m, n, g in [(0, 5, 5), (5, 0, 5), (5, 65537, 32), (65536, 32768, 32), (4, 64, 48),
                    (4, 64, 0), (-1, 4, 4)]:
        assert bk.bakron_pack4_bytes(m, n, g) == 0


def test_layout_bytes_of_the_binding(bk):
    for m, n, g in [(1, 1, 1), (16, 64, 32), (17, 65, 32), (28672, 8192, 128), (5, 700, 96),
                    (100, 65536, 32), (3, 50, 64)]:
        assert bk._packed_bytes(m, n, bk._steps(n, g)[1]) == bk.bakron_pack4_bytes(m, n, g)


def test_pack_refusals(L):
    def pack(codes=P, ldc=64, scales=P, m=8, n=64, g=32, u=0, packed=P, st=P):
        return L.bakron_pack4(codes, ldc, scales, m, n, g, u, packed, st, None)
    for bad in [dict(codes=None), dict(scales=None), dict(packed=None), dict(st=None), dict(ldc=63),
                dict(m=0), dict(n=0), dict(g=48), dict(u=2), dict(packed=ODD)]:
        assert pack(**bad) == INVALID, bad

    def unpack(packed=P, m=8, n=64, g=32, u=0, codes=P, ldc=64, scales=P):
        return L.bakron_unpack4(packed, m, n, g, u, codes, ldc, scales, None)
    for bad in [dict(codes=None), dict(scales=None), dict(packed=None), dict(ldc=63), dict(n=0),
                dict(g=0), dict(u=-1), dict(packed=ODD)]:
        assert unpack(**bad) == INVALID, bad


def test_matvec_refusals(L):
    book = (ctypes.c_float * 16)(*range(16))
    nan = (ctypes.c_float * 2)(0.0, float("nan"))

    def mv(packed=P, m=8, n=64, g=32, cb=None, bits=0, x=P, xd=2, ldx=64, xs=None, gx=64, tok=1,
           y=P, yd=2, ldy=8):
        return L.bakron_matvec4(packed, m, n, g, cb, bits, x, xd, ldx, xs, gx, tok, y, yd, ldy,
                                None)
    for bad in [dict(packed=None), dict(packed=ODD), dict(x=None), dict(y=None), dict(m=0),
                dict(n=65537, ldx=65537), dict(g=33), dict(xd=4), dict(xd=7), dict(yd=3),
                dict(ldx=63), dict(ldy=7), dict(tok=-1), dict(tok=65536), dict(xd=3),
                dict(xs=P), dict(xd=3, xs=P, gx=40), dict(xd=3, xs=P, gx=0),
                dict(cb=book, bits=0), dict(cb=book, bits=5), dict(cb=nan, bits=1),
                dict(xd=0, x=ODD), dict(yd=0, y=ODD), dict(x=ctypes.c_void_p(0x1001))]:
        assert mv(**bad) == INVALID, bad
    assert mv(tok=0, x=None, y=None) == 0       # no token: nothing to do


def test_norm_refusals(L):
    def nq(x=P, ldx=64, r=P, ldr=64, d=2, w=P, wd=2, rows=1, n=64, eps=1e-6, g=32, q=P, s=P, sm=P,
           lds=64):
        return L.bakron_rms_norm_q8(x, ldx, r, ldr, d, w, wd, rows, n, eps, g, q, s, sm, lds, None,
                                    None)
    for bad in [dict(x=None), dict(q=None), dict(s=None), dict(ldx=63), dict(ldr=63), dict(lds=63),
                dict(d=3), dict(wd=3), dict(rows=-1), dict(n=0), dict(n=65537, ldx=1 << 20,
                ldr=1 << 20, lds=1 << 20), dict(eps=0.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(g=48), dict(x=ctypes.c_void_p(0x1001)),
                dict(r=ctypes.c_void_p(0x1001)), dict(w=ODD, wd=0)]:
        assert nq(**bad) == INVALID, bad
    assert nq(rows=0, x=None) == 0


def test_distill_refusals(L):
    def ds(z=P, d=2, rows=1, V=64, ld=64, i=P, idd=4, t=P, td=0, k=3, tau=1.0, loss=P, lse=P,
           dz=None, ldd=0, st=P):
        return L.bakron_distill(z, d, rows, V, ld, i, idd, t, td, k, None, None, tau, loss, lse, dz,
                                ldd, st, None)
    for bad in [dict(z=None), dict(i=None), dict(t=None), dict(loss=None), dict(lse=None),
                dict(st=None), dict(d=3), dict(idd=0), dict(td=4), dict(k=0), dict(k=1025),
                dict(tau=0.0), dict(tau=-1.0), dict(tau=float("nan")), dict(tau=float("inf")),
                dict(tau=1e-40), dict(rows=-1), dict(V=0), dict(ld=63), dict(dz=P, ldd=63),
                dict(z=P, dz=P, ldd=65), dict(i=ODD), dict(idd=5, i=ctypes.c_void_p(0x1004)),
                dict(d=0, z=ODD)]:
        assert ds(**bad) == INVALID, bad
    assert ds(rows=0, z=None) == 0


def test_binding_refuses_what_the_library_cannot_see(bk):
    """Host tensors, other types, strided rows and wrong lengths raise in the binding."""
    z = torch.zeros(4, 64)
    for call in [lambda: bk.matvec4(z.to(torch.uint8), 4, 64, z),
                 lambda: bk.rms_norm_q8(z), lambda: bk.pack4(z.to(torch.int8), z[:, 0]),
                 lambda: bk.distill(z, z[:, :2].int(), z[:, :2])]:
        with pytest.raises((ValueError, RuntimeError)):
            call()
    with pytest.raises(ValueError, match="columns"):
        bk.matvec4(z.to(torch.uint8), 4, 63, z)
    with pytest.raises(ValueError, match="entries"):
        bk._codebook([0.0, 1.0, 2.0])
    with pytest.raises(ValueError, match="positive"):
        bk._steps(8, 0)
    meta = torch.zeros(4, 64, device="meta")
    with pytest.raises(ValueError, match="CUDA"):
        bk._rows(meta, "x", meta.get_device())


class _Stream:
    def __init__(self, device, cuda_stream=7):
        self.device, self.cuda_stream = torch.device(device), cuda_stream


def test_a_stream_handle_is_one_of_the_tensors_device(bk, monkeypatch):
    """Not of the current device, which may be another."""
    made = []
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda h, device=None: made.append((h, device)) or _Stream(device, h))
    monkeypatch.setattr(torch.cuda, "default_stream",
                        lambda device=None: made.append((0, device)) or _Stream(device, 0))
    dev = torch.device("cuda:1")
    for handle in (0x70, 0):
        assert bk._stream_on(handle, dev).device == dev
    assert made == [(0x70, dev), (0, dev)]
    own = _Stream("cuda:1")
    assert bk._stream_on(own, dev) is own
    with pytest.raises(ValueError, match="cuda:1"):
        bk._stream_on(_Stream("cuda:0"), dev)


def test_calls_take_the_device_of_their_tensors(bk, monkeypatch):
    seen = []

    class Enough(Exception):
        pass

    def stop(stream, device):
        seen.append((stream, device))
        raise Enough
    monkeypatch.setattr(bk, "_stream_on", stop)
    t = torch.zeros(4, 64, device="meta")
    for call in [lambda: bk.pack4(t, t, stream=5), lambda: bk.unpack4(t, 4, 64, stream=5),
                 lambda: bk.matvec4(t, 4, 64, t, stream=5), lambda: bk.rms_norm_q8(t, stream=5),
                 lambda: bk.distill(t, t, t, stream=5), lambda: bk.rms_norm_q8(x=t, stream=5)]:
        with pytest.raises(Enough):
            call()
    assert seen == [(5, t.device)] * 6
    with pytest.raises(ValueError, match="tensors"):
        bk.rms_norm_q8([1.0], stream=5)


def test_an_input_that_needs_a_gradient_is_refused(bk):
    """matvec4 and rms_norm_q8 have no gradient: they do not drop one in silence."""
    x = torch.zeros(4, 64, requires_grad=True)
    packed = torch.zeros(bk.bakron_pack4_bytes(4, 64, 64), dtype=torch.uint8)
    calls = [lambda: bk.matvec4(packed, 4, 64, x), lambda: bk.rms_norm_q8(x),
             lambda: bk.rms_norm_q8(x.detach(), residual=x),
             lambda: bk.matvec4(packed, 4, 64, x.detach().to(torch.int8), x_scales=x[:, :1])]
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call()
    with torch.no_grad():
        for call in calls:
            with pytest.raises(ValueError, match="CUDA"):    # host tensors: refused further on
                call()


def test_norm_in_place_takes_the_stride_of_its_input(L):
    """A sum in the buffer of x or of the residual, but with other rows: refused, for a row would be
    written while another one is read there."""
    far = ctypes.c_void_p(0x9000)

    def nq(x=P, ldx=64, r=far, ldr=64, sm=P, lds=64, rows=2):
        return L.bakron_rms_norm_q8(x, ldx, r, ldr, 2, None, 0, rows, 64, 1e-6, 32, far, far, sm, lds,
                                    None, None)
    for bad in [dict(lds=72), dict(ldx=72), dict(sm=far, lds=72), dict(sm=far, ldr=80),
                dict(r=None, lds=65)]:
        assert nq(**bad) == INVALID, bad
