"""GPU parity of the 4-bit layout, its product with a few tokens and the 8-bit norm against the fp64
oracle (run on a B200), and a run of them behind a solve.

* The layout and the codes of the norm are whole numbers: compared exactly. The codes are defined by
  the inputs alone (the norm cancels), decided in fp64 near a border.
* matvec4: with a = |x| |W|^T, the error of one result is at most
      half a step of y's type * |y| + a * (carry + (n / 64 + 24) 2^-23).
  carry is what the entry point says of its operands: nothing on the integer grid (codes and
  16-bit or 8-bit activations are exact, fp32 activations keep 24 bits), with a codebook 2^-22 (fp16,
  int8), 2^-16 (bf16) or 2^-23 (fp32). The sum takes n / 64 additions of partial sums over 64
  columns, a partial sum is 4 tensor-core steps of 16 products, each off by at most 2^-23 of its
  largest operand or of its running sum (no rounding to nearest in there), and the joining of
  partial sums adds a few more: 24 in all is more than enough.
* scales of the norm: the sum of squares (all positive) is off by at most (n / 256 + 24) 2^-24, which
  a square root halves; maximum, quotient and product add 3 half steps.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import matvec4, pack4_layout, rms_norm_q8

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
BOOK16 = [-1.0, -0.6962, -0.5251, -0.3949, -0.2844, -0.1848, -0.0911, 0.0, 0.0796, 0.1609, 0.2461,
          0.3379, 0.4407, 0.5626, 0.7230, 1.0]


@pytest.fixture(scope="module")
def bk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from two_sided_adaptive_bakron_b200 import build
    build.build()
    from two_sided_adaptive_bakron_b200 import bakron
    return bakron


def _cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def _layer(m, n, group, seed, book=None):
    """(codes, scales numpy): codes over their whole range, a row of step 0."""
    rng = np.random.default_rng(seed)
    G = 1 if group is None else -(-n // group)
    lo, hi = (-8, 8) if book is None else (0, len(book))
    codes = rng.integers(lo, hi, (m, n)).astype(np.int8)
    scales = (0.5 + rng.random((m, G))).astype(np.float32) / 64
    scales[m // 2] = 0.0
    return codes, (scales[:, 0] if group is None else scales)


# ------------------------------------------------------------------------------------ layout
@pytest.mark.parametrize("m,n,group,book", [(1, 1, None, False), (16, 64, 32, True),
                                            (17, 70, 32, False), (33, 129, None, True),
                                            (40, 200, 64, False), (15, 96, 96, False)])
def test_layout(bk, m, n, group, book):
    codes, scales = _layer(m, n, group, m + n, BOOK16 if book else None)
    packed = bk.pack4(_cuda(codes), _cuda(scales), group, unsigned=book)
    np.testing.assert_array_equal(packed.cpu().numpy(), pack4_layout(codes, scales, group))
    c, s = bk.unpack4(packed, m, n, group, unsigned=book)
    np.testing.assert_array_equal(c.cpu().numpy(), codes)
    np.testing.assert_array_equal(s.cpu().numpy(), scales)


@pytest.mark.parametrize("off,pad", [(0, 3), (1, 8), (4, 4), (8, 8)])
def test_layout_of_strided_codes(bk, off, pad):
    """Rows that start anywhere, and what lies around them is left as it was."""
    m, n = 35, 150
    codes, scales = _layer(m, n, 32, 9)
    wide = torch.full((m, n + off + pad), 77, dtype=torch.int8, device="cuda")
    view = wide[:, off:off + n]
    view.copy_(_cuda(codes))
    packed = bk.pack4(view, _cuda(scales), 32)
    np.testing.assert_array_equal(packed.cpu().numpy(), pack4_layout(codes, scales, 32))
    view.zero_()
    s = torch.empty((m, 5), device="cuda")
    assert bk.bakron_unpack4(packed, 32, False, view, s) == 0
    np.testing.assert_array_equal(view.cpu().numpy(), codes)
    assert (wide[:, :off] == 77).all() and (wide[:, off + n:] == 77).all()


@pytest.mark.parametrize("bad,unsigned", [(8, False), (-9, False), (127, False), (-1, True),
                                          (16, True), (-128, True)])
def test_codes_out_of_range_are_reported(bk, bad, unsigned):
    codes = torch.zeros((20, 70), dtype=torch.int8, device="cuda")
    codes[19, 69] = bad
    with pytest.raises(bk.BakronError):
        bk.pack4(codes, torch.ones(20, device="cuda"), unsigned=unsigned)
    st = bk.new_status("cuda")
    bk.pack4(codes, torch.ones(20, device="cuda"), unsigned=unsigned, status=st)
    assert bk.bakron_read_status(st) == bk.BAKRON_ERR_INVALID_ARG
    codes[19, 69] = 0
    bk.pack4(codes, torch.ones(20, device="cuda"), unsigned=unsigned)


# ----------------------------------------------------------------------------------- product
def _check_product(bk, m, n, tokens, x, y, group=None, book=None, x_group=None, seed=0):
    codes, scales = _layer(m, n, group, seed, book)
    rng = np.random.default_rng(seed + 1)
    xs = None
    if x == "i8":
        xv = rng.integers(-127, 128, (tokens, n)).astype(np.int8)
        Gx = 1 if x_group is None else -(-n // x_group)
        xs = (rng.random((tokens, Gx)).astype(np.float32) + 0.1) / 127
        xt = _cuda(xv)
    else:
        xt = _cuda(rng.standard_normal((tokens, n)).astype(np.float32), DT[x])
        xt[:, ::17] *= 30.0
    layer = bk.PackedLayer(_cuda(codes), _cuda(scales), group, book)
    got = layer.matvec(xt, x_scales=None if xs is None else _cuda(xs), x_group_size=x_group,
                       out_dtype=DT[y])
    assert got.dtype == DT[y] and got.shape == (tokens, m)
    ref, a = matvec4(codes, scales, xt.double().cpu().numpy(), group, book, xs, x_group)
    carry = 0.0 if book is None else {"f32": 2.0 ** -23, "bf16": 2.0 ** -16}.get(x, 2.0 ** -22)
    tol = HALF[DT[y]] * np.abs(ref) + a * (carry + (n / 64 + 24) * 2.0 ** -23)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())
    return layer, xt, xs, got


@pytest.mark.parametrize("x,y", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("i8", "f32"),
                                 ("i8", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("m,n,group,tokens", [(1, 1, None, 1), (16, 64, 32, 1), (17, 70, 32, 2),
                                              (5, 31, None, 3), (100, 1000, 96, 5),
                                              (1003, 2500, None, 3), (256, 4096, 128, 9)])
@pytest.mark.parametrize("book", [False, True])
def test_product(bk, x, y, m, n, group, tokens, book):
    _check_product(bk, m, n, tokens, x, y, group, BOOK16 if book else None,
                   x_group=64 if x == "i8" and n > 64 else None, seed=m + n)


@pytest.mark.parametrize("tokens", [1, 2, 4, 7, 8, 12, 16, 17, 31, 32, 33, 70])
@pytest.mark.parametrize("x", ["f32", "f16", "bf16", "i8"])
def test_product_over_tokens(bk, tokens, x):
    _check_product(bk, 130, 520, tokens, x, "f32", 64, seed=tokens)


@pytest.mark.parametrize("m,n,x", [(4096, 14336, "bf16"), (28672, 8192, "i8"), (64, 65536, "f16"),
                                   (48, 65536, "f32"), (70000, 96, "bf16")])
def test_product_of_large_layers(bk, m, n, x):
    """Against fp64 products of the unpacked layer on the device."""
    gen = torch.Generator(device="cuda").manual_seed(m)
    codes = torch.randint(-8, 8, (m, n), generator=gen, device="cuda", dtype=torch.int8)
    G = -(-n // 128)
    scales = torch.rand((m, G), generator=gen, device="cuda") + 0.5
    if x == "i8":
        xt = torch.randint(-127, 128, (2, n), generator=gen, device="cuda", dtype=torch.int8)
        xs = torch.rand((2, 1), generator=gen, device="cuda") + 0.5
        xd = xt.double() * xs.double()
    else:
        xt, xs = torch.randn((2, n), generator=gen, device="cuda").to(DT[x]), None
        xd = xt.double()
    layer = bk.PackedLayer(codes, scales, 128)
    got = layer.matvec(xt, x_scales=xs, out_dtype=torch.float32)
    for lo in range(0, m, 4096):
        W = codes[lo:lo + 4096].double() * \
            scales[lo:lo + 4096].double().repeat_interleave(128, dim=1)[:, :n]
        ref, a = xd @ W.T, xd.abs() @ W.abs().T
        tol = 2.0 ** -24 * ref.abs() + a * (n / 64 + 24) * 2.0 ** -23
        assert ((got[:, lo:lo + 4096].double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("book", [[-1.0, 1.0], [-1.5, -0.5, 0.5, 1.5],
                                  [float(v) for v in np.linspace(-3, 900, 8)],
                                  [v * 1e-20 for v in BOOK16], [v * 1e20 for v in BOOK16]])
def test_product_with_other_codebooks(bk, book):
    _check_product(bk, 40, 300, 2, "f16", "f32", 32, book, seed=len(book))
    _check_product(bk, 40, 300, 2, "i8", "f32", 32, book, seed=len(book))


@pytest.mark.parametrize("x", ["f32", "f16", "bf16", "i8"])
@pytest.mark.parametrize("off", [1, 3, 8])
def test_product_of_strided_activations(bk, x, off):
    """Rows of x and y that start anywhere; what lies between the rows of y stays."""
    m, n, tokens = 50, 333, 3
    codes, scales = _layer(m, n, None, 3)
    xw = torch.randint(-100, 100, (tokens, n + 13), device="cuda").to(DT[x])
    xv = xw[:, off:off + n]
    xs = torch.rand((tokens, 1), device="cuda") if x == "i8" else None
    layer = bk.PackedLayer(_cuda(codes), _cuda(scales))
    ref = layer.matvec(xv.contiguous(), x_scales=xs, out_dtype=torch.float32)
    yw = torch.full((tokens, m + 7), 5.0, device="cuda")
    assert bk.bakron_matvec4(layer.packed, None, None, xv, xs, None, yw[:, 3:3 + m]) == 0
    assert torch.equal(yw[:, 3:3 + m], ref)
    assert (yw[:, :3] == 5).all() and (yw[:, 3 + m:] == 5).all()


def test_product_one_dimension_and_no_token(bk):
    codes, scales = _layer(20, 100, None, 3)
    layer = bk.PackedLayer(_cuda(codes), _cuda(scales))
    x = torch.randn(3, 100, device="cuda")
    full = layer.matvec(x)
    one = layer.matvec(x[1])
    assert one.shape == (20,)
    ref, a = matvec4(codes, scales, x[1].double().cpu().numpy())
    assert (np.abs(one.double().cpu().numpy() - ref[0]) <= a[0] * 26 * 2.0 ** -23).all()
    assert layer.matvec(x[:0]).shape == (0, 20) and full.shape == (3, 20)


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("book", [None, BOOK16])
def test_product_keeps_a_bad_token_to_itself(bk, x, book):
    codes, scales = _layer(33, 200, 32, 8, book)
    layer = bk.PackedLayer(_cuda(codes), _cuda(scales), 32, book)
    xt = torch.randn(5, 200, device="cuda").to(DT[x])
    ref = layer.matvec(xt)
    for v in (float("nan"), float("inf"), -float("inf")):
        xb = xt.clone()
        xb[2, 199] = v
        got = layer.matvec(xb)
        assert not torch.isfinite(got[2]).any()
        keep = [0, 1, 3, 4]
        assert torch.equal(got[keep], ref[keep])


def test_product_refuses_other_devices_and_sizes(bk):
    codes, scales = _layer(32, 64, None, 1)
    layer = bk.PackedLayer(_cuda(codes), _cuda(scales))
    x = torch.randn(2, 64, device="cuda")
    with pytest.raises(ValueError):
        layer.matvec(x.cpu())
    with pytest.raises(ValueError):
        layer.matvec(x[:, :63])
    with pytest.raises(ValueError):
        layer.matvec(torch.randn(64, 2, device="cuda").T)
    with pytest.raises(ValueError):
        layer.matvec(x.double())
    with pytest.raises(ValueError):
        layer.matvec(x[:1].expand(3, 64))
    with pytest.raises(ValueError):
        bk.matvec4(layer.packed, 33, 64, x)
    with pytest.raises(bk.BakronError):
        layer.matvec(x.to(torch.int8))              # int8 without its scales
    with pytest.raises(bk.BakronError):
        layer.matvec(x, x_scales=torch.ones(2, 1, device="cuda"))
    with pytest.raises(ValueError):
        layer.matvec(x.to(torch.int8), x_scales=torch.ones(3, 1, device="cuda"))


# -------------------------------------------------------------------------------------- norm
def _check_norm(bk, x, weight, r, group=None, eps=1e-6):
    q, s, h = bk.rms_norm_q8(x, weight, eps, residual=r, group_size=group)
    f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    rq, rs, rh = rms_norm_q8(f(x), f(weight), eps, f(r), group)
    np.testing.assert_array_equal(q.cpu().numpy().reshape(rq.shape), rq)
    n = x.shape[-1]
    rtol = (n / 256 + 24) * 2.0 ** -25 + 3 * 2.0 ** -24
    np.testing.assert_allclose(s.double().cpu().numpy().reshape(rs.shape), rs, rtol=rtol, atol=1e-45)
    if r is not None:
        assert torch.equal(h, (x.float() + r.float()).to(x.dtype))
    else:
        assert h is None
    return q, s


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,n,group", [(1, 1, None), (3, 31, None), (2, 32, 32), (1, 4096, None),
                                          (5, 5003, 128), (4, 1000, 96), (7, 8192, 128),
                                          (2, 16384, None), (1, 20000, 32), (2, 65536, 128),
                                          (300, 256, None)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(bk, dt, rows, n, group, residual):
    gen = torch.Generator(device="cuda").manual_seed(rows * n)
    x = (torch.randn(rows, n, generator=gen, device="cuda") * 2).to(DT[dt])
    r = torch.randn(rows, n, generator=gen, device="cuda").to(DT[dt]) if residual else None
    w = (1 + 0.2 * torch.randn(n, generator=gen, device="cuda")).to(DT[dt])
    _check_norm(bk, x, w, r, group)


def test_norm_weight_types(bk):
    x = torch.randn(4, 777, device="cuda").bfloat16()
    w = torch.rand(777, device="cuda")
    _check_norm(bk, x, w, x)
    _check_norm(bk, x, w.half(), None, 32)
    _check_norm(bk, x, None, x, 64)
    q, s, h = bk.rms_norm_q8(x[1])
    q2, s2, _ = bk.rms_norm_q8(x)
    assert q.shape == (777,) and torch.equal(q, q2[1]) and s.shape == (1,) and h is None
    assert bk.rms_norm_q8(x[:0])[0].shape == (0, 777)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_norm_ties_go_to_even(bk, dt):
    """Quotients that are half of an odd number: 127 v / 254 with whole v."""
    x = torch.arange(-254, 255, device="cuda").float()
    x = torch.stack([x, x / 4, -x]).to(DT[dt])
    _check_norm(bk, x, None, None)


def test_norm_borders_of_near_ties(bk):
    """fp32 values one unit in the last place to either side of every border of two codes."""
    top = np.float32(1.7)
    mid = ((np.arange(-126, 126) + 0.5) * np.float64(top) / 127).astype(np.float32)
    v = np.concatenate([mid, np.nextafter(mid, np.float32(9)), np.nextafter(mid, np.float32(-9)), [top]])
    _check_norm(bk, _cuda(v.astype(np.float32)[None]), None, None)
    w = np.full(v.size, 1.0 / 3, dtype=np.float32)
    _check_norm(bk, _cuda(v.astype(np.float32)[None]), _cuda(w), None)


def test_norm_extreme_sizes(bk):
    base = torch.randn(1, 600, device="cuda")
    for f in (1e-44, 1e-39, 1e-30, 1e-18, 1e18, 1e30, 1e37):
        _check_norm(bk, base * f, None, None, 32, eps=1e-12)
    z = torch.zeros(2, 100, device="cuda")
    q, s, _ = bk.rms_norm_q8(z)
    assert not q.any() and not s.any()
    z[1, 50] = -3.0
    _check_norm(bk, z, None, None, 32)


def test_norm_of_rows_that_are_not_finite(bk):
    x = torch.randn(5, 300, device="cuda")
    x[1, 7], x[3, 299] = float("nan"), -float("inf")
    st = bk.new_status("cuda")
    q, s, _ = bk.rms_norm_q8(x, group_size=32, status=st)
    assert bk.bakron_read_status(st) == bk.BAKRON_ERR_NONFINITE
    assert not q[[1, 3]].any() and torch.isnan(s[[1, 3]]).all()
    good = [0, 2, 4]
    q2, s2, _ = bk.rms_norm_q8(x[good], group_size=32)
    assert torch.equal(q[good], q2) and torch.equal(s[good], s2)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("off", [0, 1, 4])
def test_norm_strided_and_in_place(bk, dt, off):
    rows, n = 4, 1030
    xw = torch.randn(rows, n + 11, device="cuda").to(DT[dt])
    rw = torch.randn(rows, n + 5, device="cuda").to(DT[dt])
    w = torch.rand(n, device="cuda").to(DT[dt])
    x, r = xw[:, off:off + n], rw[:, off:off + n]
    q0, s0, h0 = bk.rms_norm_q8(x.contiguous(), w, residual=r.contiguous())
    keep = rw.clone()
    q, s, h = bk.rms_norm_q8(x, w, residual=r, sum_out=r)
    assert torch.equal(q, q0) and torch.equal(s, s0) and torch.equal(r, h0) and h is r
    keep[:, off:off + n] = h0
    assert torch.equal(rw, keep)
    xc = x.clone()
    q, _, _ = bk.rms_norm_q8(x, w, sum_out=x)
    assert torch.equal(x, xc) and torch.equal(q, bk.rms_norm_q8(xc, w)[0])


# --------------------------------------------------------------------------------- together
@pytest.mark.parametrize("book", [None, BOOK16])
def test_a_solved_layer_serves_a_token(bk, book):
    """Solve, pack, norm to 8 bits, product: against the fp64 products of the round's own W."""
    from two_sided_adaptive_bakron_b200.workloads import make_workload
    Ws, HO, HI, _, bits = make_workload("small_64x128")
    s = np.abs(Ws).reshape(64, 4, 32).max(axis=2).astype(np.float32) / np.float32(1 if book else 7.5)
    solver = bk.Solver(64, 128)
    with pytest.raises(ValueError):
        solver.packed()
    solver.run(_cuda(Ws), _cuda(HO), _cuda(HI), _cuda(s), bits, group_size=32, codebook=book)
    layer = solver.packed()
    solver.check()
    codes, steps = layer.unpack()
    assert torch.equal(codes, solver.codes) and torch.equal(steps, _cuda(s))
    x = torch.randn(3, 128, device="cuda").bfloat16()
    r = torch.randn(3, 128, device="cuda").bfloat16()
    w = torch.rand(128, device="cuda").bfloat16()
    q, xs, h = bk.rms_norm_q8(x, w, residual=r, group_size=64)
    y = layer.matvec(q, xs, 64)
    xd = q.double() * xs.double().repeat_interleave(64, dim=1)
    ref, a = xd @ solver.W.double().T, xd.abs() @ solver.W.double().abs().T
    # solver.W carries one rounding of s c more (2^-24 of each term)
    assert ((y.double() - ref).abs() <= a * (26 * 2.0 ** -23 + 2.0 ** -22 + 2.0 ** -24)).all()


def test_rotated_layer_packs_its_own_steps(bk):
    from two_sided_adaptive_bakron_b200.workloads import make_workload
    Ws, HO, HI, s, bits = make_workload("small_64x128")
    solver = bk.Solver(64, 128)
    solver.run(_cuda(Ws), _cuda(HO), _cuda(HI), None, bits, incoherence=(3, 4))
    layer = solver.packed()
    x = torch.randn(2, 128, device="cuda")
    ref = x.double() @ solver.W.double().T
    a = x.double().abs() @ solver.W.double().abs().T
    assert ((layer.matvec(x).double() - ref).abs() <= a * 27 * 2.0 ** -23).all()
    solver.run(_cuda(Ws), _cuda(HO), _cuda(HI), _cuda(s), bits)     # and those of a later run
    assert torch.equal(solver.packed().unpack()[1], _cuda(s))


def test_streams_capture_and_replay(bk):
    """The same bits on another stream, and from a captured graph replayed on new values."""
    codes, scales = _layer(200, 1000, 32, 5)
    layer = bk.PackedLayer(_cuda(codes), _cuda(scales), 32)
    x = torch.randn(4, 1000, device="cuda").half()
    r = torch.randn(4, 1000, device="cuda").half()

    def step():
        q, s, h = bk.rms_norm_q8(x, None, residual=r, group_size=128)
        return q, s, h, layer.matvec(q, s, 128, torch.float16), layer.matvec(h)
    ref = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    # a stream named in the call, its outputs waited for by hand
    q, s, h = bk.rms_norm_q8(x, None, residual=r, group_size=128, stream=side)
    y = layer.matvec(q, s, 128, torch.float16, stream=side)
    side.synchronize()
    assert torch.equal(y, ref[3])
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1 = step()
    with torch.cuda.graph(g2):
        o2 = step()
    for k in range(3):
        x.copy_(torch.randn(4, 1000, device="cuda"))
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        ref = step()
        assert all(torch.equal(a, b) for a, b in zip(o1, ref))
        assert all(torch.equal(a, b) for a, b in zip(o2, ref))


@pytest.mark.parametrize("x", ["f32", "f16", "bf16", "i8"])
@pytest.mark.parametrize("book", [None, BOOK16])
def test_product_of_the_longest_rows(bk, x, book):
    """Activations that fill shared memory: fewer tokens a block."""
    _check_product(bk, 20, 65536, 9, x, "f32", 32, book, x_group=32 if x == "i8" else None, seed=2)


@pytest.mark.parametrize("args", [["--op", "pack4"], ["--op", "matvec4", "--k", "3"],
                                  ["--op", "matvec4", "--k", "1", "--dtype", "i8"],
                                  ["--op", "rms_norm_q8", "--k", "5", "--group-size", "32"],
                                  ["--op", "distill", "--k", "4", "--d", "1000", "--dtype", "f16"]])
def test_kernel_bench_runs_the_serving_calls(bk, args, capsys):
    from two_sided_adaptive_bakron_b200 import kernel_bench
    assert kernel_bench.main(args + ["--workload", "small_64x128", "--iters", "2"]) == 0
    assert " ms (mean of 1)" in capsys.readouterr().out


def _draw(rng, options):
    return options[rng.integers(len(options))]


@pytest.mark.parametrize("seed", range(24))
def test_product_of_drawn_cases(bk, seed):
    """Sizes, types, groups and tokens at random: slices that end anywhere, clusters, tails."""
    rng = np.random.default_rng(1000 + seed)
    m, n = int(np.exp(rng.uniform(0, np.log(3000)))), int(np.exp(rng.uniform(0, np.log(6000))))
    tokens = int(np.exp(rng.uniform(0, np.log(40))))
    x = _draw(rng, ["f32", "f16", "bf16", "i8"])
    group = _draw(rng, [None, 32, 64, 96, 128, 160, 256, 320, 512, 1024])
    book = _draw(rng, [None, None, BOOK16, BOOK16[:8], [-1.0, -0.25, 0.25, 1.0]])
    xg = _draw(rng, [None, 32, 64, 96, 512]) if x == "i8" else None
    _check_product(bk, m, n, tokens, x, _draw(rng, ["f32", "f16", "bf16"]) if x == "i8" else x,
                   group if group is None or group < n else None, book,
                   xg if xg is None or xg < n else None, seed=seed)


@pytest.mark.parametrize("seed", range(24))
def test_norm_of_drawn_cases(bk, seed):
    rng = np.random.default_rng(2000 + seed)
    rows = int(np.exp(rng.uniform(0, np.log(900))))
    n = int(np.exp(rng.uniform(0, np.log(20000))))
    rows = max(1, min(rows, 2_000_000 // n))
    if seed % 4 == 0:
        rows, n = 700, 8 * int(rng.integers(1, 200))      # many rows of whole chunks
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[_draw(rng, ["f32", "f16", "bf16"])]
    x = (torch.randn(rows, n, generator=gen, device="cuda") * _draw(rng, [1e-3, 1.0, 30.0])).to(dt)
    x[rows // 2] = 0
    r = _draw(rng, [None, torch.randn(rows, n, generator=gen, device="cuda").to(dt)])
    w = _draw(rng, [None, torch.randn(n, generator=gen, device="cuda").to(dt),
                    torch.randn(n, generator=gen, device="cuda")])
    _check_norm(bk, x, w, r, _draw(rng, [None, 32, 64, 96, 128, 256, 384]))


def test_calls_on_a_stream_own_what_they_write(bk):
    """Outputs made for a named stream come from that stream's memory: what the current stream still
    works on is not overwritten."""
    codes, scales = _layer(64, 256, 32, 5)
    layer = bk.PackedLayer(_cuda(codes), _cuda(scales), 32)
    x = torch.randn(8, 256, device="cuda")
    ref = layer.matvec(x)
    idx, top = torch.zeros(8, 1, dtype=torch.int32, device="cuda"), torch.zeros(8, 1, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()                             # the inputs are there for every stream
    for handle in (side, side.cuda_stream):
        busy = torch.randn(4096, 4096, device="cuda")
        keep = torch.ones(8, 64, device="cuda")
        for _ in range(4):
            busy = busy @ busy * 1e-3                    # the current stream is behind
        late = keep + busy[:8, :64] * 0
        ptr = keep.data_ptr()
        del keep                                         # its memory is free for this stream only
        y = layer.matvec(x, stream=handle)
        q, s, _ = bk.rms_norm_q8(x, stream=handle)
        loss, _, dz = bk.distill(x, idx, top, stream=handle)
        side.synchronize()
        assert y.data_ptr() != ptr and torch.equal(y, ref)
        torch.cuda.synchronize()
        assert (late == 1).all() or not torch.isfinite(busy).all()


# products whose blocks take all of shared memory, or all but a little
@pytest.mark.parametrize("m,n,group,tokens,x,book", [
    (28672, 8192, None, 16, "bf16", False), (28672, 8192, None, 9, "f16", True),
    (14336, 4096, None, 17, "bf16", True), (512, 18432, 64, 32, "bf16", False),
    (4096, 5184, 64, 20, "f32", False), (4096, 11008, 128, 5, "f32", True),
    (8192, 8192, 128, 33, "bf16", False), (28672, 8192, 128, 32, "i8", False)])
def test_product_in_full_blocks(bk, m, n, group, tokens, x, book):
    """Against fp64 products of the unpacked layer on the device."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    codes = torch.randint(0 if book else -8, 16 if book else 8, (m, n), generator=gen, device="cuda",
                          dtype=torch.int8)
    g = group or n
    scales = torch.rand((m, -(-n // g)), generator=gen, device="cuda") + 0.5
    if x == "i8":
        xt = torch.randint(-127, 128, (tokens, n), generator=gen, device="cuda", dtype=torch.int8)
        xs = torch.rand((tokens, 1), generator=gen, device="cuda") + 0.5
        xd = xt.double() * xs.double()
    else:
        xt, xs = torch.randn((tokens, n), generator=gen, device="cuda").to(DT[x]), None
        xd = xt.double()
    got = bk.PackedLayer(codes, scales, group, BOOK16 if book else None).matvec(
        xt, x_scales=xs, out_dtype=torch.float32)
    carry = 0.0 if not book else {"f32": 2.0 ** -23, "bf16": 2.0 ** -16}.get(x, 2.0 ** -22)
    table = torch.tensor(BOOK16, device="cuda").double()
    for lo in range(0, m, 4096):
        c = codes[lo:lo + 4096]
        W = (table[c.int()] if book else c.double()) * \
            scales[lo:lo + 4096].double().repeat_interleave(g, dim=1)[:, :n]
        ref, a = xd @ W.T, xd.abs() @ W.abs().T
        tol = 2.0 ** -24 * ref.abs() + a * (carry + (n / 64 + 24) * 2.0 ** -23)
        assert ((got[:, lo:lo + 4096].double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("m,n,tokens", [(128, 65536, 16), (880, 55360, 8), (2000, 65536, 1),
                                        (4096, 60000, 3)])
def test_product_of_the_longest_rows_of_many_tiles(bk, m, n, tokens):
    """fp32 activations, a codebook and steps of 32 columns: the sums of few row tiles fit."""
    gen = torch.Generator(device="cuda").manual_seed(m)
    codes = torch.randint(0, 16, (m, n), generator=gen, device="cuda", dtype=torch.int8)
    scales = torch.rand((m, -(-n // 32)), generator=gen, device="cuda") + 0.5
    xt = torch.randn((tokens, n), generator=gen, device="cuda")
    got = bk.PackedLayer(codes, scales, 32, BOOK16).matvec(xt)
    W = torch.tensor(BOOK16, device="cuda").double()[codes.int()]
    W *= scales.double().repeat_interleave(32, dim=1)[:, :n]
    ref, a = xt.double() @ W.T, xt.double().abs() @ W.abs().T
    tol = 2.0 ** -24 * ref.abs() + a * (2.0 ** -23 + (n / 64 + 24) * 2.0 ** -23)
    assert ((got.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("m,n,group,tokens", [(17, 70, 32, 1), (130, 520, 64, 8), (1003, 2500, None, 3),
                                              (100, 1000, 96, 17), (256, 4096, 128, 33),
                                              (20, 65536, 32, 9)])
@pytest.mark.parametrize("book", [BOOK16, [v * 1.0e-20 for v in BOOK16], [-1.1, 0.7]])
def test_fp32_results_of_bf16_activations_keep_the_entries(bk, m, n, group, tokens, book):
    """Codebook entries of 24 bits, as with fp32 activations (carry 2^-23), not the 16 that a 16-bit
    result is given."""
    codes, scales = _layer(m, n, group, m, book)
    x = torch.randn(tokens, n, device="cuda").bfloat16()
    got = bk.PackedLayer(_cuda(codes), _cuda(scales), group, book).matvec(x, out_dtype=torch.float32)
    ref, a = matvec4(codes, scales, x.double().cpu().numpy(), group, book)
    tol = HALF[torch.float32] * np.abs(ref) + a * (2.0 ** -23 + (n / 64 + 24) * 2.0 ** -23)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())
    # one column: the entry itself, times a power of two
    one = np.arange(len(book), dtype=np.int8)[:, None]
    got = bk.PackedLayer(_cuda(one), torch.ones(len(book), device="cuda"), None, book).matvec(
        torch.full((1, 1), 0.5, device="cuda").bfloat16(), out_dtype=torch.float32)
    want = torch.tensor(book, device="cuda") * 0.5
    assert ((got[0] - want).abs() <= 2.0 ** -23 * want.abs()).all()


def test_transposed_steps_and_lists_are_refused(bk):
    """Contiguous tensors of the right length that stand the other way round."""
    m, n, G = 48, 256, 8
    codes, steps = torch.zeros(m, n, dtype=torch.int8, device="cuda"), torch.rand(m, G, device="cuda")
    layer = bk.PackedLayer(codes, steps, 32)
    with pytest.raises(ValueError, match="48 x 8"):
        bk.PackedLayer(codes, steps.T.contiguous(), 32)
    out = torch.empty(G, m, device="cuda")
    with pytest.raises(ValueError, match="48 x 8"):
        bk.bakron_unpack4(layer.packed, 32, False, codes, out)
    q, xs, _ = bk.rms_norm_q8(torch.randn(3, n, device="cuda"), group_size=32)
    with pytest.raises(ValueError, match="3 x 8"):
        layer.matvec(q, xs.T.contiguous(), 32)
    y = layer.matvec(q, xs, 32)
    assert torch.equal(layer.matvec(q, xs.view(-1), 32), y)          # flat ones as before
    assert torch.equal(layer.matvec(q[:1], xs[0], 32), y[:1])
    z = torch.randn(5, 40, device="cuda")
    top, idx = z.topk(3, dim=1)
    ref = bk.distill(z, idx, top)
    for i, t in [(idx, top.T.contiguous()), (idx.T.contiguous(), top)]:
        with pytest.raises(ValueError):
            bk.distill(z, i, t)
    assert torch.equal(bk.distill(z, idx, top.view(-1))[0], ref[0])
