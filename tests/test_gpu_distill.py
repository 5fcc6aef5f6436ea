"""GPU parity of the distillation loss and its gradient against the fp64 oracle (run on a B200).

Tolerances. All statistics are fp32 of exact logits; per row, with L = max |z - max z| / tau over the
entries of the list and M = sum p:
* lse = max / tau + log(sum): the sum has relative error at most (V / 512 + 40) 2^-24 + 2^-21 (the
  additions of one thread, the tree, and exponentials good to 2^-21 where they count), which is its
  absolute error in the log; rounding adds 2 half steps of |lse| and |max / tau|.
* loss: sum_j p_j (log p_j - log q_j): each p_j is off by 2^-21 + (T + 4) 2^-24 where T = max |t - T|,
  each logarithm by the error of lse plus 4 half steps of its size: the bound below adds these
  up term by term in fp64 (see _loss_tol).
* gradient: (w / tau)(M q_i - p_i): each part off by the relative errors above, times their sizes,
  and one rounding to the output's type: half a step, of the value or of its smallest normal.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import distill

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -14, "bf16": 2.0 ** -126}


@pytest.fixture(scope="module")
def bk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from two_sided_adaptive_bakron_b200 import build
    build.build()
    from two_sided_adaptive_bakron_b200 import bakron
    return bakron


def _np(t):
    return None if t is None else t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def _problem(rows, V, k, dt, seed, repeat=False, scale=2.5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    z = scale * torch.randn(rows, V, generator=gen, device="cuda")
    teacher = z + 0.5 * torch.randn(rows, V, generator=gen, device="cuda")
    if repeat:
        idx = torch.randint(0, max(1, V // 3), (rows, k), generator=gen, device="cuda")
        top = teacher.gather(1, idx)
    else:
        top, idx = teacher.topk(k, dim=1)
    return z.to(DT[dt]), idx, top.contiguous(), teacher


def _check(bk, z, idx, top, tau=1.0, mass=None, w=None, grad=True, dlogits=None, dt="f32"):
    zc = _np(z)
    loss, lse, dz = bk.distill(z, idx, top, tau, mass, w, grad=grad, dlogits=dlogits)
    rl, rs, rd = distill(zc, _np(idx), _np(top), tau, _np(mass), _np(w))
    rows, V = zc.shape
    u = 2.0 ** -24
    esum = (V / 512 + 40) * u + 2.0 ** -21
    zmax = np.where(np.isfinite(zc.max(axis=1)), zc.max(axis=1), 0.0)
    elog = esum + 2 * u * (np.abs(rs) + np.abs(zmax) / tau)
    ok = rs != 0
    assert (np.abs(_np(lse) - rs) <= elog)[ok | (_np(lse) == 0)].all()
    # term by term
    i = np.where((_np(idx) >= 0) & (_np(idx) < V), _np(idx), 0)
    t = np.where((_np(idx) >= 0) & (_np(idx) < V), _np(top), -np.inf) / tau
    with np.errstate(divide="ignore", invalid="ignore"):
        tm = np.where(np.isfinite(t.max(axis=1)), t.max(axis=1), 0.0)
        T = tm + np.log(np.exp(t - tm[:, None]).sum(axis=1)) if mass is None else _np(mass)
        lp = t - T[:, None]
        p = np.where(np.isfinite(lp), np.exp(lp), 0.0)
        lp = np.where(np.isfinite(lp), lp, 0.0)
        lq = np.take_along_axis(zc, i, axis=1) / tau - rs[:, None]
        lq = np.where(np.isfinite(lq), lq, 0.0)
    big = np.abs(t[np.isfinite(t)]).max(initial=0.0) + np.abs(T[np.isfinite(T)]).max(initial=0.0)
    ep = 2.0 ** -21 + (4 * big + t.shape[1] / 512 + 44) * u
    tol = (p * ((np.abs(lp) + np.abs(lq) + 1) * (ep + 8 * u) + elog[:, None])).sum(axis=1)
    wn = np.ones(rows) if w is None else _np(w)
    err = np.abs(_np(loss) - rl)
    assert (err <= np.abs(wn) * tol + 2.0 ** -24 * np.abs(rl)).all(), float((err - wn * tol).max())
    if not grad:
        assert dz is None
        return
    sz = np.abs(rd)
    pf = np.zeros_like(rd)
    np.add.at(pf, (np.arange(rows)[:, None], i), p)
    f = np.abs(wn)[:, None] / tau
    part = sz + 2 * f * pf                       # >= f (M q + p)
    tol = HALF[dt] * np.maximum(sz, TINY[dt]) + part * (ep + esum + 8 * u)
    err = np.abs(_np(dz) - rd)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,V,k", [(1, 1, 1), (3, 2, 2), (2, 7, 3), (5, 1000, 20), (4, 4099, 64),
                                      (2, 32000, 100), (3, 50001, 7), (2, 131072, 1024),
                                      (1, 300007, 33), (40, 513, 5)])
@pytest.mark.parametrize("tau,own", [(1.0, False), (2.0, True)])
def test_loss_and_gradient(bk, dt, rows, V, k, tau, own):
    z, idx, top, teacher = _problem(rows, V, k, dt, rows * V + k)
    mass = torch.logsumexp(teacher.double() / tau, dim=1).float() if own else None
    _check(bk, z, idx, top, tau, mass, dt=dt)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_loss_alone_equals_loss_with_gradient(bk, dt):
    z, idx, top, _ = _problem(6, 9001, 9, dt, 5)
    a, la, _ = bk.distill(z, idx, top, 1.5, grad=False)
    b, lb, _ = bk.distill(z, idx, top, 1.5)
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("idx_t", [torch.int32, torch.int64])
@pytest.mark.parametrize("top_t", [torch.float32, torch.float16, torch.bfloat16])
def test_list_types(bk, idx_t, top_t):
    z, idx, top, _ = _problem(5, 700, 11, "bf16", 6)
    _check(bk, z, idx.to(idx_t), top.to(top_t), dt="bf16")


@pytest.mark.parametrize("k", [2, 31, 700, 1024])
def test_an_index_may_stand_more_than_once(bk, k):
    z, idx, top, _ = _problem(4, 90, k, "f32", k, repeat=True)
    _check(bk, z, idx, top)
    idx[:] = 5
    _check(bk, z, idx, top, 1.3)


def test_absent_entries_and_rows_that_do_not_count(bk):
    z, idx, top, _ = _problem(8, 333, 6, "f32", 7)
    idx[0, 2:], idx[1, :], idx[2, 0] = -1, -1, -7
    top[3, 1], top[4, :] = -float("inf"), -float("inf")
    w = torch.tensor([1.0, 1, 0.5, 2, 1, 0, 0, -1.5], device="cuda")
    z[5, :] = float("nan")                     # a row of weight 0 is not read
    z[6, 3] = float("inf")
    zr = z.clone()
    zr[5:7] = 0
    loss, lse, dz = bk.distill(z, idx, top, 1.0, None, w)
    l2, s2, d2 = bk.distill(zr, idx, top, 1.0, None, w)
    assert torch.equal(loss, l2) and torch.equal(lse, s2) and torch.equal(dz, d2)
    assert loss[1] == loss[4] == loss[5] == loss[6] == 0 and lse[5] == 0
    assert not dz[[1, 4, 5, 6]].any()
    _check(bk, zr, idx, top, 1.0, None, w)


def test_masked_vocabulary(bk):
    """-inf logits are entries of probability 0, the first ones of a row among them."""
    z, idx, top, _ = _problem(4, 3001, 8, "f16", 8)
    m = torch.zeros_like(z, dtype=torch.bool)
    m[:, :1500] = True
    m[1, :] = True
    for r in range(4):
        m[r, idx[r]] = False
    z[m] = -float("inf")
    _check(bk, z, idx, top, 2.0, dt="f16")
    # the teacher wants an entry that the student excludes: an infinite loss, a finite gradient
    z[2, idx[2, 0]] = -float("inf")
    loss, _, dz = bk.distill(z, idx, top)
    assert torch.isinf(loss[2]) and torch.isfinite(loss[[0, 1, 3]]).all() and torch.isfinite(dz).all()
    # masks of the type's lowest value
    z, idx, top, _ = _problem(4, 3001, 8, "bf16", 9)
    low = torch.zeros_like(z, dtype=torch.bool)
    low[:, 1000:] = True
    for r in range(4):
        low[r, idx[r]] = False
    z[low] = torch.finfo(torch.bfloat16).min
    _check(bk, z, idx, top, dt="bf16")


@pytest.mark.parametrize("bad", ["nan", "inf", "all"])
def test_bad_logits_stay_in_their_row(bk, bad):
    z, idx, top, _ = _problem(3, 5000, 4, "f32", 10)
    ref = bk.distill(z, idx, top)
    if bad == "all":
        z[1] = -float("inf")
    else:
        z[1, 4999] = float(bad)
    got = bk.distill(z, idx, top)
    assert torch.isnan(got[0][1]) and torch.isnan(got[2][1]).all()
    for a, b in zip(got, ref):
        assert torch.equal(a[[0, 2]], b[[0, 2]])


def test_index_beyond_the_vocabulary(bk):
    z, idx, top, _ = _problem(3, 500, 4, "f32", 11)
    bad = idx.clone()
    bad[1, 2] = 500
    gone = idx.clone()
    gone[1, 2] = -1
    with pytest.raises(bk.BakronError):
        bk.distill(z, bad, top)
    st = bk.new_status("cuda")
    got = bk.distill(z, bad, top, status=st)
    assert bk.bakron_read_status(st) == bk.BAKRON_ERR_INVALID_ARG
    for a, b in zip(got, bk.distill(z, gone, top)):
        assert torch.equal(a, b)
    bad[1, 2] = 2 ** 40 + 3                     # a 64-bit index does not wrap
    st.zero_()
    got = bk.distill(z, bad, top, status=st)
    assert bk.bakron_read_status(st) == bk.BAKRON_ERR_INVALID_ARG
    for a, b in zip(got, bk.distill(z, gone, top)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("off,pad", [(0, 0), (0, 8), (1, 2), (3, 5)])
def test_strides_and_in_place(bk, dt, off, pad):
    rows, V = 5, 4100
    z0, idx, top, _ = _problem(rows, V, 6, dt, 12)
    wide = torch.full((rows, V + off + pad), 9.0, device="cuda").to(DT[dt])
    z = wide[:, off:off + V]
    z.copy_(z0)
    _check(bk, z, idx, top, 1.5, dt=dt)
    ref = bk.distill(z, idx, top, 1.5)          # strides of its own for the output
    got = bk.distill(z, idx, top, 1.5, dlogits=z)
    assert got[2] is z
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    assert (wide[:, :off] == 9).all() and (wide[:, off + V:] == 9).all()


def test_gradient_against_differences(bk):
    """The loss along a direction, from the kernel's own losses: with a step of 2^-4 and central
    differences the error is the third derivative's, h^2 / 6 |d|_inf^3 / tau^3 <= 0.02 of M here, and
    the rounding of two losses, far less."""
    z, idx, top, _ = _problem(4, 600, 10, "f32", 13)
    d = torch.sign(torch.randn(4, 600, device="cuda"))
    h = 2.0 ** -4
    up, dn = bk.distill(z + h * d, idx, top, 1.5)[0], bk.distill(z - h * d, idx, top, 1.5)[0]
    along = (bk.distill(z, idx, top, 1.5)[2] * d).sum(dim=1)
    assert ((up - dn) / (2 * h) - along).abs().max() <= h * h / 6 * 8 / 1.5 ** 3 + 1e-4


def test_many_rows_and_one_row(bk):
    z, idx, top, _ = _problem(3000, 257, 3, "bf16", 14)
    _check(bk, z, idx, top, dt="bf16")
    full = bk.distill(z, idx, top)
    one = bk.distill(z[17], idx[17:18], top[17:18])
    assert one[2].shape == (257,) and one[0].shape == (1,)
    zc = _np(z[17:18])
    rl, rs, _ = distill(zc, _np(idx[17:18]), _np(top[17:18]))
    assert abs(float(one[0]) - rl[0]) <= 1e-5 and abs(float(full[0][17]) - rl[0]) <= 1e-5
    none = bk.distill(z[:0], idx[:0], top[:0])
    assert none[0].shape == (0,) and none[2].shape == (0, 257)


def test_offsets_beyond_32_bits(bk):
    """Rows whose elements lie past 2^31 from the first."""
    V, rows = 131072, 16500
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB free")
    z = torch.zeros((rows, V), dtype=torch.bfloat16, device="cuda")
    z[-3:] = (2.5 * torch.randn(3, V, device="cuda")).bfloat16()
    top, idx = z[-3:].float().topk(5, dim=1)
    idx_all = idx[:1].repeat(rows, 1)
    top_all = top[:1].repeat(rows, 1)
    idx_all[-3:], top_all[-3:] = idx, top + 0.3
    loss, lse, dz = bk.distill(z, idx_all.contiguous(), top_all.contiguous())
    l3, s3, d3 = bk.distill(z[-3:].clone(), idx, top + 0.3)
    # the order of the sums may differ with the number of rows: both are within their bounds
    tol = 2 * ((V / 512 + 40) * 2.0 ** -24 + 2.0 ** -20)
    assert (lse[-3:] - s3).abs().max() <= tol and (loss[-3:] - l3).abs().max() <= 10 * tol
    assert ((dz[-3:].float() - d3.float()).abs() <= 2.0 ** -7 * d3.float().abs() + 1e-30).all()
    # a row of equal logits: lse = log V; gradient M / V away from the list
    assert abs(float(lse[0]) - np.log(V)) <= 1e-5
    assert dz[0].float().sum().abs() <= 1e-2


def test_streams_capture_and_replay(bk):
    z, idx, top, _ = _problem(6, 10001, 12, "bf16", 15)
    st = bk.new_status("cuda")
    ref = bk.distill(z, idx, top, 2.0, status=st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = bk.distill(z, idx, top, 2.0, status=st)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = bk.distill(z, idx, top, 2.0, status=st)
    for k in range(3):
        z.copy_(2 * torch.randn(6, 10001, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, bk.distill(z, idx, top, 2.0, status=st)))
    assert bk.bakron_read_status(st) == 0


def test_a_rounded_head_against_the_original(bk):
    """The loss of a rounded output layer against its original, with the gradient carried to the
    layer's input by the library's own product of the packed transpose."""
    from two_sided_adaptive_bakron_b200.workloads import random_problem
    Ws, HO, HI, s, bits = random_problem(96, 64, 4, 3)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    solver = bk.Solver(96, 64)
    solver.run(dev(Ws), dev(HO), dev(HI), dev(s), bits)
    solver.check()
    x = torch.randn(5, 64, device="cuda")
    ref = x @ dev(Ws).T
    z = solver.packed().matvec(x)
    top, idx = ref.topk(96, dim=1)
    loss, _, dz = bk.distill(z, idx, top)
    p = torch.softmax(ref.double(), dim=1)
    kl = (p * (p.log() - torch.log_softmax(z.double(), dim=1))).sum(dim=1)
    assert ((loss.double() - kl).abs() <= 1e-5 * (1 + kl)).all() and (loss > 0).all()
    assert ((dz.double() - (torch.softmax(z.double(), dim=1) - p)).abs() <= 1e-5).all()
    back = bk.PackedLayer(solver.codes.T.contiguous(), torch.ones(64, device="cuda"))
    dx = back.matvec(dz * dev(s))
    want = dz.double() @ solver.W.double()
    a = dz.double().abs() @ solver.W.double().abs()
    assert ((dx.double() - want).abs() <= a * 30 * 2.0 ** -23).all()


# rows enough that blocks go from row to row (two an SM and more), with rows that shared memory holds
# whole, in part, and hardly at all
@pytest.mark.parametrize("dt,V,k", [("f32", 5, 3), ("f16", 257, 40), ("bf16", 8000, 32),
                                    ("bf16", 10241, 130), ("f32", 9001, 7), ("f16", 50001, 64),
                                    ("bf16", 70000, 33), ("bf16", 131072, 64),
                                    ("f32", 70003, 1024), ("f32", 140000, 9)])
@pytest.mark.parametrize("ragged", [False, True])
def test_blocks_that_go_from_row_to_row(bk, dt, V, k, ragged):
    """Every row of many against the same rows in small batches (which other kernels take), and a few
    against the oracle."""
    rows = 901 if V < 60000 else 605
    z, idx, top, _ = _problem(rows, V, k, dt, V + k, repeat=ragged and k > 2)
    w = None
    if ragged:
        gen = torch.Generator(device="cuda").manual_seed(V)
        w = (torch.rand(rows, generator=gen, device="cuda") < 0.6).float() * 1.5
        idx = torch.where(torch.rand(idx.shape, generator=gen, device="cuda") < 0.8, idx, -1)
        if V > 100:
            z[:, V // 2:V // 2 + 7] = -float("inf")
    st = bk.new_status("cuda")
    full = bk.distill(z, idx, top, 1.5, None, w, status=st)
    alone = bk.distill(z, idx, top, 1.5, None, w, grad=False, status=st)
    assert torch.equal(full[0].isinf(), alone[0].isinf()) and torch.equal(full[1], alone[1])
    assert torch.equal(full[0], alone[0])
    tol = 2 * ((V / 512 + 40) * 2.0 ** -24 + 2.0 ** -20)
    for lo in range(0, rows, 64):
        hi = min(rows, lo + 64)
        part = bk.distill(z[lo:hi], idx[lo:hi], top[lo:hi], 1.5, None,
                          None if w is None else w[lo:hi], status=st)
        fin = torch.isfinite(part[0])
        assert torch.equal(fin, torch.isfinite(full[0][lo:hi]))
        assert ((full[1][lo:hi] - part[1]).abs() <= tol * (1 + part[1].abs())).all()
        assert ((full[0][lo:hi] - part[0]).abs()[fin] <= 40 * tol).all()
        a, b = full[2][lo:hi].float(), part[2].float()
        assert ((a - b).abs() <= 2 * HALF[dt] * (b.abs() + TINY[dt]) + 40 * tol * b.abs()
                + 2.0 ** -22).all()
    assert bk.bakron_read_status(st) == 0
    if not ragged:
        _check(bk, z[-2:], idx[-2:], top[-2:], 1.5, dt=dt)
        zl = bk.distill(z, idx, top, 1.5, dlogits=z)[2]        # in place
        assert torch.equal(zl, full[2])


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", [3, 400])
def test_rows_of_nothing_but_the_lowest_value(bk, dt, rows):
    """A mask of the type's lowest value over a whole row leaves equal probabilities."""
    V = 1000
    z = torch.full((rows, V), torch.finfo(DT[dt]).min, device="cuda", dtype=DT[dt])
    z[0] = torch.randn(V, device="cuda")
    idx = torch.arange(4, device="cuda").repeat(rows, 1)
    top = torch.zeros(rows, 4, device="cuda")
    for tau in (0.5, 1.0, 3.0):
        loss, lse, dz = bk.distill(z, idx, top, tau)
        want = np.log(0.25) + np.log(V)
        if torch.finfo(DT[dt]).min / tau > -3.4e38:
            assert (loss[1:] - want).abs().max() <= 1e-5
        assert ((dz[1:, 4:].float() - 1 / V / tau).abs() <= 2 * HALF[dt] / V / tau + 1e-9).all()
        assert ((dz[1:, :4].float() - (1 / V - 0.25) / tau).abs() <= 2 * HALF[dt] / tau).all()
        assert torch.isfinite(loss[0]) and torch.isfinite(dz[0]).all()


@pytest.mark.parametrize("seed", range(20))
def test_drawn_cases(bk, seed):
    rng = np.random.default_rng(3000 + seed)
    rows = int(np.exp(rng.uniform(0, np.log(700))))
    V = int(np.exp(rng.uniform(0, np.log(60000))))
    k = min(1024, int(np.exp(rng.uniform(0, np.log(200)))))
    rows = max(1, min(rows, 4_000_000 // V))
    dt = ["f32", "f16", "bf16"][seed % 3]
    z, idx, top, teacher = _problem(rows, V, min(k, V), dt, seed, repeat=k > V or seed % 5 == 0)
    tau = [0.7, 1.0, 4.0][seed % 3]
    mass = torch.logsumexp(teacher.double() / tau, dim=1).float() if seed % 2 else None
    w = None
    if seed % 4 == 1:
        w = torch.from_numpy(rng.standard_normal(rows).astype(np.float32)).cuda()
        w[rows // 2] = 0
    _check(bk, z, idx.to(torch.int32) if seed % 3 else idx, top, tau, mass, w, dt=dt)


class _Rows:
    """Stands for the library in ``_check``: the given rows of one call over many."""

    def __init__(self, out, rows):
        self.out, self.rows = out, rows

    def distill(self, z, idx, top, tau, mass, w, grad=True, dlogits=None):
        loss, lse, dz = self.out
        return loss[self.rows], lse[self.rows], None if dz is None else dz[self.rows]


# V: rows for blocks of 128, 512 and 992 threads, which keep them whole, in part, or hardly at all
@pytest.mark.parametrize("dt,V,k", [("f32", 9, 3), ("bf16", 777, 32), ("f16", 12001, 40),
                                    ("f32", 32000, 20), ("bf16", 100003, 64), ("bf16", 131072, 64),
                                    ("f32", 100000, 33), ("f16", 200001, 7), ("bf16", 270000, 1024)])
@pytest.mark.parametrize("form", ["plain", "mass", "shifted", "in place", "repeats"])
def test_many_rows_against_the_oracle(bk, dt, V, k, form):
    """Rows from the whole of one call over many, each against the oracle under the bounds of a call
    of few: with the teacher's own log-sum-exp, with an output whose rows lie otherwise to 16-byte
    boundaries than the logits' (and apart by another stride), in place, and with indices that stand
    in a list more than once."""
    rows, tau = 611, [1.0, 1.5][k % 2]
    z, idx, top, teacher = _problem(rows, V, k, dt, V + len(form), repeat=form == "repeats" and V > 9)
    gen = torch.Generator(device="cuda").manual_seed(V)
    w = torch.randn(rows, generator=gen, device="cuda")
    w[torch.rand(rows, generator=gen, device="cuda") < 0.2] = 0
    mass = torch.logsumexp(teacher.double() / tau, dim=1).float() if form == "mass" else None
    del teacher
    pick = torch.tensor([0, 1, 147, 295, 296, 592, 609, 610], device="cuda")
    zr, ir, tr, wr = z[pick], idx[pick], top[pick], w[pick]
    mr = None if mass is None else mass[pick]
    st = bk.new_status("cuda")
    dlogits = around = None
    if form == "shifted":
        around = torch.full((rows, V + 13), 9.0, device="cuda").to(DT[dt])
        dlogits = around[:, 5:5 + V]
    elif form == "in place":
        dlogits = z
    alone = bk.distill(z, idx, top, tau, mass, w, grad=False, status=st)
    out = bk.distill(z, idx, top, tau, mass, w, dlogits=dlogits, status=st)
    _check(_Rows(out, pick), zr, ir, tr, tau, mr, wr, dt=dt)
    _check(_Rows(alone, pick), zr, ir, tr, tau, mr, wr, grad=False, dt=dt)
    assert bk.bakron_read_status(st) == 0
    assert not out[2][w == 0].any() and not out[0][w == 0].any()
    if around is not None:
        assert (around[:, :5] == 9).all() and (around[:, 5 + V:] == 9).all()
