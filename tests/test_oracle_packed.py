"""CPU pins of the fp64 restatement behind the 4-bit layer, the 8-bit norm and the distillation loss:
the layout against a vectorised form, the loss against scipy's, its gradient against differences."""
import numpy as np
import pytest

from oracle import distill, matvec4, pack4_layout, rms_norm_q8


@pytest.mark.parametrize("m,n,group", [(1, 1, None), (17, 70, 32), (16, 64, None), (33, 129, 64)])
def test_layout_vectorised(m, n, group):
    rng = np.random.default_rng(m * 100 + n)
    g = n if group is None else group
    G = -(-n // g)
    codes = rng.integers(-8, 8, (m, n))
    scales = rng.random((m, G), dtype=np.float32)
    got = pack4_layout(codes, scales, group)
    mt, kt = -(-m // 16), -(-n // 64)
    c = np.zeros((mt * 16, kt * 64), dtype=np.uint32)
    c[:m, :n] = codes & 15
    c = c.reshape(mt, 2, 8, kt, 2, 4, 8)
    word = sum(c[..., k] << (4 * p) for p, k in enumerate([0, 4, 2, 6, 1, 5, 3, 7]))
    word = word.transpose(0, 3, 2, 5, 4, 1).astype("<u4")
    np.testing.assert_array_equal(got[:mt * kt * 512], word.reshape(-1).view(np.uint8))
    s = np.zeros((mt * 16, G), dtype=np.float32)
    s[:m] = scales
    np.testing.assert_array_equal(got[mt * kt * 512:].view(np.float32),
                                  s.reshape(mt, 2, 8, G).transpose(0, 3, 2, 1).reshape(-1))


def test_matvec_scales_and_codebook():
    codes = np.array([[1, -2, 3], [0, 7, -8]])
    y, a = matvec4(codes, [2.0, 0.5], [[1.0, 10.0, 100.0]])
    np.testing.assert_array_equal(y, [[2 * 281.0, 0.5 * -730.0]])
    np.testing.assert_array_equal(a, [[2 * 321.0, 0.5 * 870.0]])
    y, _ = matvec4([[0, 3]], [1.0], [[5, 7]], codebook=[-1, 0, 1, 2], x_scales=[0.5])
    np.testing.assert_array_equal(y, [[0.5 * (-5 + 14)]])


def test_norm_codes_and_scales():
    rng = np.random.default_rng(0)
    x, r, w = rng.standard_normal((3, 100)), rng.standard_normal((3, 100)), rng.random(100)
    q, s, h = rms_norm_q8(x, w, 1e-5, r, 32)
    assert q.shape == (3, 100) and s.shape == (3, 4)
    y = h / np.sqrt((h ** 2).mean(axis=1, keepdims=True) + 1e-5) * w
    full = np.repeat(s, 32, axis=1)[:, :100]
    assert np.all(np.abs(q * full - y) <= full / 2 * (1 + 1e-12))
    assert np.abs(q).max() == 127
    q, s, _ = rms_norm_q8(np.zeros((1, 5)))
    assert not q.any() and not s.any()
    q, _, _ = rms_norm_q8(np.array([[254.0, 1.0, 3.0, -1.0, -5.0]]))   # ties to even: .5, 1.5, -2.5
    np.testing.assert_array_equal(q, [[127, 0, 2, 0, -2]])


def test_distill_against_the_full_divergence():
    """A list that holds the whole vocabulary is the KL divergence of two softmaxes."""
    from scipy.special import log_softmax, rel_entr, softmax
    rng = np.random.default_rng(1)
    z, t = rng.standard_normal((4, 20)), rng.standard_normal((4, 20))
    idx = np.tile(np.arange(20), (4, 1))
    loss, lse, _ = distill(z, idx, t, tau=1.7)
    ref = rel_entr(softmax(t / 1.7, axis=1), softmax(z / 1.7, axis=1)).sum(axis=1)
    np.testing.assert_allclose(loss, ref, rtol=1e-12)
    np.testing.assert_allclose(z / 1.7 - lse[:, None], log_softmax(z / 1.7, axis=1), rtol=1e-12)


@pytest.mark.parametrize("own_mass", [False, True])
def test_distill_gradient_against_differences(own_mass):
    rng = np.random.default_rng(2)
    z = rng.standard_normal((3, 9))
    idx = np.array([[1, 4, 4], [0, -1, 8], [-1, -1, -1]])
    t = rng.standard_normal((3, 3))
    mass = np.array([3.0, 2.5, 2.0]) if own_mass else None
    w = np.array([0.7, 1.3, 1.0])
    f = lambda z: distill(z, idx, t, 1.3, mass, w)  # noqa: E731
    _, _, dz = f(z)
    num = np.zeros_like(z)
    for i in range(3):
        for j in range(9):
            e = np.zeros_like(z)
            e[i, j] = 1e-5
            num[i, j] = (f(z + e)[0].sum() - f(z - e)[0].sum()) / 2e-5
    np.testing.assert_allclose(dz, num, rtol=0, atol=1e-9)
    assert not dz[2].any()
    loss, lse, dz = distill(z, idx, t, row_weights=[0.0, 1.0, 0.0])
    assert loss[0] == lse[0] == 0 and not dz[0].any() and loss[1] != 0
