"""Pins of the norm and rotary oracle (CPU): the rotation against matrices, the gradients against differences, the
4-bit rounding of fp64 rows against that of bf16 rows."""
import numpy as np
import pytest

from oracle import cache_oracle as C
from oracle import msa_oracle as O
from oracle import rope_oracle as R


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("pairs", [16, 48, 64])
def test_rotation_is_a_rotation_matrix(adjacent, pairs):
    rng = np.random.default_rng(0)
    pos, f = np.array([[3, -2], [0, 7], [100000, 1]]), rng.standard_normal(pairs)
    axes = rng.integers(0, 2, pairs)
    x = rng.standard_normal((3, 2, 128))
    y = R.rotate(x, R.turns(pos, f, axes), adjacent)
    for t in range(3):
        m = np.eye(128)
        for p in range(pairs):
            a, b = (2 * p, 2 * p + 1) if adjacent else (p, p + pairs)
            w = pos[t, axes[p]] * f[p]
            m[a, a] = m[b, b] = np.cos(w)
            m[a, b], m[b, a] = -np.sin(w), np.sin(w)
        assert np.allclose(y[t], x[t] @ m.T, rtol=0, atol=1e-12)


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("norm, turn, scale", [(True, True, 1.0), (True, True, 1.25), (False, True, 0.5), (True, False, 1.0)])
def test_gradients_match_differences(adjacent, norm, turn, scale):
    rng = np.random.default_rng(1)
    x, dy, w = rng.standard_normal((4, 3, 128)), rng.standard_normal((4, 3, 128)), rng.standard_normal((3, 128))
    t = R.turns(rng.integers(0, 50, (4, 1)), rng.standard_normal(32), np.zeros(32, int)) if turn else None
    w = w if norm else None
    f = lambda x, w: float((dy * R.norm_rope(x, w, t, adjacent, 1e-3, scale)).sum())
    dx, dw = R.norm_rope_grad(x, w, dy, t, adjacent, 1e-3, scale)
    h = 1e-5    # differences are off by h^2 and 1e-16 / h, times sums of a thousand values of order 1
    for _ in range(5):
        v = rng.standard_normal(x.shape)
        assert abs((f(x + h * v, w) - f(x - h * v, w)) / (2 * h) - (dx * v).sum()) < 1e-6
        if norm:
            v = rng.standard_normal(w.shape)
            assert abs((f(x, w + h * v) - f(x, w - h * v)) / (2 * h) - (dw.sum(0) * v).sum()) < 1e-6


@pytest.mark.parametrize("exp", [0, -5, 7])
def test_rounding_of_fp64_rows(exp):
    rng = np.random.default_rng(2)
    bits = O.f64_to_bf16(rng.standard_normal((40, 128)) * 2.0 ** exp * np.exp(rng.standard_normal((40, 1)) * 4))
    bits[3] = 0
    bits[4, 9], bits[5, 100] = 0x7F80, 0x7FC0
    codes, scales, _ = C.round_rows(bits, exp)
    got = R.round_values(O.bf16_to_f64(bits), exp)
    ok = np.repeat(scales != 0x7F, 16, 1)
    assert np.array_equal(got[1], scales) and np.array_equal(got[0][ok], codes[ok])
    # an fp64 value on either side of a border that no bf16 value tells apart
    x = np.full((3, 128), 0.1)
    x[:, ::16] = 6.0
    x[:, 1] = 2.5 * (1 + np.array([-1e-13, 0, 1e-13]))
    assert R.round_values(x, 0)[0][:, 1].tolist() == [4, 4, 5]
