"""Pins of the norms' fp64 oracle (oracle/norms.py): hand values and central differences."""
import numpy as np
import pytest

from oracle import norms as O

EPS = 1e-3


def _diff(f, a, dy):
    num = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep, e = a[i], 1e-6
        a[i] = keep + e
        up = (f() * dy).sum()
        a[i] = keep - e
        num[i] = (up - (f() * dy).sum()) / (2 * e)
        a[i] = keep
    return num


def test_values_by_hand():
    x = np.array([[3.0, 4.0]])
    assert np.allclose(O.gated_fwd(x, None, [1.0, 2.0], 2, 0.0, False), [[3 / 12.5 ** 0.5, 8 / 12.5 ** 0.5]])
    # group of one: x SiLU(z) normalised is its sign; SiLU(1) = 1 / (1 + 1/e) behind the norm
    assert np.allclose(O.gated_fwd(x, [[-1.0, 1.0]], [1.0, 1.0], 1, 0.0, True), [[-1.0, 1.0]])
    assert np.allclose(O.gated_fwd(x, [[0.0, 1.0]], [1.0, 1.0], 1, 0.0, False), [[0.0, 1 / (1 + np.exp(-1.0))]])
    y, r = O.residual_fwd(x, np.array([[1.0, 0.0]]), [1.0, 1.0], [2.0, 0.5], None, 0.0)
    assert np.allclose(r, [[7.0, 2.0]]) and np.allclose(y, r / (53 / 2) ** 0.5)


@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("shared", [False, True])
def test_gated_gradients(gate_first, shared):
    rng = np.random.default_rng(5)
    x, z, dy = (rng.standard_normal((3, 6)) for _ in range(3))
    w = rng.standard_normal(3 if shared else 6)
    g = O.gated_bwd(x, z, w, dy, 3, EPS, gate_first)
    f = lambda: O.gated_fwd(x, z, w, 3, EPS, gate_first)  # noqa: E731
    for name, a in (("dx", x), ("dz", z), ("dweight", w)):
        assert np.allclose(g[name], _diff(f, a, dy), rtol=1e-6, atol=1e-7), name


@pytest.mark.parametrize("post", [False, True])
def test_residual_gradients(post):
    rng = np.random.default_rng(6)
    x, r, dy, dr = (rng.standard_normal((3, 5)) for _ in range(4))
    w, sc = rng.standard_normal(5), rng.standard_normal(5)
    pw = rng.standard_normal(5) if post else None
    out = lambda: O.residual_fwd(x, r, w, sc, pw, EPS)  # noqa: E731
    g = O.residual_bwd(x, out()[1], w, dy, dr, sc, pw, EPS)
    f = lambda: np.stack(out())  # noqa: E731
    both = np.stack([dy, dr])
    for name, a in [("dx", x), ("dresidual", r), ("dweight", w), ("dscale", sc)] + ([("dpost_weight", pw)] if post
                                                                                    else []):
        assert np.allclose(g[name], _diff(f, a, both), rtol=1e-6, atol=1e-7), name
