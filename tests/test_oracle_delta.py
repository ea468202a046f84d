"""Pins of the gated delta rule's fp64 oracle (oracle/delta.py): hand-computed steps, special cases that other
oracles cover, and its adjoint against central differences."""
import numpy as np
import pytest

from oracle import delta as D
from oracle import ssd as S


def _inputs(rng, batch, L, G, H, N, P):
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
    return dict(q=unit(rng.standard_normal((batch, L, G, N))), k=unit(rng.standard_normal((batch, L, G, N))),
                v=rng.standard_normal((batch, L, H, P)), delta=rng.standard_normal((batch, L, H)),
                A=-rng.uniform(0.2, 2.0, H), beta=rng.standard_normal((batch, L, H)),
                delta_bias=rng.uniform(-2, 0, H))


def test_two_steps_by_hand():
    """One head of one channel and two states: S_0 = b v k^T; the second key equal to the first replaces the value
    (b = 1, a = 1: the state then answers the key with the new value alone)."""
    k = np.array([[[[0.6, 0.8]], [[0.6, 0.8]]]])
    v = np.array([[[[2.0]], [[-3.0]]]])
    one, zero = np.ones((1, 2, 1)), np.zeros((1, 2, 1))
    y, s = D.delta_fwd(k, k, v, zero, np.array([-1.0]), one, softplus=False, sigmoid=False, scale=1.0)
    assert np.allclose(y[0, :, 0, 0], [2.0, -3.0]) and np.allclose(s[0, 0, 0], [-1.8, -2.4])
    # b = 0.5 and a fade of 1/2 before the second: S k = 0.5 * 1 after the fade, r = -3.5, u = -1.75
    step = np.array([[[0.0], [np.log(2.0)]]])
    y, s = D.delta_fwd(k, k, v, step, np.array([-1.0]), 0.5 * one, softplus=False, sigmoid=False, scale=2.0)
    assert np.allclose(y[0, :, 0, 0], [2.0, 2 * (0.5 - 1.75)]) and np.allclose(s[0, 0, 0], [-1.25 * 0.6, -1.25 * 0.8])


def test_orthogonal_keys_are_linear_attention():
    """Keys that are distinct unit vectors never meet: the correction vanishes and y is causal attention."""
    rng = np.random.default_rng(1)
    N = L = 12
    x = _inputs(rng, 1, L, 1, 1, N, 5)
    x["k"] = np.eye(N)[rng.permutation(N)][None, :, None, :]
    y, _ = D.delta_fwd(**x, scale=0.7)
    step = np.logaddexp(x["delta"] + x["delta_bias"], 0)[0, :, 0] * x["A"][0]
    cs, b = np.cumsum(step), 1 / (1 + np.exp(-x["beta"][0, :, 0]))
    att = np.tril(np.exp(cs[:, None] - cs[None, :]) * (x["q"][0, :, 0] @ x["k"][0, :, 0].T))
    assert np.allclose(y[0, :, 0], 0.7 * att @ (b[:, None] * x["v"][0, :, 0]), atol=1e-12)


def test_vanishing_correction_is_the_ssd_layer():
    """As b -> 0 with v = w / b the write is w k^T: the SSD recurrence with C = q, B = k, x delta = w."""
    rng = np.random.default_rng(2)
    x = _inputs(rng, 2, 40, 1, 3, 8, 4)
    raw = x["delta"] + x["delta_bias"]
    step = np.logaddexp(raw, 0)
    eps = 1e-9
    y, s = D.delta_fwd(x["q"], x["k"], x["v"] * step[..., None] / eps, x["delta"], x["A"],
                       np.full_like(x["beta"], eps), delta_bias=x["delta_bias"], sigmoid=False, scale=1.0)
    yo, so = S.ssd_fwd(x["v"], x["delta"], x["A"], x["k"], x["q"], delta_bias=x["delta_bias"])
    assert np.allclose(y, yo, atol=1e-7) and np.allclose(s, so, atol=1e-7)


def test_continuation_and_packing():
    """A sequence cut in two, the second part from the first's state, equals the whole; packed sequences equal the
    separate ones; tokens of no sequence keep y."""
    rng = np.random.default_rng(3)
    x = _inputs(rng, 1, 30, 2, 4, 6, 3)
    y, s = D.delta_fwd(**x)
    cut = lambda lo, hi: {n: (a[:, lo:hi] if a.ndim > 1 else a) for n, a in x.items()}  # noqa: E731
    y1, s1 = D.delta_fwd(**cut(0, 13))
    y2, s2 = D.delta_fwd(**cut(13, 30), initial_state=s1)
    assert np.allclose(np.concatenate([y1, y2], 1), y) and np.allclose(s2, s)
    h0 = rng.standard_normal((3, 4, 3, 6))
    yp, sp = D.delta_fwd(**x, initial_state=h0, cu_seqlens=[0, 13, 13, 25], y_before=np.full(x["v"].shape, 7.0))
    a, sa = D.delta_fwd(**cut(0, 13), initial_state=h0[:1])
    b, sb = D.delta_fwd(**cut(13, 25), initial_state=h0[2:])
    assert np.allclose(yp[:, :13], a) and np.allclose(yp[:, 13:25], b) and np.all(yp[:, 25:] == 7.0)
    assert np.allclose(sp, np.concatenate([sa, h0[1:2], sb]))


@pytest.mark.parametrize("softplus,sigmoid", [(True, True), (False, False)])
def test_backward_against_central_differences(softplus, sigmoid):
    rng = np.random.default_rng(4)
    x = _inputs(rng, 1, 9, 2, 4, 4, 3)
    if not softplus:
        x["delta"] = 0.1 + 0.3 * rng.random(x["delta"].shape)   # the step itself: keep it positive
        x["delta_bias"] = 0.1 * rng.random(4)
    if not sigmoid:
        x["beta"] = rng.random(x["beta"].shape)
        x["beta"][0, 3] = 0.0                      # a token that writes nothing still has a gradient of beta
    x["initial_state"] = rng.standard_normal((2, 4, 3, 4))
    cu = [0, 5, 9]
    dy, dfs = rng.standard_normal(x["v"].shape), rng.standard_normal((2, 4, 3, 4))
    more = dict(softplus=softplus, sigmoid=sigmoid, scale=0.8, cu_seqlens=cu)
    h0 = x.pop("initial_state")

    def loss(x, h0):
        y, s = D.delta_fwd(**x, initial_state=h0, **more)
        return (y * dy).sum() + (s * dfs).sum()

    g = D.delta_bwd(**x, dy=dy, initial_state=h0, dfinal_state=dfs, **more)
    for name in list(x) + ["initial_state"]:
        a = h0 if name == "initial_state" else x[name]
        num = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            keep, e = a[i], 1e-5
            a[i] = keep + e
            up = loss(x, h0)
            a[i] = keep - e
            dn = loss(x, h0)
            a[i] = keep
            num[i] = (up - dn) / (2 * e)
        # central differences: truncation ~ e^2, rounding ~ 1e-16 |loss| / e
        assert np.allclose(g["d" + name], num, rtol=1e-6, atol=1e-8), name
