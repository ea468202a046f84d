"""fp64 CPU oracle for the RMS norms around a layer and their gradients.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).  The forwards are the
formulas of include/ssm_scan.h written out; the gradients come from the
Jacobian of t -> t / sqrt(mean t^2 + eps), applied as a matrix per group.
``tests/test_oracle_norms.py`` pins them against central differences.
"""
import numpy as np


def _silu(z):
    s = np.exp(-np.logaddexp(0.0, -z))
    return z * s, s + z * s * (1 - s)


def _rms(t, eps):
    """t / size and size over the last axis."""
    size = np.sqrt((t * t).mean(-1, keepdims=True) + eps)
    return t / size, size


def _rms_bwd(m, t, eps):
    """J^T m for t -> t / size: J = (I - t t^T / (n size^2)) / size."""
    size = _rms(t, eps)[1]
    return m / size - t * (m * t).sum(-1, keepdims=True) / (t.shape[-1] * size ** 3)


def gated_fwd(x, z, weight, group, eps, gate_first):
    x = np.asarray(x, np.float64)
    xs = x.reshape(x.shape[0], -1, group)
    w = np.asarray(weight, np.float64).reshape(1, -1, group)
    f = 1.0 if z is None else _silu(np.asarray(z, np.float64).reshape(xs.shape))[0]
    y = w * _rms(xs * f, eps)[0] if gate_first else w * _rms(xs, eps)[0] * f
    return y.reshape(x.shape)


def gated_bwd(x, z, weight, dy, group, eps, gate_first):
    x = np.asarray(x, np.float64)
    xs = x.reshape(x.shape[0], -1, group)
    w = np.asarray(weight, np.float64).reshape(1, -1, group)
    d = np.asarray(dy, np.float64).reshape(xs.shape)
    f, df = (1.0, 0.0) if z is None else _silu(np.asarray(z, np.float64).reshape(xs.shape))
    t = xs * f if gate_first else xs
    n = _rms(t, eps)[0]
    dn = d if gate_first else d * f                      # gradient of w n
    dt = _rms_bwd(dn * w, t, eps)
    dx, dz = (dt * f, dt * xs * df) if gate_first else (dt, d * w * n * df)
    dw = (dn * n).sum(0)
    if w.shape[1] == 1:
        dw = dw.sum(0)
    return dict(dx=dx.reshape(x.shape), dz=None if z is None else dz.reshape(x.shape), dweight=dw.reshape(-1))


def residual_fwd(x, residual, weight, scale, post_weight, eps):
    x = np.asarray(x, np.float64)
    a = x if post_weight is None else np.asarray(post_weight, np.float64) * _rms(x, eps)[0]
    r = (0.0 if residual is None else np.asarray(residual, np.float64)) + (
        a if scale is None else np.asarray(scale, np.float64) * a)
    return np.asarray(weight, np.float64) * _rms(r, eps)[0], r


def residual_bwd(x, residual_out, weight, dy, dresidual_out, scale, post_weight, eps):
    x, r, w, d = (np.asarray(t, np.float64) for t in (x, residual_out, weight, dy))
    dr = _rms_bwd(d * w, r, eps) + (0.0 if dresidual_out is None else np.asarray(dresidual_out, np.float64))
    pw = np.ones_like(w) if post_weight is None else np.asarray(post_weight, np.float64)
    sc = np.ones_like(w) if scale is None else np.asarray(scale, np.float64)
    n = x if post_weight is None else _rms(x, eps)[0]
    da = dr * sc
    return dict(dresidual=dr, dweight=(d * _rms(r, eps)[0]).sum(0), dscale=(dr * pw * n).sum(0),
                dpost_weight=(da * n).sum(0), dx=da if post_weight is None else _rms_bwd(da * pw, x, eps))
