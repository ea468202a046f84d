"""fp64 CPU oracle for the gated delta rule and its gradients.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py): the tests and the smoke
check may call it; the product path never does.

What it computes, token by token, per batch row (or packed sequence) and head,
with the state S (headdim x dstate):

    a_t = exp(step_t A),  step_t = softplus(delta_t + bias) or delta_t + bias,
    b_t = sigmoid(beta_t) or beta_t,
    r_t = v_t - a_t S_{t-1} k_t,  S_t = a_t S_{t-1} + b_t r_t k_t^T,  y_t = scale S_t q_t.

The backward is the hand-derived adjoint of these five lines, in reverse, from
the stored states.  ``tests/test_oracle_delta.py`` pins the forward against a
written-out example, causal linear attention and the SSD oracle, and the
backward against central differences of the forward.
"""
import numpy as np


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def _sigmoid(x):
    return np.exp(-np.logaddexp(0.0, -x))


def _rows(batch, L, cu):
    """(batch row, first token, end) of every recurrence; offsets clamped into [0, L] as the library does."""
    if cu is None:
        return [(b, 0, L) for b in range(batch)]
    out = []
    for s in range(len(cu) - 1):
        lo = min(max(int(cu[s]), 0), L)
        out.append((0, lo, max(lo, min(int(cu[s + 1]), L))))
    return out


def delta_fwd(q, k, v, delta, A, beta, delta_bias=None, softplus=True, sigmoid=True, scale=None, initial_state=None,
              cu_seqlens=None, y_before=None):
    """y [batch, L, heads, headdim] and the final states [rows, heads, headdim, dstate] in float64.

    y_before: what the rows of y hold before the call (rows of no sequence keep it; zero by default)."""
    y, S, _ = _walk(q, k, v, delta, A, beta, delta_bias, softplus, sigmoid, scale, initial_state, cu_seqlens, y_before)
    return y, S


def delta_magnitudes(q, k, v, delta, A, beta, delta_bias=None, softplus=True, sigmoid=True, scale=None,
                     initial_state=None, cu_seqlens=None):
    """The sums of magnitudes behind y and the final states: scale |S|_t |q_t| and |S|_L with |S|_t = a_t |S|_{t-1} +
    |u_t| |k_t|^T (their layouts): what roundings of single operands of their products can move them by, in units of
    the roundings' relative size."""
    x = dict(q=q, k=k, v=v, delta=delta, A=A, beta=beta, bias=delta_bias)
    _, _, (kept, rows, a, b, step, raw, kh, qh, sc) = _walk(**x, softplus=softplus, sigmoid=sigmoid, scale=scale,
                                                            h0=initial_state, cu=cu_seqlens, keep=True)
    v = _f64(v)
    out, last = np.zeros_like(v), []
    for i, (r, lo, hi) in enumerate(rows):
        M = np.abs(kept[i][0])
        for t in range(lo, hi):
            old = a[r, t, :, None, None] * kept[i][t - lo]
            u = b[r, t, :, None] * (v[r, t] - np.einsum("hpn,hn->hp", old, kh[r, t]))
            M = np.abs(a[r, t, :, None, None]) * M + np.abs(u)[..., None] * np.abs(kh[r, t])[:, None, :]
            out[r, t] = abs(sc) * np.einsum("hpn,hn->hp", M, np.abs(qh[r, t]))
        last.append(M)
    return out, np.stack(last)


def _walk(q, k, v, delta, A, beta, bias, softplus, sigmoid, scale, h0, cu, y_before=None, keep=False):
    q, k, v, delta, A, beta, bias, h0 = map(_f64, (q, k, v, delta, A, beta, bias, h0))
    batch, L, H, P = v.shape
    G, N = k.shape[2:]
    scale = N ** -0.5 if scale is None else scale
    raw = delta if bias is None else delta + bias
    step = np.logaddexp(raw, 0.0) if softplus else raw
    a, b = np.exp(step * A), _sigmoid(beta) if sigmoid else beta
    kh, qh = np.repeat(k, H // G, axis=2), np.repeat(q, H // G, axis=2)
    rows = _rows(batch, L, cu)
    y = np.zeros_like(v) if y_before is None else np.array(y_before, dtype=np.float64)
    S = np.zeros((len(rows), H, P, N)) if h0 is None else h0.copy()
    kept = []
    for i, (r, lo, hi) in enumerate(rows):
        path = [S[i].copy()]
        for t in range(lo, hi):
            old = a[r, t, :, None, None] * path[-1]
            res = v[r, t] - np.einsum("hpn,hn->hp", old, kh[r, t])
            new = old + (b[r, t, :, None] * res)[..., None] * kh[r, t][:, None, :]
            y[r, t] = scale * np.einsum("hpn,hn->hp", new, qh[r, t])
            path = path + [new] if keep else [new]
        S[i] = path[-1]
        kept.append(path)
    return y, S, (kept, rows, a, b, step, raw, kh, qh, scale)


def delta_bwd(q, k, v, delta, A, beta, dy, delta_bias=None, softplus=True, sigmoid=True, scale=None,
              initial_state=None, cu_seqlens=None, dfinal_state=None):
    """Gradients of sum(y dy) + sum(final_state dfinal_state): a dict of dq, dk, dv, ddelta, dA, dbeta, ddelta_bias,
    dinitial_state (float64).  Tokens of no sequence have zero gradients."""
    _, S, (kept, rows, a, b, step, raw, kh, qh, scale) = _walk(q, k, v, delta, A, beta, delta_bias, softplus, sigmoid,
                                                               scale, initial_state, cu_seqlens, keep=True)
    v, A, dy, beta = map(_f64, (v, A, dy, beta))
    H, P = v.shape[2:]
    G, N = k.shape[2:]
    dq, dk, dv = np.zeros_like(qh), np.zeros_like(kh), np.zeros_like(v)
    dla, db = np.zeros_like(step), np.zeros_like(step)
    dS0 = np.zeros_like(S)
    for i, (r, lo, hi) in enumerate(rows):
        dS = np.zeros((H, P, N)) if dfinal_state is None else _f64(dfinal_state)[i].copy()
        for t in reversed(range(lo, hi)):
            old, new = kept[i][t - lo], kept[i][t - lo + 1]
            at, bt, kt = a[r, t][:, None, None], b[r, t][:, None], kh[r, t]
            dq[r, t] = scale * np.einsum("hpn,hp->hn", new, dy[r, t])
            dS = dS + scale * dy[r, t][..., None] * qh[r, t][:, None, :]
            res = v[r, t] - np.einsum("hpn,hn->hp", at * old, kt)
            du = np.einsum("hpn,hn->hp", dS, kt)
            dr = bt * du
            dv[r, t] = dr
            db[r, t] = (du * res).sum(-1)
            dk[r, t] = np.einsum("hpn,hp->hn", dS, bt * res) - np.einsum("hpn,hp->hn", at * old, dr)
            dold = dS - dr[..., None] * kt[:, None, :]      # adjoint of a_t S_{t-1}
            dla[r, t] = (dold * at * old).sum((-1, -2))
            dS = at * dold
        dS0[i] = dS
    dstep = dla * A
    ddelta = dstep * _sigmoid(raw) if softplus else dstep
    grp = lambda x: x.reshape(x.shape[:2] + (G, H // G, N)).sum(3)  # noqa: E731
    return dict(dq=grp(dq), dk=grp(dk), dv=dv, ddelta=ddelta, dA=(dla * step).sum((0, 1)),
                dbeta=db * b * (1 - b) if sigmoid else db, ddelta_bias=ddelta.sum((0, 1)), dinitial_state=dS0)
