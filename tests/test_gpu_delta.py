"""GPU parity of the gated delta rule (ssm_delta_fwd, ssm_delta_update) against its fp64 oracle (oracle/delta.py).

Error measure: that of gpu_util (|g - o| over max(|o|, rms(o)), the largest).  Tolerances, derived beforehand:
  - fp32 arithmetic, token by token: a token adds a product of up to 256 terms for r and one for y, rounded at
    2^-24 of the terms' magnitudes each; with unit keys and a fading state the errors of earlier tokens fade too.
    256 x 2^-24 = 1.5e-5, twice that for r's way through the state: 3e-5 of the terms' magnitudes, for y and the
    state (or of the rms, where the terms are smaller).
  - the chunked plan keeps 22 significant bits on the state's path: three products a chunk, each off by 2 x 2^-22 of
    its terms, below the same 3e-5 for the state.
  - y of the chunked plan is a sum of products with one or two operands rounded to fp16 (the state, the scores and u;
    half a step is 2^-11 each): with M the sum of the products' magnitudes it is off by at most 2 x 2^-11 M.  Storage
    in bf16 adds half a step, 2^-8 |y|.  Both are asked element by element, M from the oracle
    (delta_magnitudes), with the fp32 part above relative to max(M, rms).
  - over all of y the roundings are independent: rounding to bf16 alone leaves a relative 2-norm of 2^-8 / sqrt(3) x
    0.72 (the mean of 1 / mantissa's share) = 1.65e-3, the fp16 operands at most a quarter of 2^-10 beside it:
    2.2e-3 is asked.
"""
import numpy as np
import pytest
import torch

from oracle import delta as D
from selective_state_space_33_amd import inputs as I
from selective_state_space_33_amd import ops

from .gpu_util import rel_err, say

pytestmark = pytest.mark.gpu

TOL_STATE = 3e-5
TOL_NORM = {"f32": 3e-5, "bf16": 2.2e-3}


def y_off(y, yo, M, dtype):
    """(largest error of y over its bound, relative 2-norm of the error); a value that is not finite fails."""
    y, yo = np.asarray(y, np.float64), np.asarray(yo, np.float64)
    if not np.all(np.isfinite(y)):
        return float("inf"), float("inf")
    rms = max(float(np.sqrt(np.mean(yo * yo))), 1e-30)
    tol = 3e-5 * np.maximum(M, rms)
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(yo) + 2.0 ** -10 * M
    return float(np.max(np.abs(y - yo) / tol)), float(np.linalg.norm(y - yo) / max(np.linalg.norm(yo), 1e-30))


def s_off(s, so, Ms):
    """Largest error of the states over max(the terms' magnitudes, rms)."""
    s, so = np.asarray(s, np.float64), np.asarray(so, np.float64)
    if not np.all(np.isfinite(s)):
        return float("inf")
    return float(np.max(np.abs(s - so) / np.maximum(Ms, max(float(np.sqrt(np.mean(so * so))), 1e-30))))


def dev(a, dtype="f32"):
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to("cuda:0")
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def tensors(x, dtype):
    return {n: dev(a, "f32" if n in ("A", "delta_bias") else dtype) for n, a in x.items()}


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def run(x, dtype, h0=None, cu=None, **kw):
    t = tensors(x, dtype)
    y, s = ops.ssm_delta_fwd(t["q"], t["k"], t["v"], t["delta"], t["A"], t["beta"], delta_bias=t["delta_bias"],
                             initial_state=dev(h0),
                             cu_seqlens=None if cu is None else torch.tensor(cu, dtype=torch.int64, device="cuda:0"),
                             **kw)
    torch.cuda.synchronize()
    return y, s


def check(x, dtype, label, h0=None, cu=None, **kw):
    say(f"delta {label} q={x['q'].shape} v={x['v'].shape} {dtype}")
    # rows of no sequence are not written: they hold the zeros that the oracle has there
    y, s = run(x, dtype, h0, cu, y=dev(np.zeros(x["v"].shape), dtype), **kw)
    yo, so = D.delta_fwd(**x, initial_state=h0, cu_seqlens=cu, **kw)
    M, Ms = D.delta_magnitudes(**x, initial_state=h0, cu_seqlens=cu, **kw)
    (ey, en), es = y_off(host(y), yo, M, dtype), s_off(host(s), so, Ms)
    print(f"[parity] delta {label}: y {ey:.2f} of its bound, norm {en:.2e}, state {es:.2e}", flush=True)
    assert ey <= 1 and en <= TOL_NORM[dtype] and es <= TOL_STATE, (ey, en, es)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,P", [(32, 16), (64, 64), (96, 48), (128, 128), (192, 32), (256, 64), (64, 37), (128, 3)])
def test_forward_shapes(N, P, dtype):
    x = I.random_delta_inputs(np.random.default_rng(1000 + N + P), 2, 75, 2, 4, N, P, dtype)
    check(x, dtype, f"N={N} P={P}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [1, 2, 15, 63, 64, 65, 127, 128, 129, 200, 321])
def test_forward_lengths(L, dtype):
    rng = np.random.default_rng(1100 + L)
    x = I.random_delta_inputs(rng, 3, L, 3, 6, 64, 32, dtype)
    check(x, dtype, f"L={L}", h0=0.3 * rng.standard_normal((3, 6, 32, 64)).astype(np.float32))


@pytest.mark.parametrize("L", [70, 500])
@pytest.mark.parametrize("opts", ["plain", "no_bias", "no_softplus", "no_sigmoid", "beta_zero", "beta_two", "scale"])
def test_forward_options(opts, L):
    rng = np.random.default_rng(1200 + len(opts) + L)
    x = I.random_delta_inputs(rng, 2, L, 2, 2, 128, 64)
    kw = {}
    if opts == "no_bias":
        x["delta_bias"] = None
    elif opts == "no_softplus":
        kw["softplus"] = False
        x["delta"] = I.round_to_bf16(np.abs(x["delta"]) * 0.05 + 0.01)  # the step itself: keep it positive
        x["delta_bias"] = np.abs(x["delta_bias"]) * 0.01
    elif opts in ("no_sigmoid", "beta_zero", "beta_two"):
        kw["sigmoid"] = False
        b = {"no_sigmoid": rng.random(x["beta"].shape), "beta_zero": np.zeros(x["beta"].shape),
             "beta_two": np.full(x["beta"].shape, 1.9375)}[opts]
        x["beta"] = I.round_to_bf16(b.astype(np.float32))
    elif opts == "scale":
        kw["scale"] = 1.75
    check(x, "bf16", f"{opts} L={L}", h0=rng.standard_normal((2, 2, 64, 128)).astype(np.float32), **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_packed_sequences(dtype):
    """Lengths of zero, one, a chunk and more, from given states; the tokens behind the last sequence and their y stay."""
    rng = np.random.default_rng(1300)
    lens = [70, 0, 1, 64, 130, 0, 17, 65]
    L = sum(lens) + 9
    cu = np.concatenate([[0], np.cumsum(lens)])
    x = I.random_delta_inputs(rng, 1, L, 2, 4, 64, 48, dtype)
    h0 = 0.5 * rng.standard_normal((len(lens), 4, 48, 64)).astype(np.float32)
    say(f"delta packed {dtype}")
    y0 = dev(np.full(x["v"].shape, 7.0), dtype)
    y, s = run(x, dtype, h0, cu, y=y0)
    yo, so = D.delta_fwd(**x, initial_state=h0, cu_seqlens=cu, y_before=np.full(x["v"].shape, 7.0))
    assert torch.equal(y[:, cu[-1]:], torch.full_like(y[:, cu[-1]:], 7.0))
    assert np.array_equal(host(s)[[1, 5]], h0[[1, 5]].astype(np.float64))
    M, Ms = D.delta_magnitudes(**x, initial_state=h0, cu_seqlens=cu)
    live = slice(0, int(cu[-1]))
    (ey, en), es = y_off(host(y)[:, live], yo[:, live], M[:, live], dtype), s_off(host(s), so, Ms)
    print(f"[parity] delta packed {dtype}: y {ey:.2f} of its bound, norm {en:.2e}, state {es:.2e}", flush=True)
    assert ey <= 1 and en <= TOL_NORM[dtype] and es <= TOL_STATE


def test_packed_offsets_outside_the_row_are_clamped():
    rng = np.random.default_rng(1310)
    x = I.random_delta_inputs(rng, 1, 150, 1, 2, 32, 32)
    check(x, "bf16", "clamped offsets", cu=[-5, 80, 400])
    check(x, "bf16", "an offset that goes back", cu=[0, 90, 40])


def test_extreme_steps_and_fades():
    """Raw steps spread over +-60: fades that underflow to 0 within a chunk next to ones that stay at 1."""
    rng = np.random.default_rng(1320)
    x = I.random_delta_inputs(rng, 2, 200, 2, 4, 64, 64)
    x["delta"] = I.round_to_bf16(x["delta"].astype(np.float64) * 20.0)
    check(x, "bf16", "extreme steps", h0=rng.standard_normal((2, 4, 64, 64)).astype(np.float32))


def test_repeated_keys():
    """The same key at every token (the chunk's triangular system at its worst): each write replaces the last one."""
    rng = np.random.default_rng(1330)
    x = I.random_delta_inputs(rng, 1, 190, 1, 2, 64, 32)
    x["k"][:] = x["k"][:, :1]
    x["delta_bias"] = np.full(2, -20.0, np.float32)     # hardly any fade
    x["delta"][:] = 0.0
    x["beta"] = I.round_to_bf16(np.full(x["beta"].shape, 1.0, np.float32))
    check(x, "bf16", "repeated keys", sigmoid=False)


def test_nan_stays_in_its_head_and_behind_its_token():
    rng = np.random.default_rng(1340)
    x = I.random_delta_inputs(rng, 2, 140, 2, 4, 64, 32)
    x["v"][1, 70, 2, 5] = np.nan
    say("delta NaN")
    y, s = run(x, "bf16")
    bad = ~np.isfinite(host(y))
    assert bad[1, 70:, 2, 5].all()
    bad[1, 70:, 2, 5] = False
    # a chunk's other tokens of that channel may share its products, nothing else does
    bad[1, 64:70, 2, 5] = False
    assert not bad.any()
    sb = ~np.isfinite(host(s))
    assert sb[1, 2, 5].all() and sb.sum() == 64


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch,G,H,N,P", [(1, 1, 1, 32, 16), (5, 2, 6, 64, 64), (33, 20, 40, 128, 128), (3, 1, 2, 96, 50),
                                           (2, 2, 2, 256, 70), (1, 4, 4, 192, 1)])
def test_step_against_oracle(batch, G, H, N, P, dtype):
    rng = np.random.default_rng(1400 + N + P)
    x = I.random_delta_inputs(rng, batch, 1, G, H, N, P, dtype)
    h0 = rng.standard_normal((batch, H, P, N)).astype(np.float32)
    say(f"delta step {batch}x{G}/{H}x{N}x{P} {dtype}")
    t = tensors(x, dtype)
    state = dev(h0)
    one = lambda a: a[:, 0].contiguous()  # noqa: E731
    y = ops.ssm_delta_update(state, one(t["q"]), one(t["k"]), one(t["v"]), one(t["delta"]), t["A"], one(t["beta"]),
                             delta_bias=t["delta_bias"])
    torch.cuda.synchronize()
    yo, so = D.delta_fwd(**x, initial_state=h0)
    M, Ms = D.delta_magnitudes(**x, initial_state=h0)
    (ey, en), es = y_off(host(y), yo[:, 0], M[:, 0], dtype), s_off(host(state), so, Ms)
    print(f"[parity] delta step: y {ey:.2f} of its bound, norm {en:.2e}, state {es:.2e}", flush=True)
    assert ey <= 1 and es <= TOL_STATE


def test_steps_continue_a_prefill():
    """A prompt through ssm_delta_fwd, then tokens one by one from its final state: the same as all of it at once."""
    rng = np.random.default_rng(1500)
    x = I.random_delta_inputs(rng, 2, 150, 2, 4, 128, 64)
    h0 = rng.standard_normal((2, 4, 64, 128)).astype(np.float32)
    say("delta prefill then steps")
    t = tensors(x, "bf16")
    cut = 145
    part = lambda a: a[:, :cut].contiguous()  # noqa: E731
    _, state = ops.ssm_delta_fwd(part(t["q"]), part(t["k"]), part(t["v"]), part(t["delta"]), t["A"], part(t["beta"]),
                                 delta_bias=t["delta_bias"], initial_state=dev(h0))
    ys = []
    for i in range(cut, 150):
        one = lambda a: a[:, i].contiguous()  # noqa: E731,B023
        ys.append(ops.ssm_delta_update(state, one(t["q"]), one(t["k"]), one(t["v"]), one(t["delta"]), t["A"],
                                       one(t["beta"]), delta_bias=t["delta_bias"]))
    torch.cuda.synchronize()
    yo, so = D.delta_fwd(**x, initial_state=h0)
    M, Ms = D.delta_magnitudes(**x, initial_state=h0)
    (ey, en), es = y_off(np.stack([host(y) for y in ys], 1), yo[:, cut:], M[:, cut:], "bf16"), s_off(host(state), so, Ms)
    print(f"[parity] delta prefill then steps: y {ey:.2f} of its bound, norm {en:.2e}, state {es:.2e}", flush=True)
    assert ey <= 1 and en <= TOL_NORM["bf16"] and es <= TOL_STATE


def test_final_state_in_the_initial_states_buffer_and_determinism():
    rng = np.random.default_rng(1510)
    x = I.random_delta_inputs(rng, 2, 300, 2, 4, 128, 64)
    h0 = rng.standard_normal((2, 4, 64, 128)).astype(np.float32)
    say("delta in place")
    y1, s1 = run(x, "bf16", h0)
    t, state = tensors(x, "bf16"), dev(h0)
    y2, s2 = ops.ssm_delta_fwd(t["q"], t["k"], t["v"], t["delta"], t["A"], t["beta"], delta_bias=t["delta_bias"],
                               initial_state=state, final_state=state)
    torch.cuda.synchronize()
    assert s2 is state and torch.equal(y1, y2) and torch.equal(s1, s2)


def test_without_final_state():
    x = I.random_delta_inputs(np.random.default_rng(1520), 1, 100, 1, 2, 64, 64)
    say("delta without a final state")
    y1, _ = run(x, "bf16")
    y2, s2 = run(x, "bf16", return_final_state=False)
    assert s2 is None and torch.equal(y1, y2)


@pytest.mark.parametrize("L", [1, 2, 16, 17, 40, 64])
def test_chunked_plan_on_short_sequences(L, monkeypatch):
    monkeypatch.setenv("SSM_DELTA_CHUNKED", "1")
    rng = np.random.default_rng(1600 + L)
    x = I.random_delta_inputs(rng, 3, L, 3, 6, 96, 48)
    check(x, "bf16", f"chunked L={L}", h0=0.3 * rng.standard_normal((3, 6, 48, 96)).astype(np.float32))


@pytest.mark.parametrize("P", [16, 64, 80, 128, 144, 272])
def test_chunked_plan_channel_tiles(P):
    """Channel tiles that fill a wavefront, a workgroup and several of them only in part."""
    rng = np.random.default_rng(1620 + P)
    x = I.random_delta_inputs(rng, 1, 150, 2, 2, 64, P)
    check(x, "bf16", f"P={P}", h0=rng.standard_normal((1, 2, P, 64)).astype(np.float32))


def test_plans_agree(monkeypatch):
    """The chunked plan and the one token by token (y differs by their roundings to bf16)."""
    rng = np.random.default_rng(1640)
    x = I.random_delta_inputs(rng, 2, 700, 2, 4, 128, 128)
    say("delta plans agree")
    y1, s1 = run(x, "bf16")
    monkeypatch.setenv("SSM_DELTA_CHUNKED", "0")
    y2, s2 = run(x, "bf16")
    a, b, es = host(y1), host(y2), rel_err(host(s1), host(s2))
    en = np.linalg.norm(a - b) / np.linalg.norm(b)
    print(f"[parity] delta plans: y norm {en:.2e} state {es:.2e}", flush=True)
    assert 0 < en <= 2 * TOL_NORM["bf16"] and es <= 2 * TOL_STATE


def test_long_sequence_against_oracle():
    """2048 tokens of slowly fading heads: errors of the state would pile up."""
    rng = np.random.default_rng(1650)
    x = I.random_delta_inputs(rng, 1, 2048, 1, 2, 64, 32)
    x["A"] = np.float32([-0.01, -0.5])
    check(x, "bf16", "long, slow fade")


@pytest.mark.parametrize("size", [1e-12, 1e-5, 3e4, 1e9])
def test_values_of_any_magnitude(size):
    """Values, states and y scale together (by a power of two per row and head): as exact at 1e-12 as at 1, beside a row
    of zeros and one of ordinary size."""
    rng = np.random.default_rng(1600)
    x = I.random_delta_inputs(rng, 3, 200, 2, 4, 64, 48)
    size = np.array([size, 0.0, 1.0]).reshape(3, 1, 1, 1)
    x["v"] = I.round_to_bf16((x["v"] * size).astype(np.float32))
    h0 = (size * rng.standard_normal((3, 4, 48, 64))).astype(np.float32)
    say(f"delta values of size {size[0, 0, 0, 0]}")
    y, s = run(x, "bf16", h0)
    yo, so = D.delta_fwd(**x, initial_state=h0)
    M, Ms = D.delta_magnitudes(**x, initial_state=h0)
    for b in (0, 2):
        (ey, en), es = y_off(host(y)[b], yo[b], M[b], "bf16"), s_off(host(s)[b], so[b], Ms[b])
        print(f"[parity] row {b}: y {ey:.2f} of its bound, norm {en:.2e}, state {es:.2e}", flush=True)
        assert ey <= 1 and en <= TOL_NORM["bf16"] and es <= TOL_STATE, (b, ey, en, es)
    assert not host(y)[1].any() and not host(s)[1].any()


@pytest.mark.parametrize("scale", [1e-9, 1e6])
def test_scale_of_any_magnitude(scale):
    rng = np.random.default_rng(1610)
    x = I.random_delta_inputs(rng, 1, 150, 1, 2, 32, 32)
    check(x, "bf16", f"scale {scale}", scale=scale)


@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("where", ["q", "k", "v", "delta", "beta"])
@pytest.mark.parametrize("token", [0, 69, 111, 128])
def test_garbage_in_padding_leaves_what_is_before_it(where, token, value):
    """A NaN or an infinity in a token (of padding, say) reaches it and what follows it, and no token before it, other
    row, head or (from v) channel: there the results are those of the clean call, bit for bit."""
    rng = np.random.default_rng(1620)
    x = I.random_delta_inputs(rng, 2, 140, 2, 4, 64, 48)
    say(f"delta {value} in {where} at {token}")
    y0, s0 = run(x, "bf16")
    head = 1 if where in "qk" else 2
    x[where] = x[where].copy()
    x[where][(1, token, head) + ((5,) if where in "qkv" else ())] = -value if where == "delta" else value
    y, s = run(x, "bf16")
    same = y == y0
    heads = [2, 3] if where in "qk" else [2]
    if where == "v":
        assert not torch.isfinite(y[1, token:, 2, 5]).any() and not torch.isfinite(s[1, 2, 5]).any()
        same[1, token:, 2, 5] = True
    elif where in "qk" or np.isnan(value):
        assert not torch.isfinite(y[1, token, heads]).any()
        same[1, token:, heads] = True
    else:       # an infinite step or beta is a fade or a gate of its limit: nothing, 0 or 1
        same[1, token:, heads] = True
    assert bool(same.all())
    if where == "k" or (where in ("delta", "beta") and np.isnan(value)):
        assert not torch.isfinite(s[1, heads]).any()


@pytest.mark.parametrize("N,P", [(32, 80), (96, 80), (64, 144), (128, 96)])
@pytest.mark.parametrize("L", [65, 130])
def test_wide_workgroups_give_what_narrow_ones_do(N, P, L):
    """A batch large enough for eight wavefronts a workgroup, its last row ending where its tensors do, one token into a
    chunk: each row as alone, where the workgroups have four, bit for bit."""
    rng = np.random.default_rng(1630 + N)
    B, H = 16, 24
    x = I.random_delta_inputs(rng, B, L, H // 2, H, N, P)
    say(f"delta wide N={N} P={P} L={L}")
    t = tensors(x, "bf16")
    h0 = dev(rng.standard_normal((B, H, P, N)))

    def call(s):
        return ops.ssm_delta_fwd(*(t[n][s].contiguous() for n in ("q", "k", "v", "delta")), t["A"],
                                 t["beta"][s].contiguous(), delta_bias=t["delta_bias"], initial_state=h0[s].contiguous())

    y, S = call(slice(0, B))
    for b in (0, 7, B - 1):
        yb, Sb = call(slice(b, b + 1))
        assert torch.equal(y[b:b + 1], yb) and torch.equal(S[b:b + 1], Sb), b


def test_values_that_outgrow_their_scale_beside_a_nan():
    """From the second chunk on the values are a million times larger, and one of them a NaN: its channel is lost, the
    others of its tile are those of the clean call."""
    rng = np.random.default_rng(1640)
    x = I.random_delta_inputs(rng, 1, 200, 1, 2, 64, 32)
    x["v"][:, :64] = I.round_to_bf16((x["v"][:, :64] * 1e-6).astype(np.float32))
    x["v"][0, 70, 1, 5] = 0.25
    say("delta NaN where the scale changes")
    y0, s0 = run(x, "bf16")
    yo, so = D.delta_fwd(**x)
    M, Ms = D.delta_magnitudes(**x)
    ey, _ = y_off(host(y0), yo, M, "bf16")
    assert ey <= 1 and s_off(host(s0), so, Ms) <= TOL_STATE
    x["v"][0, 70, 1, 5] = np.nan
    y, s = run(x, "bf16")
    assert not torch.isfinite(y[0, 70:, 1, 5]).any() and not torch.isfinite(s[0, 1, 5]).any()
    y[0, 70:, 1, 5], s[0, 1, 5] = y0[0, 70:, 1, 5], s0[0, 1, 5]
    assert torch.equal(y, y0) and torch.equal(s, s0)
