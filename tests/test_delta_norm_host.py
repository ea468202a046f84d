"""Host-side checks of the gated delta rule's and the norms' entry points (no GPU): arguments that must be refused
are refused before any HIP call.  The pointers are made up and never read."""
import pytest
import torch

from selective_state_space_33_amd import ops

F32, BF16 = ops.SSM_DTYPE_F32, ops.SSM_DTYPE_BF16
INVALID, UNSUPPORTED = ops.SSM_ERR_INVALID_ARG, ops.SSM_ERR_UNSUPPORTED


def _delta(**kw):
    a = dict(q=0x1000, k=0x2000, v=0x3000, delta=0x4000, A=0x5000, beta=0x6000, bias=None, h0=None, cu=None, nseq=0,
             y=0x7000, fs=None, batch=1, L=8, H=4, P=64, G=2, N=64, dt=BF16, ws=None, wsb=0)
    a.update(kw)
    return ops.lib().ssm_delta_fwd(a["q"], a["k"], a["v"], a["delta"], a["A"], a["beta"], a["bias"], 1, 1, 1.0,
                                   a["h0"], a["cu"], a["nseq"], a["y"], a["fs"], a["batch"], a["L"], a["H"], a["P"],
                                   a["G"], a["N"], a["dt"], a["ws"], a["wsb"], None)


SHARED = [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(delta=None), INVALID),
    (dict(A=None), INVALID), (dict(beta=None), INVALID), (dict(batch=0), INVALID), (dict(H=0), INVALID),
    (dict(P=-1), INVALID), (dict(G=0), INVALID), (dict(G=3), INVALID), (dict(N=0), INVALID), (dict(dt=4), INVALID),
    (dict(q=0x1008), INVALID), (dict(k=0x2004), INVALID), (dict(v=0x3001), INVALID), (dict(beta=0x6001), INVALID),
    (dict(A=0x5002), INVALID), (dict(y=0x7001), INVALID),
    (dict(N=16), UNSUPPORTED), (dict(N=80), UNSUPPORTED), (dict(N=160), UNSUPPORTED), (dict(N=288), UNSUPPORTED),
    (dict(batch=1 << 20, H=1 << 14), UNSUPPORTED), (dict(P=1 << 21), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,expect", SHARED + [
    (dict(y=None), INVALID), (dict(L=0), INVALID), (dict(h0=0x8008), INVALID), (dict(fs=0x8004), INVALID),
    (dict(cu=0x9004, nseq=2), INVALID), (dict(cu=0x9000, nseq=0), INVALID), (dict(cu=0x9000, nseq=2, batch=2), INVALID),
    (dict(nseq=2), INVALID),
])
def test_delta_fwd_refuses(kw, expect):
    assert _delta(**kw) == expect


@pytest.mark.parametrize("kw,expect", SHARED + [(dict(state=None), INVALID), (dict(state=0x8008), INVALID),
                                                (dict(y=None), INVALID)])
def test_delta_update_refuses(kw, expect):
    a = dict(q=0x1000, k=0x2000, v=0x3000, delta=0x4000, A=0x5000, beta=0x6000, bias=None, state=0x8000, y=0x7000,
             batch=1, H=4, P=64, G=2, N=64, dt=BF16)
    a.update(kw)
    assert ops.lib().ssm_delta_update(a["state"], a["q"], a["k"], a["v"], a["delta"], a["A"], a["beta"], a["bias"], 1,
                                      1, 1.0, a["y"], a["batch"], a["H"], a["P"], a["G"], a["N"], a["dt"],
                                      None) == expect


GATED = [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(rows=0), INVALID), (dict(dim=0), INVALID),
    (dict(group=0), INVALID), (dict(group=48), INVALID), (dict(dt=3), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(x=0x1001), INVALID),
    (dict(z=0x2001), INVALID), (dict(w=0x3002), INVALID), (dict(dim=8200, group=8200), UNSUPPORTED),
    (dict(rows=1 << 32), UNSUPPORTED),
]


def _gated(bwd, **kw):
    a = dict(x=0x1000, z=0x2000, w=0x3000, eps=1e-5, y=0x4000, dy=0x5000, dx=0x6000, dz=0x7000, dw=0x8000, rows=4,
             dim=128, group=64, dt=BF16, ws=0x100000, wsb=1 << 30)
    a.update(kw)
    L = ops.lib()
    if bwd:
        return L.ssm_gated_norm_bwd(a["x"], a["z"], a["w"], 0, 0, a["eps"], a["dy"], a["dx"], a["dz"], a["dw"],
                                    a["rows"], a["dim"], a["group"], a["dt"], a["ws"], a["wsb"], None)
    return L.ssm_gated_norm_fwd(a["x"], a["z"], a["w"], 0, 0, a["eps"], a["y"], a["rows"], a["dim"], a["group"],
                                a["dt"], None)


@pytest.mark.parametrize("kw,expect", GATED + [(dict(y=None), INVALID), (dict(y=0x4001), INVALID)])
def test_gated_norm_fwd_refuses(kw, expect):
    assert _gated(False, **kw) == expect


@pytest.mark.parametrize("kw,expect", GATED + [
    (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(dw=None), INVALID), (dict(dz=0x7001), INVALID),
    (dict(dw=0x8002), INVALID), (dict(ws=None), INVALID), (dict(ws=0x100010), INVALID), (dict(wsb=100), INVALID)])
def test_gated_norm_bwd_refuses(kw, expect):
    assert _gated(True, **kw) == expect


RESIDUAL = [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(rows=-1), INVALID), (dict(dim=0), INVALID),
    (dict(dt=3), INVALID), (dict(rdt=3), INVALID), (dict(eps=-1.0), INVALID), (dict(x=0x1001), INVALID),
    (dict(sc=0x2002), INVALID), (dict(pw=0x2002), INVALID), (dict(w=0x3001), INVALID), (dict(r=0x9002), INVALID),
    (dict(dim=8193), UNSUPPORTED), (dict(dt=F32, rdt=BF16), UNSUPPORTED),
]


def _residual(bwd, **kw):
    a = dict(x=0x1000, r=0x9000, sc=0x2000, pw=None, w=0x3000, eps=1e-5, y=0x4000, ro=0xa000, dy=0x5000, dro=0xb000,
             dx=0x6000, dr=0xc000, dsc=0x7000, dpw=None, dw=0x8000, rows=4, dim=128, dt=BF16, rdt=F32, ws=0x100000,
             wsb=1 << 30)
    a.update(kw)
    L = ops.lib()
    if bwd:
        return L.ssm_residual_norm_bwd(a["x"], a["r"], a["sc"], a["pw"], a["w"], a["eps"], a["dy"], a["dro"], a["dx"],
                                       a["dr"], a["dsc"], a["dpw"], a["dw"], a["rows"], a["dim"], a["dt"], a["rdt"],
                                       a["ws"], a["wsb"], None)
    return L.ssm_residual_norm_fwd(a["x"], a["r"], a["sc"], a["pw"], a["w"], a["eps"], a["y"], a["ro"], a["rows"],
                                   a["dim"], a["dt"], a["rdt"], None)


@pytest.mark.parametrize("kw,expect", RESIDUAL + [(dict(y=None), INVALID), (dict(ro=None), INVALID),
                                                  (dict(ro=0xa002), INVALID)])
def test_residual_norm_fwd_refuses(kw, expect):
    assert _residual(False, **kw) == expect


@pytest.mark.parametrize("kw,expect", RESIDUAL + [
    (dict(r=None), INVALID), (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(dw=None), INVALID),
    (dict(dro=0xb002), INVALID), (dict(dr=0xc001), INVALID), (dict(ws=None), INVALID), (dict(ws=0x100080), INVALID),
    (dict(wsb=300), INVALID)])
def test_residual_norm_bwd_refuses(kw, expect):
    assert _residual(True, **kw) == expect


def test_workspace_sizes():
    L = ops.lib()
    assert L.ssm_gated_norm_bwd_workspace_size(1000, 256, 64, BF16) % 256 == 0
    assert L.ssm_gated_norm_bwd_workspace_size(1000, 256, 64, BF16) >= 256 + 256 * 4
    assert L.ssm_gated_norm_bwd_workspace_size(1000, 256, 60, BF16) == 0
    assert L.ssm_gated_norm_bwd_workspace_size(0, 256, 64, BF16) == 0
    assert L.ssm_residual_norm_bwd_workspace_size(1, 100, BF16, F32) >= 256 + 3 * 100 * 4
    assert L.ssm_residual_norm_bwd_workspace_size(1, 100, F32, BF16) == 0
    assert L.ssm_delta_fwd_workspace_size(0, 100, 2, 64, 2, 64, 0, BF16) == 0
    assert L.ssm_delta_fwd_workspace_size(2, 100, 2, 64, 2, 64, 3, BF16) == 0       # packed needs batch 1


def test_binding_checks_tensors():
    """The Python binding names the tensor that does not fit (on the CPU, before the library is asked)."""
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError, match="weight"):
        ops.ssm_gated_norm_fwd(x, None, torch.zeros(8, dtype=torch.float64))
    with pytest.raises(ValueError, match="z has shape"):
        ops.ssm_gated_norm_fwd(x, torch.zeros(4, 7), torch.zeros(8))
    with pytest.raises(ValueError, match="contiguous"):
        ops.ssm_residual_norm_fwd(torch.zeros(8, 4).t(), None, torch.zeros(8))
    with pytest.raises(ValueError, match="k has shape|q has shape"):
        ops.ssm_delta_fwd(torch.zeros(1, 3, 2, 32), torch.zeros(1, 4, 2, 32), torch.zeros(1, 4, 4, 16),
                          torch.zeros(1, 4, 4), torch.zeros(4), torch.zeros(1, 4, 4))


@pytest.mark.parametrize("kw,expect", SHARED + [
    (dict(dy=None), INVALID), (dict(dq=None), INVALID), (dict(dk=None), INVALID), (dict(dv=None), INVALID),
    (dict(dd=None), INVALID), (dict(dA=None), INVALID), (dict(db=None), INVALID), (dict(L=0), INVALID),
    (dict(v=0x3008), INVALID), (dict(dy=0x8008), INVALID), (dict(dv=0xb008), INVALID), (dict(dq=0x9001), INVALID),
    (dict(dA=0xd002), INVALID), (dict(dfs=0xe008), INVALID), (dict(dh0=0xf008), INVALID),
    (dict(dt=F32), UNSUPPORTED), (dict(N=192), UNSUPPORTED), (dict(P=40), UNSUPPORTED),
    (dict(H=1 << 16, P=128), UNSUPPORTED), (dict(cu=0x9000, nseq=2, batch=2), INVALID),
    (dict(ws=None), INVALID), (dict(ws=0x100010), INVALID), (dict(wsb=4096), INVALID),
])
def test_delta_bwd_refuses(kw, expect):
    a = dict(q=0x1000, k=0x2000, v=0x3000, delta=0x4000, A=0x5000, beta=0x6000, bias=None, dy=0x8000, dfs=None,
             h0=None, cu=None, nseq=0, dq=0x9000, dk=0xa000, dv=0xb000, dd=0xc000, dA=0xd000, db=0xe000, dbias=None,
             dh0=None, y=0, batch=1, L=100, H=4, P=64, G=2, N=64, dt=BF16, ws=0x100000, wsb=1 << 40)
    a.update(kw)
    if "y" in kw:       # the shared list's misaligned y is this call's dy
        a["dy"] = kw["y"]
    rc = ops.lib().ssm_delta_bwd(a["q"], a["k"], a["v"], a["delta"], a["A"], a["beta"], a["bias"], 1, 1, 1.0, a["dy"],
                                 a["dfs"], a["h0"], a["cu"], a["nseq"], a["dq"], a["dk"], a["dv"], a["dd"], a["dA"],
                                 a["db"], a["dbias"], a["dh0"], a["batch"], a["L"], a["H"], a["P"], a["G"], a["N"],
                                 a["dt"], a["ws"], a["wsb"], None)
    assert rc == expect
