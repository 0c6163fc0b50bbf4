"""Argument checks of the block operators (gated scan, conv1d gradient, block norm), all before any GPU work (CPU)."""
import pytest
import torch

from tests.test_abi_cpu import P, _lib

Q = P + 0x10000000   # outputs lie away from the inputs


def gated_fwd(lib, **kw):
    a = dict(x=P, r=P, i=P, A=P, reset=None, h0=None, y=Q, hf=None, st=None, batch=2, seqlen=5, dim=6, form=0, act=1,
             ws=None, wsb=0)
    a.update(kw)
    return lib.ssm_gated_scan_fwd(*(a[k] for k in ("x", "r", "i", "A", "reset", "h0", "y", "hf", "st", "batch", "seqlen",
                                                   "dim", "form", "act", "ws", "wsb")), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(r=None), 1), (dict(i=None), 1), (dict(A=None), 1), (dict(y=None), 1),
    (dict(batch=-1), 2), (dict(seqlen=-1), 2), (dict(dim=-1), 2), (dict(form=1), 2), (dict(y=P), 2), (dict(y=P + 100), 2),
    (dict(batch=1 << 31, seqlen=1 << 30, dim=16), 2),
    (dict(act=2), 3), (dict(form=2), 4), (dict(dim=1 << 28, batch=1, seqlen=1, y=P + (1 << 40)), 4),
    (dict(x=P + 1), 7), (dict(A=P + 2), 7), (dict(h0=P + 1), 7), (dict(st=P + 2), 7), (dict(y=Q + 2, act=0), 7),
])
def test_gated_fwd_refusals(kw, code):
    lib = _lib()
    assert gated_fwd(lib, **kw) == code
    assert lib.ssm_last_error() != b""


S = Q + 0x1000000   # and one output from the other


@pytest.mark.parametrize("kw", [
    dict(st=Q), dict(st=P), dict(st=S, hf=S), dict(st=S, h0=S), dict(hf=Q), dict(hf=P), dict(hf=Q + 116), dict(h0=Q),
    dict(st=S, hf=S + 44), dict(reset=Q), dict(reset=S, st=S), dict(A=Q), dict(A=S, hf=S),
])
def test_gated_fwd_refuses_buffers_that_share_memory(kw):
    # 2 x 5 x 6: y is 120 bytes, h0, h_final and states (one row of states) 48, A 24, reset 10
    assert gated_fwd(_lib(), **kw) == 2


@pytest.mark.parametrize("kw", [dict(state=P), dict(x=Q + 4), dict(A=Q), dict(A=Q + 0x100000), dict(r=Q + 44), dict(i=Q)])
def test_gated_step_refuses_buffers_that_share_memory(kw):
    assert step(_lib(), **kw) == 2


def gated_bwd(lib, **kw):
    a = dict(x=P, r=P, i=P, A=P, reset=None, h0=None, st=P, dout=P, dhf=None, dx=Q, dr=Q, di=Q, dA=Q, dh0=None, batch=2,
             seqlen=5, dim=6, form=0, act=1, ws=None, wsb=0)
    a.update(kw)
    return lib.ssm_gated_scan_bwd(*(a[k] for k in ("x", "r", "i", "A", "reset", "h0", "st", "dout", "dhf", "dx", "dr", "di",
                                                   "dA", "dh0", "batch", "seqlen", "dim", "form", "act", "ws", "wsb")), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(i=None), 1), (dict(dout=None), 1), (dict(dx=None), 1), (dict(dr=None), 1), (dict(di=None), 1),
    (dict(dA=None), 1), (dict(form=1), 2), (dict(seqlen=-4), 2), (dict(dx=P), 2), (dict(di=P + 50), 2), (dict(act=9), 3),
    (dict(form=-1), 4), (dict(dr=Q + 1), 7), (dict(dhf=P + 2), 7), (dict(ws=Q, wsb=16), 5),
])
def test_gated_bwd_refusals(kw, code):
    lib = _lib()
    assert gated_bwd(lib, **kw) == code
    assert lib.ssm_last_error() != b""


def step(lib, **kw):
    a = dict(x=P, r=P, i=P, A=P, state=Q, y=Q + 0x100000, batch=3, dim=4, form=0, act=1)
    a.update(kw)
    return lib.ssm_gated_state_update(*(a[k] for k in ("x", "r", "i", "A", "state", "y", "batch", "dim", "form", "act")), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(state=None), 1), (dict(y=None), 1), (dict(A=None), 1), (dict(form=1), 2), (dict(batch=-1), 2),
    (dict(y=Q), 2), (dict(y=Q + 20), 2), (dict(y=P), 2), (dict(act=7), 3), (dict(form=5), 4), (dict(state=Q + 2), 7),
])
def test_gated_step_refusals(kw, code):
    assert step(_lib(), **kw) == code


def conv_bwd(lib, **kw):
    a = dict(x=P, w=P, bias=P, si=None, silu=1, dout=P, dso=None, dx=Q, dw=Q, db=Q, dsi=None, batch=2, seqlen=5, dim=6,
             width=4, act=1, ws=None, wsb=0)
    a.update(kw)
    return lib.ssm_causal_conv1d_bwd(*(a[k] for k in ("x", "w", "bias", "si", "silu", "dout", "dso", "dx", "dw", "db", "dsi",
                                                      "batch", "seqlen", "dim", "width", "act", "ws", "wsb")), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(dout=None), 1), (dict(dx=None), 1), (dict(dw=None), 1), (dict(db=None), 1),
    (dict(width=0), 2), (dict(silu=2), 2), (dict(dim=-1), 2), (dict(dx=P), 2), (dict(dsi=Q + 4096, dso=Q + 4100), 2),
    (dict(act=3), 3), (dict(width=9), 4), (dict(x=P + 1), 7), (dict(dw=Q + 2), 7), (dict(ws=Q, wsb=1), 5),
])
def test_conv_bwd_refusals(kw, code):
    assert conv_bwd(_lib(), **kw) == code


def norm_fwd(lib, **kw):
    a = dict(y=P, z=P, res=P, wpost=P, scale=P, wpre=P, rng=P, p=0.1, eps=1e-5, ro=Q, out=Q + 0x100000, rows=3, dim=8, act=1,
             rdt=0)
    a.update(kw)
    return lib.ssm_block_norm_fwd(*(a[k] for k in ("y", "z", "res", "wpost", "scale", "wpre", "rng", "p", "eps", "ro", "out",
                                                   "rows", "dim", "act", "rdt")), None)


@pytest.mark.parametrize("kw,code", [
    (dict(y=None), 1), (dict(rng=None), 1), (dict(out=None), 1), (dict(wpre=None), 1), (dict(ro=None, wpre=None, out=None), 1),
    (dict(rows=-1), 2), (dict(p=1.0), 2), (dict(p=-0.1), 2), (dict(p=float("nan")), 2), (dict(eps=0.0), 2),
    (dict(eps=float("nan")), 2), (dict(eps=float("inf")), 2), (dict(ro=P + 4), 2), (dict(out=P), 2), (dict(out=Q), 2),
    (dict(act=2), 3), (dict(rdt=2), 3), (dict(dim=16385), 4), (dict(p=0.999999), 4), (dict(rng=P + 4), 7),
    (dict(wpost=P + 2), 7), (dict(res=P + 2), 7),
])
def test_norm_fwd_refusals(kw, code):
    lib = _lib()
    assert norm_fwd(lib, **kw) == code
    assert lib.ssm_last_error() != b""


def norm_bwd(lib, **kw):
    a = dict(y=P, z=P, res=P, wpost=P, scale=P, wpre=P, rng=P, p=0.1, eps=1e-5, dres=P, dout=P, dy=Q, dz=Q, dr=Q, dwpost=Q,
             dscale=Q, dwpre=Q, rows=3, dim=8, act=1, rdt=0, ws=None, wsb=0)
    a.update(kw)
    return lib.ssm_block_norm_bwd(*(a[k] for k in ("y", "z", "res", "wpost", "scale", "wpre", "rng", "p", "eps", "dres", "dout",
                                                   "dy", "dz", "dr", "dwpost", "dscale", "dwpre", "rows", "dim", "act", "rdt",
                                                   "ws", "wsb")), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), 1), (dict(dz=None), 1), (dict(dr=None), 1), (dict(dwpost=None), 1), (dict(dscale=None), 1),
    (dict(dwpre=None), 1), (dict(dout=None), 1), (dict(wpre=None), 1), (dict(dres=None, dout=None, wpre=None), 1),
    (dict(dy=P), 2), (dict(dr=P + 32), 2), (dict(p=2.0), 2), (dict(rdt=5), 3), (dict(dim=20000), 4), (dict(dz=Q + 1), 7),
    (dict(ws=Q, wsb=8), 5),
])
def test_norm_bwd_refusals(kw, code):
    assert norm_bwd(_lib(), **kw) == code


def test_empty_calls_are_noops():
    lib = _lib()
    assert gated_fwd(lib, batch=0, x=None, r=None, i=None, y=None) == 0
    assert gated_fwd(lib, dim=0, x=None, r=None, i=None, y=None, A=None) == 0
    assert gated_bwd(lib, dim=0) == 0
    assert step(lib, batch=0) == 0
    assert conv_bwd(lib, dim=0) == 0
    assert norm_fwd(lib, rows=0) == 0
    assert norm_bwd(lib, dim=0) == 0


def test_workspace_queries_of_empty_and_unsupported_sizes():
    lib = _lib()
    assert lib.ssm_gated_scan_workspace_bytes(0, 5, 5, 1) == 0 == lib.ssm_gated_scan_workspace_bytes(1, 0, 5, 1)
    assert lib.ssm_gated_scan_states_bytes(3, 129, 10) == 3 * 3 * 10 * 4
    assert lib.ssm_gated_scan_bwd_workspace_bytes(3, 129, 10, 1, 0) == lib.ssm_gated_scan_bwd_workspace_bytes(3, 129, 10, 1, 1) + 360
    assert lib.ssm_causal_conv1d_bwd_workspace_bytes(1, 5, 5, 9) == 0
    assert lib.ssm_block_norm_bwd_workspace_bytes(5, 16385) == 0 == lib.ssm_block_norm_bwd_workspace_bytes(0, 5)
    # few rows of few channels: a long sequence is split into chunks that run in parallel, a short one is not
    assert lib.ssm_gated_scan_workspace_bytes(1, 100000, 64, 1) > 0
    assert lib.ssm_gated_scan_workspace_bytes(1, 100, 64, 1) == 0


def test_binding_refuses_before_the_library():
    import selective_state_space_58_amd as ssm
    x = torch.zeros(2, 3, 4)
    for call in (lambda: ssm.ssm_gated_scan_fwd(x, x), lambda: ssm.ssm_gated_scan_bwd(x, x, x),
                 lambda: ssm.ssm_gated_scan_fwd_train(x, x), lambda: ssm.ssm_gated_state_update(x[0], x[0], x[0]),
                 lambda: ssm.ssm_causal_conv1d_bwd(x, x[0], x), lambda: ssm.ssm_block_norm_fwd(x),
                 lambda: ssm.ssm_block_norm_bwd(x, x)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(TypeError, match="torch.Tensor"):
        ssm.ssm_gated_scan_fwd([1.0], x)
