"""Host-side checks of the gated linear recurrence's and the RMS norm's entry
points: sizes, refusals before any launch, empty calls (no GPU needed)."""
import ctypes

import pytest
import torch

import gated_delta_rule_37_gb300 as gdr
from gated_delta_rule_37_gb300 import build as gbuild

P = ctypes.c_void_p
BF16, F32, E4M3 = gdr.GDR_BF16, gdr.GDR_F32, gdr.GDR_E4M3
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdr.load()


def _fwd(lib, **kw):
    a = dict(x=P(16), ldx=64, g=P(32), ldg=64, h0=None, cu=P(48), N=1, T=8, D=64, dtype=BF16, gate=F32, flags=0,
             y=P(64), ldy=64, hT=None, ws=P(256), wn=1 << 40)
    a.update(kw)
    return lib.gdr_linrec_fwd(a["x"], a["ldx"], a["g"], a["ldg"], a["h0"], a["cu"], a["N"], a["T"], a["D"],
                              a["dtype"], a["gate"], a["flags"], a["y"], a["ldy"], a["hT"], a["ws"], a["wn"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INVALID), (dict(g=None), INVALID), (dict(y=None), INVALID), (dict(cu=None), INVALID),
    (dict(x=P(17)), INVALID),                              # bf16 at an odd address
    (dict(g=P(34)), INVALID),                              # fp32 off its 4 bytes
    (dict(ldx=-64), INVALID), (dict(ldy=63), INVALID),
    (dict(h0=P(20)), INVALID), (dict(hT=P(20)), INVALID), (dict(cu=P(50)), INVALID),
    (dict(D=(1 << 24) + 1, ldx=1 << 25, ldg=1 << 25, ldy=1 << 25), UNSUPPORTED),
    (dict(D=0), INVALID), (dict(N=-1), INVALID), (dict(T=-1), INVALID), (dict(N=0), INVALID),
    (dict(dtype=E4M3), UNSUPPORTED), (dict(gate=7), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED),
    (dict(T=(1 << 31) - 511), UNSUPPORTED), (dict(T=(1 << 31) - 512, wn=16), WORKSPACE),
    (dict(flags=gdr.GDR_COMMIT), INVALID), (dict(flags=0x40), INVALID),
    (dict(h0=P(512), hT=P(512)), INVALID), (dict(h0=P(512), hT=P(512), T=0), INVALID),   # the state in place
])
def test_linrec_fwd_rejects_before_launch(lib, kw, code):
    assert _fwd(lib, **kw) == code
    assert lib.gdr_last_error().decode()


def test_linrec_workspace(lib):
    with pytest.raises(gdr.GdrError):
        gdr.linrec_workspace_size(1, 8, 0, dtype=BF16, gate_dtype=F32)
    with pytest.raises(gdr.GdrError):
        gdr.linrec_workspace_size(1, 8, 8, dtype=E4M3, gate_dtype=F32)
    assert lib.gdr_linrec_workspace_size(1, 8, 8, BF16, F32, None) == INVALID
    need = gdr.linrec_workspace_size(1, 1 << 20, 4096, dtype=BF16, gate_dtype=F32)
    assert need % 256 == 0
    if need:
        assert _fwd(lib, T=1 << 20, D=4096, ldx=4096, ldg=4096, ldy=4096, wn=need - 1) == WORKSPACE
        assert _fwd(lib, T=1 << 20, D=4096, ldx=4096, ldg=4096, ldy=4096, ws=None) == WORKSPACE
        assert _fwd(lib, T=1 << 20, D=4096, ldx=4096, ldg=4096, ldy=4096, ws=P(128)) == INVALID


def test_linrec_fwd_empty_is_ok(lib):
    assert _fwd(lib, N=0, T=0) == 0
    assert _fwd(lib, N=3, T=0) == 0                        # no final state wanted: nothing to do


def _bwd(lib, **kw):
    a = dict(dy=P(16), ldd=64, g=P(32), ldg=64, y=P(48), ldy=64, h0=None, df=None, cu=P(64), N=1, T=8, D=64,
             dtype=BF16, gate=F32, flags=0, dx=P(80), ldx=64, dg=P(96), lddg=64, d0=None, ws=P(256), wn=1 << 40)
    a.update(kw)
    return lib.gdr_linrec_bwd(a["dy"], a["ldd"], a["g"], a["ldg"], a["y"], a["ldy"], a["h0"], a["df"], a["cu"],
                              a["N"], a["T"], a["D"], a["dtype"], a["gate"], a["flags"], a["dx"], a["ldx"], a["dg"],
                              a["lddg"], a["d0"], a["ws"], a["wn"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), INVALID), (dict(g=None), INVALID), (dict(y=None), INVALID), (dict(dx=None), INVALID),
    (dict(dg=None), INVALID), (dict(cu=None), INVALID), (dict(y=P(49)), INVALID), (dict(dg=P(98)), INVALID),
    (dict(ldx=8), INVALID), (dict(lddg=8), INVALID), (dict(df=P(8)), INVALID), (dict(d0=P(8)), INVALID),
    (dict(h0=P(8)), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(flags=4), INVALID), (dict(N=0), INVALID),
    (dict(df=P(512), d0=P(512)), INVALID), (dict(h0=P(512), d0=P(512)), INVALID),        # the state in place
])
def test_linrec_bwd_rejects_before_launch(lib, kw, code):
    assert _bwd(lib, **kw) == code
    assert lib.gdr_last_error().decode()


def _step(lib, **kw):
    a = dict(x=P(16), ldx=64, g=P(32), ldg=64, pool=P(48), pt=F32, slots=8, idx=P(64), cu=P(80), N=4, T=4, D=64,
             dtype=BF16, gate=F32, flags=gdr.GDR_COMMIT, y=P(96), ldy=64, ib=None, steps=0)
    a.update(kw)
    return lib.gdr_linrec_step(a["x"], a["ldx"], a["g"], a["ldg"], a["pool"], a["pt"], a["slots"], a["idx"], a["cu"],
                               a["N"], a["T"], a["D"], a["dtype"], a["gate"], a["flags"], a["y"], a["ldy"], a["ib"],
                               a["steps"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INVALID), (dict(pool=None), INVALID), (dict(idx=None), INVALID), (dict(cu=None), INVALID),
    (dict(y=None), INVALID), (dict(pool=P(50)), INVALID), (dict(ib=P(112)), INVALID),
    (dict(ib=P(113), steps=2), INVALID), (dict(idx=P(66)), INVALID), (dict(slots=0), INVALID), (dict(pt=2), UNSUPPORTED),
    (dict(flags=gdr.GDR_QK_L2NORM), INVALID), (dict(ldy=1), INVALID), (dict(D=-1), INVALID),
])
def test_linrec_step_rejects_before_launch(lib, kw, code):
    assert _step(lib, **kw) == code
    assert lib.gdr_last_error().decode()


def test_linrec_step_empty_is_ok(lib):
    assert _step(lib, N=0, T=0) == 0
    assert _step(lib, T=0) == 0


def _norm(lib, **kw):
    a = dict(x=P(16), ldx=64, r=P(32), ldr=64, w=P(48), M=4, D=64, eps=1e-6, dtype=BF16, ro=P(64), ldo=64, y=P(80),
             ldy=64, yt=BF16, sc=None, group=0)
    a.update(kw)
    return lib.gdr_rmsnorm_fwd(a["x"], a["ldx"], a["r"], a["ldr"], a["w"], a["M"], a["D"], a["eps"], a["dtype"],
                               a["ro"], a["ldo"], a["y"], a["ldy"], a["yt"], a["sc"], a["group"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID),
    (dict(r=None), INVALID), (dict(ro=None), INVALID),     # residual and residual_out go together
    (dict(x=P(17)), INVALID), (dict(w=P(52)), INVALID), (dict(ldo=63), INVALID), (dict(ldr=-1), INVALID),
    (dict(M=-1), INVALID), (dict(D=0), INVALID), (dict(D=32769, ldo=1 << 20, ldy=1 << 20), UNSUPPORTED),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(dtype=E4M3), UNSUPPORTED), (dict(yt=F32), UNSUPPORTED), (dict(yt=9), UNSUPPORTED),
    (dict(group=32), INVALID),                             # groups without codes
    (dict(sc=P(96)), INVALID),                             # scales without codes
    (dict(yt=E4M3), INVALID),                              # codes without scales
    (dict(yt=E4M3, sc=P(96), group=48), INVALID), (dict(yt=E4M3, sc=P(96), group=-1), INVALID),
])
def test_rmsnorm_fwd_rejects_before_launch(lib, kw, code):
    assert _norm(lib, **kw) == code
    assert lib.gdr_last_error().decode()


def test_rmsnorm_empty_is_ok(lib):
    assert _norm(lib, M=0) == 0
    assert _norm_bwd(lib, M=0, dw=None) == 0


def _norm_bwd(lib, **kw):
    a = dict(dy=P(16), ldd=64, s=P(32), lds=64, w=P(48), ds=None, ldds=0, M=4, D=64, eps=1e-6, dtype=BF16, dx=P(64),
             ldx=64, dw=P(80), ws=P(256), wn=1 << 40)
    a.update(kw)
    return lib.gdr_rmsnorm_bwd(a["dy"], a["ldd"], a["s"], a["lds"], a["w"], a["ds"], a["ldds"], a["M"], a["D"],
                               a["eps"], a["dtype"], a["dx"], a["ldx"], a["dw"], a["ws"], a["wn"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), INVALID), (dict(s=None), INVALID), (dict(w=None), INVALID), (dict(dx=None), INVALID),
    (dict(ds=P(33), ldds=64), INVALID), (dict(ldx=63), INVALID), (dict(dw=P(84)), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wn=100), WORKSPACE), (dict(ws=P(128)), INVALID),
    (dict(D=32769), UNSUPPORTED), (dict(eps=-0.5), INVALID), (dict(dtype=2), UNSUPPORTED),
])
def test_rmsnorm_bwd_rejects_before_launch(lib, kw, code):
    assert _norm_bwd(lib, **kw) == code
    assert lib.gdr_last_error().decode()


def test_rmsnorm_bwd_workspace(lib):
    assert gdr.rmsnorm_bwd_workspace_size(0, 64) == 0
    n = [gdr.rmsnorm_bwd_workspace_size(M, 1001) for M in (1, 100, 100000)]
    assert n[0] >= 1001 * 4 and sorted(n) == n and all(v % 256 == 0 for v in n)


def test_binding_refuses_cpu_tensors():
    x, w = torch.zeros(2, 8), torch.zeros(8)
    cu = torch.tensor([0, 2], dtype=torch.int32)
    with pytest.raises(ValueError):
        gdr.linrec_fwd(x, x, cu)
    with pytest.raises(ValueError):
        gdr.linrec_bwd(x, x, x, cu)
    with pytest.raises(ValueError):
        gdr.linrec_step(x, x, x, cu, cu)
    with pytest.raises(ValueError):
        gdr.rmsnorm_fwd(x, w)
    with pytest.raises(ValueError):
        gdr.rmsnorm_bwd(x, x, w)
