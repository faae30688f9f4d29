"""Host-side checks of the attention layer's entry points: refusals before any launch, empty calls, workspace
sizes (no GPU needed)."""
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


def _append(lib, **kw):
    a = dict(q=P(16), ldq=512, k=P(32), ldk=128, v=P(48), ldv=128, f=P(64), R=64, lens=P(80), table=P(96), ldt=4, mp=4,
             cu=P(112), N=2, T=4, Hq=8, Hkv=2, D=64, dtype=BF16, flags=0, qo=P(128), ldqo=512, ko=P(144), ldko=128,
             kc=P(160), vc=P(176), pages=9, ps=16)
    a.update(kw)
    return lib.gdr_kv_append(a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"], a["f"], a["R"], a["lens"],
                             a["table"], a["ldt"], a["mp"], a["cu"], a["N"], a["T"], a["Hq"], a["Hkv"], a["D"],
                             a["dtype"], a["flags"], a["qo"], a["ldqo"], a["ko"], a["ldko"], a["kc"], a["vc"],
                             a["pages"], a["ps"], None)


HEADS = [
    (dict(N=-1), INVALID), (dict(T=-1), INVALID), (dict(N=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=7), INVALID),
    (dict(Hq=-8), INVALID), (dict(Hq=258), UNSUPPORTED), (dict(Hq=65538), UNSUPPORTED), (dict(D=96), UNSUPPORTED),
    (dict(dtype=E4M3), UNSUPPORTED), (dict(N=65536), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED),
    (dict(cu=None), INVALID), (dict(cu=P(113)), INVALID), (dict(flags=0x80), INVALID),
    (dict(q=None), INVALID), (dict(q=P(18)), INVALID), (dict(ldq=4), INVALID), (dict(ldq=-512), INVALID),
]

PAGED = [
    (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(kc=P(168)), INVALID), (dict(vc=P(168)), INVALID),
    (dict(table=None), INVALID), (dict(table=P(98)), INVALID), (dict(ldt=3), INVALID), (dict(mp=0), INVALID),
    (dict(lens=None), INVALID), (dict(lens=P(81)), INVALID), (dict(pages=0), INVALID), (dict(ps=8), UNSUPPORTED),
    (dict(ps=48), UNSUPPORTED), (dict(ps=512), UNSUPPORTED), (dict(pages=1 << 30), UNSUPPORTED),
    (dict(mp=1 << 27, ldt=1 << 27), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", HEADS + PAGED + [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=P(40)), INVALID), (dict(ldv=12), INVALID),
    (dict(qo=None), INVALID), (dict(Hq=0), INVALID), (dict(ldqo=504), INVALID), (dict(ldko=120), INVALID),
    (dict(R=-16), INVALID), (dict(R=80), INVALID), (dict(R=24), INVALID), (dict(f=None), INVALID),
    (dict(R=3, flags=gdr.GDR_ROPE_PAIRS), INVALID), (dict(f=P(66)), INVALID),
    (dict(qo=P(16), ldqo=520), INVALID), (dict(ko=P(32), ldko=136), INVALID),
])
def test_append_rejects_before_launch(lib, kw, code):
    assert _append(lib, **kw) == code
    assert lib.gdr_last_error().decode()


def _fwd(lib, **kw):
    a = dict(q=P(16), ldq=512, k=P(32), ldk=128, v=P(48), ldv=128, cu=P(112), N=2, T=4, Hq=8, Hkv=2, D=64, scale=0.1,
             dtype=BF16, flags=0, o=P(128), ldo=512)
    a.update(kw)
    return lib.gdr_attn_fwd(a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"], a["cu"], a["N"], a["T"], a["Hq"],
                            a["Hkv"], a["D"], a["scale"], a["dtype"], a["flags"], a["o"], a["ldo"], None)


@pytest.mark.parametrize("kw,code", HEADS + [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(o=None), INVALID), (dict(o=P(130)), INVALID),
    (dict(ldo=504), INVALID), (dict(ldo=516), INVALID), (dict(o=P(16)), INVALID), (dict(o=P(48)), INVALID),
    (dict(Hq=0), INVALID), (dict(flags=gdr.GDR_ROPE_PAIRS), INVALID), (dict(ldk=1 << 32), INVALID),
    (dict(T=(1 << 28), Hq=8), UNSUPPORTED), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
])
def test_fwd_rejects_before_launch(lib, kw, code):
    assert _fwd(lib, **kw) == code
    assert lib.gdr_last_error().decode()


def _step(lib, **kw):
    a = dict(q=P(16), ldq=512, kc=P(160), vc=P(176), pages=9, ps=16, table=P(96), ldt=4, mp=4, lens=P(80), pp=P(192),
             pl=20, cu=P(112), N=2, T=4, Hq=8, Hkv=2, D=64, scale=0.1, dtype=BF16, flags=0, o=P(128), ldo=512,
             ws=P(256), wn=1 << 40)
    a.update(kw)
    return lib.gdr_attn_step(a["q"], a["ldq"], a["kc"], a["vc"], a["pages"], a["ps"], a["table"], a["ldt"], a["mp"],
                             a["lens"], a["pp"], a["pl"], a["cu"], a["N"], a["T"], a["Hq"], a["Hkv"], a["D"],
                             a["scale"], a["dtype"], a["flags"], a["o"], a["ldo"], a["ws"], a["wn"], None)


@pytest.mark.parametrize("kw,code", HEADS + PAGED + [
    (dict(o=None), INVALID), (dict(o=P(16)), INVALID), (dict(ldo=504), INVALID), (dict(pl=-1), INVALID),
    (dict(pl=0), INVALID), (dict(pp=None), INVALID), (dict(pp=P(193)), INVALID), (dict(ws=None), WORKSPACE),
    (dict(wn=16), WORKSPACE), (dict(ws=P(128)), INVALID), (dict(Hq=0), INVALID), (dict(flags=gdr.GDR_COMMIT), INVALID),
    (dict(scale=0.0), INVALID),
])
def test_step_rejects_before_launch(lib, kw, code):
    assert _step(lib, **kw) == code
    assert lib.gdr_last_error().decode()


def test_empty_is_ok(lib):
    for call in (_append, _fwd, _step):
        assert call(lib, T=0) == 0
        assert call(lib, N=0, T=0) == 0


def test_step_workspace(lib):
    def size(N, T, Hq=8, Hkv=2, D=128, prefix_len=0, dtype=BF16):
        return gdr.attn_step_workspace_size(N, T, Hq, Hkv, D, prefix_len=prefix_len, dtype=dtype)

    assert size(0, 0) == size(3, 0) == 0
    n = size(4, 4)
    assert n > 0 and n % 256 == 0
    assert size(4, 4, prefix_len=100) > n
    assert _step(lib, wn=size(2, 4, D=64, prefix_len=20) - 1) == WORKSPACE
    assert lib.gdr_attn_step_workspace_size(1, 1, 8, 2, 64, 0, BF16, None) == INVALID
    for bad in (dict(Hq=3), dict(D=80), dict(dtype=E4M3), dict(prefix_len=-1)):
        with pytest.raises(gdr.GdrError):
            size(4, 4, **bad)


def test_binding_refuses_cpu_tensors():
    x, cu = torch.zeros(2, 1, 64), torch.tensor([0, 2], dtype=torch.int32)
    cache = torch.zeros(1, 1, 16, 64)
    with pytest.raises(ValueError):
        gdr.attn_fwd(x, x, x, cu)
    with pytest.raises(ValueError):
        gdr.attn_step(x, cache, cache, cu[None], cu[:1], cu)
    with pytest.raises(ValueError):
        gdr.kv_append(x, x, cache, cache, cu[None], cu[:1], cu)
