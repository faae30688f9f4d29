"""What a call leaves behind when copies do not land, without a fault: one
tile's barrier is made to expect bytes that nothing copies, its bounded wait runs
out, and every output is then either the call's value or as it was."""
import ctypes

import pytest
import torch

import gated_delta_rule_37_gb300 as gdr
from tests.gpu_util import Guarded, bits_equal, sentinel_like

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdr.load()
    assert gdr.device_status() == 0, "error word not clean before the test"


def ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def status():
    torch.cuda.synchronize()
    w = ctypes.c_int(0)
    code = gdr.load().gdr_get_device_status(None, ctypes.byref(w))
    assert code in (0, 5)
    return w.value


# one row of tiles; a cluster of rows; rows that look back, few and many of them
@pytest.mark.parametrize("T,D,lost", [(100, 64, 0), (100, 65, 0), (900, 64, 0), (900, 64, 1), (1100, 65, 3),
                                      (900, 65, 5), (4000, 64, 2), (4000, 65, 0), (60000, 72, 100), (40000, 129, 30)])
def test_scan(T, D, lost):
    r = torch.Generator().manual_seed(T + D)
    x, g = torch.randn(T, D, generator=r).to(DEV), (-torch.rand(T, D, generator=r)).to(DEV)
    cu = torch.tensor([0, T // 3, T // 3, T], dtype=torch.int32, device=DEV)
    want, last = gdr.linrec_fwd(x, g, cu)
    y, hT = (Guarded(s, F, DEV, fill_bytes=sentinel_like(s, F)) for s in ((T, D), (3, D)))
    n = gdr.linrec_workspace_size(3, T, D, dtype=gdr.GDR_F32, gate_dtype=gdr.GDR_F32)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    assert gdr.load().gdr_selftest_linrec_lost_copy(ptr(x), ptr(g), ptr(cu), 3, T, D, lost, ptr(y.view), ptr(hT.view),
                                                    ptr(ws), n, None) == 0
    assert status() == 0x200 and y.guards_intact() and hT.guards_intact()
    tokens = 320 if D % 8 == 0 else 160
    for got, right in ((y.view, want), (hT.view, last)):
        bits, blank = got.view(torch.int32), sentinel_like((1,), F).view(torch.int32).to(DEV)
        assert ((bits == blank) | (bits == right.view(torch.int32))).all(), "neither the call's value nor untouched"
    blank = y.view.view(torch.int32) == sentinel_like((1,), F).view(torch.int32).to(DEV)
    assert blank[lost * tokens:(lost + 1) * tokens].all(), "the tile that lost its copies"
    assert status() == 0
    assert all(bits_equal(a, b) for a, b in zip(gdr.linrec_fwd(x, g, cu), (want, last)))   # the context is intact
    assert status() == 0


# one to eight rows at a time in a CTA; the first row of a CTA and later ones, the last of all
@pytest.mark.parametrize("M,D,lost", [(1, 4096, 0), (5, 512, 3), (3000, 4096, 0), (3000, 4096, 2999), (6000, 512, 2500),
                                      (4000, 1024, 1300), (2000, 2048, 700)])
def test_norm_backward(M, D, lost):
    r = torch.Generator().manual_seed(M + D)
    dy, s = (torch.randn(M, D, generator=r).to(BF).to(DEV) for _ in range(2))
    w = torch.randn(D, generator=r).to(DEV)
    want, dw = gdr.rmsnorm_bwd(dy, s, w)
    dx = Guarded((M, D), BF, DEV, fill_bytes=sentinel_like((M, D), BF))
    got_dw = torch.zeros(D, device=DEV)
    n = gdr.rmsnorm_bwd_workspace_size(M, D)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    assert gdr.load().gdr_selftest_rmsnorm_lost_copy(ptr(dy), ptr(s), ptr(w), M, D, lost, ptr(dx.view), ptr(got_dw),
                                                     ptr(ws), n, None) == 0
    assert status() == 0x400 and dx.guards_intact()
    blank = (dx.view.view(torch.int16) == sentinel_like((1,), BF).view(torch.int16).to(DEV)).all(1)
    right = (dx.view.view(torch.int16) == want.view(torch.int16)).all(1)
    assert blank[lost] and (blank | right).all(), "neither the call's rows nor untouched"
    assert torch.isnan(got_dw).all()
    assert all(bits_equal(a, b) for a, b in zip(gdr.rmsnorm_bwd(dy, s, w), (want, dw)))
    assert status() == 0
