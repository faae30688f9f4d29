"""GPU parity of the residual RMS norm (types of its own and e4m3, backward)
against the fp64 oracle.

Tolerances, per element.  A row's sum of squares runs over at most 128 terms in
a thread and a tree above: its relative error is below 144 * 2^-24, half of
that in 1 / sqrt, and a few roundings in the products: 80 * 2^-24 of the value
(eps / 2 of the type on top where it is stored).  The backward adds two
products of such factors and a row's dot product: 160 * 2^-24 of the sum of the
terms' magnitudes; dweight adds its rows and the CTAs' parts, at most 400
roundings of the magnitudes' sum.  The residual's addition is exact: one fp32
sum, rounded once.  e4m3: half a step is 2^-4 of the value, 2^-10 below 2^-6.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_37_gb300 as gdr
import oracle
from tests.gpu_util import Guarded, bits_equal, sentinel_like

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24
EPS = 1e-6
WIDTHS = [1, 7, 8, 64, 100, 128, 129, 1000, 1001, 2048, 4096, 5000, 8192, 16384, 32768, 32767]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdr.load()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


def make(seed, M, D, dtype):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=r)  # noqa: E731
    row = torch.exp2(8 * torch.rand(M, 1, generator=r) - 4)
    return dict(x=(n(M, D) * row).to(dtype), r=(2 * n(M, D) * row).to(dtype), w=1 + 0.3 * n(D), dy=n(M, D).to(dtype),
                ds=n(M, D).to(dtype))


def check(got, want, tol, what):
    got = f64(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}, " \
        f"{got[bad][0]} for {want[bad][0]} within {np.broadcast_to(tol, want.shape)[bad][0]}"


def guarded(shape, dtype):
    if dtype == E4:
        return Guarded(shape, dtype, DEV, fill_bytes=torch.full(shape, 0x5A, dtype=torch.uint8))
    return Guarded(shape, dtype, DEV, fill_bytes=sentinel_like(shape, dtype))


def total(c, residual=True):
    return (c["x"].float() + c["r"].float()).to(c["x"].dtype) if residual else c["x"]


def check_codes(codes, scales, y, group, what):
    """codes * scales against y = the exact norm [M, D]."""
    M, D = y.shape
    group = group or D
    groups = -(-D // group)
    assert scales.shape == (M, groups)
    wide = np.zeros((M, groups * group))
    wide[:, :D] = np.abs(y)
    want = np.maximum(wide.reshape(M, groups, group).max(2), 1e-12) / 448
    check(scales, want, 90 * U * want, what + " scales")
    v = y / np.repeat(want, group, 1)[:, :D]
    # the code of a value within 1e-5 of v: half a step away from it at most
    check(codes, v, np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10) + 1e-5 * np.abs(v), what + " codes")


def run_fwd(c, *, residual, y_dtype, group=0):
    M, D = c["x"].shape
    y, ro = guarded((M, D), y_dtype), guarded((M, D), c["x"].dtype)
    sc = guarded((M, -(-D // group) if group else 1), F) if y_dtype == E4 else None
    gdr.rmsnorm_fwd(c["x"].to(DEV), c["w"].to(DEV), residual=c["r"].to(DEV) if residual else None, eps=EPS,
                    y_dtype=y_dtype, scale_group=group, y=y.view, residual_out=ro.view if residual else None,
                    scales=sc.view if sc else None)
    torch.cuda.synchronize()
    assert y.guards_intact() and ro.guards_intact() and (sc is None or sc.guards_intact())
    return y.view.cpu(), ro.view.cpu() if residual else None, sc.view.cpu() if sc else None


def check_fwd(c, y, ro, sc, *, residual, group=0):
    s = total(c, residual)
    if residual:
        assert bits_equal(ro, s), "residual_out"
    want = oracle.rmsnorm(f64(s), c["w"], EPS)
    if y.dtype == E4:
        check_codes(y, sc, want, group, "y")
    else:
        check(y, want, (80 * U + half_step(y.dtype)) * np.abs(want), "y")


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", WIDTHS)
def test_fwd(D, dtype):
    c = make(D, 5 if D > 8192 else 37, D, dtype)
    for residual in (True, False):
        check_fwd(c, *run_fwd(c, residual=residual, y_dtype=dtype), residual=residual)


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", WIDTHS)
def test_fwd_e4m3(D, dtype, group):
    c = make(D + 1, 3 if D > 8192 else 21, D, dtype)
    residual = group != 32
    check_fwd(c, *run_fwd(c, residual=residual, y_dtype=E4, group=group), residual=residual, group=group)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,D", [(1, 128), (3, 1), (700, 8), (5000, 128), (2000, 520), (1500, 1001), (300, 4096),
                                 (40, 16384), (3, 32768), (4, 32767), (33, 8200)])
def test_bwd(M, D, dtype):
    c = make(M + D, M, D, dtype)
    s, dy, w = f64(c["x"]), f64(c["dy"]), f64(c["w"])
    rs, rw = oracle.rmsnorm_bwd(dy, s, w, EPS)
    r = 1 / np.sqrt((s * s).mean(1, keepdims=True) + EPS)
    terms = r * np.abs(w * dy) + r ** 3 * np.abs(s) * np.abs(s * w * dy).mean(1, keepdims=True)
    w_terms = np.abs(r * dy * s).sum(0)
    for ds in (True, False):
        dx, dw = guarded((M, D), dtype), guarded((D,), F)
        gdr.rmsnorm_bwd(c["dy"].to(DEV), c["x"].to(DEV), c["w"].to(DEV), eps=EPS,
                        d_residual_out=c["ds"].to(DEV) if ds else None, dx=dx.view, dweight=dw.view)
        torch.cuda.synchronize()
        assert dx.guards_intact() and dw.guards_intact()
        want = rs + f64(c["ds"]) if ds else rs
        check(dx.view.cpu(), want, 160 * U * terms + (U + half_step(dtype)) * np.abs(want), "dx")
        check(dw.view.cpu(), rw, 400 * U * w_terms, "dweight")
        only, none = gdr.rmsnorm_bwd(c["dy"].to(DEV), c["x"].to(DEV), c["w"].to(DEV), eps=EPS, output_dweight=False,
                                     d_residual_out=c["ds"].to(DEV) if ds else None)
        assert none is None and bits_equal(only, dx.view)


@pytest.mark.parametrize("D", [2080, 2081])
def test_offsets_beyond_32_bits(D):
    """Rows whose elements' numbers pass 2^31: the last ones against 64 bits."""
    M, n = (1 << 20) + 5, 50
    assert (M - n) * D > 1 << 31
    c = make(41, n, D, BF)
    big = {}
    for k in ("x", "r", "dy", "ds"):
        big[k] = torch.zeros(M, D, dtype=BF, device=DEV)
        big[k][M - n:] = c[k].to(DEV)
    w = c["w"].to(DEV)
    for y_dtype, group in ((BF, 0), (E4, 32)):
        y, ro, sc = gdr.rmsnorm_fwd(big["x"], w, residual=big["r"], eps=EPS, y_dtype=y_dtype, scale_group=group)
        check_fwd(c, y[M - n:].cpu(), ro[M - n:].cpu(), sc[M - n:].cpu() if group else None, residual=True, group=group)
        assert not ro[:M - n].any() and not (y[:M - n].view(torch.int8) & 0x7f).any()
        del y, ro, sc
    s, dy = f64(c["x"]), f64(c["dy"])
    rs, rw = oracle.rmsnorm_bwd(dy, s, f64(c["w"]), EPS)
    r = 1 / np.sqrt((s * s).mean(1, keepdims=True) + EPS)
    terms = r * np.abs(f64(c["w"]) * dy) + r ** 3 * np.abs(s) * np.abs(s * f64(c["w"]) * dy).mean(1, keepdims=True)
    dx, dw = gdr.rmsnorm_bwd(big["dy"], big["x"], w, eps=EPS, d_residual_out=big["ds"])
    want = rs + f64(c["ds"])
    check(dx[M - n:].cpu(), want, 160 * U * terms + (U + half_step(BF)) * np.abs(want), "dx")
    check(dw.cpu(), rw, 400 * U * np.abs(r * dy * s).sum(0), "dweight")
    assert not dx[:M - n].any()


@pytest.mark.parametrize("D", [64, 1001, 4096])
def test_gradient_against_differences(D):
    """The kernel's gradient against differences of the kernel's own forward, in fp32."""
    c = make(7, 3, D, F)
    x, w, dy = c["x"].to(DEV), c["w"].to(DEV), c["dy"].to(DEV)
    dx, dw = gdr.rmsnorm_bwd(dy, x, w, eps=EPS)
    r = torch.Generator().manual_seed(1)
    for arg, grad in ((x, dx), (w, dw)):
        way = torch.randn(arg.shape, generator=r).to(DEV) * arg.abs().mean()
        h = 2.0 ** -7
        val = [(dy.double() * gdr.rmsnorm_fwd(*((x + k * way, w) if arg is x else (x, w + k * way)), eps=EPS)[0].double())
               .sum() for k in (h, -h)]
        diff, along = float(val[0] - val[1]) / (2 * h), float((grad.double() * way.double()).sum())
        # third-order term h^2 |way|^3 and fp32 roundings 80 * 2^-24 |y| sqrt(n) / h, both well under 2 % of the
        # magnitude that the terms of the sum add up to
        scale = float((grad.double() * way.double()).abs().sum())
        assert abs(diff - along) <= 0.02 * scale


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_in_place(dtype):
    """residual_out on residual or on x, dx on dy or on d_residual_out."""
    for D in (1001, 4096):
        c = make(40 + D, 50, D, dtype)
        x, r, w, dy, ds = (c[k].to(DEV) for k in ("x", "r", "w", "dy", "ds"))
        y, ro, _ = gdr.rmsnorm_fwd(x, w, residual=r, eps=EPS)
        for into in (1, 0):
            ops = [x.clone(), r.clone()]
            y2, ro2, _ = gdr.rmsnorm_fwd(ops[0], w, residual=ops[1], eps=EPS, residual_out=ops[into])
            assert ro2 is ops[into] and bits_equal(ro2, ro) and bits_equal(y2, y)
        dx, dw = gdr.rmsnorm_bwd(dy, x, w, eps=EPS, d_residual_out=ds)
        for into in (0, 1):
            ops = [dy.clone(), ds.clone()]
            dx2, dw2 = gdr.rmsnorm_bwd(ops[0], x, w, eps=EPS, d_residual_out=ops[1], dx=ops[into])
            assert bits_equal(dx2, dx) and bits_equal(dw2, dw)


@pytest.mark.parametrize("M,D", [(3000, 1024), (2000, 4096), (1, 4096), (700, 512)])
def test_in_place_with_rows_on_their_way(M, D):
    """dx written over dy while later rows are being fetched; rows more than a
    CTA's, and fewer than it can hold."""
    c = make(45, M, D, BF)
    x, w, dy, ds = (c[k].to(DEV) for k in ("x", "w", "dy", "ds"))
    dx, dw = gdr.rmsnorm_bwd(dy, x, w, eps=EPS, d_residual_out=ds)
    for into in (0, 1):
        ops = [dy.clone(), ds.clone()]
        dx2, dw2 = gdr.rmsnorm_bwd(ops[0], x, w, eps=EPS, d_residual_out=ops[1], dx=ops[into])
        assert bits_equal(dx2, dx) and bits_equal(dw2, dw)


def test_in_place_with_another_stride_is_refused():
    wide = torch.randn(6, 32, device=DEV)
    x, w = torch.randn(6, 8, device=DEV), torch.ones(8, device=DEV)
    flat = wide.view(-1)[:48].view(6, 8)                   # the same address, rows 8 apart instead of 32
    with pytest.raises(gdr.GdrError, match="stride"):
        gdr.rmsnorm_fwd(x, w, residual=wide[:, :8], residual_out=flat)
    with pytest.raises(gdr.GdrError, match="stride"):
        gdr.rmsnorm_bwd(wide[:, :8], x, w, dx=flat)


def test_strides_and_alignment():
    for off, width, D in ((0, 256, 128), (128, 256, 128), (3, 200, 128), (1, 140, 131)):
        c = make(50 + off, 90, D, BF)
        wide = torch.full((90, 7 * width), float("nan"), dtype=BF, device=DEV)
        cut = [wide[:, i * width + off:i * width + off + D] for i in range(7)]
        for t, k in zip(cut, ("x", "r", "dy", "ds")):
            t.copy_(c[k])
        w = c["w"].to(DEV)
        y, ro, _ = gdr.rmsnorm_fwd(cut[0], w, residual=cut[1], eps=EPS, y=cut[4], residual_out=cut[5])
        check_fwd(c, y.cpu(), ro.cpu(), None, residual=True)
        dx, dw = gdr.rmsnorm_bwd(cut[2], cut[0], w, eps=EPS, d_residual_out=cut[3], dx=cut[6])
        plain, dw0 = gdr.rmsnorm_bwd(c["dy"].to(DEV), c["x"].to(DEV), w, eps=EPS, d_residual_out=c["ds"].to(DEV))
        assert (dx.float() - plain.float()).abs().max() <= 2.0 ** -7 * plain.float().abs().max()
        assert (dw - dw0).abs().max() <= 400 * U * dw0.abs().max() * 90
        other = torch.ones_like(wide, dtype=torch.bool)
        for i in range(7):
            other[:, i * width + off:i * width + off + D] = False
        assert torch.isnan(wide[other]).all(), "written outside the column blocks"
        # codes at any byte offset
        raw = torch.full((90, width + D), 0x5A, dtype=torch.uint8, device=DEV)
        codes = raw[:, off:off + D].view(E4)
        q, _, sc = gdr.rmsnorm_fwd(cut[0], w, eps=EPS, y_dtype=E4, scale_group=64, y=codes)
        check_codes(q.cpu(), sc.cpu(), oracle.rmsnorm(f64(c["x"]), w, EPS), 64, "strided")
        assert (raw[:, :off] == 0x5A).all() and (raw[:, off + D:] == 0x5A).all()
    # one row for every row
    x = torch.randn(1, 256, device=DEV)
    y, _, _ = gdr.rmsnorm_fwd(x.expand(9, 256), torch.ones(256, device=DEV))
    assert all(bits_equal(y[i], y[0]) for i in range(9))


def test_zeros_and_bad_values():
    """Rows of zeros have codes of 0 and a scale; what is not finite stays in its row."""
    c = make(60, 6, 256, F)
    c["x"][1] = 0
    c["x"][2, 7] = np.nan
    c["x"][3, 9] = np.inf
    x, w = c["x"].to(DEV), c["w"].to(DEV)
    want = oracle.rmsnorm(f64(c["x"][[0, 4, 5]]), w, EPS)
    for dt in (None, E4):
        y, _, sc = gdr.rmsnorm_fwd(x, w, eps=EPS, y_dtype=dt, scale_group=64 if dt else 0)
        y = y.float().cpu()
        assert (y[1] == 0).all() and torch.isnan(y[2]).all() and torch.isnan(y[3, 9])
        if dt:
            check_codes(y[[0, 4, 5]], sc.cpu()[[0, 4, 5]], want, 64, "beside bad rows")
            assert torch.allclose(sc[1].cpu(), torch.full((4,), 1e-12 / 448), rtol=1e-6)
        else:
            check(y[[0, 4, 5]], want, 81 * U * np.abs(want), "beside bad rows")
    zero, _, _ = gdr.rmsnorm_fwd(torch.zeros(2, 64, device=DEV), torch.ones(64, device=DEV), eps=0.0)
    assert torch.isnan(zero).all()                          # 0 / 0, as the formula says
    dx, dw = gdr.rmsnorm_bwd(c["dy"].to(DEV), x, w, eps=EPS)
    assert torch.isfinite(dx[[0, 1, 4, 5]]).all()
    # values far below the floor of the scale
    tiny = torch.full((1, 64), 1e-20, device=DEV)
    q, _, sc = gdr.rmsnorm_fwd(tiny, torch.full((64,), 1e-16, device=DEV), eps=1.0, y_dtype=E4)
    assert (q.float() == 0).all() and float(sc) == pytest.approx(1e-12 / 448, rel=1e-6)


@pytest.mark.parametrize("M,D", [(3000, 512), (77, 1001)])
def test_same_bits_every_time_and_in_a_graph(M, D):
    c = make(70, M, D, BF)
    x, r, w, dy, ds = (c[k].to(DEV) for k in ("x", "r", "w", "dy", "ds"))
    ws = torch.empty(gdr.rmsnorm_bwd_workspace_size(M, D), dtype=torch.uint8, device=DEV)

    def both(ws=None):
        return gdr.rmsnorm_fwd(x, w, residual=r, y_dtype=E4, scale_group=128) + \
            gdr.rmsnorm_bwd(dy, x, w, d_residual_out=ds, workspace=ws)

    want = [t.clone() for t in both()]
    for _ in range(5):
        ws.random_(0, 256)
        for a, b in zip(both(ws), want):
            assert bits_equal(a, b)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(both(ws))
        graphs.append(graph)
    for _ in range(2):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(o, want):
            assert bits_equal(a, b)


def test_empty_and_stream():
    w = torch.ones(16, device=DEV)
    y, ro, _ = gdr.rmsnorm_fwd(torch.empty(0, 16, device=DEV), w, residual=torch.empty(0, 16, device=DEV))
    assert y.shape == ro.shape == (0, 16)
    dx, dw = gdr.rmsnorm_bwd(torch.empty(0, 16, device=DEV), torch.empty(0, 16, device=DEV), w)
    assert dx.shape == (0, 16) and not dw.any()
    c = make(80, 500, 512, BF)
    x, dy, w = c["x"].to(DEV), c["dy"].to(DEV), c["w"].to(DEV)
    want = gdr.rmsnorm_fwd(x, w)[0], *gdr.rmsnorm_bwd(dy, x, w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = gdr.rmsnorm_fwd(x, w, stream=side)[0], *gdr.rmsnorm_bwd(dy, x, w, stream=side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert bits_equal(a, b)


def test_binding_refusals():
    x, w = torch.randn(6, 8, device=DEV), torch.ones(8, device=DEV)
    for bad in (dict(residual=x[:5]), dict(residual_out=x), dict(scales=w), dict(y=torch.empty(6, 9, device=DEV)),
                dict(residual=x.t().contiguous().t()), dict(residual=x.cpu())):
        with pytest.raises(ValueError):
            gdr.rmsnorm_fwd(x, w, **bad)
    with pytest.raises(TypeError):
        gdr.rmsnorm_fwd(x, w.to(BF))
    with pytest.raises(TypeError):
        gdr.rmsnorm_fwd(x.half(), w)
    with pytest.raises(TypeError):
        gdr.rmsnorm_bwd(x, x.to(BF), w)
    for bad in (dict(y_dtype=BF), dict(y_dtype=E4, scale_group=48), dict(eps=-1.0), dict(scale_group=32)):
        with pytest.raises(gdr.GdrError):
            gdr.rmsnorm_fwd(x, w, **bad)
    with pytest.raises(gdr.GdrError):
        gdr.rmsnorm_fwd(torch.zeros(1, 32769, device=DEV), torch.ones(32769, device=DEV))
