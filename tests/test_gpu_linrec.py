"""GPU parity of the gated linear recurrence (forward, backward, slot-pool
step) against the fp64 oracle.

Tolerances, per element.  With S the recurrence of |x| and W the recurrence of
S (the same terms, each weighted by the steps it has come through), a chain of
fp32 steps is off by at most

    4 * 2^-24 W       a step's decay is exp to 1 ulp (2^-23), its fused
                      multiply-add half an ulp (2^-24); one to spare
  + 32 * 2^-24 max S  where decays of a run are formed from the sum G of the
                      gates: k additions leave k 2^-24 |G| in the exponent and
                      |G| e^-|G| <= 0.37, so 0.37 k 2^-24 of the state it
                      multiplies; k <= 16 over a tile's runs and a handful of
                      such products on the way to any row
  + half a step of the stored type, eps / 2 of the value
  + 2^-126 times what a decay multiplies: exp(g) below 2^-126 (g < -87.3) is
                      below fp32's normal numbers and may be stored with any
                      rounding down to 0, off by less than 2^-126.

The backward recurrence is the same one from the end; dg multiplies mu by a
stored y, one more rounding.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_37_gb300 as gdr
import oracle
from tests.gpu_util import Guarded, bits_equal, sentinel_like

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F = torch.bfloat16, torch.float32
U = 2.0 ** -24
TINY = 2.0 ** -126
TYPES = [(BF, F), (F, F), (BF, BF), (F, BF)]
LENS = {
    "one token": [1],
    "empty ones": [0, 1, 0, 0, 7, 0],
    "short": [5, 64, 3],
    "around 64s": [63, 65, 128, 1],
    "around 256": [255, 1, 257, 256],
    "one of 700": [700],
    "many": [1 + (i * 7) % 9 for i in range(150)],
}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdr.load()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


def make(seed, lens, D, dtype, gate, *, pad=0, g_lo=-1.0):
    r = torch.Generator().manual_seed(seed)
    T = sum(lens) + pad
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    # channels of long, middling and short memory
    per = g_lo * torch.rand(D, generator=r) ** 4
    return dict(cu=cu, x=torch.randn(T, D, generator=r).to(dtype), g=(per * torch.rand(T, D, generator=r)).to(gate),
                h0=torch.randn(len(lens), D, generator=r), df=torch.randn(len(lens), D, generator=r),
                y=torch.randn(T, D, generator=r).to(dtype), lens=lens, T=T, D=D)


def chain_tol(x, g, cu, start):
    """Bound on the fp32 error of the recurrence, per row, and of its last states."""
    S, s_last = oracle.linrec(np.abs(f64(x)), g, cu, initial_state=None if start is None else np.abs(f64(start)))
    W, w_last = oracle.linrec(S, g, cu)
    cu = [int(v) for v in cu]
    top = np.concatenate([np.broadcast_to(S[a:b].max(0), (b - a, S.shape[1])) for a, b in zip(cu, cu[1:]) if b > a]
                         + [np.zeros((0, S.shape[1]))])
    tol = np.full(S.shape, np.nan)
    tol[:cu[-1]] = 4 * U * W[:cu[-1]] + (32 * U + TINY) * top
    last = np.zeros(s_last.shape)
    for n, (a, b) in enumerate(zip(cu, cu[1:])):
        if b > a:
            last[n] = tol[b - 1]
    return tol, last


def check(got, want, tol, what):
    got = f64(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}, " \
        f"{got[bad][0]} for {want[bad][0]} within {np.broadcast_to(tol, want.shape)[bad][0]}"


def run_fwd(c, *, h0=True, workspace=None):
    y = Guarded((c["T"], c["D"]), c["x"].dtype, DEV, fill_bytes=sentinel_like((c["T"], c["D"]), c["x"].dtype))
    hT = Guarded(c["h0"].shape, F, DEV, fill_bytes=sentinel_like(c["h0"].shape, F))
    gdr.linrec_fwd(c["x"].to(DEV), c["g"].to(DEV), c["cu"].to(DEV), initial_state=c["h0"].to(DEV) if h0 else None,
                   y=y.view, final_state=hT.view, workspace=workspace)
    torch.cuda.synchronize()
    assert y.guards_intact() and hT.guards_intact()
    return y.view.cpu(), hT.view.cpu()


def check_fwd(c, y, hT, *, h0=True):
    n = int(c["cu"][-1])
    start = c["h0"] if h0 else None
    ry, rT = oracle.linrec(f64(c["x"]), f64(c["g"]), c["cu"], initial_state=start)
    tol, last = chain_tol(c["x"], f64(c["g"]), c["cu"], start)
    check(y[:n], ry[:n], tol[:n] + half_step(y.dtype) * np.abs(ry[:n]), "y")
    check(hT, rT, last, "final state")
    assert bits_equal(y[n:], sentinel_like((c["T"] - n, c["D"]), y.dtype)), "rows behind the last sequence"


def run_bwd(c, *, h0=True, df=True):
    dx = Guarded((c["T"], c["D"]), c["x"].dtype, DEV, fill_bytes=sentinel_like((c["T"], c["D"]), c["x"].dtype))
    dg = Guarded((c["T"], c["D"]), c["g"].dtype, DEV, fill_bytes=sentinel_like((c["T"], c["D"]), c["g"].dtype))
    d0 = Guarded(c["h0"].shape, F, DEV, fill_bytes=sentinel_like(c["h0"].shape, F))
    gdr.linrec_bwd(c["x"].to(DEV), c["g"].to(DEV), c["y"].to(DEV), c["cu"].to(DEV),
                   initial_state=c["h0"].to(DEV) if h0 else None, d_final_state=c["df"].to(DEV) if df else None,
                   dx=dx.view, dg=dg.view, d_initial_state=d0.view)
    torch.cuda.synchronize()
    assert dx.guards_intact() and dg.guards_intact() and d0.guards_intact()
    return dx.view.cpu(), dg.view.cpu(), d0.view.cpu()


def check_bwd(c, dx, dg, d0, *, h0=True, df=True):
    n, cu = int(c["cu"][-1]), [int(v) for v in c["cu"]]
    g, y = f64(c["g"]), f64(c["y"])
    start = c["h0"] if h0 else None
    rx, rg, r0 = oracle.linrec_bwd(f64(c["x"]), g, y, c["cu"], initial_state=start,
                                   d_final_state=c["df"] if df else None)
    # lam is the recurrence, from the end, of dy with the decay of the token behind (0 at a sequence's end,
    # where the final state's gradient is added to dy): the same bound
    back = np.full(g.shape, -np.inf)
    back[:-1] = g[1:]
    b = np.abs(f64(c["x"]))
    for k, e in enumerate(cu[1:]):
        if e > cu[k]:
            back[e - 1] = -np.inf
            if df:
                b[e - 1] += np.abs(f64(c["df"])[k])
    rev = lambda a: a[:n][::-1].copy()  # noqa: E731
    cr = np.concatenate([[0], np.cumsum(c["lens"][::-1])])
    tol = chain_tol(torch.from_numpy(rev(b)), rev(back), cr, None)[0][::-1]
    check(dx[:n], rx[:n], tol + half_step(dx.dtype) * np.abs(rx[:n]), "dx")
    before = np.zeros((n, c["D"]))
    before[1:] = np.abs(y[:n - 1]) if n > 1 else 0
    mu_tol = np.exp(g[:n]) * (tol + 4 * U * np.abs(rx[:n])) + TINY * np.abs(rx[:n])
    tol0 = np.zeros(r0.shape)
    for k, a in enumerate(cu[:-1]):
        if cu[k + 1] > a:
            before[a] = np.abs(f64(c["h0"])[k]) if h0 else 0
            tol0[k] = mu_tol[a]
    check(dg[:n], rg[:n], mu_tol * before + (U + half_step(dg.dtype)) * np.abs(rg[:n]) + TINY, "dg")
    check(d0, r0, tol0, "d_initial_state")
    for t in (dx, dg):
        assert bits_equal(t[n:], sentinel_like((c["T"] - n, c["D"]), t.dtype)), "rows behind the last sequence"


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(d)[6:] for d in t))
@pytest.mark.parametrize("D", [1, 8, 65, 128, 200])
@pytest.mark.parametrize("lens", LENS, ids=lambda k: k.replace(" ", "_"))
def test_fwd_and_bwd(lens, D, types):
    c = make(D + len(lens), LENS[lens], D, *types, pad=3 if D == 65 else 0)
    check_fwd(c, *run_fwd(c))
    check_bwd(c, *run_bwd(c))


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(d)[6:] for d in t))
@pytest.mark.parametrize("D", [72, 65])
@pytest.mark.parametrize("lens", [[192, 192, 320, 448, 1], [448], [320, 0, 320, 0], [191, 1, 193, 447, 1, 449, 319, 321],
                                  [192 * 35], [64, 1, 64 * 105 - 1]],
                         ids=["ends of tiles", "one", "two", "around", "whole tiles", "a token before"])
def test_sequences_that_end_with_tiles(lens, D, types):
    """Tiles are 96 to 448 tokens, by type and direction: sequences that end
    with them, just before and just behind, in calls of one row of tiles, of a
    few and of many."""
    c = make(26 + len(lens), lens, D, *types)
    check_fwd(c, *run_fwd(c))
    check_bwd(c, *run_bwd(c))


@pytest.mark.parametrize("D", [2080, 2081])
def test_offsets_beyond_32_bits(D):
    """Rows whose elements' numbers pass 2^31 (and bytes 2^32): the last
    sequence of a long batch, against 64 bits."""
    T, n = (1 << 20) + 5, 700
    assert (T - n) * D > 1 << 31
    big = {}
    for k in ("x", "y"):
        big[k] = torch.zeros(T, D, dtype=BF, device=DEV)
    big["g"] = torch.full((T, D), -1.0, dtype=BF, device=DEV)
    c = make(31, [n], D, BF, BF)
    for k, v in big.items():
        v[T - n:] = c[k].to(DEV)
    cu = torch.tensor([0, T - n, T], dtype=torch.int32, device=DEV)
    h0 = torch.cat([torch.zeros(1, D), c["h0"]]).to(DEV)
    df = torch.cat([torch.zeros(1, D), c["df"]]).to(DEV)
    y, hT = gdr.linrec_fwd(big["x"], big["g"], cu, initial_state=h0)
    check_fwd(c, y[T - n:].cpu(), hT[1:].cpu())
    assert not y[:T - n].any() and not hT[0].any()
    del y
    dx, dg, d0 = gdr.linrec_bwd(big["x"], big["g"], big["y"], cu, initial_state=h0, d_final_state=df)
    check_bwd(c, dx[T - n:].cpu(), dg[T - n:].cpu(), d0[1:].cpu())
    assert not dx[:T - n].any() and not dg[:T - n].any() and not d0[0].any()


def test_without_states():
    c = make(3, [40, 0, 300], 72, BF, F)
    check_fwd(c, *run_fwd(c, h0=False), h0=False)
    check_bwd(c, *run_bwd(c, h0=False, df=False), h0=False, df=False)
    y, none = gdr.linrec_fwd(c["x"].to(DEV), c["g"].to(DEV), c["cu"].to(DEV), output_final_state=False)
    assert none is None and bits_equal(y, run_fwd(c, h0=False)[0])
    dx, dg, none = gdr.linrec_bwd(c["x"].to(DEV), c["g"].to(DEV), c["y"].to(DEV), c["cu"].to(DEV),
                                  output_d_initial_state=False)
    assert none is None and bits_equal(dx, run_bwd(c, h0=False, df=False)[0])


@pytest.mark.parametrize("types", [(BF, F), (F, F), (BF, BF)], ids=["bf16", "f32", "bf16-gates"])
def test_long_memory(types):
    """8200 tokens of channels that forget over hundreds to thousands of tokens: many tiles, one carry."""
    c = make(11, [8200], 72, *types, g_lo=-0.01)
    check_fwd(c, *run_fwd(c))
    check_bwd(c, *run_bwd(c))


@pytest.mark.parametrize("types", [(BF, BF), (F, F)], ids=["bf16", "f32"])
def test_long_unaligned_rows(types):
    """The same with rows of every alignment."""
    c = make(22, [4000, 1, 4199], 65, *types, g_lo=-0.02, pad=1)
    check_fwd(c, *run_fwd(c))
    check_bwd(c, *run_bwd(c))


@pytest.mark.parametrize("lens,pad", [([100], 900), ([5, 0, 300], 4000), ([3000], 3000), ([0, 0], 700), ([0], 9000)])
@pytest.mark.parametrize("D", [64, 65])
def test_padded_batches(D, lens, pad):
    """Whole tiles behind the last sequence, in calls of every size."""
    c = make(23, lens, D, BF, F, pad=pad)
    check_fwd(c, *run_fwd(c))
    check_bwd(c, *run_bwd(c))


@pytest.mark.parametrize("T,D", [(400, 64), (1500, 72), (3000, 200), (3000, 65)])
def test_workspace_is_kept_to(T, D):
    """The stated size is enough, and nothing around it is written."""
    c = make(24, [T], D, BF, F)
    n = gdr.linrec_workspace_size(1, T, D, dtype=gdr.GDR_BF16, gate_dtype=gdr.GDR_F32)
    ws = Guarded((n,), torch.uint8, DEV, fill_bytes=torch.full((n,), 0x3C, dtype=torch.uint8))
    y, hT = run_fwd(c, workspace=ws.view)
    assert ws.guards_intact()
    check_fwd(c, y, hT)
    if n:
        with pytest.raises(gdr.GdrError, match="workspace"):
            run_fwd(c, workspace=ws.view[:n - 1])
    assert gdr.device_status() == 0


def test_many_sequences():
    """More sequences than a grid axis holds, most of them one token or none."""
    c = make(12, [(i * 5) % 3 for i in range(70000)], 8, BF, F)
    check_fwd(c, *run_fwd(c))
    check_bwd(c, *run_bwd(c))


def test_wide_rows():
    c = make(13, [70, 33], 8192, BF, BF)
    check_fwd(c, *run_fwd(c))
    check_bwd(c, *run_bwd(c))


@pytest.mark.parametrize("g", [0.0, -2.0, -30.0, -200.0, -np.inf])
def test_extreme_decays(g):
    """Sums, underflowing products of decays, resets."""
    c = make(14, [300, 1, 290], 64, F, F)
    c["g"][:, ::2] = g
    check_fwd(c, *run_fwd(c))
    check_bwd(c, *run_bwd(c))


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_a_bad_value_stays_in_its_sequence_and_channel(value):
    lens = [40, 300, 0, 500, 9]
    c = make(15, lens, 64, F, F)
    y0, h0 = run_fwd(c)
    dx0, dg0, d00 = run_bwd(c)
    cu = [int(v) for v in c["cu"]]
    t, ch = cu[1] + 30, 5
    c["x"][t, ch] = value
    y, hT = run_fwd(c)
    dx, dg, d0 = run_bwd(c)
    row = torch.arange(c["T"])
    hit = torch.zeros(c["T"], c["D"], dtype=torch.bool)
    hit[:, ch] = (row >= t) & (row < cu[2])
    assert bits_equal(y[~hit], y0[~hit]) and not torch.isfinite(y[t, ch])
    if np.isnan(value):
        assert torch.isnan(y[hit]).all() and torch.isnan(hT[1, ch])
    other = torch.ones_like(hT, dtype=torch.bool)
    other[1, ch] = False
    assert bits_equal(hT[other], h0[other])
    hit[:, ch] = (row >= cu[1]) & (row <= t)
    assert bits_equal(dx[~hit], dx0[~hit]) and bits_equal(dg[~hit], dg0[~hit]) and bits_equal(d0[other], d00[other])
    assert not torch.isfinite(dx[t, ch])


def test_rows_behind_the_last_sequence_are_not_read():
    c = make(16, [100, 200], 64, BF, F, pad=77)
    want = run_fwd(c), run_bwd(c)
    for k in ("x", "g", "y"):
        c[k][300:] = np.nan
    got = run_fwd(c), run_bwd(c)
    for a, b in zip(want[0] + want[1], got[0] + got[1]):
        assert bits_equal(a, b)


def test_strides_and_alignment():
    """Column blocks of one wide matrix, at aligned and unaligned offsets, an
    expanded row of gates, and a row of one token with a stride of its own."""
    c = make(17, [37, 270], 64, BF, BF)
    want = run_fwd(c) + run_bwd(c)
    cu, h0, df = c["cu"].to(DEV), c["h0"].to(DEV), c["df"].to(DEV)
    for off, width in ((0, 256), (64, 256), (3, 201), (1, 64 * 3 + 1)):
        wide = torch.full((c["T"], 5 * width), float("nan"), dtype=BF, device=DEV)
        cut = [wide[:, i * width + off:i * width + off + 64] for i in range(5)]
        for t, k in zip(cut, ("x", "g", "y")):
            t.copy_(c[k])
        y, hT = gdr.linrec_fwd(cut[0], cut[1], cu, initial_state=h0, y=cut[3])
        dx, dg, d0 = gdr.linrec_bwd(cut[0], cut[1], cut[2], cu, initial_state=h0, d_final_state=df,
                                    dx=torch.empty_strided((c["T"], 64), (65, 1), dtype=BF, device=DEV), dg=cut[4])
        for a, b in zip((y, hT, dx, dg, d0), want):
            assert (a.cpu().double() - b.double()).abs().max() <= 1e-2 * b.double().abs().max()
        other = torch.ones_like(wide, dtype=torch.bool)
        for i in range(5):
            other[:, i * width + off:i * width + off + 64] = False
        assert torch.isnan(wide[other]).all(), "written outside the column blocks"
    c["g"] = c["g"][:1].expand(c["T"], 64)
    one = gdr.linrec_fwd(c["x"].to(DEV), c["g"][:1].to(DEV).expand(c["T"], 64), cu, initial_state=h0)
    check_fwd(c, one[0].cpu(), one[1].cpu())
    row = torch.randn(1, 128, device=DEV).to(BF)
    y, _ = gdr.linrec_fwd(row[:, ::1][:, :64], torch.zeros(1, 64, device=DEV), torch.tensor([0, 1], dtype=torch.int32,
                                                                                          device=DEV))
    assert bits_equal(y, row[:, :64])


@pytest.mark.parametrize("lens,D", [([3000], 256), ([1, 500, 700], 65)])
def test_same_bits_every_time_and_in_a_graph(lens, D):
    """Equal bits from call to call, from a captured and replayed call, and
    from two graphs that share a workspace and run one after the other."""
    c = make(18, lens, D, BF, F)
    args = [c[k].to(DEV) for k in ("x", "g", "cu")]
    h0, df, yy = c["h0"].to(DEV), c["df"].to(DEV), c["y"].to(DEV)
    ws = torch.empty(max(1, gdr.linrec_workspace_size(len(lens), c["T"], D, dtype=gdr.GDR_BF16,
                                                      gate_dtype=gdr.GDR_F32)), dtype=torch.uint8, device=DEV)

    def both(ws=None):
        return gdr.linrec_fwd(*args, initial_state=h0, workspace=ws) + \
            gdr.linrec_bwd(args[0], args[1], yy, args[2], initial_state=h0, d_final_state=df, workspace=ws)

    want = [t.clone() for t in both()]
    for _ in range(20):
        ws.random_(0, 256)                                 # a workspace needs no initialisation
        for a, b in zip(both(ws), want):
            assert bits_equal(a, b)
    graphs, outs = [], []
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both(ws)
    torch.cuda.synchronize()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(both(ws))
        graphs.append(graph)
    for _ in range(3):
        for o in outs:
            for t in o:
                t.fill_(-1)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for o in outs:
            for a, b in zip(o, want):
                assert bits_equal(a, b)


def test_streams():
    """A call on a stream of its own: its outputs and workspace belong to that
    stream; two calls at once do not disturb one another."""
    c = make(19, [5000], 128, BF, F)
    x, g, cu, h0 = (c[k].to(DEV) for k in ("x", "g", "cu", "h0"))
    want = gdr.linrec_fwd(x, g, cu, initial_state=h0)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[gdr.linrec_fwd(x, g, cu, initial_state=h0, stream=s) for _ in range(5)] for s in streams]
    torch.cuda.synchronize()
    for runs in got:
        for y, hT in runs:
            assert bits_equal(y, want[0]) and bits_equal(hT, want[1])


def test_calls_that_share_the_gpu():
    """Calls of several times the GPU's size at once, on streams and workspaces
    of their own: tiles wait only for tiles that are running, so all end, with
    the bits of a call alone."""
    c = make(25, [9000, 11000], 1024, BF, BF)
    x, g, y, cu, h0, df = (c[k].to(DEV) for k in ("x", "g", "y", "cu", "h0", "df"))
    want = gdr.linrec_fwd(x, g, cu, initial_state=h0) + \
        gdr.linrec_bwd(x, g, y, cu, initial_state=h0, d_final_state=df)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s in streams:
            got.append(gdr.linrec_fwd(x, g, cu, initial_state=h0, stream=s) +
                       gdr.linrec_bwd(x, g, y, cu, initial_state=h0, d_final_state=df, stream=s))
    torch.cuda.synchronize()
    for run in got:
        for a, b in zip(run, want):
            assert torch.equal(a, b)
    assert gdr.device_status() == 0


def test_empty_calls():
    cu = torch.zeros(4, dtype=torch.int32, device=DEV)
    x, g, h0 = torch.empty(0, 8, device=DEV), torch.empty(0, 8, device=DEV), torch.randn(3, 8, device=DEV)
    y, hT = gdr.linrec_fwd(x, g, cu, initial_state=h0)
    assert y.shape == (0, 8) and bits_equal(hT, h0)
    assert not gdr.linrec_fwd(x, g, cu)[1].any()
    dx, dg, d0 = gdr.linrec_bwd(x, g, y, cu, d_final_state=h0)
    assert dx.shape == dg.shape == (0, 8) and bits_equal(d0, h0)
    # rows, but none of them in a sequence
    x, out = torch.randn(40, 8, device=DEV), torch.full((40, 8), 7.0, device=DEV)
    _, hT = gdr.linrec_fwd(x, -x.abs(), cu, initial_state=h0, y=out)
    assert (out == 7).all() and bits_equal(hT, h0)


def test_validate():
    c = make(20, [10, 20], 16, F, F, pad=2)
    x, g, cu = c["x"].to(DEV), c["g"].to(DEV), c["cu"].to(DEV)
    fwd = lambda g=g, cu=cu: gdr.linrec_fwd(x, g, cu, flags=gdr.GDR_VALIDATE)  # noqa: E731
    fwd()
    for bad_cu in ([1, 10, 30], [0, 31, 30], [0, 10, 33], [0, -1, 30]):
        with pytest.raises(gdr.GdrError, match="cu_seqlens"):
            fwd(cu=torch.tensor(bad_cu, dtype=torch.int32, device=DEV))
    for v in (0.5, np.nan):
        bad = g.clone()
        bad[29, 15] = v
        with pytest.raises(gdr.GdrError, match="gate"):
            fwd(g=bad)
        with pytest.raises(gdr.GdrError, match="gate"):
            gdr.linrec_bwd(x, bad, x, cu, flags=gdr.GDR_VALIDATE)
        bad[29, 15], bad[31, 0] = -np.inf, v               # a reset is a gate, a row behind the last sequence is not read
        fwd(g=bad)


def test_malformed_lengths_stay_inside_the_tensors():
    """What is written is unspecified, where it is not."""
    for cu in ([5, 20, 10, 400], [0, 1000, 20, 300], [-7, 20, 300, 300], [300, 200, 100, 0], [0, 300, 300, 2 ** 31 - 1]):
        c = make(21, [100, 100, 100], 64, BF, F)
        c["cu"] = torch.tensor(cu, dtype=torch.int32)
        run_fwd(c)
        run_bwd(c)
    y, hT = run_fwd(make(21, [100, 100, 100], 64, BF, F))
    check_fwd(make(21, [100, 100, 100], 64, BF, F), y, hT)


def test_binding_refusals():
    x, g = torch.randn(6, 8, device=DEV), -torch.rand(6, 8, device=DEV)
    cu = torch.tensor([0, 6], dtype=torch.int32, device=DEV)
    for bad in (dict(initial_state=torch.zeros(2, 8, device=DEV)), dict(y=torch.empty(6, 9, device=DEV)),
                dict(final_state=torch.empty(1, 8)), dict(workspace=torch.empty(8, device=DEV))):
        with pytest.raises(ValueError):
            gdr.linrec_fwd(x, g, cu, **bad)
    for bad in (dict(initial_state=torch.zeros(1, 8, device=DEV, dtype=BF)), dict(y=torch.empty(6, 8, device=DEV,
                                                                                              dtype=BF))):
        with pytest.raises(TypeError):
            gdr.linrec_fwd(x, g, cu, **bad)
    with pytest.raises(TypeError):
        gdr.linrec_fwd(x, g, cu.long())
    with pytest.raises(TypeError):
        gdr.linrec_fwd(x.half(), g, cu)
    with pytest.raises(ValueError):
        gdr.linrec_fwd(x.t().contiguous().t(), g, cu)      # not dense along its last axis
    with pytest.raises(ValueError):
        gdr.linrec_fwd(x, g[:5], cu)
    with pytest.raises(gdr.GdrError):
        gdr.linrec_fwd(x, g, cu, y=torch.empty(8, device=DEV).expand(6, 8))   # rows written over one another


# ---- the slot-pool step ------------------------------------------------------


def pool_case(seed, lens, D, dtype, gate, pool_dtype, skip=()):
    c = make(seed, lens, D, dtype, gate)
    r = torch.Generator().manual_seed(seed)
    N = len(lens)
    idx = torch.randperm(N + 3, generator=r)[:N].to(torch.int32)
    for k, v in dict(skip).items():
        idx[k] = v
    return dict(c, idx=idx, pool=torch.randn(N + 3, D, generator=r).to(pool_dtype))


def run_step(c, *, commit, steps=0, rows=None):
    N = len(c["lens"])
    pool = Guarded(c["pool"].shape, c["pool"].dtype, DEV, fill_bytes=c["pool"])
    y = Guarded((c["T"], c["D"]), c["x"].dtype, DEV, fill_bytes=sentinel_like((c["T"], c["D"]), c["x"].dtype))
    ib = None
    if steps:
        shape = (rows or N, steps, c["D"])
        ib = Guarded(shape, c["pool"].dtype, DEV, fill_bytes=sentinel_like(shape, c["pool"].dtype))
    gdr.linrec_step(c["x"].to(DEV), c["g"].to(DEV), pool.view, c["idx"].to(DEV), c["cu"].to(DEV),
                    flags=gdr.GDR_COMMIT if commit else 0, y=y.view, intermediate_states=ib.view if ib else None)
    torch.cuda.synchronize()
    assert pool.guards_intact() and y.guards_intact() and (ib is None or ib.guards_intact())
    return pool.view.cpu(), y.view.cpu(), None if ib is None else ib.view.cpu()


def check_step(c, pool, y, ib, *, commit):
    cu, idx = [int(v) for v in c["cu"]], c["idx"].tolist()
    slots = c["pool"].shape[0]
    start = torch.stack([c["pool"][min(max(i, 0), slots - 1)] for i in idx]).float()
    ry, rT = oracle.linrec(f64(c["x"]), f64(c["g"]), c["cu"], initial_state=start)
    tol, last = chain_tol(c["x"], f64(c["g"]), c["cu"], start)
    written = set()
    for n, i in enumerate(idx):
        a, b = cu[n], cu[n + 1]
        if not 0 <= i < slots:
            assert bits_equal(y[a:b], sentinel_like((b - a, c["D"]), y.dtype))
        elif b > a:
            check(y[a:b], ry[a:b], tol[a:b] + half_step(y.dtype) * np.abs(ry[a:b]), "y")
            if commit:
                written.add(i)
                check(pool[i], rT[n], last[n] + half_step(pool.dtype) * np.abs(rT[n]), "slot")
        if ib is not None:
            kept = min(b - a, ib.shape[1]) if 0 <= i < slots else 0
            w = ry[a:a + kept]
            check(ib[n, :kept], w, tol[a:a + kept] + half_step(ib.dtype) * np.abs(w), "states")
            assert bits_equal(ib[n, kept:], sentinel_like(tuple(ib[n, kept:].shape), ib.dtype))
    for i in range(slots):
        if i not in written:
            assert bits_equal(pool[i], c["pool"][i]), "a slot that must stay as it was"


@pytest.mark.parametrize("pool_dtype", [F, BF], ids=["f32-pool", "bf16-pool"])
@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(d)[6:] for d in t))
@pytest.mark.parametrize("D", [1, 8, 65, 256, 4096])
def test_step(D, types, pool_dtype):
    c = pool_case(D, [1, 3, 0, 12, 1, 7, 2], D, *types, pool_dtype, skip={1: -1, 4: -5})
    check_step(c, *run_step(c, commit=True, steps=12), commit=True)
    check_step(c, *run_step(c, commit=False), commit=False)
    check_step(c, *run_step(c, commit=False, steps=5, rows=9), commit=False)   # later states dropped


def test_step_decode_batch():
    c = pool_case(30, [1] * 256, 520, BF, F, F, skip={i: -1 for i in range(0, 256, 10)})
    check_step(c, *run_step(c, commit=True), commit=True)


def test_step_skips_slots_out_of_range_and_reports_them():
    c = pool_case(31, [2, 2, 2], 64, BF, F, F, skip={1: 10 ** 6})
    check_step(c, *run_step(c, commit=True), commit=True)
    dev = {k: c[k].to(DEV) for k in ("x", "g", "pool", "idx", "cu")}
    call = lambda flags, idx, **kw: gdr.linrec_step(dev["x"], dev["g"], dev["pool"], idx, dev["cu"],  # noqa: E731
                                                    flags=flags | gdr.GDR_VALIDATE, **kw)
    with pytest.raises(gdr.GdrError, match="num_slots"):
        call(0, dev["idx"])
    twice = torch.tensor([0, 3, 3], dtype=torch.int32, device=DEV)
    with pytest.raises(gdr.GdrError, match="duplicate"):
        call(gdr.GDR_COMMIT, twice)
    call(0, twice)                                         # read twice, written by none
    with pytest.raises(gdr.GdrError, match="steps"):
        call(0, twice, intermediate_states=torch.empty(3, 1, 64, device=DEV))


def test_step_without_decay_slots_shared_for_reading():
    c = pool_case(32, [3, 3, 3], 40, F, F, BF, skip={0: 2, 1: 2, 2: 2})
    check_step(c, *run_step(c, commit=False, steps=3), commit=False)


def test_prefill_then_steps_is_one_long_sequence():
    """A prompt through linrec_fwd, its final states put into a pool, then a
    verify step and single tokens: together the recurrence over all of it."""
    lens, more = [30, 1, 400], [4, 1, 6]
    whole = make(33, [a + b for a, b in zip(lens, more)], 96, F, F)
    cu = [int(v) for v in whole["cu"]]
    head = torch.cat([torch.arange(cu[n], cu[n] + lens[n]) for n in range(3)])
    d = lambda t: t.to(DEV)  # noqa: E731
    cu_of = lambda ls: torch.tensor([0] + list(np.cumsum(ls)), dtype=torch.int32, device=DEV)  # noqa: E731
    y0, hT = gdr.linrec_fwd(d(whole["x"][head]), d(whole["g"][head]), cu_of(lens), initial_state=d(whole["h0"]))
    pool = torch.full((5, 96), float("nan"), device=DEV)
    idx = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    pool[idx.long()] = hT
    got = {n: [y0[sum(lens[:n]):sum(lens[:n + 1])]] for n in range(3)}
    take = [m - 1 for m in more]                           # all but one token as a verify, the last as a decode
    for first, counts in ((0, take), (1, [1, 1, 1])):
        rows = torch.cat([torch.arange(cu[n] + lens[n] + (take[n] if first else 0),
                                       cu[n] + lens[n] + (take[n] if first else 0) + counts[n]) for n in range(3)])
        y = gdr.linrec_step(d(whole["x"][rows]), d(whole["g"][rows]), pool, idx, cu_of(counts))
        for n in range(3):
            got[n].append(y[sum(counts[:n]):sum(counts[:n + 1])])
    y = torch.cat([torch.cat(got[n]) for n in range(3)]).cpu()
    check_fwd(whole, y, pool[idx.long()].cpu())
