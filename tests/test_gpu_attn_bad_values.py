"""Infinities and NaN in the attention layer: rows that do not see them keep their bits where no product reaches them,
and rows that see them cost no more than others."""
import pytest
import torch

import gated_delta_rule_37_gb300 as gdr
import oracle
from tests.attn_util import DEV, Pool, check_attention, ints, normal, starts
from tests.gpu_util import bits_equal

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def _no_wait_gave_up():
    yield
    assert gdr.device_status() == 0


def _prompt(T, Hq, Hkv, D, dtype=BF16):
    return [normal(s, T, H, D, dtype=dtype) for s, H in ((1, Hq), (2, Hkv), (3, Hkv))]


# ---- prompts: what lies behind a sequence ----------------------------------------------


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (16, 2), (3, 1), (2, 2), (128, 1)])
@pytest.mark.parametrize("L", [380, 129, 1, 700])
def test_values_behind_a_sequence_change_no_bit(L, Hq, Hkv, D):
    """Every row tile whose last key tile goes on into the next sequence or the padding, not the last one alone."""
    behind = 200
    q, k, v = _prompt(L + behind, Hq, Hkv, D)
    cu = starts([L, behind])
    clean = gdr.attn_fwd(q, k, v, cu)
    for what in (NAN, INF):
        kb, vb = k.clone(), v.clone()
        kb[L:], vb[L:] = what, what
        for c in (cu, starts([L]), starts([L, 0, 0])):
            assert bits_equal(gdr.attn_fwd(q, kb, vb, c)[:L], clean[:L])


# ---- missing pages -----------------------------------------------------------------------


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_missing_pages_read_no_other(page, D):
    """The cache's first rows, NaN and not any sequence's, change no bit where the prefix or a sequence lacks a page."""
    prefix, lens, lengths = 4 * page + 5, [4 * page + 20, 6 * page, 4 * page + 5], [1, 3, 2]
    cu = starts(lengths)
    pool = Pool(2, [a + n for a, n in zip(lens, lengths)], 2, D, page, BF16, prefix)
    for name in ("k", "v"):  # a page of nobody's in front
        c = getattr(pool, name)
        setattr(pool, name, torch.cat([torch.zeros_like(c[:1]), c]))
    pool.table = torch.where(pool.table >= 0, pool.table + 1, pool.table)
    pool.prefix_pages = pool.prefix_pages + 1
    pool.prefix_pages[1], pool.prefix_pages[3] = -1, pool.k.shape[0]
    pool.table[1, 5] = -3
    pool.table_list, pool.prefix_list = pool.table.tolist(), pool.prefix_pages.tolist()
    q = normal(1, sum(lengths), 8, D, dtype=BF16)
    clean = pool.step(q, lens, cu)
    check_attention(clean, pool.reference(q, lens, cu), max(lens) + 3)
    for what in (NAN, INF):
        pool.k[0], pool.v[0] = what, what
        assert bits_equal(pool.step(q, lens, cu), clean)


# ---- rows that see them --------------------------------------------------------------------


def _time(f, calls=4):
    """The shortest of several runs of a few calls, in ms."""
    f()
    best = 1e9
    for _ in range(4):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(calls):
            f()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) / calls)
    return best


def _spoil(k, v, what):
    """One bad channel of key head 0, as `what` says; the heads' share of the result that it reaches."""
    k, v = k.clone(), v.clone()
    if what == "key":
        k[0, 0, 5] = NAN
        return k, v, slice(None)
    if what == "value":
        v[0, 0, 5] = NAN
    elif what == "infinite value":
        v[0, 0, 5] = INF
    elif what == "infinite channel":
        v[:, 0, 5] = -INF
    else:
        v[:, 0, 5] = NAN
    return k, v, 5


BAD = ["key", "value", "infinite value", "channel", "infinite channel"]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("what", BAD)
def test_prompt_of_rows_that_see_a_bad_value(what, D):
    """They are right to have met it: no row is computed once more for it, other channels and heads keep their bits,
    and the call takes about as long (one row after the other it would take a thousand times as long)."""
    T, Hq, Hkv = 8192, 8, 2
    q, k, v = _prompt(T, Hq, Hkv, D)
    kb, vb, channel = _spoil(k, v, what)
    cu = starts([T])
    clean, o = gdr.attn_fwd(q, k, v, cu), gdr.attn_fwd(q, kb, vb, cu)
    hit = torch.zeros(o.shape, dtype=torch.bool, device=DEV)
    hit[:, :Hq // Hkv, channel] = True
    assert not torch.isfinite(o[hit]).any()
    if not what.startswith("infinite"):
        assert torch.isnan(o[hit]).all()
    else:
        assert (o[hit] == (INF if what == "infinite value" else -INF)).all()
    assert bits_equal(torch.where(hit, 0, o), torch.where(hit, 0, clean))
    good, bad = _time(lambda: gdr.attn_fwd(q, k, v, cu, o=clean)), _time(lambda: gdr.attn_fwd(q, kb, vb, cu, o=o))
    assert bad < 4 * good, f"{bad:.3f} ms against {good:.3f}"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefix", [0, 4096])
@pytest.mark.parametrize("what", BAD)
def test_step_of_rows_that_see_a_bad_value(what, prefix, D):
    """The same of decode, the bad token in the prefix or at the beginning of every sequence."""
    N, Hq, Hkv, own = 64, 32, 8, 4096
    lens, cu = [prefix + own - 1] * N, starts([1] * N)
    pool = Pool(1, [prefix + own] * N, Hkv, D, 64, BF16, prefix)
    q = normal(2, N, Hq, D, dtype=BF16)
    clean = pool.step(q, lens, cu)
    good = _time(lambda: pool.step(q, lens, cu))
    pages = pool.prefix_list[:1] if prefix else [t[0] for t in pool.table_list]
    if what == "key":
        pool.k[pages, 0, 0, 5] = NAN
    elif what.endswith("channel"):
        pool.v[:, 0, :, 5] = NAN if what == "channel" else -INF
    else:
        pool.v[pages, 0, 0, 5] = NAN if what == "value" else INF
    o = pool.step(q, lens, cu)
    hit = torch.zeros(o.shape, dtype=torch.bool, device=DEV)
    hit[:, :Hq // Hkv, slice(None) if what == "key" else 5] = True
    assert not torch.isfinite(o[hit]).any()
    assert bits_equal(torch.where(hit, 0, o), torch.where(hit, 0, clean))
    bad = _time(lambda: pool.step(q, lens, cu))
    assert bad < 4 * good, f"{bad:.3f} ms against {good:.3f}"


@pytest.mark.parametrize("D", [64, 128])
def test_verify_of_rows_that_see_a_bad_value(D):
    """Several tokens of a sequence: those that see the last one's NaN, those that see the first one's, and a channel
    that is NaN throughout."""
    N, m, Hq, Hkv, own = 32, 12, 32, 8, 4096
    lens, cu = [own - m] * N, starts([m] * N)
    pool = Pool(1, [own] * N, Hkv, D, 64, BF16)
    q = normal(2, N * m, Hq, D, dtype=BF16)
    clean = pool.step(q, lens, cu)
    good = _time(lambda: pool.step(q, lens, cu))
    pool.v[:, 0, :, 5] = NAN
    o = pool.step(q, lens, cu)
    hit = torch.zeros(o.shape, dtype=torch.bool, device=DEV)
    hit[:, :4, 5] = True
    assert torch.isnan(o[hit]).all()
    assert bits_equal(torch.where(hit, 0, o), torch.where(hit, 0, clean))
    bad = _time(lambda: pool.step(q, lens, cu))
    assert bad < 4 * good, f"{bad:.3f} ms against {good:.3f}"


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_of_scores_of_minus_infinity(D):
    """Many rows that see scores of -inf alone: 0, whatever the values, and as fast as others."""
    T, Hq, Hkv = 8192, 8, 2
    q, k, v = _prompt(T, Hq, Hkv, D)
    cu = starts([T])
    good = _time(lambda: gdr.attn_fwd(q, k, v, cu))
    q[..., 0] = 1
    k[:, :, 0] = -INF
    v[3, 0, 2], v[T // 2, 1, 2] = NAN, INF
    o = gdr.attn_fwd(q, k, v, cu)
    assert (o == 0).all()
    bad = _time(lambda: gdr.attn_fwd(q, k, v, cu, o=o))
    assert bad < 4 * good, f"{bad:.3f} ms against {good:.3f}"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,m", [(2, 1), (2, 3), (16, 1), (16, 5)])
def test_scores_of_minus_infinity_of_bad_values(m, Hq, D, dtype):
    """A row all of whose scores are -inf is 0 also where the values are not finite: prompts, the step in each of its
    tiles, in one run and cut into several, with a prefix and without."""
    T = 900
    q, k, v = torch.ones(T, Hq, D, dtype=dtype, device=DEV), normal(1, T, 1, D, dtype=dtype), normal(2, T, 1, D, dtype=dtype)
    k[:, :, 0] = -INF
    v[0, 0, 3], v[500, 0, 4], v[T - 1, 0, 5] = NAN, INF, NAN
    assert (gdr.attn_fwd(q, k, v, starts([T])) == 0).all()
    for prefix in (0, 200):
        pool = Pool(1, [T, T], 1, D, 64, dtype, prefix)
        for n in range(2):
            for p in range(-(-T // 64)):
                pages = pool.prefix_list if (p + 1) * 64 <= prefix or pool.table_list[n][p] < 0 else pool.table_list[n]
                rows = slice(p * 64, min((p + 1) * 64, T))
                pool.k[pages[p], 0, :rows.stop - rows.start], pool.v[pages[p], 0, :rows.stop - rows.start] = k[rows, 0], v[rows, 0]
        if prefix:  # the page that it ends in is the prefix's and each sequence's
            pool.k[pool.prefix_list[3], 0], pool.v[pool.prefix_list[3], 0] = k[192:256, 0], v[192:256, 0]
        o = pool.step(q[:2 * m], [T - m, T - m], starts([m, m]))
        assert (o == 0).all(), prefix


# ---- values near the type's largest -----------------------------------------------------------


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128])
def test_values_whose_weighted_sum_fits(D, dtype):
    """Values of up to 2^119: 300 of them with weights of at most 1 stay below 2^128, with the 2^6.5 by which the scores
    rise behind the first tile they would not."""
    T, Hq, Hkv = 300, 4, 1
    q, k = torch.ones(T, Hq, D, dtype=dtype, device=DEV), torch.zeros(T, Hkv, D, dtype=dtype, device=DEV)
    k[128:, :, 0] = 4.5 * D ** 0.5
    v = ((normal(3, T, Hkv, D).abs().clamp(max=1) / 2 + 0.5) * 2.0 ** 119).to(dtype)
    cu = starts([T])
    ref = oracle.attn_fwd(q, k, v, cu, D ** -0.5)
    check_attention(gdr.attn_fwd(q, k, v, cu), ref, T, "prompt")
    for prefix in (0, 256):
        pool = Pool(1, [T], Hkv, D, 64, dtype, prefix)
        for t in range(T):
            row = (pool.prefix_list if t < prefix else pool.table_list[0])[t // 64], slice(None), t % 64
            pool.k[row], pool.v[row] = k[t], v[t]
        check_attention(pool.step(q[T - 5:], [T - 5], starts([5])), [x[T - 5:] for x in ref], T, f"step {prefix}")


# ---- rows that do not see them ------------------------------------------------------------------


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("what", [NAN, INF, -INF])
def test_rows_before_bad_values(what, D):
    """Bad values of several tokens of one tile, in one channel or in all: each row has those that it sees."""
    T, Hq, Hkv = 600, 8, 2
    q, k, v = _prompt(T, Hq, Hkv, D)
    clean = v.clone()
    v[300, 0, 7], v[333, 0, 9], v[333, 1], v[340, 0, 7] = what, what, what, what
    cu = starts([T])
    o, good = gdr.attn_fwd(q, k, v, cu), gdr.attn_fwd(q, k, clean, cu)
    hit = torch.zeros(o.shape, dtype=torch.bool, device=DEV)
    hit[300:, :4, 7], hit[333:, :4, 9], hit[333:, 4:] = True, True, True
    assert not torch.isfinite(o[hit]).any()
    assert (o[300, :4, 7] == what).all() or what != what
    ref = [x.copy() for x in oracle.attn_fwd(q, k, clean, cu, D ** -0.5)]
    ref[0][hit.cpu().numpy()] = NAN
    check_attention(o, ref, T)
    assert bits_equal(o[:128], good[:128])  # row tiles before the tokens' key tile are as they were


@pytest.mark.parametrize("prefix", [0, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("m", [5, 40])
def test_step_rows_before_bad_values(m, D, prefix):
    """The same of several tokens over the cache; one sequence ends within the prefix."""
    lens, lengths = [500, 60], [m, 3]
    cu = starts(lengths)
    pool = Pool(3, [a + n for a, n in zip(lens, lengths)], 2, D, 64, BF16, prefix)
    q = normal(2, m + 3, 8, D, dtype=BF16)
    ref = [x.copy() for x in pool.reference(q, lens, cu)]

    def at(n, t):
        return (pool.prefix_list if t < prefix else pool.table_list[n])[t // 64], 0, t % 64

    pool.v[at(0, 503)][7] = NAN
    pool.v[at(1, 62)][9] = NAN  # with a prefix its token 62, which the first sequence sees as well
    o = pool.step(q, lens, cu)
    hit = torch.zeros(o.shape, dtype=torch.bool, device=DEV)
    hit[3:m, :4, 7], hit[m + 2, :4, 9] = True, True
    if prefix:
        hit[:m, :4, 9] = True
    assert torch.isnan(o[hit]).all()
    ref[0][hit.cpu().numpy()] = NAN
    check_attention(o, ref, 600)
