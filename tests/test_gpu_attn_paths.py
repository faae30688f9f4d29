"""Calls of the attention layer that its documentation allows and that take other ways through the kernels: many and
empty sequences, tokens that share a row, captured prompts, streams at once, lengths beyond the table, rows that are
computed once more."""
import numpy as np
import pytest
import torch

import gated_delta_rule_37_gb300 as gdr
import oracle
from tests.attn_util import DEV, Pool, check_attention, ints, normal, starts
from tests.gpu_util import bits_equal

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _reference(q, k, v, cu, scale=None):
    return oracle.attn_fwd(q, k, v, cu, q.shape[2] ** -0.5 if scale is None else scale)


@pytest.fixture(autouse=True)
def _no_wait_gave_up():
    yield
    assert gdr.device_status() == 0


# ---- sequences -------------------------------------------------------------------


@pytest.mark.parametrize("N", [64, 65, 1000])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 1, 64), (3, 3, 128)])
def test_prompt_of_mostly_empty_sequences(N, Hq, Hkv, D):
    """Up to 64 sequences are taken in the order of their lengths, more by search; most are empty here."""
    lengths = [0] * N
    for i, n in enumerate((1, 130, 17, 257, 64, 1, 300)):
        lengths[(i * 37 + 5) % N] = n
    lengths[N - 1] = 33
    T, cu = sum(lengths), starts(lengths)
    q, k, v = normal(1, T + 5, Hq, D, dtype=BF16), normal(2, T + 5, Hkv, D, dtype=BF16), normal(3, T + 5, Hkv, D, dtype=BF16)
    o = torch.full_like(q, 7.0)
    gdr.attn_fwd(q, k, v, cu, o=o, flags=gdr.GDR_VALIDATE)
    check_attention(o[:T], _reference(q[:T], k[:T], v[:T], cu), 300)
    assert (o[T:] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("prefix", [0, 150])
def test_step_of_many_sequences(dtype, prefix):
    """More sequences than a block has threads: empty ones, padding, some within the prefix."""
    N, Hq, Hkv, D = 700, 2, 1, 64
    lengths = [(0, 1, 1, 2)[i * 7 % 4] if i % 5 else 0 for i in range(N)]
    lens = [-1 if i % 11 == 3 else (i * 29) % 190 for i in range(N)]
    T, cu = sum(lengths), starts(lengths)
    pool = Pool(8, [a + n if a >= 0 and n else 0 for a, n in zip(lens, lengths)], Hkv, D, 16, dtype, prefix)
    q = normal(9, T, Hq, D, dtype=dtype, std=2.0)
    o = torch.full_like(q, 5.0)
    pool.step(q, lens, cu, o=o, flags=gdr.GDR_VALIDATE)
    ref = pool.reference(q, lens, cu)
    check_attention(o, ref, 192)
    assert (o.cpu()[torch.isnan(torch.from_numpy(ref[0]))] == 5.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_step_within_the_prefix(dtype):
    """No sequence has a key of its own."""
    lens, lengths = [10, 0, 150, 197], [3, 1, 2, 2]
    pool = Pool(4, [0] * 4, 2, 128, 32, dtype, 200)
    q, cu = normal(9, 8, 6, 128, dtype=dtype, std=2.0), starts(lengths)
    check_attention(pool.step(q, lens, cu), pool.reference(q, lens, cu), 200)


@pytest.mark.parametrize("T,Hq,Hkv,prefix,page", [
    (1, 4, 1, 9000, 64),      # one row tile, cut along the keys as often as it may be
    (1300, 32, 32, 130, 16),  # more blocks of rows than CTAs: several of each
    (70, 12, 4, 1, 256),      # a prefix of one key
    (33, 16, 2, 1000, 128),
])
@pytest.mark.parametrize("D", [64, 128])
def test_prefix_shared_out_over_the_gpu(T, Hq, Hkv, prefix, page, D):
    """Against the fp64 softmax over the prefix and the one or two keys behind it (checked on some rows)."""
    N = max(1, T // 2)
    lengths = [T // N + (i < T % N) for i in range(N)]
    lens = [prefix] * N
    pool = Pool(3, [a + n for a, n in zip(lens, lengths)], Hkv, D, page, BF16, prefix)
    q, cu = normal(5, T, Hq, D, dtype=BF16, std=2.0), starts(lengths)
    o = pool.step(q, lens, cu)
    assert bits_equal(o, pool.step(q, lens, cu))
    first = np.cumsum([0, *lengths])
    for n in {0, N // 3, N // 2, N - 1}:
        part = slice(first[n], first[n + 1])
        pages = (prefix + lengths[n] - 1) // page + 1
        k, v = (torch.cat([c[p].transpose(0, 1) for p in
                           [pool.prefix_list[i] if (i + 1) * page <= prefix or i * page < prefix and
                            pool.table_list[n][i] < 0 else pool.table_list[n][i] for i in range(pages)]])
                for c in (pool.k, pool.v))
        # the page that the prefix ends in: its keys from the prefix's, the others from the sequence's
        cut = prefix // page * page
        if cut < prefix:
            for x, c in ((k, pool.k), (v, pool.v)):
                x[cut:prefix] = c[pool.prefix_list[-1]].transpose(0, 1)[:prefix - cut]
        m = lengths[n]
        k, v = k[:prefix + m].double(), v[:prefix + m].double()
        qs = q[part].double().view(m, Hkv, -1, D)
        s = torch.einsum("mhgd,jhd->mhgj", qs, k) * D ** -0.5
        late = torch.arange(prefix + m, device=DEV) > torch.arange(prefix, prefix + m, device=DEV)[:, None]
        p = torch.softmax(s.masked_fill(late[:, None, None], -np.inf), -1)
        ref = torch.einsum("mhgj,jhd->mhgd", p, v).reshape(m, Hq, D)
        weight = torch.einsum("mhgj,jhd->mhgd", p, v.abs()).reshape(m, Hq, D)
        score = torch.einsum("mhgd,jhd->mhgj", qs.abs(), k.abs()).amax(-1).reshape(m, Hq) * D ** -0.5
        check_attention(o[part], [x.cpu().numpy() for x in (ref, weight, score)], prefix + m, str(n))


def test_prefix_pages_that_are_missing():
    lens, cu = [301, 310], starts([1, 2])
    pool = Pool(2, [302, 312], 1, 128, 16, BF16, 290)
    pages = pool.prefix_pages.clone()
    pages[3], pages[9], pages[18] = -1, pool.k.shape[0], -7
    pool.prefix_pages, pool.prefix_list = pages, pages.tolist()
    q = normal(1, 3, 4, 128, dtype=BF16)
    check_attention(pool.step(q, lens, cu), pool.reference(q, lens, cu), 312)
    with pytest.raises(gdr.GdrError, match="prefix page"):
        pool.step(q, lens, cu, flags=gdr.GDR_VALIDATE)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_lengths_beyond_the_table(dtype):
    """A length near 2^31: the keys that have a place are seen, the others are not there."""
    pool = Pool(2, [96, 40], 2, 64, 32, dtype, spare=0)
    cu, q = starts([3, 1]), normal(1, 4, 8, 64, dtype=dtype)
    o = pool.step(q, [2 ** 31 - 2, 39], cu)
    for t in range(3):
        check_attention(o[t:t + 1], pool.reference(q[t:t + 1], [95], starts([1])), 96, str(t))
    check_attention(o[3:], Pool.reference(_only(pool, 1), q[3:], [39], starts([1])), 40)
    k = normal(3, 4, 2, 64, dtype=dtype)
    before = pool.k.clone()
    gdr.kv_append(k[:3], k[:3], pool.k, pool.v, pool.table[:1], ints([2 ** 31 - 2]), starts([3]))
    assert bits_equal(before, pool.k)


def _only(pool, n):
    other = object.__new__(Pool)
    other.__dict__.update(pool.__dict__)
    other.table = pool.table[n:n + 1]
    return other


# ---- tensors -----------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128])
def test_tokens_that_share_a_row(dtype, D):
    """Inputs that are one row for all tokens (a token stride of 0), or rows that overlap (half a row apart)."""
    T, Hq, Hkv = 90, 4, 2
    cu = starts([50, 40])
    one = normal(1, 1, Hkv, D, dtype=dtype).expand(T, Hkv, D)
    flat = normal(2, (T + 1) * Hkv * D // 2, dtype=dtype)
    half = flat.as_strided((T, Hkv, D), (Hkv * D // 2, D, 1))
    q = normal(3, T, Hq, D, dtype=dtype)
    q1 = normal(4, 1, Hq, D, dtype=dtype).expand(T, Hq, D)
    for a, b, c in ((q, one, half), (q, half, one), (q1, half, half)):
        check_attention(gdr.attn_fwd(a, b, c, cu), _reference(a, b, c, cu), 50)
    pool = Pool(3, [70 + 6, 90 + 6], Hkv, D, 32, dtype, 40)
    lens, cu = [70, 90], starts([6, 6])
    check_attention(pool.step(q1[:12], lens, cu), pool.reference(q1[:12], lens, cu), 96)
    k, v = gdr.kv_append(one[:12], half[:12], pool.k, pool.v, pool.table, ints(lens), cu, output_k=True)[1], half[:12]
    assert bits_equal(k, one[:12].contiguous())
    row = pool.table_list[1][90 // 32], slice(None), 90 % 32
    assert bits_equal(pool.v[row].contiguous(), v[6].contiguous())


# ---- rows that are computed once more ------------------------------------------------


@pytest.mark.parametrize("D", [64, 128])
def test_an_early_nan_reaches_one_channel_of_all_later_rows(D):
    """Every row of the prompt and of the step behind it is computed once more, by many CTAs at once."""
    T, Hq, Hkv = 700, 8, 2
    q, k, v = normal(1, T, Hq, D, dtype=BF16), normal(2, T, Hkv, D, dtype=BF16), normal(3, T, Hkv, D, dtype=BF16)
    v[1, 0, 3] = float("nan")
    cu = starts([T])
    o = gdr.attn_fwd(q, k, v, cu)
    assert torch.isnan(o[1:, :4, 3]).all()
    clean = v.clone()
    clean[1, 0, 3] = 0
    keep = np.ones((T, Hq, D), bool)
    keep[1:, :4, 3] = False
    ref = [x.copy() for x in _reference(q, k, clean, cu)]
    ref[0][~keep] = np.nan
    check_attention(o, ref, T)
    pool = Pool(1, [T + 4], Hkv, D, 64, BF16, 128)
    pool.v[pool.prefix_list[0], 0, 1, 3] = float("nan")
    a = pool.step(q[:4], [T], starts([4]))
    assert torch.isnan(a[:, :4, 3]).all()
    pool.v[pool.prefix_list[0], 0, 1, 3] = 0
    ref = [x.copy() for x in pool.reference(q[:4], [T], starts([4]))]
    ref[0][:, :4, 3] = np.nan
    check_attention(a, ref, T + 4)


def test_scores_of_minus_infinity_alone():
    """A row all of whose scores are -inf is 0, in each path; one with a finite score has only that."""
    for dtype in (BF16, F32):
        q = torch.ones(40, 2, 64, dtype=dtype, device=DEV)
        k, v = normal(1, 40, 1, 64, dtype=dtype), normal(2, 40, 1, 64, dtype=dtype)
        k[:20, 0, 0] = -float("inf")
        o = gdr.attn_fwd(q, k, v, starts([40]))
        assert (o[:20] == 0).all()
        check_attention(o[20:], _reference(q[20:], k[20:], v[20:], starts([20])), 20)
        pool = Pool(1, [40], 1, 64, 16, dtype)
        for t in range(40):
            row = pool.table_list[0][t // 16], slice(None), t % 16
            pool.k[row], pool.v[row] = k[t], v[t]
        o = torch.cat([pool.step(q[:1], [19], starts([1])), pool.step(q[:1], [20], starts([1]))])
        assert (o[0] == 0).all()
        check_attention(o[1:], _reference(q[20:21], k[20:21], v[20:21], starts([1])), 1)


# ---- streams and graphs ----------------------------------------------------------------


def test_prompts_captured_and_on_two_streams():
    """Two graphs of prompts of many row tiles, replayed at once and beside an eager call."""
    Hq, Hkv, D = 14, 2, 64
    lengths = [(i * 53) % 200 + 1 for i in range(100)]
    T, cu = sum(lengths), starts(lengths)
    x = [[normal(i * 3 + j, T, H, D, dtype=BF16) for j, H in enumerate((Hq, Hkv, Hkv))] for i in range(3)]
    want = [gdr.attn_fwd(*a, cu) for a in x]
    out = [torch.zeros_like(a[0]) for a in x]
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                gdr.attn_fwd(*x[i], cu, o=out[i])
        graphs.append(g)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        for i, g in enumerate(graphs):
            with torch.cuda.stream(side[i]):
                g.replay()
        gdr.attn_fwd(*x[2], cu, o=out[2], stream=side[2])
    torch.cuda.synchronize()
    assert all(bits_equal(a, b) for a, b in zip(out, want))


def test_layer_in_place_in_one_projection():
    """q and k turned where they lie, column blocks of one projection's output, then the prompt over them."""
    T, Hq, Hkv, D = 130, 4, 2, 64
    rows = normal(1, T, (Hq + 2 * Hkv) * D, dtype=BF16)
    kept = rows.clone()
    q, k, v = (rows[:, a * D:b * D].unflatten(1, (-1, D)) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    f = (100.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().to(DEV)
    pool = Pool(1, [T], Hkv, D, 64, BF16)
    cu, zero = starts([T]), ints([0])
    qa, ka = gdr.kv_append(k.contiguous(), v.contiguous(), pool.k, pool.v, pool.table, zero, cu, q=q.contiguous(),
                           freqs=f, output_k=True)
    gdr.kv_append(k, v, pool.k, pool.v, pool.table, zero, cu, q=q, freqs=f, q_out=q, k_out=k)
    assert bits_equal(q.contiguous(), qa) and bits_equal(k.contiguous(), ka)
    assert bits_equal(rows[:, (Hq + Hkv) * D:].contiguous(), kept[:, (Hq + Hkv) * D:].contiguous())
    assert bits_equal(gdr.attn_fwd(q, k, v, cu), gdr.attn_fwd(qa, ka, v.contiguous(), cu))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv,D,R,pairs", [(2, 2, 128, 128, False), (8, 1, 64, 32, True), (0, 1, 64, 64, False),
                                              (16, 2, 128, 64, False)])
def test_append_of_many_tokens_is_that_of_few(Hq, Hkv, D, R, pairs, dtype):
    """Blocks that have several tokens give the bits of blocks that have one: rows behind the last sequence, empty
    sequences, padding, missing pages and places beyond the table among them."""
    page, N = 32, 61
    lengths = [(0, 1, 400, 7, 233, 64, 331)[i % 7] for i in range(N)]
    lens = [-1 if i % 10 == 4 else (i * 37) % 90 for i in range(N)]
    T, first = sum(lengths), np.cumsum([0, *lengths])
    assert T // 2 >= 152 * 8 and max(lengths) < 2 * 152 * 8
    width = max(-(-(a + n) // page) for a, n in zip(lens, lengths)) - 1  # the longest lacks its last page
    order = np.random.default_rng(1).permutation(N * width)
    table = torch.from_numpy(order.reshape(N, width).astype(np.int32)).to(DEV)
    table[3, 1], table[5, 0] = -1, N * width
    q, k, v = (normal(i, T + 5, H, D, dtype=dtype) if H else None for i, H in ((1, Hq), (2, Hkv), (3, Hkv)))
    f = normal(4, R // 2, std=0.3)
    flags = gdr.GDR_ROPE_PAIRS if pairs else 0

    def call(kc, vc, a, b, q_out, k_out):
        part = slice(first[a], first[b] if b < N else T + 5)
        cut = lambda t: None if t is None else t[part]
        gdr.kv_append(k[part], v[part], kc, vc, table[a:b], ints(lens[a:b]), starts(lengths[a:b]), q=cut(q), freqs=f,
                      flags=flags, q_out=cut(q_out), k_out=k_out[part])

    out = []
    for cuts in ([0, N], [*range(0, N, 4), N]):
        kc = torch.full((N * width, Hkv, page, D), 9.0, dtype=dtype, device=DEV)
        vc = kc.clone()
        q_out, k_out = (torch.full_like(t, 5.0) if t is not None else None for t in (q, k))
        for a, b in zip(cuts[:-1], cuts[1:]):
            call(kc, vc, a, b, q_out, k_out)
        out.append([t for t in (kc, vc, q_out, k_out) if t is not None])
    assert all(bits_equal(x, y) for x, y in zip(*out))
    assert (out[0][-1][T:] == 5.0).all() and (out[0][0] == 9.0).any()
