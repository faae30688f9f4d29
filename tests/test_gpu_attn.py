"""Causal attention over packed prompts, and over the paged cache, against the fp64 oracle."""
import numpy as np
import pytest
import torch

import gated_delta_rule_37_gb300 as gdr
import oracle
from tests.attn_util import DEV, Pool, check_attention, ints, normal, starts
from tests.gpu_util import Guarded, bits_equal, sentinel_like

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _reference(q, k, v, cu, scale=None):
    return oracle.attn_fwd(q, k, v, cu, q.shape[2] ** -0.5 if scale is None else scale)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lengths,Hq,Hkv", [
    ([1], 1, 1),
    ([1, 2, 0, 63, 64, 65], 2, 2),
    ([127, 128, 129, 1, 0], 4, 2),
    ([255, 257, 3], 3, 1),            # a group that does not divide the tile
    ([200, 31], 14, 2),
    ([33, 150], 8, 1),
    ([40], 128, 1),                   # a row tile for every token
    ([5, 1, 7, 2], 200, 2),           # 100 rows a token
])
def test_prompt_matches_oracle(lengths, Hq, Hkv, D, dtype):
    T, cu = sum(lengths), starts(lengths)
    q, k, v = normal(1, T, Hq, D, dtype=dtype, std=2.0), normal(2, T, Hkv, D, dtype=dtype), normal(3, T, Hkv, D, dtype=dtype)
    o = gdr.attn_fwd(q, k, v, cu, flags=gdr.GDR_VALIDATE)
    check_attention(o, _reference(q, k, v, cu), max(lengths), "prompt")
    assert bits_equal(o, gdr.attn_fwd(q, k, v, cu))


@pytest.mark.parametrize("Hq,Hkv", [(14, 2), (8, 8), (64, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_many_short_sequences(Hq, Hkv, D):
    """Many times more row tiles than the GPU has CTAs, of one to five key tiles: whole problems fit into the copies'
    ring, which is then ahead by more than one."""
    lengths = [(37 * i) % 150 + 1 if i % 9 else 600 - i for i in range(400)]
    T, cu = sum(lengths), starts(lengths)
    q, k, v = normal(1, T, Hq, D, dtype=BF16, std=2.0), normal(2, T, Hkv, D, dtype=BF16), normal(3, T, Hkv, D, dtype=BF16)
    o = gdr.attn_fwd(q, k, v, cu)
    assert gdr.device_status() == 0
    for n in range(0, 400, 13):
        part = slice(sum(lengths[:n]), sum(lengths[:n + 1]))
        check_attention(o[part], _reference(q[part], k[part], v[part], starts(lengths[n:n + 1])), lengths[n], str(n))
    for _ in range(5):
        assert bits_equal(o, gdr.attn_fwd(q, k, v, cu))
    assert gdr.device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_rows_behind_and_strides(dtype):
    """Column blocks of one projection, rows behind the last sequence (of NaN), redzones, a scale of its own."""
    T, Hq, Hkv, D = 150, 4, 2, 128
    rows = normal(4, T + 9, (Hq + 2 * Hkv) * D, dtype=dtype)
    rows[T:] = float("nan")
    q, k, v = (rows[:, a * D:b * D].unflatten(1, (-1, D)) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    cu = starts([100, 50])
    out = Guarded((T + 9, Hq * D + 16), dtype, DEV, sentinel_like((T + 9, Hq * D + 16), dtype))
    kept = out.view.clone()
    o = out.view[:, :Hq * D].unflatten(1, (Hq, D))
    gdr.attn_fwd(q, k, v, cu, scale=0.3, o=o)
    check_attention(o[:T], _reference(q[:T], k[:T], v[:T], cu, 0.3), 100)
    assert out.guards_intact() and bits_equal(out.view[T:], kept[T:])
    assert bits_equal(out.view[:, Hq * D:].contiguous(), kept[:, Hq * D:].contiguous())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_prompt_keeps_bad_values_to_the_rows_that_see_them(dtype, what):
    lengths = [90, 200, 60]
    T, cu = sum(lengths), starts(lengths)
    q, k, v = normal(1, T, 4, 64, dtype=dtype), normal(2, T, 2, 64, dtype=dtype), normal(3, T, 2, 64, dtype=dtype)
    clean = gdr.attn_fwd(q, k, v, cu)
    bad = 90 + 70  # a token inside a tile of the second sequence
    kb, vb = k.clone(), v.clone()
    kb[bad, 0, 5] = what
    vb[bad, 1, 7] = what
    o = gdr.attn_fwd(q, kb, vb, cu)
    rows = torch.ones(T, dtype=torch.bool, device=DEV)
    rows[bad:290] = False
    assert torch.isfinite(o[rows]).all()
    check_attention(o[:90], _reference(q[:90], k[:90], v[:90], starts([90])), 90)
    check_attention(o[90:bad], _reference(q[90:bad], k[90:bad], v[90:bad], starts([70])), 200)
    assert bits_equal(o[290:], clean[290:])
    assert not torch.isfinite(o[bad:290, 2:, 7]).any()  # the value is seen from its token on
    finite = torch.arange(64, device=DEV) != 7
    assert torch.isfinite(o[90:290, 2:][..., finite]).all()
    if what != what:
        assert torch.isnan(o[bad:290, :2]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_large_scores(dtype):
    """Scores of hundreds, growing along the keys so that the maximum moves in every tile, and equal ones."""
    T = 400
    q, k, v = normal(1, T, 2, 128, dtype=dtype), normal(2, T, 2, 128, dtype=dtype), normal(3, T, 2, 128, dtype=dtype)
    cu = starts([T])
    ramp = (q.float().mean(0, keepdim=True).sign() * torch.linspace(0, 3, T, device=DEV)[:, None, None]).to(dtype)
    q2 = (q.float().mean(0, keepdim=True).sign().expand(T, 2, 128) * 2).to(dtype)
    check_attention(gdr.attn_fwd(q2, ramp, v, cu), _reference(q2, ramp, v, cu), T, "growing")
    check_attention(gdr.attn_fwd(q2, -ramp, v, cu), _reference(q2, -ramp, v, cu), T, "falling")
    zero = torch.zeros_like(k)
    check_attention(gdr.attn_fwd(q, zero, v, cu), _reference(q, zero, v, cu), T, "equal")
    far = torch.full_like(k, 1e30)
    far[:, :, 1:] = 0
    neg = torch.full_like(q, -1e6)  # every score far below fp32's exponentials of 0: the row's own maximum counts
    check_attention(gdr.attn_fwd(neg, (far * 1e-27).to(dtype), v, cu), _reference(neg, (far * 1e-27).to(dtype), v, cu), T)


# ---- the step over the cache ---------------------------------------------------

STEPS = [
    # lengths, lens, Hq, Hkv, page, prefix
    ([1], [0], 1, 1, 16, 0),
    ([1] * 5, [0, 5, -1, 63, 64], 4, 2, 16, 0),
    ([1, 1, 1], [300, 1000, 17], 8, 1, 64, 0),
    ([4, 1, 0, 12, 7], [100, 0, 5, 250, -1], 8, 2, 32, 0),
    ([1] * 6, [100, 101, 140, -1, 99, 100], 4, 1, 16, 100),
    ([3, 12, 1], [130, 128, 700], 6, 2, 128, 128),
    ([5, 2], [10, 300], 7, 1, 64, 200),          # a sequence that ends within the prefix
    ([70, 130], [0, 33], 4, 2, 256, 0),          # many rows of a sequence
    ([1, 1], [2000, 3], 16, 16, 32, 0),
    ([1] * 40, [400 + i for i in range(40)], 14, 2, 64, 390),
    ([1], [5000], 128, 1, 64, 0),
    ([2, 1], [900, 800], 2, 2, 64, 777),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("case", range(len(STEPS)))
def test_step_matches_oracle(case, D, dtype):
    lengths, lens, Hq, Hkv, page, prefix = STEPS[case]
    T, cu = sum(lengths), starts(lengths)
    ends = [a + n if a >= 0 and n else 0 for a, n in zip(lens, lengths)]
    pool = Pool(case, ends, Hkv, D, page, dtype, prefix)
    q = normal(9, T + 3, Hq, D, dtype=dtype, std=2.0)
    out = Guarded((T + 3, Hq, D), dtype, DEV, sentinel_like((T + 3, Hq, D), dtype))
    kept = out.view.clone()
    need = gdr.attn_step_workspace_size(len(lens), T + 3, Hq, Hkv, D, prefix_len=prefix,
                                        dtype=gdr.GDR_BF16 if dtype == BF16 else gdr.GDR_F32)
    ws = Guarded((need,), torch.uint8, DEV)
    ws.view.fill_(255)  # a workspace of NaN
    o = pool.step(q, lens, cu, o=out.view, workspace=ws.view, flags=gdr.GDR_VALIDATE)
    ref = pool.reference(q, lens, cu)
    check_attention(o, ref, max(ends), "step")
    skipped = torch.isnan(torch.from_numpy(ref[0]))
    assert bits_equal(o.cpu()[skipped], kept.cpu()[skipped])
    assert out.guards_intact() and ws.guards_intact()
    assert bits_equal(o, pool.step(q, lens, cu, o=kept.clone()))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_step_cut_into_many_runs(dtype):
    """One long sequence beside short ones: its keys lie in many CTAs' runs, with and without a prefix."""
    lens, lengths = [20000, 3, 511], [1, 2, 1]
    cu = starts(lengths)
    for prefix in (0, 3):
        pool = Pool(7, [a + n for a, n in zip(lens, lengths)], 2, 64, 64, dtype, prefix)
        q = normal(3, 4, 8, 64, dtype=dtype, std=2.0)
        check_attention(pool.step(q, lens, cu), pool.reference(q, lens, cu), 20001)


@pytest.mark.parametrize("group,D", [(4, 128), (4, 64), (20, 128), (40, 128), (40, 64)])
def test_step_long_runs(group, D):
    """Runs of many tiles per CTA, many times over: the copies' ring laps often, and every call gives the same bits."""
    Hkv, lens = 4, [60000, 25000]
    cu = starts([1, 1])
    pool = Pool(5, [a + 1 for a in lens], Hkv, D, 64, BF16)
    q = normal(3, 2, Hkv * group, D, dtype=BF16, std=2.0)
    o = pool.step(q, lens, cu)
    for n, a in enumerate(lens):
        k, v = (c[pool.table[n, :-(-(a + 1) // 64)].long()].transpose(1, 2).flatten(0, 1)[:a + 1].double()
                for c in (pool.k, pool.v))
        s = torch.einsum("hgd,jhd->hgj", q[n].double().view(Hkv, group, D), k) * D ** -0.5
        p = torch.softmax(s, -1)
        ref = torch.einsum("hgj,jhd->hgd", p, v).view(1, -1, D)
        weight = torch.einsum("hgj,jhd->hgd", p, v.abs()).view(1, -1, D)
        score = torch.einsum("hgd,jhd->hgj", q[n].double().view(Hkv, group, D).abs(), k.abs()).amax(-1) * D ** -0.5
        check_attention(o[n:n + 1], [x.cpu().numpy() for x in (ref, weight, score.view(1, -1))], a + 1)
    for _ in range(40):
        assert bits_equal(o, pool.step(q, lens, cu))
    assert gdr.device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("prefix", [0, 70])
def test_step_leaves_unwritten_cache_rows_alone(dtype, prefix):
    """Everything that no row sees is NaN: rows behind a sequence's end in its last page, other pages, and of a
    verify's later tokens what the earlier ones do not see."""
    lens, lengths, Hkv, D, page = [75, 100, 70], [1, 9, 3], 2, 128, 32
    cu = starts(lengths)
    pool = Pool(11, [a + n for a, n in zip(lens, lengths)], Hkv, D, page, dtype, prefix)
    full = (pool.k.clone(), pool.v.clone())
    pool.k.fill_(float("nan"))
    pool.v.fill_(float("nan"))
    for n, (a, m) in enumerate(zip(lens, lengths)):
        for p in range(a + m):
            pages = pool.prefix_list if p < prefix else pool.table_list[n]
            at = pages[p // page], slice(None), p % page
            pool.k[at], pool.v[at] = full[0][at], full[1][at]
    q = normal(3, sum(lengths), 4, D, dtype=dtype)
    ref = pool.reference(q, lens, cu)
    check_attention(pool.step(q, lens, cu), ref, 110)
    # the last token of the second sequence holds an infinity: only its own row sees it
    at = pool.table_list[1][108 // page], 1, 108 % page, 5
    pool.v[at] = float("inf")
    o = pool.step(q, lens, cu)
    hit = torch.zeros(o.shape, dtype=torch.bool, device=DEV)
    hit[9, 2:, 5] = True
    assert (o[hit] == float("inf")).all()
    check_attention(torch.where(hit, 0, o), (np.where(hit.cpu(), 0, ref[0]), ref[1], ref[2]), 110)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_step_pages_that_are_missing(dtype):
    """Keys without a page are not seen; a row that sees none is 0; validation names them."""
    pool = Pool(2, [100, 40, 60], 1, 64, 16, dtype)
    table = pool.table.clone()
    table[0, 2], table[0, 4] = -1, pool.k.shape[0]
    table[1, :] = -5
    pool.table, pool.table_list = table, table.tolist()
    lens, cu = [99, 39, 200], starts([1, 1, 1])  # the third: longer than its table
    q = normal(1, 3, 4, 64, dtype=dtype)
    o = pool.step(q, lens, cu)
    check_attention(o, pool.reference(q, lens, cu), 100)
    assert (o[1] == 0).all()
    with pytest.raises(gdr.GdrError, match="page number outside.*longer"):
        pool.step(q, lens, cu, flags=gdr.GDR_VALIDATE)


def test_step_prefix_is_the_same_as_pages_of_each():
    """With the prefix's pages in every row of the table the result is the same operator."""
    lens, Hkv, D, page, prefix = [500, 640, 530, 512], 2, 128, 64, 512
    pool = Pool(4, [a + 2 for a in lens], Hkv, D, page, F32, prefix)
    cu, q = starts([2] * 4), normal(5, 8, 8, D, std=2.0)
    shared = pool.step(q, lens, cu)
    pool.table[:, :8] = pool.prefix_pages
    pool.prefix_pages, pool.prefix_len = None, 0
    apart = pool.step(q, lens, cu)
    assert (shared - apart).abs().max() < 1e-5


def test_offsets_beyond_32_bits():
    """A cache of more than 2^31 elements, the sequence in its last pages."""
    pages, page, Hkv, D = 70000, 256, 1, 128
    k = torch.empty(pages, Hkv, page, D, dtype=BF16, device=DEV)
    v = torch.empty(pages, Hkv, page, D, dtype=BF16, device=DEV)
    used = [pages - 1, 3, pages - 2]
    for i, p in enumerate(used):
        k[p], v[p] = normal(i, Hkv, page, D, dtype=BF16), normal(i + 10, Hkv, page, D, dtype=BF16)
    small = Pool(1, [3 * page], Hkv, D, page, BF16, spare=0)
    small.table_list = [[0, 1, 2]]
    small.table = ints(small.table_list)
    small.k, small.v = k[used].clone(), v[used].clone()
    q = normal(5, 2, 8, D, dtype=BF16)
    cu = starts([2])
    o = gdr.attn_step(q, k, v, ints([used]), ints([700]), cu)
    check_attention(o, small.reference(q, [700], cu), 702)
    new = normal(6, 2, 1, D, dtype=BF16)
    gdr.kv_append(new, new, k, v, ints([used]), ints([700]), cu)
    assert bits_equal(k[used[2], 0, 700 - 512:702 - 512], new[:, 0])


# ---- the layer as it is used -----------------------------------------------------


def _freqs(R):
    return (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float().to(DEV)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefill_then_decode_equals_the_whole_prompt(dtype):
    """append + prompt attention over the first tokens, then append + step for the rest, a few at a time, against the
    prompt attention over everything."""
    Hq, Hkv, D, page, N = 8, 2, 128, 32, 3
    first, steps = [70, 33, 128], [1, 4, 1, 7]
    total = [a + sum(steps) for a in first]
    f = _freqs(D)
    q, k, v = ([normal(s * 10 + n, t, H, D, dtype=dtype) for n, t in enumerate(total)]
               for s, H in ((1, Hq), (2, Hkv), (3, Hkv)))
    whole = Pool(1, total, Hkv, D, page, dtype)
    qa, ka = gdr.kv_append(torch.cat(k), torch.cat(v), whole.k, whole.v, whole.table, ints([0] * N), starts(total),
                           q=torch.cat(q), freqs=f, output_k=True)
    full = gdr.attn_fwd(qa, ka, torch.cat(v), starts(total))
    ref = _reference(qa, ka, torch.cat(v), starts(total))
    check_attention(full, ref, max(total))
    base = np.cumsum([0, *total])
    pool = Pool(2, total, Hkv, D, page, dtype, fill=float("nan"))
    at, got = [0] * N, []
    for i, m in enumerate([None, *steps]):
        take = first if m is None else [m] * N
        part = [torch.cat([x[n][at[n]:at[n] + take[n]] for n in range(N)]) for x in (q, k, v)]
        cu, lens = starts(take), ints(at)
        qo, ko = gdr.kv_append(part[1], part[2], pool.k, pool.v, pool.table, lens, cu, q=part[0], freqs=f,
                               output_k=i == 0)
        o = gdr.attn_fwd(qo, ko, part[2], cu) if i == 0 else gdr.attn_step(qo, pool.k, pool.v, pool.table, lens, cu)
        rows = np.concatenate([base[n] + at[n] + np.arange(take[n]) for n in range(N)])
        check_attention(o, [x[rows] for x in ref], max(total), f"part {i}")
        at = [a + b for a, b in zip(at, take)]
        got.append(o)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_captured_step_replays_with_other_lengths(dtype):
    """A graph of append and step, replayed as the sequences grow, on a stream of its own; two graphs share nothing."""
    N, Hq, Hkv, D, page, prefix = 4, 8, 2, 64, 16, 40
    lens = [45, 100, -1, 60]
    pool = Pool(3, [a + 8 if a >= 0 else 0 for a in lens], Hkv, D, page, dtype, prefix)
    eager = Pool(3, [a + 8 if a >= 0 else 0 for a in lens], Hkv, D, page, dtype, prefix)
    live, cu = ints(lens), starts([1] * N)
    q, k, v = normal(1, N, Hq, D, dtype=dtype), normal(2, N, Hkv, D, dtype=dtype), normal(3, N, Hkv, D, dtype=dtype)
    f = _freqs(D)
    qo, o = torch.zeros_like(q), torch.zeros_like(q)

    def step(c, n, o):
        gdr.kv_append(k, v, c.k, c.v, c.table, n, cu, q=q, freqs=f, q_out=qo)
        return gdr.attn_step(qo, c.k, c.v, c.table, n, cu, prefix_pages=c.prefix_pages, prefix_len=prefix, o=o)

    step(pool, live, o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(pool, live, o)
    for i in range(6):
        q.copy_(normal(20 + i, N, Hq, D, dtype=dtype))
        k.copy_(normal(30 + i, N, Hkv, D, dtype=dtype))
        graph.replay()
        want = step(eager, live.clone(), torch.zeros_like(q))
        assert bits_equal(o, want)
        live += (live >= 0).to(torch.int32)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_two_streams_at_once(dtype):
    lens, cu = [3000, 2000], starts([1, 1])
    pool = Pool(1, [3001, 2001], 2, 64, 64, dtype, 1000)
    q = [normal(i, 2, 8, 64, dtype=dtype) for i in range(2)]
    want = [pool.step(x, lens, cu) for x in q]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in q]
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            got[i].append(pool.step(q[i], lens, cu, stream=side[i]))
    torch.cuda.synchronize()
    assert all(bits_equal(o, want[i]) for i in range(2) for o in got[i])


def test_no_sequences_or_tokens():
    pool = Pool(1, [5], 1, 64, 16, BF16)
    q, k = torch.empty(0, 2, 64, dtype=BF16, device=DEV), torch.empty(0, 1, 64, dtype=BF16, device=DEV)
    none = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert gdr.attn_fwd(q, k, k, none).shape == (0, 2, 64)
    assert gdr.attn_fwd(q, k, k, ints([0, 0])).shape == (0, 2, 64)
    assert pool.step(q, [3], ints([0, 0])).shape == (0, 2, 64)
    q = normal(1, 3, 2, 64, dtype=BF16)
    o = torch.full_like(q, 3.0)
    assert (pool.step(q, [-1], ints([0, 3]), o=o) == 3.0).all()
    assert (pool.step(q, [2], ints([0, 0]), o=o) == 3.0).all()
    assert (gdr.attn_fwd(q, q, q, ints([0, 0]), o=o) == 3.0).all()
