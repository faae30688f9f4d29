"""The paged cache's append with rotary positions against the fp64 oracle."""
import numpy as np
import pytest
import torch

import gated_delta_rule_37_gb300 as gdr
import oracle
from tests.attn_util import DEV, HALF, Pool, ints, normal, starts
from tests.gpu_util import bits_equal

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _freqs(R):
    return (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float().to(DEV) if R else None


def _close(got, ref, x, what):
    """A turned pair is two products and a sum in fp32 with sines off by 2^-22 (two steps of their own rounding, and
    the reduced angle's), rounded once: 2^-21 of the pair's magnitude and half a step of the result."""
    g, size = got.double().cpu().numpy(), np.abs(x.double().cpu().numpy()).max(-1, keepdims=True)
    live = ~np.isnan(ref)
    bound = HALF[got.dtype] * np.abs(ref) + 2.0 ** -21 * 2 * np.broadcast_to(size, ref.shape)
    assert (np.abs(g - ref) <= bound)[live].all(), f"{what}: {np.nanmax(np.abs(g - ref) / bound)}"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lengths,lens,Hq,Hkv,D,R,page,pairs", [
    ([1], [0], 2, 2, 64, 64, 16, False),
    ([1] * 9, [0, 1, 15, 16, 17, -1, 31, 100, 63], 8, 2, 128, 128, 16, False),
    ([5, 0, 1, 40, 3], [14, 3, 7, 30, -1], 12, 4, 64, 32, 16, False),
    ([130, 2], [0, 62], 7, 1, 128, 64, 64, True),
    ([3, 70], [5, 250], 6, 6, 128, 6, 128, True),
    ([20, 20], [5, 250], 2, 1, 64, 0, 256, False),
    ([300], [0], 14, 2, 64, 64, 32, False),
])
def test_append_matches_oracle(lengths, lens, Hq, Hkv, D, R, page, pairs, dtype):
    T, cu = sum(lengths), starts(lengths)
    pool = Pool(3, [max(0, a + n) if a >= 0 else 0 for a, n in zip(lens, lengths)], Hkv, D, page, dtype)
    before_k, before_v = pool.k.clone(), pool.v.clone()
    # two rows behind the last sequence, which stay as they were
    q, k, v = (normal(s, T + 2, H, D, dtype=dtype) for s, H in ((4, Hq), (5, Hkv), (6, Hkv)))
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    f = _freqs(R)
    got = gdr.kv_append(k, v, pool.k, pool.v, pool.table, ints(lens), cu, q=q, freqs=f,
                        flags=gdr.GDR_VALIDATE | (gdr.GDR_ROPE_PAIRS if pairs else 0), q_out=qo, k_out=ko)
    assert got[0] is qo and got[1] is ko
    rq, rk, rkc, rvc = oracle.kv_append(k, v, before_k, before_v, pool.table.cpu(), lens, cu, q=q,
                                        freqs=[] if f is None else f, pairs=pairs)
    _close(qo, rq, q, "q")
    _close(ko, rk, k, "k")
    for out, ref in ((qo, rq), (ko, rk)):
        assert (out[torch.isnan(torch.from_numpy(ref)).to(DEV)] == 7.0).all()
    # channels that do not turn, values and all other rows of the caches keep their bits
    if R < D:
        live = ~torch.isnan(torch.from_numpy(rq[..., 0]))
        assert bits_equal(qo[..., R:].cpu()[live], q[..., R:].cpu()[live])
    assert bits_equal(pool.v, torch.from_numpy(rvc).to(dtype))
    same = torch.from_numpy((rkc == before_k.double().cpu().numpy()).all(-1))
    assert bits_equal(pool.k.cpu()[same], before_k.cpu()[same])
    _close(pool.k, rkc, torch.full_like(pool.k, float(k.abs().max())), "k_cache")
    # the cached key is the dense one
    for n, (a, c) in enumerate(zip(lens, cu.tolist())):
        if a >= 0 and lengths[n]:
            p = oracle.cache_row(page, pool.table_list[n], a, pool.k.shape[0])
            assert bits_equal(pool.k[p[0], :, p[1]], ko[c])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_far_positions(dtype):
    """Positions up to 2^31 - 2: the angle is reduced exactly.  The far ones lie behind the table's only page, so
    that nothing of them is cached."""
    far = [0, 1, 1 << 16, (1 << 20) + 1, (1 << 24) + 1, (1 << 30) + 12345, (1 << 31) - 2]
    pool = Pool(1, [1] * len(far), 1, 128, 16, dtype)
    before = pool.k.clone()
    q, k = normal(1, len(far), 3, 128, dtype=dtype), normal(2, len(far), 1, 128, dtype=dtype)
    f = _freqs(128)
    qo, ko = gdr.kv_append(k, k, pool.k, pool.v, pool.table, ints(far), starts([1] * len(far)), q=q, freqs=f,
                           output_k=True)
    _close(qo, oracle.rotate(q, far, f), q, "q")
    _close(ko, oracle.rotate(k, far, f), k, "k")
    written = [pool.table_list[0][0], pool.table_list[1][0]]  # positions 0 and 1 alone have a row
    rest = [p for p in range(before.shape[0]) if p not in written]
    assert bits_equal(pool.k[rest], before[rest])


@pytest.mark.parametrize("R,pairs", [(128, False), (64, False), (62, True)])
def test_in_place_and_column_blocks(R, pairs):
    """q, k and v as column blocks of one projection's rows, turned in place."""
    T, Hq, Hkv, D = 50, 6, 2, 128
    rows = normal(9, T, (Hq + 2 * Hkv) * D, dtype=BF16)
    kept = rows.clone()
    q, k, v = (rows[:, a * D:b * D].unflatten(1, (-1, D)) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    pool = Pool(3, [60], Hkv, D, 16, BF16)
    flags = gdr.GDR_ROPE_PAIRS if pairs else 0
    kw = dict(freqs=_freqs(R), flags=flags)
    args = (pool.table, ints([10]), starts([T]))
    qo, ko = gdr.kv_append(k.contiguous(), v.contiguous(), pool.k, pool.v, *args, q=q.contiguous(), output_k=True, **kw)
    kc, vc = pool.k.clone(), pool.v.clone()
    pool.k.zero_(), pool.v.zero_()
    a, b = gdr.kv_append(k, v, pool.k, pool.v, *args, q=q, q_out=q, k_out=k, **kw)
    assert a is q and b is k
    assert bits_equal(q.contiguous(), qo) and bits_equal(k.contiguous(), ko)
    assert bits_equal(rows[:, (Hq + Hkv) * D:].contiguous(), kept[:, (Hq + Hkv) * D:].contiguous())
    used = pool.table_list[0]
    used = used[1:3]  # the pages whose rows all are new: positions 16 .. 47 of 10 .. 59
    assert bits_equal(pool.k[used], kc[used]) and bits_equal(pool.v[used], vc[used])


def test_bad_pages_are_left_out():
    """Page numbers outside the cache: the token's key is not written; validation names them."""
    pool = Pool(5, [1] * 4, 2, 64, 16, F32)
    before = pool.k.clone()
    k = normal(2, 4, 2, 64)
    bad = ints([[-1], [pool.k.shape[0]], [2 ** 31 - 1], [pool.spare[0]]])
    q, _ = gdr.kv_append(k, k, pool.k, pool.v, bad, ints([0, 0, 0, 3]), starts([1] * 4), q=k)
    assert bits_equal(q, k)
    changed = (pool.k != before).any(-1).any(1).nonzero().tolist()
    assert changed == [[pool.spare[0], 3]]
    with pytest.raises(gdr.GdrError, match="page number"):
        gdr.kv_append(k, k, pool.k, pool.v, bad, ints([0, 0, 0, 3]), starts([1] * 4), flags=gdr.GDR_VALIDATE)
    with pytest.raises(gdr.GdrError, match="longer"):
        gdr.kv_append(k, k, pool.k, pool.v, pool.table, ints([0, 16, 0, 0]), starts([1] * 4), flags=gdr.GDR_VALIDATE)
    with pytest.raises(gdr.GdrError, match="cu_seqlens"):
        gdr.kv_append(k, k, pool.k, pool.v, pool.table, ints([0] * 4), ints([0, 2, 1, 3, 4]), flags=gdr.GDR_VALIDATE)


def test_many_sequences():
    """More sequences than the search looks at in one trip, empty ones among them."""
    r = np.random.default_rng(0)
    lengths = r.integers(0, 3, 20000).tolist()
    T = sum(lengths)
    lens = r.integers(0, 15, 20000).tolist()
    cu = starts(lengths)
    k = torch.arange(T, device=DEV, dtype=F32)[:, None, None].expand(T, 1, 64).contiguous()
    table = torch.randperm(20000, generator=torch.Generator().manual_seed(1)).to(torch.int32)[:, None].to(DEV)
    kc, vc = torch.full((20000, 1, 32, 64), -1.0, device=DEV), torch.full((20000, 1, 32, 64), -1.0, device=DEV)
    gdr.kv_append(k, k, kc, vc, table, ints(lens), cu)
    want = torch.full((20000, 32), -1.0)
    t = 0
    for n, (a, b) in enumerate(zip(lens, lengths)):
        for i in range(b):
            want[n, a + i] = t
            t += 1
    want = want[torch.argsort(table[:, 0].cpu().long())]
    assert torch.equal(kc[:, 0, :, 0].cpu(), want) and torch.equal(vc[:, 0, :, 63].cpu(), want)
