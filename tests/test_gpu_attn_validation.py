"""GDR_VALIDATE of the attention step asks for no more than the step reads."""
import pytest
import torch

import gated_delta_rule_37_gb300 as gdr
from tests.attn_util import Pool, check_attention, ints, normal, starts
from tests.gpu_util import bits_equal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("prefix,lens,lengths", [
    (100, [89], [1]),               # ends within the prefix's last page
    (100, [99], [1]),               # with the prefix
    (100, [60, 130, 97], [3, 2, 3]),
    (70, [65, 10], [1, 1]),
])
def test_a_sequence_within_the_prefix_needs_no_page(prefix, lens, lengths, dtype):
    """The page that the prefix ends in is asked of the sequences that go beyond it alone."""
    page, cu = 64, starts(lengths)
    ends = [a + n for a, n in zip(lens, lengths)]
    pool = Pool(1, [e if e > prefix else 0 for e in ends], 2, 64, page, dtype, prefix)
    for n, e in enumerate(ends):
        if e <= prefix:
            assert all(p == -1 for p in pool.table_list[n])
    pool.table = torch.cat([pool.table, torch.full_like(pool.table, -1)], 1)  # the entry is there, and holds no page
    pool.table_list = pool.table.tolist()
    q = normal(2, sum(lengths), 4, 64, dtype=dtype)
    o = pool.step(q, lens, cu, flags=gdr.GDR_VALIDATE)
    check_attention(o, pool.reference(q, lens, cu), max(ends))
    assert bits_equal(o, pool.step(q, lens, cu))


def test_a_sequence_beyond_the_prefix_does():
    pool = Pool(1, [130, 0], 1, 64, 64, torch.bfloat16, 100)
    cu, q = starts([1, 1]), normal(2, 2, 2, 64, dtype=torch.bfloat16)
    pool.step(q, [129, 99], cu, flags=gdr.GDR_VALIDATE)
    with pytest.raises(gdr.GdrError, match="page number outside"):
        pool.step(q, [129, 100], cu, flags=gdr.GDR_VALIDATE)
    with pytest.raises(gdr.GdrError, match="longer than its pages"):
        pool.step(q, [64 * pool.table.shape[1], 99], cu, flags=gdr.GDR_VALIDATE)
    pool.table[0, 1] = -1
    with pytest.raises(gdr.GdrError, match="page number outside"):
        pool.step(q, [129, 99], cu, flags=gdr.GDR_VALIDATE)
    with pytest.raises(gdr.GdrError, match="page number outside"):  # an append writes to its own pages, shared or not
        k = normal(3, 2, 1, 64, dtype=torch.bfloat16)
        gdr.kv_append(k, k, pool.k, pool.v, pool.table, ints([128, 99]), cu, flags=gdr.GDR_VALIDATE)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,prefix,m", [(16, 105, 1), (16, 48, 3), (32, 100, 20), (64, 200, 1)])
def test_entries_within_the_prefix_hold_anything(page, prefix, m, dtype):
    """Of pages that end within the prefix: no page, one that is not there, one of NaN, another sequence's."""
    lens, cu = [prefix + 40, prefix, prefix + 700], starts([m] * 3)
    pool = Pool(1, [a + m for a in lens], 2, 64, page, dtype, prefix)
    q = normal(2, 3 * m, 8, 64, dtype=dtype)
    want = pool.step(q, lens, cu, flags=gdr.GDR_VALIDATE)
    for spare in pool.spare:
        pool.k[spare], pool.v[spare] = float("nan"), float("inf")
    for entry in (pool.k.shape[0], -7, pool.spare[0], pool.table_list[2][prefix // page + 1]):
        pool.table[:, :prefix // page] = entry
        assert bits_equal(pool.step(q, lens, cu, flags=gdr.GDR_VALIDATE), want)
