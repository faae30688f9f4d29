"""Infinities and NaN in the attention layer: rows that do not see them."""
import pytest
import torch

import gated_delta_rule_37_gb300 as gdr
from tests.attn_util import Pool, check_attention, normal, starts
from tests.gpu_util import bits_equal

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
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
