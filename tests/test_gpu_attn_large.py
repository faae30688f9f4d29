"""Prompts of so many rows that the CUDA cores' kernels take their large tiles: fp32, and bf16 tokens that share rows."""
import pytest
import torch

import gated_delta_rule_37_gb300 as gdr
import oracle
from tests.attn_util import DEV, check_attention, normal, starts
from tests.gpu_util import bits_equal

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _reference(q, k, v, cu, rows, scale):
    """The oracle's three results for some tokens' rows, by its formula for a row."""
    import numpy as np

    group, begin = q.shape[1] // k.shape[1], cu.tolist()
    q, k, v = (x.double().cpu().numpy() for x in (q, k, v))
    out = []
    for t in rows:
        first = max(b for b in begin if b <= t)
        for h in range(q.shape[1]):
            seen = slice(first, t + 1), h // group
            out.append(oracle.attend(q[t, h], k[seen], v[seen], scale))
    shape = len(rows), q.shape[1]
    return [np.array([x[i] for x in out]).reshape(shape + (() if i == 2 else (q.shape[2],))) for i in range(3)]


def _tokens(T, H, D, dtype, seed, shared):
    """[T, H, D]; with `shared` rows that begin half a row apart, or with "one" a single row for all tokens."""
    if shared == "one":
        return normal(seed, 1, H, D, dtype=dtype).expand(T, H, D)
    if shared == "half":
        return normal(seed, (T + 1) * H * D // 2, dtype=dtype).as_strided((T, H, D), (H * D // 2, D, 1))
    return normal(seed, T, H, D, dtype=dtype)


@pytest.mark.parametrize("dtype,shared", [(F32, None), (F32, "half"), (BF16, "half"), (BF16, "one")])
@pytest.mark.parametrize("D,Hq,Hkv", [
    (128, 32, 8),   # 128 rows a tile: 64000 (token, head) rows
    (64, 32, 8),    # 64 rows
    (128, 6, 2),    # 64 rows, of a group that does not divide them
    (64, 14, 2),
])
def test_large_tiles(D, Hq, Hkv, dtype, shared):
    """Rows at the tiles' borders and beside them, of sequences that end and begin within tiles."""
    lengths = [700, 1, 0, 333, 64, 902] if Hq == 32 else [1200, 1, 0, 333, 64, 900]
    T, cu = sum(lengths), starts(lengths)
    rows_per_tile = 128 if D == 128 and Hq == 32 else 64
    tiles = lambda rows: -(-T * (Hq // Hkv) // rows) * Hkv
    assert tiles(rows_per_tile) >= 152 and (D == 64 or rows_per_tile == 128 or tiles(128) < 152)
    q, k, v = (_tokens(T, H, D, dtype, s, x) for s, H, x in ((1, Hq, None), (2, Hkv, None), (3, Hkv, shared)))
    if shared == "one":
        q = _tokens(T, Hq, D, dtype, 4, "half")
    o = torch.full((T + 3, Hq, D), 7.0, dtype=dtype, device=DEV)
    gdr.attn_fwd(q, k, v, cu, o=o[:T], flags=gdr.GDR_VALIDATE)
    assert (o[T:] == 7.0).all() and torch.isfinite(o).all()
    first = cu.tolist()
    rows = sorted({t for b, e in zip(first[:-1], first[1:]) if e > b
                   for t in (b, b + 15, b + 16, b + 31, b + 32, b + 63, b + 64, b + 127, b + 128, (b + e) // 2, e - 2, e - 1)
                   if b <= t < e})
    check_attention(o[rows], _reference(q, k, v, cu, rows, D ** -0.5), max(lengths))
    assert bits_equal(o[:T], gdr.attn_fwd(q, k, v, cu))


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 32, 8), (64, 16, 4)])
def test_large_tiles_keep_bad_values_to_the_rows_that_see_them(D, Hq, Hkv):
    lengths = [700, 300, 1000] if D == 128 else [1300, 300, 1100]
    T, cu = sum(lengths), starts(lengths)
    q, k, v = (normal(s, T, H, D) for s, H in ((1, Hq), (2, Hkv), (3, Hkv)))
    clean = gdr.attn_fwd(q, k, v, cu)
    bad = lengths[0] + 150
    v[bad, 1, 3] = float("nan")
    k[bad + 9, 0, 2] = float("inf")
    o = gdr.attn_fwd(q, k, v, cu)
    group, end = Hq // Hkv, lengths[0] + lengths[1]
    hit = torch.zeros(o.shape, dtype=torch.bool, device=DEV)
    hit[bad:end, group:2 * group, 3] = True
    assert torch.isnan(o[hit]).all()
    hit[bad + 9:end, :group] = True
    assert bits_equal(torch.where(hit, 0, o), torch.where(hit, 0, clean))
