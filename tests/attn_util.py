"""Cases and bounds of the attention layer's tests."""
import numpy as np
import torch

import gated_delta_rule_37_gb300 as gdr
import oracle

DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def starts(lengths):
    return ints(np.cumsum([0, *lengths]).tolist())


def normal(seed, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).to(DEV)


def check_attention(got, ref, keys: int, what: str = ""):
    """|got - o| within what the arithmetic allows.  With u the type's half step and e = 2^-23 (a truncated fp32
    step): a score of D products is off by (D + 4) e times the sum of their magnitudes (`score`), its exponential
    relatively by as much and by 2^-21 of its own, a sum over n keys by n e, the weights by u where they are rounded
    to bf16.  All of it is in proportion to sum p |v| (`weight`), once for the numerator and, but for the weights'
    rounding, once for the sum below it; the result is rounded once.  Rows that the oracle gives as NaN are not
    compared here."""
    o, weight, score = (np.asarray(x) for x in ref)
    g = got.detach().double().cpu().numpy()
    D, e, u = o.shape[-1], 2.0 ** -23, HALF[got.dtype]
    rounded = u if got.dtype == torch.bfloat16 else 0.0
    rel = rounded + 2 * ((D + 4) * e * score[..., None] + 2.0 ** -21 + (keys + 8) * e)
    bound = u * np.abs(o) * (1 + rel) + rel * weight + 1e-37
    live = ~np.isnan(o)
    assert np.isfinite(g[live]).all(), f"{what}: not finite"
    worst = (np.abs(g - o) / bound)[live].max() if live.any() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"


class Pool:
    """A paged cache for sequences of `ends` tokens, pages in random order, and spare pages."""

    def __init__(self, seed, ends, Hkv, D, page, dtype, prefix=0, spare=3, fill=None):
        r = np.random.default_rng(seed)
        first = prefix // page
        own = [max(0, -(-e // page) - first) for e in ends]
        shared = -(-prefix // page)
        count = shared + sum(own) + spare
        order = r.permutation(count)
        self.prefix_len = prefix
        self.prefix_list = order[:shared].tolist()
        at = shared
        self.table_list = []
        width = max(1, first + max(own, default=0))
        for c in own:
            self.table_list.append([-1] * first + order[at:at + c].tolist() + [-1] * (width - first - c))
            at += c
        self.spare = order[at:].tolist()
        self.table = ints(self.table_list).reshape(len(ends), width)
        self.prefix_pages = ints(self.prefix_list) if prefix else None
        shape = (count, Hkv, page, D)
        if fill is None:
            self.k, self.v = normal(seed + 1, *shape, dtype=dtype), normal(seed + 2, *shape, dtype=dtype)
        else:
            self.k = torch.full(shape, fill, dtype=dtype, device=DEV)
            self.v = torch.full(shape, fill, dtype=dtype, device=DEV)

    def step(self, q, lens, cu, **kw):
        return gdr.attn_step(q, self.k, self.v, self.table, ints(lens), cu, prefix_pages=self.prefix_pages,
                             prefix_len=self.prefix_len, **kw)

    def reference(self, q, lens, cu, scale=None):
        return oracle.attn_step(q.float().cpu(), self.k.float().cpu(), self.v.float().cpu(), self.table.cpu(), lens,
                                cu.cpu(), q.shape[2] ** -0.5 if scale is None else scale, self.prefix_list,
                                self.prefix_len)
