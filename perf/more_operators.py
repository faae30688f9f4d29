"""Measured cases of the attention layer that stands between delta-rule layers: its paged cache, the prompt's
attention and the step over the cache.

    append   token i of sequence n has position p = cache_lens[n] + i.  Channels j and j + R/2 (or 2j and 2j + 1) of
             a head, j < R/2, turn by the angle p freqs[j]; the others stay.  The turned key and the value go to row
             p % page_size of page table[n, p // page_size] of the caches [pages, Hkv, page_size, D]; the turned
             query, and for a prompt the turned key, are returned as dense rows too.
    prompt   o_t = sum_j softmax_j(scale q_t . k_j) v_j over the tokens j <= t of t's own sequence; query head h
             reads key head h / (Hq / Hkv).
    step     the same for token i of sequence n over the keys 0 .. cache_lens[n] + i of the cache.  The first
             `prefix` keys are the same for every sequence and lie in pages of their own; a sequence with
             cache_lens[n] < 0 is padding, its rows stay as they are.

``run`` computes them in plain torch operations, or with ``own`` set through the library's entry points.
"""
import itertools
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
DEV = "cuda"


def listed():
    return [
        # one user's decode step: the latency of a call
        dict(name="append decode 4", op="append", N=4, L=1, ctx=500, Hq=32, Hkv=8, D=128, R=128, page=64, io="bf16",
             pairs=False, k_out=False),
        # the decode batch of the benchmark, a tenth of it padding
        dict(name="append decode 256", op="append", N=256, L=1, ctx=500, Hq=32, Hkv=16, D=128, R=128, page=64,
             io="bf16", pairs=False, k_out=False),
        # one long prompt, the keys returned for its attention
        dict(name="append prompt 32768", op="append", N=1, T=32768, ctx=0, Hq=32, Hkv=8, D=128, R=128, page=64,
             io="bf16", pairs=False, k_out=True),
        # a packed batch in full precision behind far positions, half of the channels turned, in neighbouring pairs
        dict(name="append packed f32", op="append", N=37, T=7001, ctx=900, Hq=12, Hkv=4, D=64, R=32, page=16,
             io="f32", pairs=True, k_out=True),
        # the library's tiny parity shape, 2 heads of 64, in full precision
        dict(name="prompt tiny f32", op="prompt", N=1, T=128, Hq=2, Hkv=2, D=64, io="f32"),
        # the benchmark's ragged prefill, 16 heads of 128
        dict(name="prompt varlen", op="prompt", N=4, T=6113, Hq=16, Hkv=16, D=128, io="bf16"),
        # many short prompts, 7 heads of 64 on each key head
        dict(name="prompt packed short", op="prompt", N=64, T=16001, Hq=14, Hkv=2, D=64, io="bf16"),
        # one long prompt
        dict(name="prompt long", op="prompt", N=1, T=32768, Hq=32, Hkv=8, D=128, io="bf16"),
        # one user's decode step far into a conversation: few rows, a long axis
        dict(name="step decode 1 long", op="step", N=1, L=1, ctx=65536, prefix=0, Hq=32, Hkv=8, D=128, page=64,
             io="bf16"),
        # a decode batch of ragged lengths, a tenth of it padding
        dict(name="step decode 256", op="step", N=256, L=1, ctx=4096, prefix=0, Hq=32, Hkv=8, D=128, page=64,
             io="bf16"),
        # the same batch behind a long system prompt
        dict(name="step decode 256 prefix", op="step", N=256, L=1, ctx=1024, prefix=16000, Hq=32, Hkv=8, D=128,
             page=64, io="bf16"),
        # a speculative verify of 1..12 tokens each behind a shared prompt
        dict(name="step verify 64 prefix", op="step", N=64, L=12, ctx=1024, prefix=8192, Hq=16, Hkv=2, D=128, page=32,
             io="bf16"),
    ]


HEADS = ((16, 16), (32, 16), (32, 8), (16, 2), (12, 4), (14, 2), (8, 1), (2, 2))


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "prompt", "prompt", "step", "step"))
    Hq, Hkv = rng.choice(HEADS)
    D, io = rng.choice((64, 128, 128)), rng.choice(("bf16", "bf16", "bf16", "f32"))
    page = rng.choice((16, 32, 64, 128))
    if op == "append":
        case = dict(op=op, ctx=_spread(rng, 1, 2000), Hq=Hq, Hkv=Hkv, D=D, R=rng.choice((D, D, D // 2, 0)), page=page,
                    io=io, pairs=rng.random() < 0.3, k_out=rng.random() < 0.5)
        if rng.random() < 0.5:
            return dict(case, N=_spread(rng, 1, 256), L=rng.choice((1, 1, 4, 12)))
        T = _spread(rng, 1, 16000)
        return dict(case, N=min(T, _spread(rng, 1, 64)), T=T)
    if op == "prompt":
        T = _spread(rng, 1, 16000 if io == "bf16" else 4000)
        return dict(op=op, N=min(T, _spread(rng, 1, 64)), T=T, Hq=Hq, Hkv=Hkv, D=D, io=io)
    case = dict(op=op, N=_spread(rng, 1, 256), L=rng.choice((1, 1, 4, 12)), ctx=_spread(rng, 1, 30000),
                prefix=rng.choice((0, 0, 1)) * _spread(rng, 1, 16000), Hq=Hq, Hkv=Hkv, D=D, page=page, io=io)
    while case["N"] * case["ctx"] * Hkv * D * SIZE[io] > 256 * 4096 * 8 * 128 * 2:
        case["ctx"] = (case["ctx"] + 1) // 2
    while case["N"] * (case["L"] + 1) // 2 * case["prefix"] * Hq * D > 64 * 6 * 8192 * 32 * 128:
        case["prefix"] = (case["prefix"] + 1) // 2
    return case


def _shape(case):
    """(tokens of each sequence, tokens that each has in the cache before them, -1 for padding): part of the shape,
    the same for every seed."""
    N = case["N"]
    r = torch.Generator().manual_seed(N * 64 + case.get("T", case.get("L", 0)))
    if "T" not in case:
        lengths = torch.randint(1, case["L"] + 1, (N,), generator=r).tolist()
    elif N == 4 and case["T"] == 6113:
        lengths = [65, 1000, 2048, 3000]
    else:
        cuts = (torch.randperm(case["T"] - 1, generator=r)[: N - 1] + 1).sort().values.tolist()
        lengths = [b - a for a, b in zip([0] + cuts, cuts + [case["T"]])]
    if case["op"] == "prompt":
        return lengths, [0] * N
    before = torch.randint(0, case["ctx"] + 1, (N,), generator=r)
    if N == 1:
        before[:] = case["ctx"]
    before += case.get("prefix", 0)
    if "T" not in case and N > 8:
        before[torch.rand(N, generator=r) < 0.1] = -1
    return lengths, before.tolist()


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, Hq, Hkv, D, io = case["op"], case["Hq"], case["Hkv"], case["D"], DTYPES[case["io"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device=DEV, dtype=io)
                * std).to(io)

    lengths, before = _shape(case)
    T = sum(lengths)
    s = {"op": op, "cu": _ints([0, *itertools.accumulate(lengths)])}
    # scores of a few units: some keys carry most of a row, as in trained heads
    s["q"] = normal(T, Hq, D, std=2.0)
    if op != "step":
        s["k"], s["v"] = normal(T, Hkv, D), normal(T, Hkv, D)
    if op == "prompt":
        return s
    page, prefix = case["page"], case.get("prefix", 0)
    ends = [b + n if b >= 0 else 0 for b, n in zip(before, lengths)]
    first = prefix // page  # a sequence's own pages: those from the end of the prefix on
    counts = [max(0, -(-e // page) - first) for e in ends]
    shared = -(-prefix // page)
    pages = torch.randperm(shared + sum(counts) + 3, generator=gen, device=DEV).to(torch.int32)
    s["prefix"], s["prefix_pages"] = prefix, pages[:shared].contiguous()
    table = torch.full((len(ends), first + max(counts)), -1, dtype=torch.int32)
    own_pages, at = pages[shared:].tolist(), 0
    for n, c in enumerate(counts):
        table[n, first:first + c] = torch.tensor(own_pages[at:at + c], dtype=torch.int32)
        at += c
    s["table"], s["before"] = table.to(DEV), _ints(before)
    s["k_cache"], s["v_cache"] = normal(pages.numel(), Hkv, page, D), normal(pages.numel(), Hkv, page, D)
    if op == "append":
        R = case["R"]
        s["pairs"] = case["pairs"]
        s["q_out"], s["k_out"] = torch.zeros_like(s["q"]), torch.zeros_like(s["k"]) if case["k_out"] else None
        s["freqs"] = None if R == 0 else (10000.0 ** (-torch.arange(0, R, 2, device=DEV, dtype=torch.float64) / R)
                                          ).float()
    else:
        s["o"] = torch.zeros_like(s["q"])
    return s


def work(case):
    Hq, Hkv, D, e = case["Hq"], case["Hkv"], case["D"], SIZE[case["io"]]
    lengths, before = _shape(case)
    alive = [(n, b) for n, b in zip(lengths, before) if b >= 0]
    T = sum(n for n, _ in alive)
    if case["op"] == "append":
        heads = 2 * Hq + 4 * Hkv + (Hkv if case["k_out"] else 0)
        return {"bytes": T * heads * D * e, "flops": 3 * T * (Hq + Hkv) * case["R"]}
    seen = sum(n * b + n * (n + 1) // 2 for n, b in alive)
    if case["op"] == "prompt":
        rows = T
    else:
        rows = case["prefix"] + sum(b + n - case["prefix"] for n, b in alive)
    return {"bytes": (2 * T * Hq + 2 * rows * Hkv) * D * e, "flops": 4 * seen * Hq * D}


# ---- the operators in plain torch operations -------------------------------


def _rows(s):
    """Of every token: its sequence and its position (negative for padding)."""
    cu = s["cu"].long()
    token = torch.arange(s["q"].shape[0], device=DEV)
    row = torch.searchsorted(cu, token, right=True) - 1
    before = s["before"].long()[row]
    return row, torch.where(before >= 0, before + token - cu[row], -1)


def _turn(x, position, freqs, pairs):
    if freqs is None:
        return x.clone()
    # angles of far positions lose their fraction in 32 bits
    angle = position.double()[:, None] * freqs.double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    half, y = freqs.numel(), x.float()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if pairs else (slice(0, half), slice(half, 2 * half))
    out = y.clone()
    out[..., a] = y[..., a] * cos - y[..., b] * sin
    out[..., b] = y[..., b] * cos + y[..., a] * sin
    return out.to(x.dtype)


def _plain_append(s):
    row, position = _rows(s)
    live = (position >= 0).nonzero()[:, 0]
    row, position = row[live], position[live]
    k = _turn(s["k"][live], position, s["freqs"], s["pairs"])
    s["q_out"][live] = _turn(s["q"][live], position, s["freqs"], s["pairs"])
    if s["k_out"] is not None:
        s["k_out"][live] = k
    page = s["k_cache"].shape[2]
    at = (s["table"][row, position // page].long(), slice(None), position % page)
    s["k_cache"][at] = k
    s["v_cache"][at] = s["v"][live]
    return [s["q_out"], s["k_out"], s["k_cache"], s["v_cache"]]


def _plain_prompt(s):
    q, k, v = s["q"], s["k"], s["v"]
    (T, Hq, D), Hkv, cu = q.shape, k.shape[1], s["cu"].tolist()
    o = torch.empty_like(q)
    for begin, end in zip(cu[:-1], cu[1:]):
        ks = k[begin:end].float().permute(1, 2, 0)                       # [Hkv, D, L]
        vs = v[begin:end].float().transpose(0, 1)                        # [Hkv, L, D]
        rows = max(1, min(end - begin, (1 << 28) // (Hq * (end - begin))))
        for a in range(begin, end, rows):
            b = min(a + rows, end)
            n = b - begin
            qs = q[a:b].float().view(b - a, Hkv, -1, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D) * D ** -0.5
            p = (qs @ ks[..., :n]).view(Hkv, -1, b - a, n)
            late = torch.arange(n, device=DEV) > torch.arange(a - begin, n, device=DEV)[:, None]
            p.masked_fill_(late, -math.inf)
            p = (p - p.amax(-1, keepdim=True)).exp_()
            total = p.sum(-1, keepdim=True)
            r = (p.view(Hkv, -1, n) @ vs[:, :n]).view(Hkv, -1, b - a, D) / total
            o[a:b] = r.permute(2, 0, 1, 3).reshape(b - a, Hq, D).to(o.dtype)
    return [o]


def _plain_step(s):
    """Sequences of similar lengths together, each padded to the longest of them; the prefix's scores beside theirs."""
    q, o, page, prefix = s["q"], s["o"], s["k_cache"].shape[2], s["prefix"]
    (T, Hq, D), Hkv, cu = q.shape, s["k_cache"].shape[1], s["cu"].long()
    g, first, N = Hq // Hkv, prefix // page, cu.numel() - 1
    row, position = _rows(s)
    columns = s["table"].shape[1] - first
    longest = int((cu[1:] - cu[:-1]).max())
    pk, pv = (c[s["prefix_pages"].long()].transpose(0, 1).flatten(1, 2)[:, :prefix].float()
              for c in (s["k_cache"], s["v_cache"]))
    step = max(1, (1 << 28) // (max(1, columns) * page * Hkv * D + longest * Hq * (prefix + columns * page)))
    for a in range(0, N, step):
        b = min(a + step, N)
        # the sequences' tokens as [b - a, longest] with the ones that are missing repeated
        token = torch.minimum(cu[a:b, None] + torch.arange(longest, device=DEV), cu[a + 1:b + 1, None] - 1)
        seen = position[token]
        qs = q[token].float().view(b - a, longest, Hkv, g, D).permute(0, 2, 1, 3, 4) * D ** -0.5
        qs = qs.reshape(b - a, Hkv, longest * g, D)
        pages = s["table"][a:b, first:].long().clamp(min=0)
        ks, vs = (c[pages].transpose(2, 3).reshape(b - a, columns * page, Hkv, D).transpose(1, 2).float()
                  for c in (s["k_cache"], s["v_cache"]))
        flat = qs.transpose(0, 1).reshape(Hkv, -1, D)
        near = qs @ ks.transpose(2, 3)
        far = (flat @ pk.transpose(1, 2)).view(Hkv, b - a, longest * g, prefix).transpose(0, 1)
        key = torch.arange(first * page, (first + columns) * page, device=DEV)
        hide = (key > seen[:, :, None]) | (key < prefix)
        near = near.view(b - a, Hkv, longest, g, -1).masked_fill(hide[:, None, :, None], -math.inf)
        p = torch.cat((far, near.view(b - a, Hkv, longest * g, -1)), -1)
        p = (p - p.amax(-1, keepdim=True)).exp_()
        total = p.sum(-1, keepdim=True)
        r = p[..., prefix:] @ vs
        lead = p[..., :prefix].transpose(0, 1).reshape(Hkv, (b - a) * longest * g, prefix)
        r += (lead @ pv).view(Hkv, b - a, -1, D).transpose(0, 1)
        r = (r / total).view(b - a, Hkv, longest, g, D).permute(0, 2, 1, 3, 4).reshape(b - a, longest, Hq, D)
        live = s["before"][a:b] >= 0
        # rows that were repeated write their token's value once more
        o[token[live]] = r[live].to(o.dtype)
    return [o]


def run(state):
    s, op = state, state["op"]
    if own:
        import gated_delta_rule_37_gb300 as gdr

        if op == "append":
            gdr.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["before"], s["cu"], q=s["q"],
                          freqs=s["freqs"], flags=gdr.GDR_ROPE_PAIRS if s["pairs"] else 0, q_out=s["q_out"],
                          k_out=s["k_out"])
            return [s["q_out"], s["k_out"], s["k_cache"], s["v_cache"]]
        if op == "prompt":
            return [gdr.attn_fwd(s["q"], s["k"], s["v"], s["cu"])]
        return [gdr.attn_step(s["q"], s["k_cache"], s["v_cache"], s["table"], s["before"], s["cu"],
                              prefix_pages=s["prefix_pages"] if s["prefix"] else None, prefix_len=s["prefix"],
                              o=s["o"])]
    return _plain_append(s) if op == "append" else _plain_prompt(s) if op == "prompt" else _plain_step(s)


# ---- the definitions in 64 bits --------------------------------------------


def exact(case, seed):
    s, op, D = prepare(case, seed), case["op"], case["D"]
    lengths, before = _shape(case)
    starts = [0, *itertools.accumulate(lengths)]
    group = case["Hq"] // case["Hkv"]
    if op == "append":
        q, k = torch.zeros_like(s["q"]).double(), torch.zeros_like(s["k"]).double()
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
        R, page = case["R"], case["page"]
        for n, b in enumerate(before):
            if b < 0:
                continue
            part = slice(starts[n], starts[n + 1])
            p = torch.arange(b, b + lengths[n], device=DEV)
            for x, y in ((s["q"], q), (s["k"], k)):
                z = x[part].double()
                if R:
                    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                                       torch.outer(p.double(), s["freqs"].double()))[:, None]
                    if case["pairs"]:
                        w = torch.view_as_complex(z[..., :R].reshape(*z.shape[:-1], R // 2, 2).contiguous()) * turn
                        z[..., :R] = torch.view_as_real(w).flatten(-2)
                    else:
                        w = torch.complex(z[..., :R // 2], z[..., R // 2:R]) * turn
                        z[..., :R] = torch.cat((w.real, w.imag), -1)
                y[part] = z
            where = s["table"][n].long()[p // page]
            k_cache[where, :, p % page] = k[part]
            v_cache[where, :, p % page] = s["v"][part].double()
        return [q, k if case["k_out"] else None, k_cache, v_cache]
    if op == "step":
        o = s["o"].double()
        lead = [c[s["prefix_pages"].long()].transpose(1, 2).flatten(0, 1)[:s["prefix"]].double()
                for c in (s["k_cache"], s["v_cache"])]
    else:
        o = torch.zeros_like(s["q"]).double()
    for n, b in enumerate(before):
        if b < 0:
            continue
        part, end = slice(starts[n], starts[n + 1]), b + lengths[n]
        if op == "prompt":
            k, v = s["k"][part].double(), s["v"][part].double()
        else:
            cut = s["prefix"] // case["page"]
            k, v = (torch.cat((c, x[s["table"][n, cut:].long().clamp(min=0)].transpose(1, 2).flatten(0, 1)
                               [s["prefix"] - cut * case["page"]:end - cut * case["page"]].double()))
                    for c, x in zip(lead, (s["k_cache"], s["v_cache"])))
        q = s["q"][part].double() / math.sqrt(D)
        for h in range(case["Hq"]):
            kh, vh = k[:, h // group], v[:, h // group]
            for i in range(0, lengths[n], 4096):
                j = min(i + 4096, lengths[n])
                score = q[i:j, h] @ kh[:b + j].T
                score = torch.where(torch.ones_like(score, dtype=torch.bool).tril(b + i), score, -math.inf)
                o[starts[n] + i:starts[n] + j, h] = torch.softmax(score, 1) @ vh[:b + j]
    return [o]
