"""Measured cases of the gated linear recurrence and of the residual RMS norm.

Per channel c of a packed sequence n (tokens cu[n] .. cu[n+1]-1), with the
natural-log decay g <= 0:

    scan_fwd   h_t = exp(g_t) h_{t-1} + x_t, from h0[n];  y_t = h_t;  final[n] = last h
    scan_bwd   lam_t = dy_t + mu_{t+1}, mu_t = exp(g_t) lam_t, mu after the last token = dfinal[n];
               dx_t = lam_t;  dg_t = mu_t y_{t-1} (h0 before the first token);  dh0[n] = first mu
    step       scan_fwd of a few tokens per sequence from a slot of a state pool (slot < 0: skipped),
               with the last state committed to the pool or every token's state kept

and per row of a [M, D] matrix:

    norm_fwd   s = round(x + residual);  y = s w / sqrt(mean(s^2) + eps), in the input's type or as
               e4m3 codes with one scale a / 448 per group of a row, a = max(max |y|, 1e-12)
    norm_bwd   gradients of x (and of the residual) and of w, from dy, s and the gradient that
               arrives at s along the residual stream

``run`` computes them in plain torch operations, or with ``own`` set through
the library's entry points.
"""
import itertools
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6
DEV = "cuda"


def listed():
    return [
        # one user's decode step through one layer: the latency of a call
        dict(name="step decode 4", op="step", N=4, L=1, D=2048, io="bf16", gate="f32", pool="f32", commit=True,
             keep=False),
        # the decode batch of the benchmark (256 sequences, 32 heads of 128), a tenth of it padding
        dict(name="step decode 256", op="step", N=256, L=1, D=4096, io="bf16", gate="f32", pool="f32", commit=True,
             keep=False),
        # the speculative verify of the benchmark: 1..12 tokens each, states kept, nothing committed
        dict(name="step verify 64", op="step", N=64, L=12, D=4096, io="bf16", gate="f32", pool="bf16", commit=False,
             keep=True),
        # a short prompt in full precision: the smallest scan, the library's tiny parity shape with 2 heads of 64
        dict(name="scan_fwd tiny f32", op="scan_fwd", N=1, T=128, D=128, io="f32", gate="f32", memory=50.0),
        # the benchmark's ragged prefill, 16 heads of 128
        dict(name="scan_fwd varlen", op="scan_fwd", N=4, T=6113, D=2048, io="bf16", gate="f32", memory=50.0),
        # one long prompt, 32 heads of 128
        dict(name="scan_fwd long", op="scan_fwd", N=1, T=32768, D=4096, io="bf16", gate="f32", memory=1000.0),
        # training on a packed batch of many short documents, a channel count that is odd
        dict(name="scan_bwd packed odd", op="scan_bwd", N=37, T=7001, D=1001, io="f32", gate="f32", memory=20.0),
        # training on one long document with gates in the activations' type
        dict(name="scan_bwd long", op="scan_bwd", N=1, T=32768, D=4096, io="bf16", gate="bf16", memory=1000.0),
        # the norm of a decode step
        dict(name="norm_fwd 8 rows", op="norm_fwd", M=8, D=4096, io="bf16", out="same", group=0, residual=True),
        # the norm before 8-bit projections over a long prompt
        dict(name="norm_fwd e4m3 long", op="norm_fwd", M=32768, D=4096, io="bf16", out="e4m3", group=128,
             residual=True),
        # rows of an odd width, one scale for each
        dict(name="norm_fwd e4m3 odd", op="norm_fwd", M=3001, D=1001, io="f32", out="e4m3", group=0, residual=False),
        # a training step's norm
        dict(name="norm_bwd 16k", op="norm_bwd", M=16384, D=4096, io="bf16", residual=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Channel counts: multiples of 128, of 8, or any number at all."""
    D, unit = _spread(rng, lo, hi), rng.choice((128, 8, 1))
    return max(unit, D // unit * unit)


def draw(rng):
    op = rng.choice(("step", "scan_fwd", "scan_fwd", "scan_bwd", "norm_fwd", "norm_fwd", "norm_bwd"))
    io = rng.choice(("bf16", "bf16", "f32"))
    if op == "step":
        return dict(op=op, N=_spread(rng, 1, 512), L=rng.choice((1, 1, 4, 12)), D=_width(rng, 16, 8192), io=io,
                    gate=rng.choice(("f32", io)), pool=rng.choice(("f32", "bf16")), commit=rng.random() < 0.6,
                    keep=rng.random() < 0.4)
    if op in ("scan_fwd", "scan_bwd"):
        T, D = _spread(rng, 1, 32768), _width(rng, 16, 8192)
        while T * D > 30000 * 2048:
            T = (T + 1) // 2
        return dict(op=op, N=min(T, _spread(rng, 1, 64)), T=T, D=D, io=io, gate=rng.choice(("f32", io)),
                    memory=float(_spread(rng, 5, 2000)))
    M, D = _spread(rng, 1, 32768), _width(rng, 16, 16384)
    while M * D > 16384 * 2048:
        M = (M + 1) // 2
    if op == "norm_bwd":
        return dict(op=op, M=M, D=D, io=io, residual=rng.random() < 0.7)
    return dict(op=op, M=M, D=D, io=io, out=rng.choice(("same", "e4m3")), group=rng.choice((0, 32, 64, 128)),
                residual=rng.random() < 0.7)


def _lengths(case, seed):
    """Lengths of the packed sequences: for `step` 1..L each, the same ones for every seed (the rows in all
    are part of the shape), else a random split of T into N parts."""
    N = case["N"]
    r = torch.Generator().manual_seed(N * 64 + case["L"] if case["op"] == "step" else seed)
    if case["op"] == "step":
        if case["L"] == 1:
            return [1] * N
        return torch.randint(1, case["L"] + 1, (N,), generator=r).tolist()
    if N == 4 and case["T"] == 6113:
        return [65, 1000, 2048, 3000]
    cuts = (torch.randperm(case["T"] - 1, generator=r)[: N - 1] + 1).sort().values.tolist()
    return [b - a for a, b in zip([0] + cuts, cuts + [case["T"]])]


def _starts(lengths):
    return torch.tensor([0, *itertools.accumulate(lengths)], dtype=torch.int32, device=DEV)


def _gates(T, D, memory, dtype, gen):
    """Decays of channels that remember from a few tokens to several times `memory` tokens."""
    scale = memory ** -1.0 * torch.exp2(4 * torch.rand(D, generator=gen, device=DEV) - 2)
    return (-scale * (0.1 + 1.8 * torch.rand(T, D, generator=gen, device=DEV))).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, D, io = case["op"], case["D"], DTYPES[case["io"]]

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)

    s = {"op": op}
    if op == "step":
        lengths, N = _lengths(case, seed), case["N"]
        T, slots = sum(lengths), 2 * N + 1
        s["cu"] = _starts(lengths)
        s["x"], s["g"] = normal(T, D, dtype=io), _gates(T, D, 20.0, DTYPES[case["gate"]], gen)
        s["pool"] = normal(slots, D, dtype=DTYPES[case["pool"]], std=3.0)
        index = torch.randperm(slots, generator=gen, device=DEV)[:N].to(torch.int32)
        index[torch.rand(N, generator=gen, device=DEV) < 0.1] = -1
        s["index"], s["commit"] = index, case["commit"]
        s["y"] = torch.zeros(T, D, dtype=io, device=DEV)
        s["states"] = torch.zeros(N, case["L"], D, dtype=s["pool"].dtype, device=DEV) if case["keep"] else None
    elif op in ("scan_fwd", "scan_bwd"):
        T, N = case["T"], case["N"]
        s["cu"] = _starts(_lengths(case, seed))
        s["g"] = _gates(T, D, case["memory"], DTYPES[case["gate"]], gen)
        s["h0"] = normal(N, D, std=3.0)
        if op == "scan_fwd":
            s["x"] = normal(T, D, dtype=io)
        else:
            s["dy"], s["y"] = normal(T, D, dtype=io), normal(T, D, dtype=io, std=3.0)
            s["dfinal"] = normal(N, D)
    else:
        M = case["M"]
        s["w"] = 1.0 + normal(D, std=0.2)
        s["x"] = normal(M, D, dtype=io)
        s["residual"] = normal(M, D, dtype=io, std=2.0) if case["residual"] else None
        if op == "norm_bwd":
            s["dy"] = normal(M, D, dtype=io)
        else:
            s["e4m3"], s["group"] = case["out"] == "e4m3", case["group"]
    return s


def work(case):
    op, D, e = case["op"], case["D"], SIZE[case["io"]]
    if op == "step":
        # about nine in ten sequences are not padding, each of (1 + L) / 2 tokens on average
        n = 0.9 * case["N"]
        T, p = n * (1 + case["L"]) / 2, SIZE[case["pool"]]
        per_token = 2 * e + SIZE[case["gate"]] + (p if case["keep"] else 0)
        return {"bytes": T * D * per_token + n * D * p * (2 if case["commit"] else 1), "flops": 3 * T * D}
    if op == "scan_fwd":
        return {"bytes": case["T"] * D * (2 * e + SIZE[case["gate"]]) + 8 * case["N"] * D, "flops": 3 * case["T"] * D}
    if op == "scan_bwd":
        return {"bytes": case["T"] * D * (3 * e + 2 * SIZE[case["gate"]]) + 12 * case["N"] * D,
                "flops": 4 * case["T"] * D}
    n = case["M"] * D
    if op == "norm_bwd":
        return {"bytes": n * e * (4 if case["residual"] else 3) + 8 * D, "flops": 9 * n}
    out = e if case["out"] == "same" else 1
    scales = 0 if case["out"] == "same" else 4 * case["M"] * (-(-D // case["group"]) if case["group"] else 1)
    return {"bytes": n * (e * (3 if case["residual"] else 1) + out) + scales + 4 * D, "flops": 6 * n}


# ---- the operators in plain torch operations -------------------------------


def _scan(g, b):
    """h_t = exp(g_t) h_{t-1} + b_t along the first axis, h before it 0: the pairs
    of neighbours are composed, the half as long scan of them gives every second
    h, and those give the ones between.  The composed decays are kept as sums of
    logarithms: a product of thousands of rounded factors near 1 drifts."""
    if b.shape[0] == 1:
        return b.clone()
    n = b.shape[0] // 2 * 2
    odd = _scan(g[1:n:2] + g[0:n:2], g[1:n:2].exp() * b[0:n:2] + b[1:n:2])
    h = torch.empty_like(b)
    h[1:n:2] = odd
    h[0] = b[0]
    h[2::2] = g[2::2].exp() * odd[: (b.shape[0] - 1) // 2] + b[2::2]
    return h


def _scan_from(g, x, first, start):
    """The scan over packed sequences whose first rows are `first`, each from its row of `start`."""
    g, b = g.float().clone(), x.float().clone()
    b[first] += g[first].exp() * start
    g[first] = -math.inf
    return _scan(g, b)


def _plain_scan_fwd(x, g, h0, cu):
    h = _scan_from(g, x, cu[:-1].long(), h0)
    return h.to(x.dtype), h[cu[1:].long() - 1]


def _plain_scan_bwd(dy, g, y, h0, dfinal, cu):
    # lam_t = dy_t + exp(g_{t+1}) lam_{t+1}, dfinal in the place of the product after a last token: a scan from the end
    first, last = cu[:-1].long(), cu[1:].long() - 1
    b, after = dy.float().clone(), torch.full_like(g, -math.inf, dtype=torch.float32)
    b[last] += dfinal
    after[:-1] = g[1:].float()
    after[last] = -math.inf
    lam = _scan(after.flip(0), b.flip(0)).flip(0)
    mu = g.float().exp() * lam
    before = torch.zeros_like(b)
    before[1:] = y[:-1].float()
    before[first] = h0
    return lam.to(dy.dtype), (mu * before).to(g.dtype), mu[first]


def _plain_step(s):
    cu, pool = s["cu"].long(), s["pool"]
    T = s["x"].shape[0]
    token = torch.arange(T, device=DEV)
    row = torch.searchsorted(cu, token, right=True) - 1
    h0 = pool[s["index"].long().clamp(min=0)].float()
    h = _scan_from(s["g"], s["x"], cu[:-1], h0)
    kept = (s["index"] >= 0)[row]
    s["y"].copy_(torch.where(kept[:, None], h.to(s["y"].dtype), s["y"]))
    if s["states"] is not None:
        at = (row, token - cu[row])
        s["states"][at] = torch.where(kept[:, None], h.to(pool.dtype), s["states"][at])
    if s["commit"]:
        # skipped sequences write their old value back to a slot of their own: the spare last row
        spare = torch.cat((pool, pool[:1]))
        slot = torch.where(s["index"] >= 0, s["index"].long(), pool.shape[0])
        spare[slot] = h[cu[1:] - 1].to(pool.dtype)
        pool.copy_(spare[:-1])
    return [s["y"], s["pool"], s["states"]]


def _plain_norm_fwd(s):
    x = s["x"]
    if s["residual"] is not None:
        x = (x.float() + s["residual"].float()).to(x.dtype)
    v = x.float()
    y = v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS) * s["w"]
    total = x if s["residual"] is not None else None
    if not s["e4m3"]:
        return [y.to(x.dtype), total]
    M, D = y.shape
    group = s["group"] or D
    wide = torch.zeros(M, -(-D // group) * group, device=DEV)
    wide[:, :D] = y
    wide = wide.view(M, -1, group)
    scale = wide.abs().amax(2).clamp(min=1e-12) / 448
    codes = (wide / scale[:, :, None]).view(M, -1)[:, :D].to(torch.float8_e4m3fn)
    return [codes, total, scale]


def _plain_norm_bwd(s):
    x, dy, w = s["x"].float(), s["dy"].float(), s["w"]
    r = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    z, unit = dy * w, x * r
    dx = r * (z - unit * (z * unit).mean(1, keepdim=True))
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    return [dx.to(s["dy"].dtype), (dy * unit).sum(0)]


def run(state):
    s, op = state, state["op"]
    if own:
        import gated_delta_rule_37_gb300 as gdr

        if op == "step":
            gdr.linrec_step(s["x"], s["g"], s["pool"], s["index"], s["cu"], flags=gdr.GDR_COMMIT if s["commit"] else 0,
                            y=s["y"], intermediate_states=s["states"])
            return [s["y"], s["pool"], s["states"]]
        if op == "scan_fwd":
            return list(gdr.linrec_fwd(s["x"], s["g"], s["cu"], initial_state=s["h0"]))
        if op == "scan_bwd":
            return list(gdr.linrec_bwd(s["dy"], s["g"], s["y"], s["cu"], initial_state=s["h0"],
                                       d_final_state=s["dfinal"]))
        if op == "norm_fwd":
            y, total, scale = gdr.rmsnorm_fwd(s["x"], s["w"], residual=s["residual"], eps=EPS,
                                              y_dtype=torch.float8_e4m3fn if s["e4m3"] else None,
                                              scale_group=s["group"] if s["e4m3"] else 0)
            return [y, total, scale] if s["e4m3"] else [y, total]
        return list(gdr.rmsnorm_bwd(s["dy"], s["x"], s["w"], eps=EPS, d_residual_out=s["residual"]))
    if op == "step":
        return _plain_step(s)
    if op == "scan_fwd":
        return list(_plain_scan_fwd(s["x"], s["g"], s["h0"], s["cu"]))
    if op == "scan_bwd":
        return list(_plain_scan_bwd(s["dy"], s["g"], s["y"], s["h0"], s["dfinal"], s["cu"]))
    return _plain_norm_fwd(s) if op == "norm_fwd" else _plain_norm_bwd(s)


# ---- the definitions in 64 bits, token by token -----------------------------


def exact(case, seed):
    def walk(x, decay, start, cu):
        """Every h of the recurrence, one token after the other; start [N, D]."""
        out = torch.empty_like(x)
        for n in range(len(cu) - 1):
            h = start[n].clone()
            for t in range(cu[n], cu[n + 1]):
                h.mul_(decay[t]).add_(x[t])
                out[t] = h
        return out

    def walk_back(dy, decay, dfinal, cu):
        """lam and mu of the backward recurrence, from the last token of each sequence to its first."""
        lam, mu = torch.empty_like(dy), torch.empty_like(dy)
        for n in range(len(cu) - 1):
            m = dfinal[n]
            for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
                torch.add(dy[t], m, out=lam[t])
                m = torch.mul(lam[t], decay[t], out=mu[t])
        return lam, mu

    s, op = prepare(case, seed), case["op"]
    if op == "step":
        cu, index = s["cu"].tolist(), s["index"].tolist()
        start = torch.stack([s["pool"][max(i, 0)] for i in index]).double()
        h = walk(s["x"].double(), torch.exp(s["g"].double()), start, cu)
        y, pool = s["y"].double(), s["pool"].double()
        states = None if s["states"] is None else s["states"].double()
        for n, i in enumerate(index):
            if i < 0:
                continue
            y[cu[n]:cu[n + 1]] = h[cu[n]:cu[n + 1]]
            if states is not None:
                states[n, :cu[n + 1] - cu[n]] = h[cu[n]:cu[n + 1]]
            if s["commit"]:
                pool[i] = h[cu[n + 1] - 1]
        return [y, pool, states]
    if op == "scan_fwd":
        cu = s["cu"].tolist()
        h = walk(s["x"].double(), torch.exp(s["g"].double()), s["h0"].double(), cu)
        return [h, torch.stack([h[e - 1] for e in cu[1:]])]
    if op == "scan_bwd":
        cu = s["cu"].tolist()
        lam, mu = walk_back(s["dy"].double(), torch.exp(s["g"].double()), s["dfinal"].double(), cu)
        dh0 = torch.stack([mu[b] for b in cu[:-1]])
        y = s["y"].double()
        for b, h0 in zip(cu[:-1], s["h0"].double()):
            mu[b] *= h0
        inner = torch.ones(y.shape[0], dtype=torch.bool, device=DEV)
        inner[torch.tensor(cu[:-1], device=DEV)] = False
        at = inner.nonzero()[:, 0]
        mu[at] = mu[at] * y[at - 1]
        return [lam, mu, dh0]
    w, D = s["w"].double(), case["D"]
    if op == "norm_bwd":
        x, dy = s["x"].double(), s["dy"].double()
        inv = 1.0 / torch.sqrt((x * x).sum(1, keepdim=True) / D + EPS)
        dot = (dy * w * x).sum(1, keepdim=True)
        dx = dy * w * inv - x * (inv ** 3) * dot / D
        if s["residual"] is not None:
            dx += s["residual"].double()
        return [dx, (dy * x * inv).sum(0)]
    x, total = s["x"], None
    if s["residual"] is not None:
        # the sum's rounding to the row's type is part of the definition; the sum itself is returned unrounded
        total = x.double() + s["residual"].double()
        x = total.to(x.dtype) if case["io"] == "f32" else total.float().to(x.dtype)
    x = x.double()
    y = x * w / torch.sqrt((x * x).sum(1, keepdim=True) / D + EPS)
    if not s["e4m3"]:
        return [y, total]
    # the codes' values before their rounding
    scales, codes, group = [], torch.empty_like(y), case["group"] or D
    for b in range(0, D, group):
        part = y[:, b:b + group]
        scale = part.abs().max(1).values.clamp(min=1e-12) / 448
        codes[:, b:b + group] = part / scale[:, None]
        scales.append(scale)
    return [codes, total, torch.stack(scales, 1)]
