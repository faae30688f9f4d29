"""One recurrent block as a user runs it: the residual's addition and norm, the
gates from raw projections, the gated linear recurrence; forward and backward
over packed sequences against automatic differentiation in 64 bits, and its
serving form, where prefill and decode steps share the norm and the pool."""
import numpy as np
import pytest
import torch

import gated_delta_rule_37_gb300 as gdr

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdr.load()


def params(seed, width, D):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=r)  # noqa: E731
    p = dict(w=1 + 0.2 * n(width), wa=n(width, D) / width ** 0.5, wb=n(width, D) / width ** 0.5,
             wx=n(width, D) / width ** 0.5, A_log=0.5 * n(D), dt_bias=n(D) - 2)
    return {k: v.to(DEV) for k, v in p.items()}, n


def mixer(p, u):
    """Raw projections of the normed rows and what the recurrence takes from them."""
    return u @ p["wa"], u @ p["wb"], u @ p["wx"]


def plain(p, x, res, h0, cu):
    """The block in 64 bits, differentiable."""
    s = x + res
    u = s / torch.sqrt((s * s).mean(1, keepdim=True) + EPS) * p["w"]
    a, b, v = mixer(p, u)
    g = -torch.exp(p["A_log"]) * torch.nn.functional.softplus(a + p["dt_bias"])
    inp = torch.sigmoid(b) * v
    rows, last = [], []
    for n in range(len(cu) - 1):
        h = h0[n]
        for t in range(cu[n], cu[n + 1]):
            h = torch.exp(g[t]) * h + inp[t]
            rows.append(h)
        last.append(h)
    return s, torch.stack(rows), torch.stack(last)


def test_training_step():
    lens, width, D = [50, 1, 130], 96, 72
    p, n = params(1, width, D)
    T, cu = sum(lens), [0] + list(np.cumsum(lens))
    x, res, h0 = n(T, width).to(DEV), n(T, width).to(DEV), n(3, D).to(DEV)
    ws, wy, wh = n(T, width).to(DEV), n(T, D).to(DEV), n(3, D).to(DEV)
    dcu = torch.tensor(cu, dtype=torch.int32, device=DEV)

    # 64 bits, automatic
    q = {k: v.double().requires_grad_() for k, v in dict(p, x=x, res=res, h0=h0).items()}
    s, y, last = plain(q, q["x"], q["res"], q["h0"], cu)
    loss = (ws * s).sum() + (wy * y).sum() + (wh * last).sum()
    names = ["x", "res", "h0", "w", "wa", "wb", "wx", "A_log", "dt_bias"]
    want = dict(zip(names, torch.autograd.grad(loss, [q[k] for k in names])))

    # the library's operators, and plain products between them
    u, s1, _ = gdr.rmsnorm_fwd(x, p["w"], residual=res, eps=EPS)
    a, b, v = mixer(p, u)
    g, beta = gdr.gating_fwd(a, p["dt_bias"], p["A_log"], b)
    inp = beta * v
    y1, last1 = gdr.linrec_fwd(inp, g, dcu, initial_state=h0)
    d_inp, dg, dh0 = gdr.linrec_bwd(wy, g, y1, dcu, initial_state=h0, d_final_state=wh)
    da = dg * -torch.exp(p["A_log"]) * torch.sigmoid(a + p["dt_bias"])
    db, dv = d_inp * v * beta * (1 - beta), d_inp * beta
    du = da @ p["wa"].t() + db @ p["wb"].t() + dv @ p["wx"].t()
    dx, dw = gdr.rmsnorm_bwd(du, s1, p["w"], eps=EPS, d_residual_out=ws)
    got = dict(x=dx, res=dx, h0=dh0, w=dw, wa=u.t() @ da, wb=u.t() @ db, wx=u.t() @ dv, A_log=(dg * g).sum(0),
               dt_bias=da.sum(0))
    # every path is a few hundred fp32 roundings long (2^-24 each, 130 tokens, sums of 181 rows): 1e-4 of the largest
    # element leaves a factor of ten over 180 * 2^-24
    for k, r in dict(want, y=y, last=last, s=s).items():
        o = dict(got, y=y1, last=last1, s=s1)[k].double()
        assert (o - r).abs().max() <= 1e-4 * r.abs().max(), k


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_serving(dtype):
    """Prompts through the prefill, then tokens one at a time through the pool,
    in a captured graph, against all tokens at once in the same types."""
    lens, steps, width, D = [20, 300, 1], 5, 128, 64
    p, n = params(2, width, D)
    T = sum(lens) + 3 * steps
    x, res = n(T, width).to(DEV).to(dtype), n(T, width).to(DEV).to(dtype)
    whole = [m + steps for m in lens]
    cu = [0] + list(np.cumsum(whole))
    on = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731

    def gates(rows_x, rows_res):
        u, s, _ = gdr.rmsnorm_fwd(rows_x, p["w"], residual=rows_res, eps=EPS)
        a, b, v = (t.to(dtype) for t in mixer(p, u.float()))
        g, beta = gdr.gating_fwd(a, p["dt_bias"], p["A_log"], b)
        return (beta * v).contiguous(), g

    inp, g = gates(x, res)
    want, _ = gdr.linrec_fwd(inp, g, on(cu))
    head = torch.cat([torch.arange(cu[i], cu[i] + lens[i]) for i in range(3)]).to(DEV)
    inp, g = gates(x[head], res[head])
    got, last = gdr.linrec_fwd(inp, g, on([0] + list(np.cumsum(lens))))
    tol = 2.0 ** -6 if dtype == torch.bfloat16 else 1e-5   # of the largest: the products' own rounding at other shapes
    assert (got.float() - want[head].float()).abs().max() <= tol * want.abs().max()
    pool, idx = torch.zeros(7, D, device=DEV), on([6, 1, 3])
    pool[idx.long()] = last
    tx, tr = torch.empty(3, width, device=DEV, dtype=dtype), torch.empty(3, width, device=DEV, dtype=dtype)
    one = on([0, 1, 2, 3])

    def token():
        i, g = gates(tx, tr)
        return gdr.linrec_step(i, g, pool, idx, one)

    tx.zero_(), tr.zero_()
    keep = pool.clone()
    token()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token()
    pool.copy_(keep)
    for k in range(steps):
        rows = torch.tensor([cu[i] + lens[i] + k for i in range(3)], device=DEV)
        tx.copy_(x[rows]), tr.copy_(res[rows])
        graph.replay()
        assert (out.float() - want[rows].float()).abs().max() <= tol * want.abs().max()
