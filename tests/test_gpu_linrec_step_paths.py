"""The slot-pool step over its variants (1, 2, 4 and 8 channels per thread, chosen
by N * D and the SMs) and over all gates.

Bounds are those of tests/test_gpu_linrec.py.  The exponential by itself: its
argument is reduced by two fused steps to |r| <= 0.35, each off by 2^-26 at most;
the polynomial's last step rounds by 2^-24 of the result, the ones before by
0.35 * 2^-24 and less, its first omitted term is 0.1 * 2^-24: 2.2 * 2^-24 of the
value, 3 * 2^-24 allowed."""
import numpy as np
import pytest
import torch

import gated_delta_rule_37_gb300 as gdr
from tests.gpu_util import sentinel_like
from tests.test_gpu_linrec import BF, DEV, F, TYPES, check_step, f64, pool_case, run_step

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdr.load()


def sizes():
    """N and D on both sides of the two thresholds (152 SMs: 466,944 and 933,888 channels in all)."""
    return [(228, 2040), (228, 2048), (455, 2048), (456, 2048), (256, 4096), (57, 16384), (150, 8192)]


def lengths(N, most):
    r = torch.Generator().manual_seed(N)
    return torch.randint(0 if most > 1 else 1, most + 1, (N,), generator=r).tolist()


@pytest.mark.parametrize("pool_dtype", [F, BF], ids=["f32-pool", "bf16-pool"])
@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(d)[6:] for d in t))
@pytest.mark.parametrize("N,D", sizes())
def test_decode(N, D, types, pool_dtype):
    c = pool_case(N + D, [1] * N, D, *types, pool_dtype, skip={i: -1 for i in range(0, N, 11)})
    check_step(c, *run_step(c, commit=True), commit=True)


@pytest.mark.parametrize("pool_dtype", [F, BF], ids=["f32-pool", "bf16-pool"])
@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(d)[6:] for d in t))
@pytest.mark.parametrize("N,D", [(228, 2040), (228, 2048), (456, 2048), (150, 8192)])
def test_verify(N, D, types, pool_dtype):
    """0 to 5 tokens: whole and half groups of those loaded at once; states kept,
    more and fewer than there are tokens; committed or not."""
    c = pool_case(N + D, lengths(N, 5), D, *types, pool_dtype, skip={0: -1, 7: -3, N - 1: -1})
    check_step(c, *run_step(c, commit=False, steps=5), commit=False)
    check_step(c, *run_step(c, commit=True, steps=3, rows=N + 2), commit=True)


GATES = [0.0, -0.0, -2.0, -30.0, -87.2, -87.4, -200.0, -np.inf]


@pytest.mark.parametrize("types", [(F, F), (BF, BF)], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 65])
@pytest.mark.parametrize("gate", GATES)
def test_extreme_decays(gate, D, types):
    c = pool_case(64, [1, 4, 0, 7, 12], D, *types, F, skip={1: -1})
    c["g"][:, ::2] = gate
    check_step(c, *run_step(c, commit=True, steps=12), commit=True)


@pytest.mark.parametrize("D", [64, 65])
def test_wide_range_of_decays(D):
    c = pool_case(65, [3, 12, 1, 9], D, F, F, F)
    c["g"] = -100 * torch.rand(c["T"], D, generator=torch.Generator().manual_seed(1)) ** 3
    check_step(c, *run_step(c, commit=True, steps=12), commit=True)


@pytest.mark.parametrize("D", [64, 65])
def test_a_bad_gate_stays_in_its_sequence_and_channel(D):
    lens = [2, 6, 3]
    c = pool_case(66, lens, D, F, F, F)
    pool0, y0, _ = run_step(c, commit=True)
    at = int(c["cu"][1]) + 2
    c["g"][at, 5] = np.nan
    pool, y, _ = run_step(c, commit=True)
    hit = torch.zeros(c["T"], D, dtype=torch.bool)
    hit[at:int(c["cu"][2]), 5] = True
    assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], y0[~hit])
    slot = torch.zeros_like(pool, dtype=torch.bool)
    slot[int(c["idx"][1]), 5] = True
    assert torch.isnan(pool[slot]).all() and torch.equal(pool[~slot], pool0[~slot])


@pytest.mark.parametrize("D", [4096, 4095])
def test_exponential(D):
    """States of 1 and rows of 0: every output is a decay, exp(g) of any g that gives a normal number."""
    r = torch.Generator().manual_seed(67)
    N = 256
    g = -87.3 * torch.rand(N, D, generator=r)
    g[: N // 2] = -(2.0 ** -(30 * torch.rand(N // 2, D, generator=r)))
    one = torch.ones(N, D, device=DEV)
    cu, idx = torch.arange(N + 1, dtype=torch.int32, device=DEV), torch.arange(N, dtype=torch.int32, device=DEV)
    y = gdr.linrec_step(torch.zeros(N, D, device=DEV), g.to(DEV), one, idx, cu)
    scan, last = gdr.linrec_fwd(torch.zeros(N, D, device=DEV), g.to(DEV), cu, initial_state=torch.ones(N, D, device=DEV))
    want = np.exp(f64(g))
    for got in (y, one, scan, last):
        assert (np.abs(f64(got) - want) <= 3 * U * want).all()


@pytest.mark.parametrize("D", [4096, 4095])
def test_offsets_beyond_32_bits(D):
    """Slots, rows and kept states whose elements' numbers pass 2^31: the last ones against 64 bits."""
    N, n, steps = (1 << 31) // (3 * D) + 40, 30, 3
    c = pool_case(68, [1 + i % 3 for i in range(n)], D, BF, BF, BF, skip={4: -1})
    T, slots = N - n + c["T"], (1 << 31) // D + 50
    assert (N - n) * steps * D > 1 << 31 and (slots - 40) * D > 1 << 31
    # sequences before: padding of one token each
    big = {k: torch.zeros(T, D, dtype=BF, device=DEV) for k in ("x", "g")}
    for k, v in big.items():
        v[T - c["T"]:] = c[k].to(DEV)
    pool = torch.zeros(slots, D, dtype=BF, device=DEV)
    first = slots - c["pool"].shape[0]
    pool[first:] = c["pool"].to(DEV)
    idx = torch.full((N,), -1, dtype=torch.int32)
    idx[N - n:] = torch.where(c["idx"] >= 0, c["idx"] + first, c["idx"])
    cu = torch.cat([torch.arange(N - n, dtype=torch.int32), c["cu"] + (N - n)])
    states = torch.zeros(N, steps, D, dtype=BF, device=DEV)
    y = torch.zeros(T, D, dtype=BF, device=DEV)
    gdr.linrec_step(big["x"], big["g"], pool, idx.to(DEV), cu.to(DEV), y=y, intermediate_states=states)
    assert not y[:N - n].any() and not states[:N - n].any() and not pool[:first].any()
    tail = sentinel_like((c["T"], D), BF)
    kept = sentinel_like((n, steps, D), BF)
    got_y, got_s = y[N - n:].cpu(), states[N - n:].cpu()
    at = [int(v) for v in c["cu"]]
    for k, i in enumerate(c["idx"].tolist()):
        if i >= 0:
            tail[at[k]:at[k + 1]] = got_y[at[k]:at[k + 1]]
            kept[k, :at[k + 1] - at[k]] = got_s[k, :at[k + 1] - at[k]]
        else:
            assert not got_y[at[k]:at[k + 1]].any()
        assert not got_s[k, at[k + 1] - at[k] if i >= 0 else 0:].any()
    check_step(c, pool[first:].cpu(), tail, kept, commit=True)
