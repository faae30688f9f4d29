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
