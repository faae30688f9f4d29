"""The accuracy of channels of long memory, in the 2-norm.

A decay near 1 is applied thousands of times: an error of its that has a mean of
0.3 * 2^-24 leaves 0.3 * 2^-24 * 4000 = 7e-5 of a state with a memory of 4000
tokens, well inside the element-wise bounds of tests/test_gpu_linrec.py, which add
the worst case of every step.  Without a mean, roundings add up as a random walk.
A state passes one composition per run of R tokens, so memory / R of them, the
k-th last weighted by e^-(k R / memory) in the state and by e^-(2 k R / memory)
in its variance, which sums to memory / (2 R).  The roundings of a composition's
decay (0.3 of 2^-24 on average) and of its fused multiply-add (0.4) are together
0.5 * 2^-24 = 2^-25.  Allowed is twice that walk: 2 * 2^-25 * sqrt(memory / (2 R)),
0.6e-6 to 1.6e-6 here."""
import numpy as np
import pytest
import torch

import gated_delta_rule_37_gb300 as gdr
import oracle
from tests.test_gpu_linrec import BF, DEV, F, f64

pytestmark = pytest.mark.gpu
MEMORY, T = 4000, 16000
# tokens of a run: (aligned, unaligned) by type and direction
RUN = {(BF, "fwd"): (7, 24), (BF, "bwd"): (5, 16), (F, "fwd"): (5, 20), (F, "bwd"): (3, 12)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdr.load()


def case(D, dtype, gate):
    r = torch.Generator().manual_seed(D)
    g = (-(0.1 + 1.8 * torch.rand(T, D, generator=r)) / MEMORY).to(gate)
    return dict(g=g, x=torch.randn(T, D, generator=r).to(dtype), y=torch.randn(T, D, generator=r).to(dtype),
                h0=100 * torch.randn(1, D, generator=r), cu=torch.tensor([0, T], dtype=torch.int32))


def allowed(dtype, way, D):
    return 2 * 2.0 ** -25 * (MEMORY / (2 * RUN[dtype, way][D % 8 != 0])) ** 0.5


def off(got, want):
    return np.linalg.norm(f64(got) - want) / np.linalg.norm(want)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("gate", [BF, F], ids=["bf16-gates", "f32-gates"])
@pytest.mark.parametrize("D", [64, 65])
def test_long_memory(D, gate, dtype):
    c = case(D, dtype, gate)
    dev = {k: v.to(DEV) for k, v in c.items()}
    y, last = gdr.linrec_fwd(dev["x"], dev["g"], dev["cu"], initial_state=dev["h0"])
    want, want_last = oracle.linrec(f64(c["x"]), f64(c["g"]), c["cu"], initial_state=c["h0"])
    assert off(last, want_last) <= allowed(dtype, "fwd", D)
    dx, dg, first = gdr.linrec_bwd(dev["x"], dev["g"], dev["y"], dev["cu"], initial_state=dev["h0"],
                                   d_final_state=dev["h0"])
    wx, wg, wf = oracle.linrec_bwd(f64(c["x"]), f64(c["g"]), f64(c["y"]), c["cu"], initial_state=c["h0"],
                                   d_final_state=c["h0"])
    assert off(first, wf) <= allowed(dtype, "bwd", D)
    if dtype == F:
        assert off(y, want) <= allowed(dtype, "fwd", D) and off(dx, wx) <= allowed(dtype, "bwd", D)
        if gate == F:
            assert off(dg, wg) <= allowed(dtype, "bwd", D) + 2.0 ** -24


def test_the_bound_sees_a_mean_error():
    """The oracle with decays that are 0.3 * 2^-24 low on average is far outside."""
    c = case(64, F, F)
    g, want = f64(c["g"]), oracle.linrec(f64(c["x"]), f64(c["g"]), c["cu"], initial_state=c["h0"])[1]
    low = oracle.linrec(f64(c["x"]), g - 0.3 * 2.0 ** -24, c["cu"], initial_state=c["h0"])[1]
    assert np.linalg.norm(low - want) / np.linalg.norm(want) > 5 * allowed(F, "bwd", 64)


@pytest.mark.parametrize("D", [64, 65])
def test_long_memory_of_the_step(D):
    """All tokens through the slot pool, one composition each."""
    c = case(D, F, F)
    pool = c["h0"].to(DEV)
    gdr.linrec_step(c["x"].to(DEV), c["g"].to(DEV), pool, torch.zeros(1, dtype=torch.int32, device=DEV), c["cu"].to(DEV))
    want = oracle.linrec(f64(c["x"]), f64(c["g"]), c["cu"], initial_state=c["h0"])[1]
    assert off(pool, want) <= 2 * 2.0 ** -25 * (MEMORY / 2) ** 0.5
