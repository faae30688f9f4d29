"""The norm's e4m3 output where a code's choice is exact: rows of +-1 with
eps = 0 have a norm of exactly +-1, so that y is the weight to the last bit, and
weights are made of a group's scale times numbers of few bits.  No tolerance."""
import pytest
import torch

import gated_delta_rule_37_gb300 as gdr
from tests.gpu_util import bits_equal

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdr.load()


def signs(M, D, dtype, aligned, r):
    """Rows of +-1, 16-byte aligned or not."""
    one = (2.0 * torch.randint(0, 2, (M, D), generator=r) - 1).to(dtype)
    wide = torch.zeros(M, D + 9, dtype=dtype, device=DEV)
    out = wide[:, 1:1 + D] if not aligned else torch.zeros(M, D, dtype=dtype, device=DEV)
    out.copy_(one)
    return one.float(), out


def midpoints():
    """The numbers half-way between two neighbouring magnitudes of e4m3."""
    v = torch.arange(0, 127, dtype=torch.uint8).view(E4).double()
    return (v[1:] + v[:-1]) / 2


@pytest.mark.parametrize("aligned", [True, False], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("D", [128, 2048, 16384])
def test_values_half_way_between_codes(D, group, dtype, aligned):
    """scale = max / 448 exactly, and every quotient a midpoint exactly: the even code."""
    r = torch.Generator().manual_seed(D + group)
    span = group or D
    mids = midpoints()
    m = mids[torch.randint(0, len(mids), (D,), generator=r)].view(-1, span)
    m[:, 5] = 448                                          # a group's largest
    # 19 bits: times a midpoint's 5 or 448's 3, a number of 24
    s = torch.randint(1 << 18, 1 << 19, (D // span, 1), generator=r).double() * 2.0 ** -20
    w = (m * s).float()
    assert (w.double() == m * s).all() and ((w[:, 5:6] / 448).double() == s).all()
    sign, x = signs(7, D, dtype, aligned, r)
    q, _, scales = gdr.rmsnorm_fwd(x, w.flatten().to(DEV), eps=0.0, y_dtype=E4, scale_group=group)
    assert bits_equal(scales, s.float().view(1, -1).expand(7, -1))
    want = (sign * m.flatten().float()).to(E4)
    assert bits_equal(q.cpu().view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("aligned", [True, False], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("D", [256, 2048, 16384])
def test_a_bad_value_in_a_group(D, group, dtype, aligned):
    """A NaN among a group's values makes its scale and its codes NaN, an
    infinity its scale infinite, its own code NaN and the others 0; the other
    groups are as they were."""
    r = torch.Generator().manual_seed(D + group)
    span = group or D
    w = torch.randn(D, generator=r)
    _, x = signs(5, D, dtype, aligned, r)
    call = lambda w: [t.cpu() for t in gdr.rmsnorm_fwd(x, w.to(DEV), eps=0.0, y_dtype=E4, scale_group=group)[::2]]  # noqa: E731
    q0, s0 = call(w)
    for value in (float("nan"), float("inf"), -float("inf")):
        bad = w.clone()
        bad[D - 3] = value                                 # in the last group
        q, s = call(bad)
        hit = torch.arange(D) >= D - span
        assert bits_equal(q.view(torch.uint8)[:, ~hit], q0.view(torch.uint8)[:, ~hit])
        assert bits_equal(s[:, :-1], s0[:, :-1])
        own = q.float()[:, hit]
        if value != value:
            assert torch.isnan(s[:, -1]).all() and torch.isnan(own).all()
        else:
            assert (s[:, -1] == float("inf")).all() and torch.isnan(own[:, span - 3]).all()
            own[:, span - 3] = 0
            assert (own == 0).all()


@pytest.mark.parametrize("aligned", [True, False], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("dtype,ints", [(BF, torch.int16), (F, torch.int32)], ids=["bf16", "f32"])
def test_residual_addition_of_any_bits(dtype, ints, aligned):
    """The stored sum is the rounded sum for all exponents: subnormal numbers,
    sums that overflow or cancel, infinities, NaN."""
    r = torch.Generator().manual_seed(5)
    M, D = 1500, 1000
    a, b = (torch.randint(-(1 << 8 * dtype.itemsize - 1), 1 << 8 * dtype.itemsize - 1, (M, D), generator=r).to(ints).view(dtype)
            for _ in range(2))
    b[: M // 3] = (a[: M // 3].view(ints) ^ torch.randint(0, 4, (M // 3, D), generator=r).to(ints)).view(dtype).neg()
    near = torch.randint(-300, 300, (M // 3, D), generator=r).to(ints)
    b[M // 3: 2 * (M // 3)] = (a[M // 3: 2 * (M // 3)].view(ints) + near * (1 << 8 * dtype.itemsize - 12)).view(dtype)
    wide = torch.zeros(2, M, D + 8, dtype=dtype, device=DEV)
    at = 0 if aligned else 1
    x, res = wide[0, :, at:at + D], wide[1, :, at:at + D]
    x.copy_(a)
    res.copy_(b)
    got = gdr.rmsnorm_fwd(x, torch.ones(D, device=DEV), residual=res)[1].cpu()
    want = (a.double() + b.double()).to(dtype) if dtype == F else (a.float() + b.float()).to(dtype)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan) and torch.equal(got.view(ints)[~nan], want.view(ints)[~nan])
