"""Pins of the fp64 oracle of the gated linear recurrence and the row norm:
closed forms, an explicit sum, and gradients against central differences."""
import numpy as np
import pytest

import oracle


def _case(seed, lens, D, g_lo=-1.0):
    r = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lens)])
    T = int(cu[-1])
    return r, cu, r.standard_normal((T, D)), r.uniform(g_lo, 0, (T, D)), r.standard_normal((len(lens), D))


def test_linrec_equals_the_explicit_sum():
    _, cu, x, g, h0 = _case(1, [3, 0, 5, 1], 4)
    y, final = oracle.linrec(x, g, cu, initial_state=h0)
    for n in range(4):
        for t in range(cu[n], cu[n + 1]):
            G = lambda s: g[s:t + 1].sum(0)  # noqa: E731  decay from before token s to token t
            want = np.exp(G(cu[n])) * h0[n] + sum(np.exp(G(s + 1)) * x[s] for s in range(cu[n], t + 1))
            np.testing.assert_allclose(y[t], want, rtol=1e-13, atol=1e-13)
        want = y[cu[n + 1] - 1] if cu[n + 1] > cu[n] else h0[n]
        np.testing.assert_array_equal(final[n], want)


def test_linrec_closed_forms():
    _, cu, x, _, h0 = _case(2, [6, 4], 3)
    zero, gone = np.zeros_like(x), np.full_like(x, -np.inf)
    y, _ = oracle.linrec(x, zero, cu)                      # no decay: running sums
    np.testing.assert_allclose(y[:6], np.cumsum(x[:6], 0), rtol=1e-13)
    np.testing.assert_allclose(y[6:], np.cumsum(x[6:], 0), rtol=1e-13)
    y, final = oracle.linrec(x, gone, cu, initial_state=h0)  # full decay: the input alone
    np.testing.assert_array_equal(y, x)
    y, _ = oracle.linrec(zero, zero - 0.5, cu, initial_state=h0)  # no input: geometric
    np.testing.assert_allclose(y[9], h0[1] * np.exp(-2.0), rtol=1e-13)


def test_linrec_bwd_against_differences():
    r, cu, x, g, h0 = _case(3, [4, 0, 1, 6], 3)
    wy, wf = r.standard_normal(x.shape), r.standard_normal(h0.shape)

    def loss(x, g, h0):
        y, f = oracle.linrec(x, g, cu, initial_state=h0)
        return (wy * y).sum() + (wf * f).sum()

    y, _ = oracle.linrec(x, g, cu, initial_state=h0)
    got = oracle.linrec_bwd(wy, g, y, cu, initial_state=h0, d_final_state=wf)
    for k, grad in enumerate(got):
        arg = [x, g, h0][k]
        for i in np.ndindex(arg.shape):
            args = [[a.copy() for a in (x, g, h0)] for _ in range(2)]
            args[0][k][i] += 1e-5
            args[1][k][i] -= 1e-5
            d = (loss(*args[0]) - loss(*args[1])) / 2e-5
            # central differences: error h^2 f''' / 6 ~ 1e-10 and roundoff 1e-16 |loss| / 1e-5 ~ 1e-10
            assert abs(d - grad[i]) < 1e-7 * (1 + abs(d))


@pytest.mark.parametrize("eps", [0.0, 1e-6, 0.5])
def test_rmsnorm_and_gradient_against_differences(eps):
    r = np.random.default_rng(4)
    s, w, dy = r.standard_normal((3, 5)), r.standard_normal(5), r.standard_normal((3, 5))
    y = oracle.rmsnorm(s, w, eps)
    np.testing.assert_allclose(((y / w) ** 2).mean(1), (s ** 2).mean(1) / ((s ** 2).mean(1) + eps), rtol=1e-12)
    ds, dw = oracle.rmsnorm_bwd(dy, s, w, eps)
    for arg, grad in ((s, ds), (w, dw)):
        for i in np.ndindex(arg.shape):
            keep = arg[i]
            arg[i] = keep + 1e-5
            hi = (dy * oracle.rmsnorm(s, w, eps)).sum()
            arg[i] = keep - 1e-5
            lo = (dy * oracle.rmsnorm(s, w, eps)).sum()
            arg[i] = keep
            assert abs((hi - lo) / 2e-5 - grad[i]) < 1e-7 * (1 + abs(grad[i]))


def test_rmsnorm_matches_the_gated_norm_of_decode():
    r = np.random.default_rng(5)
    o, w = r.standard_normal((2, 3, 8)), r.standard_normal(8)
    big = np.full(o.shape, 60.0)                            # sigmoid(60) = 1 to 1e-26
    np.testing.assert_allclose(oracle.gated_rmsnorm(o, w, big, 1e-6), oracle.rmsnorm(o, w, 1e-6), rtol=1e-12)
