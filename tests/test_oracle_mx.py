"""The float64 reference of the 4-bit floating-point operators and the token
statistics: values worked out by hand, and gradients against differences.

Central differences in float64 with step h = 1e-5 on smooth functions: the
truncation error is h^2 / 6 times a third derivative of order one (2e-11
of the values), the rounding 2^-53 / h of them (1e-11); 1e-7 leaves room
for third derivatives and values in the hundreds."""

import numpy as np
import pytest

import oracle as orc

H, TOL = 1e-5, 1e-7


def differences(f, x):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + H
        up = f()
        x[i] = keep - H
        down = f()
        x[i] = keep
        g[i] = (up - down) / (2 * H)
    return g


def test_a_block_by_hand():
    # largest magnitude 7 = 1.75 2^2: power 0; ties go to the even code
    x = np.zeros((1, 33))
    x[0, :12] = [7.0, -6.5, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.2, 0.26, 4.99]
    x[0, 32] = -0.75                                  # its own block: power -3, 6 of them
    codes, scales, hat = orc.mx_quantize(x)
    assert codes.shape == (1, 32) and scales.tolist() == [[127, 124]]
    want = [6, -6, 4, 4, 2, 2, 1, 1, 0, 0, 0.5, 4]
    assert hat[0, :12].tolist() == want and hat[0, 32] == -0.75
    assert codes[0, 0] == 7 | (15 << 4) and codes[0, 4] == 0 | (8 << 4) and codes[0, 16] == 15
    assert not codes[0, 17:].any()


def test_powers_zeros_and_what_is_not_finite():
    x = np.zeros((5, 32))
    x[0, 3] = 2.0 ** -10
    x[1, 3] = 2.0 ** -140
    x[2, 5] = np.nan
    x[3, 5] = -np.inf
    codes, scales, hat = orc.mx_quantize(x)
    assert scales[:, 0].tolist() == [127 - 12, 0, 255, 255, 0]
    assert hat[0, 3] == 2.0 ** -10 and hat[1, 3] == 0.0 and not codes[2:].any()
    assert np.isnan(hat[2:4]).all() and not hat[4].any()


def test_values_of_all_codes():
    codes = (np.arange(0, 16, 2) | (np.arange(1, 16, 2) << 4)).astype(np.uint8)[None]
    codes = np.concatenate([codes, np.zeros((1, 8), np.uint8)], 1)
    v = orc.mx_values(codes, np.array([[128]], np.uint8), 16)[0]
    assert v[:8].tolist() == [0, 1, 2, 3, 4, 6, 8, 12] and (v[8:] == -v[:8]).all()


@pytest.mark.parametrize("act", ["none", "relu", "silu"])
def test_gated_gradients_are_differences(act):
    rng = np.random.default_rng(3)
    X, Wg, Wu = rng.normal(size=(3, 5)), rng.normal(size=(4, 5)), rng.normal(size=(4, 5))
    dY = rng.normal(size=(3, 4))
    value = lambda: float((dY * orc.mx_gate(X @ Wg.T, act) * (X @ Wu.T)).sum())  # noqa: E731
    dX, dG, dU = orc.mx_gated_backward(dY, X @ Wg.T, X @ Wu.T, Wg, Wu, act)
    assert np.abs(dX - differences(value, X)).max() < TOL
    G, U = X @ Wg.T, X @ Wu.T
    value = lambda: float((dY * orc.mx_gate(G, act) * U).sum())  # noqa: E731
    assert np.abs(dG - differences(value, G)).max() < TOL
    assert np.abs(dU - differences(value, U)).max() < TOL


def test_token_statistics_by_hand():
    z = np.log(np.array([[1.0, 2.0, 1.0, 4.0], [1.0, 1.0, 1.0, 1.0]]))
    z[1, 2] = -np.inf
    logp, entropy, lse, top, idx = orc.token_stats(z, [1, -1], 3, 1.0)
    assert np.allclose(logp, [np.log(0.25), 0.0]) and np.allclose(lse, np.log([8.0, 3.0]))
    assert np.allclose(entropy, [1.75 * np.log(2.0), np.log(3.0)])
    assert idx.tolist() == [[3, 1, 0], [0, 1, 3]] and np.allclose(top[0], np.log([4.0, 2.0, 1.0]))
    logp, _, lse, top, idx = orc.token_stats(np.array([[np.nan, 1.0], [-np.inf, -np.inf]]), [0, 0], 2, 1.0)
    assert np.isnan(logp).all() and lse[1] == -np.inf and idx.tolist() == [[1, -1], [0, 1]]


def test_token_gradient_is_differences():
    rng = np.random.default_rng(4)
    z, T = rng.normal(size=(4, 7)), 1.3
    tokens, g, h = [3, -1, 6, 0], rng.normal(size=4), rng.normal(size=4)
    g[3] = h[3] = 0.0

    def value():
        logp, entropy, *_ = orc.token_stats(z, tokens, 0, T)
        return float((g * logp + h * entropy).sum())

    assert np.abs(orc.token_grad(z, tokens, g, h, T) - differences(value, z)).max() < TOL
