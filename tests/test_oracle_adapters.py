"""The float64 reference of the adapter products and the distillation loss
against differences of its own forward values and against values worked out
by hand.

Central differences in float64 with step h = 1e-5 on smooth functions: the
truncation error is h^2 / 6 times a third derivative of order one (2e-11
of the values), the rounding 2^-53 / h of them (1e-11); 1e-7 leaves room
for third derivatives and values in the hundreds."""

import numpy as np
import pytest

import oracle as orc

H = 1e-5
TOL = 1e-7


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


def test_lora_gradients_are_differences():
    rng = np.random.default_rng(1)
    n, m, d, r, L = 5, 4, 6, 2, 3
    X, W = rng.normal(size=(n, d)), rng.normal(size=(m, d))
    A, B, alpha = rng.normal(size=(L, r, d)), rng.normal(size=(L, m, r)), rng.uniform(1, 2, L)
    ids = np.array([2, -1, 0, 2, 7])          # adapter 1 has no row, two rows have no adapter
    dY = rng.normal(size=(n, m))
    value = lambda: float((dY * orc.lora_matmul(X, W, A, B, alpha, ids)[0]).sum())  # noqa: E731
    hidden = orc.lora_matmul(X, W, A, B, alpha, ids)[1]
    dX, dA, dB = orc.lora_backward(dY, X, hidden, W, A, B, alpha, ids)
    assert np.abs(dX - differences(value, X)).max() < TOL
    assert np.abs(dA - differences(value, A)).max() < TOL
    assert np.abs(dB - differences(value, B)).max() < TOL
    assert not dA[1].any() and not dB[1].any()


@pytest.mark.parametrize("tail", [False, True])
def test_distill_gradient_is_differences(tail):
    rng = np.random.default_rng(2)
    n, vocab, k, T = 4, 9, 3, 1.5
    z = rng.normal(size=(n, vocab))
    teacher = rng.normal(size=(n, vocab))
    idx = np.argsort(-teacher, axis=1)[:, :k]
    t = np.take_along_axis(teacher, idx, 1)
    idx[1, 2] = -1
    t_lse = np.log(np.exp(teacher / T).sum(1)) if tail else None
    w = np.array([1.0, 0.5, 0.0, 2.0])
    value = lambda: float(orc.distill(z, idx, t, T, t_lse, w)[0].sum())  # noqa: E731
    grad = orc.distill(z, idx, t, T, t_lse, w)[1]
    assert np.abs(grad - differences(value, z)).max() < TOL
    assert not grad[2].any()


def test_distill_zero_where_student_is_teacher():
    z = np.log(np.array([[0.5, 0.25, 0.125, 0.125]]))
    for t_lse in (np.array([0.0]), None):
        idx = np.array([[0, 1]]) if t_lse is not None else np.array([[0, 1, 2, 3]])
        t = z[:, : idx.shape[1]]
        loss, grad = orc.distill(z, idx, t, 1.0, t_lse)
        assert abs(loss[0]) < 1e-15 and np.abs(grad).max() < 1e-15


def test_distill_by_hand():
    # q = (1/2, 1/4, 1/4); the teacher knows id 0 alone with p = 3/4
    z = np.log(np.array([[0.5, 0.25, 0.25]]))
    loss, grad = orc.distill(z, np.array([[0]]), np.array([[np.log(0.75)]]), 1.0, np.array([0.0]))
    assert abs(loss[0] - (0.75 * np.log(1.5) + 0.25 * np.log(0.5))) < 1e-15
    assert np.abs(grad[0] - np.array([-0.25, 0.125, 0.125])).max() < 1e-15
    # renormalised, the one known id has probability 1
    loss, grad = orc.distill(z, np.array([[0]]), np.array([[5.0]]), 1.0)
    assert abs(loss[0] - np.log(2.0)) < 1e-15
    assert np.abs(grad[0] - np.array([-0.5, 0.25, 0.25])).max() < 1e-15


@pytest.mark.parametrize("case", ["masked", "whole", "over"])
def test_distill_gradient_without_the_rest_class_is_differences(case):
    """The class of all others is left out where the student has no mass there
    (every other cell -inf, or no other cell) and where the known ids' own
    probabilities reach 1 or more: their sum, not 1, multiplies q."""
    rng = np.random.default_rng(3)
    n, vocab, k, T = 3, 7, 4, 1.5
    z = rng.normal(size=(n, vocab))
    if case == "whole":
        z = z[:, :k].copy()
    idx = np.stack([rng.permutation(z.shape[1])[:k] for _ in range(n)])
    t = rng.normal(size=(n, k))
    if case == "masked":
        for r in range(n):
            z[r, np.setdiff1d(np.arange(vocab), idx[r])] = -np.inf
    known = np.log(np.exp(t / T).sum(1))
    t_lse = known + np.array([0.3, 0.7, 1.5]) * (-1 if case == "over" else 1)
    w = np.array([1.0, 0.5, 2.0])
    value = lambda: float(orc.distill(z, idx, t, T, t_lse, w)[0].sum())  # noqa: E731
    grad = orc.distill(z, idx, t, T, t_lse, w)[1]
    assert np.abs(grad - differences(value, z)).max() < TOL
    assert np.abs(grad.sum(1)).max() < 1e-14        # the loss does not see a common shift


def test_distill_without_the_rest_class_by_hand():
    # p = (.4, .2, .1) on all that is not masked: d = q * 0.7 - p
    z = np.array([[0.3, -0.2, 0.1, -np.inf, -np.inf]])
    p = np.array([0.4, 0.2, 0.1])
    grad = orc.distill(z, np.array([[0, 1, 2]]), np.log(p)[None], 1.0, np.array([0.0]))[1]
    q = np.exp(z[0, :3]) / np.exp(z[0, :3]).sum()
    assert np.abs(grad[0, :3] - (0.7 * q - p)).max() < 1e-15 and not grad[0, 3:].any()
    assert np.abs(grad[0, :3] - np.array([-0.1114, -0.0249, 0.1363])).max() < 1e-4
