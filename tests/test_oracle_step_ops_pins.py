"""Pins of the fp64 oracle of the operators before and behind the LM head:
closed forms, torch's own operators, central differences."""
import numpy as np
import pytest
import torch

from oracle import step_ops as O

RNG = np.random.Generator(np.random.PCG64(7))


def test_norms_closed_forms():
    x = np.array([[3.0, 1.0, 3.0, 1.0]])  # mean 2, deviation 1
    y, n, mean, rstd = O.norm_forward(x, None, None, 0.0, True)
    assert mean[0] == 2.0 and rstd[0] == 1.0 and np.array_equal(y, [[1, -1, 1, -1]])
    x = np.array([[6.0, 8.0]])  # mean square 50
    y, _, _, rstd = O.norm_forward(x, np.array([2.0, 1.0]), None, 0.0, False)
    assert rstd[0] == pytest.approx(1 / np.sqrt(50)) and np.allclose(y, [[12 / np.sqrt(50), 8 / np.sqrt(50)]])
    # a constant row: the deviation is the eps alone
    y, _, _, rstd = O.norm_forward(np.full((1, 5), 7.0), None, np.ones(5), 0.25, True)
    assert rstd[0] == 2.0 and np.array_equal(y, np.ones((1, 5)))


def test_norms_against_torch():
    x, w, b = RNG.normal(size=(6, 11)) * 3 + 1, RNG.normal(size=11), RNG.normal(size=11)
    want = torch.nn.functional.layer_norm(torch.tensor(x), (11,), torch.tensor(w), torch.tensor(b), 1e-3).numpy()
    assert np.allclose(O.norm_forward(x, w, b, 1e-3, True)[0], want, rtol=1e-13, atol=1e-13)
    want = torch.nn.functional.rms_norm(torch.tensor(x), (11,), torch.tensor(w), 1e-3).numpy()
    assert np.allclose(O.norm_forward(x, w, None, 1e-3, False)[0], want, rtol=1e-13, atol=1e-13)


@pytest.mark.parametrize("center", [False, True])
def test_norm_gradients_against_differences(center):
    x, w, b, g = RNG.normal(size=(3, 7)), RNG.normal(size=7), RNG.normal(size=7), RNG.normal(size=(3, 7))
    eps, h = 1e-2, 1e-6

    def loss(x, w, b):
        return (g * O.norm_forward(x, w, b, eps, center)[0]).sum()

    gx, gw, gb = O.norm_backward(x, w, g, eps, center)
    for at in np.ndindex(3, 7):
        e = np.zeros((3, 7))
        e[at] = h
        assert gx[at] == pytest.approx((loss(x + e, w, b) - loss(x - e, w, b)) / (2 * h), abs=1e-7)
    for j in range(7):
        e = np.eye(7)[j] * h
        assert gw[j] == pytest.approx((loss(x, w + e, b) - loss(x, w - e, b)) / (2 * h), abs=1e-7)
        assert gb[j] == pytest.approx((loss(x, w, b + e) - loss(x, w, b - e)) / (2 * h), abs=1e-7)
    if center:  # a shift of a row changes nothing
        assert np.allclose(gx.sum(axis=1), 0, atol=1e-12)
    # nor does a scaling, but for eps
    g0, _, _ = O.norm_backward(x, w, g, 0.0, center)
    assert np.allclose((g0 * x).sum(axis=1), 0, atol=1e-12)


def test_embedding():
    E = RNG.normal(size=(9, 4))
    ids = np.array([3, 0, -100, 3, 8, 9, -1, 2 ** 40, 3])
    out = O.embed_forward(ids, E, 0.5)
    assert np.array_equal(out[[0, 1, 3, 4]], 0.5 * E[[3, 0, 3, 8]]) and not out[2].any()
    assert np.isnan(out[5:8]).all()
    g = RNG.normal(size=(9, 4))
    grad = O.embed_backward(ids, g, 9, 0.5)
    assert np.allclose(grad[3], 0.5 * (g[0] + g[3] + g[8])) and np.allclose(grad[8], 0.5 * g[4])
    assert not grad[[1, 2, 4, 5, 6, 7]].any()
    # the gradient of sum(g * out) over live rows
    live = [0, 1, 3, 4, 8]
    for at in [(3, 1), (0, 0), (8, 3), (5, 2)]:
        e = np.zeros((9, 4))
        e[at] = 1e-6
        d = sum((g[t] * (O.embed_forward(ids, E + e, 0.5) - O.embed_forward(ids, E - e, 0.5))[t]).sum() for t in live)
        assert grad[at] == pytest.approx(d / 2e-6, abs=1e-8)


def test_norm_and_clipping():
    ts = [np.array([3.0]), np.zeros((0, 4)), np.array([[0.0, 4.0]])]
    assert O.grad_norm(ts) == 5.0
    assert O.clip_factor(ts, 5.0) == 1.0 and O.clip_factor(ts, 1.0) == 0.2 and O.clip_factor(ts, np.inf) == 1.0
    assert O.grad_norm([np.array([3e200, 4e200]) * 1e-100]) == pytest.approx(5e100)
