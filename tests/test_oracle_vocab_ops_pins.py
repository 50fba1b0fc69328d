"""Pins of oracle/vocab_ops.py to something other than itself (CPU)."""
import math

import numpy as np
import pytest

from oracle import vocab_ops as O


def draw(T=4, H=6, V=11, seed=0):
    r = np.random.Generator(np.random.PCG64(seed))
    return r, r.standard_normal((T, H)), r.standard_normal((V, H))


def test_uniform_distribution_closed_forms():
    V, K = 9, 4
    h, W, y = np.zeros((3, 5)), np.ones((V, 5)), np.array([0, 8, -100])
    logp, lse, ent, top, ids = O.top_forward(h, W, y, K)
    assert np.allclose(logp, [-math.log(V)] * 2 + [0]) and np.allclose(ent, [math.log(V)] * 2 + [0])
    assert (ids[:2] == np.arange(K)).all() and (ids[2] == -1).all()       # ties to the lowest id
    assert np.allclose(top[:2], -math.log(V)) and (top[2] == -np.inf).all()
    # a teacher of n equal tokens against the uniform student: KL = log V - log n
    loss, _, lp = O.distill_forward(h, W, np.array([[3, 1, -1]] * 3), np.zeros((3, 3)), 2.0)
    assert np.allclose(loss, math.log(V) - math.log(2)) and (lp[:, 2] == -np.inf).all()


def test_student_equal_to_the_teacher_has_no_loss():
    _, h, W = draw(V=6)
    z = O.logits(h, W)
    ids = np.tile(np.arange(6), (4, 1))
    loss, _, _ = O.distill_forward(h, W, ids, z, 1.5)
    dz, _ = O.distill_dz(h, W, ids, z, np.ones(4), 1.5)
    assert np.abs(loss).max() < 1e-12 and np.abs(dz).max() < 1e-12


def test_alternatives_and_entropy_by_brute_force():
    _, h, W = draw(seed=3)
    logp, lse, ent, top, ids = O.top_forward(h, W, np.array([2, 5, 0, 10]), 13)
    for t in range(4):
        z = [float(h[t] @ W[v]) for v in range(11)]
        s = sum(math.exp(x) for x in z)
        assert math.isclose(lse[t], math.log(s), abs_tol=1e-12)
        assert math.isclose(ent[t], -sum(math.exp(x) / s * math.log(math.exp(x) / s) for x in z), abs_tol=1e-12)
        assert ids[t, :11].tolist() == sorted(range(11), key=lambda v: (-z[v], v)) and (ids[t, 11:] == -1).all()
        assert math.isclose(np.exp(top[t, :11]).sum(), 1.0, abs_tol=1e-12)


@pytest.mark.parametrize("tau", [1.0, 0.5, 3.0])
def test_gradients_by_central_differences(tau):
    r, h, W = draw(seed=5)
    y = np.array([1, -100, 7, 3])
    g, ge = r.standard_normal(4), r.standard_normal(4)
    ids = np.array([[4, 2, 4], [-1, -1, 0], [0, 9, 5], [1, 8, 2]])  # a token twice; an empty row below
    tl = r.standard_normal((4, 3))
    tl[1] = -np.inf
    f_top = lambda a, b: (lambda o: (g * o[0]).sum() + (ge * o[2]).sum())(O.top_forward(a, b, y, 0))  # noqa: E731
    f_dis = lambda a, b: (g * O.distill_forward(a, b, ids, tl, tau)[0]).sum()  # noqa: E731
    for f, dz in ((f_top, O.top_dz(h, W, y, g, ge)[0]), (f_dis, O.distill_dz(h, W, ids, tl, g, tau)[0])):
        for x, grad in ((h, dz @ W), (W, dz.T @ h)):
            for at in np.ndindex(x.shape):
                d = 1e-5
                keep = x[at]
                x[at] = keep + d
                up = f(h, W)
                x[at] = keep - d
                down = f(h, W)
                x[at] = keep
                assert math.isclose((up - down) / (2 * d), grad[at], abs_tol=1e-7)
