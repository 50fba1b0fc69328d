"""linear_logp_top, linear_distill and linear_logp on values at the edges: a
teacher's undefined logits and those near the type's ends, -inf and NaN among
the student's.  Against the fp64 oracle (oracle/vocab_ops.py) where a result
is defined, with the inputs and the tolerances of test_gpu_vocab_ops.py.
"""
import numpy as np
import pytest
import torch

import selected_token_lm_amd as rlk
from oracle import vocab_ops as O
from tests.gpu_util import DEV, f32_dev, i32_dev, say
from tests.test_gpu_vocab_ops import LOGP_TOL, LOSS_TOL, Case, check_grads, check_top, close

pytestmark = pytest.mark.gpu

BF16_LOWEST = float(torch.finfo(torch.bfloat16).min)
F32_LOWEST = float(torch.finfo(torch.float32).min)


def distinct_teacher(c, K, of=None):
    """K distinct ids a row (of those given, else of all) and logits."""
    of = np.arange(c.V) if of is None else of
    ids = np.stack([c.r.permutation(of)[:K] for _ in range(c.T)]).astype(np.int32)
    return ids, (2 * c.r.standard_normal((c.T, K))).astype(np.float32)


@pytest.mark.parametrize("T", [20, 150])  # few rows and row tiles
@pytest.mark.parametrize("value", ["nan", "inf"])
def test_a_teachers_undefined_logit_makes_every_gradient_nan(T, value):
    """As an id outside the vocabulary does: the row's grad_h, and all of
    grad_W, which sums over the rows.  In an empty slot it says nothing."""
    c = Case(T, 64, 500, seed=3)
    h, W = c.dev()
    n_ids, n_lg = distinct_teacher(c, 4)
    n_lg[4, 2] = float(value)
    ids, lg, g = i32_dev(n_ids), f32_dev(n_lg), f32_dev(c.g)
    bad = torch.zeros(T, dtype=torch.bool, device=DEV)
    bad[4] = True
    loss, lse, lp = rlk.linear_distill_fwd(h, W, ids, lg)
    assert loss[bad].isnan().all() and loss[~bad].isfinite().all()
    for dt in (torch.float32, torch.bfloat16):
        gh, gW = rlk.linear_distill_bwd(h, W, ids, lg, lse, lp, g, grad_W_dtype=dt)
        assert gh[bad].isnan().all() and gh[~bad].isfinite().all()
        assert gW.isnan().all()
    ids[4, 2] = -1
    loss, lse, lp = rlk.linear_distill_fwd(h, W, ids, lg)
    gh, gW = rlk.linear_distill_bwd(h, W, ids, lg, lse, lp, g)
    assert all(x.isfinite().all() for x in (loss, gh, gW))


def column_sets(V):
    """Sets of tokens (not 0) that are whole chunks, whole splits, or neither."""
    S = -(-V // 32)
    sets = {"one": [1], "spread": list(range(1, V, 3)), "last": [V - 1]}
    if S > 128:
        sets["first chunk"] = list(range(7 * S, 7 * S + 128))
        sets["second chunk"] = list(range(7 * S + 128, min(7 * S + 256, 8 * S)))
    if V > 2 * S:
        sets["split"] = list(range(S, 2 * S))
        sets["splits"] = [v for v in range(V) if v // S % 2]
    return sets


@pytest.mark.parametrize("T", [20, 150])
@pytest.mark.parametrize("V", [5, 20, 621, 20011])  # splits of 1, 1, 20 and 626 columns; the third's last is 1 wide
def test_logits_of_minus_infinity_count_nothing(T, V):
    """A masked vocabulary: a constant 1 in h, -inf in W for the tokens masked."""
    for name, off in column_sets(V).items():
        say(f"[-inf] T={T} V={V}: {name}")
        c = Case(T, 64, V, seed=5)
        opened = np.setdiff1d(np.arange(V), off)
        c.h[:, 0], c.W[:, 0] = 1.0, 0.0
        c.W[off, 0] = -np.inf
        c.y = opened[c.r.integers(0, len(opened), T)].astype(np.int32)
        check_top(c, min(8, len(opened)), grads=False)  # (and linear_logp_fwd's bits)
        n_ids, n_lg = distinct_teacher(c, 3, opened)
        h, W = c.dev()
        got = rlk.linear_distill_fwd(h, W, i32_dev(n_ids), f32_dev(n_lg), 2.0)
        want = O.distill_forward(c.h, c.W, n_ids, n_lg, 2.0)
        for what, a, b, tol in zip(("loss", "lse", "logp_ids"), got, want, (LOSS_TOL, LOGP_TOL, LOGP_TOL)):
            close(what, a, b, tol)
        y = i32_dev(c.y)
        parts = torch.stack([rlk.lse_partial(h, W, y, 0, V)])
        for a, b in zip(rlk.lse_merge(parts, y), rlk.linear_logp_fwd_save(h, W, y)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T", [20, 150])
def test_a_vocabulary_masked_with_the_lowest_value_and_a_temperature(T):
    """z / temperature passes fp32's range in the masked tokens: they count
    nothing, and the gradients stay defined."""
    V, tau = 20011, 0.5
    c = Case(T, 64, V, seed=6)
    off = np.concatenate([column_sets(V)[n] for n in ("split", "second chunk")])
    opened = np.setdiff1d(np.arange(V), off)
    c.h[:, 0], c.W[:, 0] = 1.0, 0.0
    c.W[off, 0] = BF16_LOWEST
    n_ids, n_lg = distinct_teacher(c, 6, opened)
    h, W = c.dev()
    ids, lg, g = i32_dev(n_ids), f32_dev(n_lg), f32_dev(c.g)
    loss, lse, lp = rlk.linear_distill_fwd(h, W, ids, lg, tau)
    want = O.distill_forward(c.h, c.W, n_ids, n_lg, tau)
    close("loss", loss, want[0], LOSS_TOL)
    close("lse", lse, want[1], LOGP_TOL)
    close("logp_ids", lp, want[2], LOGP_TOL / tau)
    dz, size = O.distill_dz(c.h, c.W, n_ids, n_lg, c.g, tau)
    check_grads(c, dz, size, *rlk.linear_distill_bwd(h, W, ids, lg, lse, lp, g, tau))


@pytest.mark.parametrize("T", [20, 150])
def test_rows_of_minus_infinity_alone(T):
    """No distribution: an lse of -inf, the rest NaN; the alternatives are the first tokens."""
    c = Case(T, 64, 500, seed=8)
    c.h[:, 0] = 1.0
    h, W = c.dev()
    W[:, 0] = -np.inf
    logp, lse, ent, top, ids = rlk.linear_logp_top_fwd(h, W, i32_dev(c.y), 6)
    assert logp.isnan().all() and lse.eq(-np.inf).all() and ent.isnan().all()
    assert torch.equal(ids, torch.arange(6, device=DEV, dtype=torch.int32).expand(T, 6))


@pytest.mark.parametrize("T", [20, 150])
@pytest.mark.parametrize("V", [5, 20, 621, 20011])
def test_a_nan_logit_is_never_lost(T, V):
    """Wherever it lies in the order of the statistics: first or alone in its
    chunk or split.  Results without it would look sound."""
    for name, off in column_sets(V).items():
        say(f"[NaN] T={T} V={V}: {name}")
        c = Case(T, 64, V, seed=7)
        opened = np.setdiff1d(np.arange(V), off)
        c.y = opened[c.r.integers(0, len(opened), T)].astype(np.int32)
        n_ids, n_lg = distinct_teacher(c, 3, opened)
        h, W = c.dev()
        W[torch.tensor(off, device=DEV)] = float("nan")
        y, ids, lg, g = i32_dev(c.y), i32_dev(n_ids), f32_dev(n_lg), f32_dev(c.g)
        K = min(8, len(opened))
        logp, lse, ent, top, best = rlk.linear_logp_top_fwd(h, W, y, K)
        for x in (logp, lse, ent, top):
            assert x.isnan().all()
        assert best.ge(0).all() and not torch.isin(best, torch.tensor(off, device=DEV, dtype=torch.int32)).any()
        for x in rlk.linear_distill_fwd(h, W, ids, lg):
            assert x.isnan().all()
        for x in (*rlk.linear_logp_fwd(h, W, y), *rlk.linear_logp_fwd_save(h, W, y)[:2]):
            assert x.isnan().all()
        P = 2
        S = -(-V // 32)
        parts = [rlk.lse_partial(h, W[16 * S * p: min(V, 16 * S * (p + 1))], y, 16 * S * p, V)
                 for p in range(P) if 16 * S * p < V]
        for x in rlk.lse_merge(torch.stack(parts), y):
            assert x.isnan().all()
        gh, gW = rlk.linear_logp_top_bwd(h, W, y, lse, ent, g, g)
        assert gh.isnan().all() and gW.isnan().all()


@pytest.mark.parametrize("T", [20, 150])
@pytest.mark.parametrize("V", [5, 621, 20011])
def test_a_logit_of_plus_infinity(T, V):
    """No distribution, as with torch's log_softmax; the token is the first alternative."""
    for at in (0, V // 2, V - 1):
        c = Case(T, 64, V, seed=10)
        c.h[:, 0], c.W[:, 0] = 1.0, 0.0
        c.W[at, 0] = np.inf
        c.y[:] = (at + 1) % V
        n_ids, n_lg = distinct_teacher(c, 3)
        h, W = c.dev()
        y, ids, lg = i32_dev(c.y), i32_dev(n_ids), f32_dev(n_lg)
        logp, lse, ent, top, best = rlk.linear_logp_top_fwd(h, W, y, 3)
        for x in (logp, lse, ent, top, *rlk.linear_distill_fwd(h, W, ids, lg), *rlk.linear_logp_fwd(h, W, y)):
            assert x.isnan().all()
        assert best[:, 0].eq(at).all()


@pytest.mark.parametrize("T", [20, 150])
def test_rows_of_nan_alone(T):
    c = Case(T, 64, 500, seed=8)
    h, W = c.dev()
    logp, lse, ent, top, ids = rlk.linear_logp_top_fwd(torch.full_like(h, float("nan")), W, i32_dev(c.y), 6)
    assert logp.isnan().all() and lse.isnan().all() and ent.isnan().all() and ids.eq(-1).all() and top.eq(-np.inf).all()


@pytest.mark.parametrize("T", [20, 150])
@pytest.mark.parametrize("tau", [0.5, 1.0, 0.001, 8.0])
def test_a_teachers_logits_near_the_types_ends(T, tau):
    """Rows masked with the lowest value as a whole (uniform over their
    slots), in part, and logits whose quotient by the temperature passes
    fp32: all are finite logits, and their q is defined."""
    K = 5
    c = Case(T, 64, 700, seed=9)
    n_ids, n_lg = distinct_teacher(c, K)
    n_lg[1] = F32_LOWEST
    n_lg[2] = BF16_LOWEST
    n_lg[3, 1:] = F32_LOWEST
    n_lg[4] = [3e38, -3e38, 2e38, 0.0, 3e38]
    n_lg[5] = [F32_LOWEST, F32_LOWEST, -np.inf, F32_LOWEST, -np.inf]
    n_lg[6] = -F32_LOWEST
    h, W = c.dev()
    ids, lg, g = i32_dev(n_ids), f32_dev(n_lg), f32_dev(c.g)
    loss, lse, lp = rlk.linear_distill_fwd(h, W, ids, lg, tau)
    with np.errstate(over="ignore"):
        want = O.distill_forward(c.h, c.W, n_ids, n_lg, tau)
        dz, size = O.distill_dz(c.h, c.W, n_ids, n_lg, c.g, tau)
    # z / tau: logits of up to 64 / tau, and the teacher's slots as far apart
    scale = max(1.0, 1.0 / tau)
    close("loss", loss, want[0], LOSS_TOL * scale)
    close("lse", lse, want[1], LOGP_TOL * scale)
    close("logp_ids", lp, want[2], LOGP_TOL * scale)
    if tau >= 0.5:  # (the bounds of check_grads are of exponents up to 64)
        check_grads(c, dz, size, *rlk.linear_distill_bwd(h, W, ids, lg, lse, lp, g, tau))


def test_the_same_id_in_several_slots():
    """Each slot keeps its own log q in the loss, which is then below the
    divergence of the ids' summed q by a constant of the teacher: two slots
    of weight 1/2 on one token against a uniform student of V tokens give
    log V - log 2.  The gradient is that of the sum."""
    V = 900
    for T in (3, 140):
        h, W = torch.zeros((T, 64), dtype=torch.bfloat16, device=DEV), torch.ones((V, 64), dtype=torch.bfloat16, device=DEV)
        twice, once = (torch.full((T, k), 7, dtype=torch.int32, device=DEV) for k in (2, 1))
        zero = torch.zeros((T, 2), device=DEV)
        a = rlk.linear_distill_fwd(h, W, twice, zero)
        b = rlk.linear_distill_fwd(h, W, once, zero[:, :1])
        close("loss of two slots", a[0], np.full(T, np.log(V) - np.log(2)), LOSS_TOL)
        close("loss of one", b[0], np.full(T, np.log(V)), LOSS_TOL)
        one = torch.ones(T, device=DEV)
        ga = rlk.linear_distill_bwd(h, W, twice, zero, a[1], a[2], one)
        gb = rlk.linear_distill_bwd(h, W, once, zero[:, :1], b[1], b[2], one)
        assert torch.equal(ga[0], gb[0]) and torch.equal(ga[1], gb[1])
