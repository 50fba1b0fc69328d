"""linear_logp_top and linear_distill on the GPU against the fp64 oracle
(oracle/vocab_ops.py).

Inputs lie on dyadic grids (h in 1/16, W in 2^-k): every partial sum of a
logit is exact in fp32, so the alternatives' order, ties included, is a fact
of the inputs and ids are compared exactly.

Tolerances, derived for such inputs with |z - max| <= 64 and |lse| <= 32:
  e(x) = exp2(x log2 e): the product's half step 2^-24 |x log2 e| <= 2^-24 *
    93 of the exponent, times ln 2, and exp2's ulp: 64 * 2^-24 + 2^-23 < 4e-6
    relative; a sum passes <= 8 levels in a chunk, its split's chunks and 5
    levels, each 2^-24 and (folding) one more e(x) near 1: < 1e-5 relative.
  logp = (z - m) - log s: 1e-5 from s, and the half steps of z - m, of
    log2 s, of its product and of the difference, 4 * 2^-24 * 64: 2.5e-5.
  entropy = log s - u / s: 1e-5 from log s, 2e-5 of |u / s| <= 16: 4e-4.
  loss = sum q (lq - lp): the q (2e-5 of terms <= 64, summing to 1): 1.5e-3.
  dz: its fp32 terms 5e-5 relative (e(z - lse), lse's 2^-24 * 32 * 2 in the
    exponent), then half a bf16 step, 2^-8.  A gradient element is off by at
    most sum |factor| (5e-5 terms + 2^-8 |dz|), 2^-8 of itself where it is
    bf16, and its fp32 chain's n 2^-24 of the sum of magnitudes (n = V or T
    steps; below 1e-2 of the 2^-8 term for the sizes here: 5 % are added).
"""
import math

import numpy as np
import pytest
import torch

import selected_token_lm_amd as rlk
from oracle import vocab_ops as O
from tests.gpu_util import DEV, f32_dev, i32_dev, say

pytestmark = pytest.mark.gpu

LOGP_TOL, ENT_TOL, LOSS_TOL, STEP = 2.5e-5, 4e-4, 1.5e-3, 2.0 ** -8


class Case:
    """Grid inputs: a row leans towards one token by 0 .. 12; `mask` of the rows inactive."""

    def __init__(self, T, H, V, mask=0.0, seed=0, lean=12.0, dup=False):
        r = np.random.Generator(np.random.PCG64(seed))
        steps = 2.0 ** round(math.log2(16 * math.sqrt(H)))
        grid = lambda x, s: np.clip(np.round(x * s), -127, 127) / s  # noqa: E731
        self.T, self.H, self.V, self.r = T, H, V, r
        self.W = grid(r.standard_normal((V, H)) / math.sqrt(H), steps)
        if dup:  # every token's row again, and again: ties in threes
            self.W = self.W[np.arange(V) % max(1, V // 3)]
        t = r.integers(0, V, T)
        self.h = grid(r.standard_normal((T, H)) + lean * r.random((T, 1)) * self.W[t], 16.0)
        self.y = np.where(r.random(T) < 0.5, t, r.integers(0, V, T)).astype(np.int32)
        off = np.zeros(T, dtype=bool)
        off[r.permutation(T)[: int(round(mask * T))]] = True
        self.off, self.lean = off, t
        self.y[off] = -100
        self.g, self.ge = r.standard_normal(T).astype(np.float32), r.standard_normal(T).astype(np.float32)

    def dev(self):
        b = lambda x: torch.from_numpy(x).to(torch.bfloat16).to(DEV)  # noqa: E731
        return b(self.h), b(self.W)

    def teacher(self, K, empty=0.2):
        """Ids with repeats, the leaning token among them, empty slots by id
        and by logit (with NaN and inf where an id says empty), and rows
        without any."""
        r, T, V = self.r, self.T, self.V
        ids = r.integers(0, V, (T, K))
        ids[:, K // 2] = self.lean
        if K > 2:
            ids[:, K - 1] = ids[:, 0]
        lg = (2 * r.standard_normal((T, K))).astype(np.float32)
        a, b = r.random((T, K)) < empty / 2, r.random((T, K)) < empty / 2
        lg[b] = -np.inf
        ids[a] = -1 - r.integers(0, 50, (T, K))[a]
        lg[a] = np.where(r.random((T, K)) < 0.5, np.nan, np.inf)[a]
        ids[self.off] = -1
        return ids.astype(np.int32), lg


def np64(t):
    return t.detach().double().cpu().numpy()


def close(name, got, want, tol):
    got, want = np64(got), np.asarray(want)
    assert np.array_equal(np.isfinite(got), np.isfinite(want)), name
    f = np.isfinite(want)
    assert np.array_equal(got[~f], want[~f]), name
    d = np.abs(got[f] - want[f]).max(initial=0.0)
    say(f"  {name}: max error {d:.3e} of {tol:.1e}")
    assert d <= tol, name


def check_grads(c, dz, size, gh, gW):
    off = 5e-5 * size + STEP * np.abs(dz)
    for name, got, want, bound in (("grad_h", gh, dz @ c.W, off @ np.abs(c.W)),
                                   ("grad_W", gW, dz.T @ c.h, off.T @ np.abs(c.h))):
        bound = 1.05 * bound + (STEP * np.abs(want) if got.dtype == torch.bfloat16 else 0) + 1e-30
        worst = (np.abs(np64(got) - want) / bound).max()
        say(f"  {name} ({got.dtype}): {worst:.3f} of the bound")
        assert worst <= 1, name


def check_top(c, K, grads=True):
    h, W = c.dev()
    y, g, ge = i32_dev(c.y), f32_dev(c.g), f32_dev(c.ge)
    logp, lse, ent, top, ids = rlk.linear_logp_top_fwd(h, W, y, K)
    want = O.top_forward(c.h, c.W, c.y, K)
    assert np.array_equal(ids.cpu().numpy(), want[4])
    close("logp", logp, want[0], LOGP_TOL)
    close("lse", lse, want[1], LOGP_TOL)
    close("entropy", ent, want[2], ENT_TOL)
    close("top_logp", top, want[3], LOGP_TOL)
    base_logp, base_lse = rlk.linear_logp_fwd(h, W, y)  # the operator beside it: the same bits
    assert torch.equal(logp, base_logp) and torch.equal(lse, base_lse)
    if grads:
        dz, size = O.top_dz(c.h, c.W, c.y, c.g, c.ge)
        for dt in (torch.float32, torch.bfloat16):
            gh, gW = rlk.linear_logp_top_bwd(h, W, y, lse, ent, g, ge, grad_W_dtype=dt)
            assert gW.dtype == dt and gh.dtype == torch.bfloat16
            check_grads(c, dz, size, gh, gW)
            assert torch.count_nonzero(gh[y == -100]) == 0


def check_distill(c, K, tau, grads=True):
    h, W = c.dev()
    n_ids, n_lg = c.teacher(K)
    ids, lg, g = i32_dev(n_ids), f32_dev(n_lg), f32_dev(c.g)
    loss, lse, lp = rlk.linear_distill_fwd(h, W, ids, lg, tau)
    with np.errstate(invalid="ignore"):
        want = O.distill_forward(c.h, c.W, n_ids, n_lg, tau)
        close("loss", loss, want[0], LOSS_TOL)
        close("lse", lse, want[1], LOGP_TOL)
        close("logp_ids", lp, want[2], LOGP_TOL * max(1.0, 1 / tau))
        if not grads:
            return
        dz, size = O.distill_dz(c.h, c.W, n_ids, n_lg, c.g, tau)
    for dt in (torch.float32, torch.bfloat16):
        gh, gW = rlk.linear_distill_bwd(h, W, ids, lg, lse, lp, g, tau, grad_W_dtype=dt)
        assert gW.dtype == dt
        check_grads(c, dz, size, gh, gW)


# the few-row kernels end at 128 rows (by 16, 32, 64); the others' row tiles hold
# 256, and more than 256 of their tiles run in rounds, the last one in halves
SHAPES = [(1, 64, 1, 0.0), (1, 64, 5, 0.0), (7, 128, 33, 0.0), (64, 256, 4096, 0.0), (37, 64, 1000, 0.3),
          (17, 2048, 700, 0.0), (100, 192, 2500, 0.2), (321, 448, 2500, 0.0), (448, 64, 1000, 0.0), (128, 64, 12_345, 0.1),
          (300, 192, 5000, 0.2), (129, 320, 20011, 0.15), (600, 64, 9000, 0.5), (5, 64, 300_000, 0.0)]


@pytest.mark.parametrize("T,H,V,mask", SHAPES)
@pytest.mark.parametrize("K", [0, 1, 8, 64, 65, 128])
def test_top(T, H, V, mask, K):
    say(f"[top] T={T} H={H} V={V} mask={mask} K={K}")
    check_top(Case(T, H, V, mask, seed=K), K, grads=K in (0, 8))


@pytest.mark.parametrize("T,H,V,mask", SHAPES)
@pytest.mark.parametrize("K,tau", [(1, 1.0), (8, 2.0), (65, 0.5), (128, 1.0)])
def test_distill(T, H, V, mask, K, tau):
    say(f"[distill] T={T} H={H} V={V} mask={mask} K={K} tau={tau}")
    check_distill(Case(T, H, V, mask, seed=K), K, tau, grads=K != 1)


def test_ties_go_to_the_lowest_id():
    say("[top] ties")
    for K in (3, 20, 128):
        check_top(Case(40, 64, 3000, 0.1, seed=K, dup=True), K, grads=False)
    # every logit equal: the list of candidates overflows and is cut
    h, W = torch.ones((3, 64), dtype=torch.bfloat16, device=DEV), torch.zeros((70_000, 64), dtype=torch.bfloat16, device=DEV)
    logp, lse, ent, top, ids = rlk.linear_logp_top_fwd(h, W, i32_dev(np.array([0, -100, 69_999])), 128)
    assert ids[0].tolist() == list(range(128)) == ids[2].tolist() and ids[1].eq(-1).all()
    close("entropy", ent, [math.log(70_000), 0, math.log(70_000)], ENT_TOL)


def test_tiles_in_rounds():
    """576 tiles of 256 columns and rows: two rounds of 256 units, and 64 in halves."""
    check_top(Case(300, 64, 70_000, seed=21), 30)
    check_distill(Case(300, 64, 70_000, seed=22), 30, 1.0)


@pytest.mark.parametrize("T,H", [(300, 128), (40, 128), (200, 448)])
@pytest.mark.parametrize("budget", ["1", "2", "12", "40"])
def test_groups_of_splits_change_no_bit(budget, T, H, monkeypatch):
    """The workspace budget sets how many splits are processed together."""
    c = Case(T, H, 20_011, 0.2, seed=4)
    h, W = c.dev()
    y, g, ge = i32_dev(c.y), f32_dev(c.g), f32_dev(c.ge)
    n_ids, n_lg = c.teacher(20)
    ids, lg = i32_dev(n_ids), f32_dev(n_lg)

    def everything():
        out = list(rlk.linear_logp_top_fwd(h, W, y, 50))
        out += rlk.linear_logp_top_bwd(h, W, y, out[1], out[2], g, ge)
        d = rlk.linear_distill_fwd(h, W, ids, lg, 1.5)
        return out + list(d) + list(rlk.linear_distill_bwd(h, W, ids, lg, d[1], d[2], g, 1.5, grad_W_dtype=torch.bfloat16))

    want = everything()
    monkeypatch.setenv("RLK_DZ_BUDGET_MB", budget)
    sizes = rlk.vocab_workspace_bytes(rlk.VOP_TOP_FWD, T, H, 20_011, 50)
    say(f"[groups] budget {budget} MiB: {sizes} bytes")
    for a, b in zip(everything(), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("H", [128, 448])
def test_a_row_does_not_depend_on_its_batch(H):
    """Alone, in a small batch, in a large one, in another order: the same
    bits, grad_h among them; and twice the same."""
    c = Case(700, H, 6001, 0.1, seed=9)
    h, W = c.dev()
    y, g, ge = i32_dev(c.y), f32_dev(c.g), f32_dev(c.ge)
    n_ids, n_lg = c.teacher(30)
    ids, lg = i32_dev(n_ids), f32_dev(n_lg)

    def rows(at):
        a = [x[at].contiguous() for x in (h, y, g, ge, ids, lg)]
        out = list(rlk.linear_logp_top_fwd(a[0], W, a[1], 12))
        out.append(rlk.linear_logp_top_bwd(a[0], W, a[1], out[1], out[2], a[2], a[3], need_grad_W=False)[0])
        d = list(rlk.linear_distill_fwd(a[0], W, a[4], a[5], 2.0))
        d.append(rlk.linear_distill_bwd(a[0], W, a[4], a[5], d[1], d[2], a[2], 2.0, need_grad_W=False)[0])
        return out + d

    every = torch.arange(700, device=DEV)
    want = rows(every)
    assert all(torch.equal(a, b) for a, b in zip(rows(every), want))
    r = np.random.Generator(np.random.PCG64(1))
    for n in (1, 2, 17, 48, 65, 97, 145, 190, 256, 285, 290, 300, 340, 400, 500):
        at = torch.from_numpy(r.permutation(700)[:n].copy()).to(DEV)
        say(f"[batch] {n} rows")
        for a, b in zip(rows(at), want):
            assert torch.equal(a.view(torch.int16), b[at].contiguous().view(torch.int16))


def test_inactive_rows_and_masked_values():
    """Rows without a target, or without a kept slot, may hold anything."""
    c = Case(50, 64, 700, 0.4, seed=2)
    h, W = c.dev()
    y = i32_dev(c.y)
    n_ids, n_lg = c.teacher(9)
    ids, lg = i32_dev(n_ids), f32_dev(n_lg)
    want = list(rlk.linear_logp_top_fwd(h, W, y, 5)) + list(rlk.linear_distill_fwd(h, W, ids, lg))
    h[y == -100] = float("nan")
    got = list(rlk.linear_logp_top_fwd(h, W, y, 5)) + list(rlk.linear_distill_fwd(h, W, ids, lg))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    g = f32_dev(c.g)
    g[y == -100] = float("inf")
    gh, gW = rlk.linear_logp_top_bwd(h, W, y, got[1], got[2], g, g)
    assert torch.isfinite(gh).all() and torch.isfinite(gW).all() and gh[y == -100].eq(0).all()
    gh, gW = rlk.linear_distill_bwd(h, W, ids, lg, got[6], got[7], g)
    assert torch.isfinite(gh).all() and torch.isfinite(gW).all() and gh[y == -100].eq(0).all()
    # nothing active at all
    none = torch.full_like(y, -100)
    out = rlk.linear_logp_top_fwd(h, W, none, 4)
    assert all(x.eq(0).all() for x in out[:3]) and out[3].eq(-math.inf).all() and out[4].eq(-1).all()
    gh, gW = rlk.linear_logp_top_bwd(h, W, none, out[1], out[2], g, g, grad_W_dtype=torch.bfloat16)
    assert gh.eq(0).all() and gW.eq(0).all()
    loss, lse, lp = rlk.linear_distill_fwd(h, W, torch.full_like(ids, -1), lg)
    assert loss.eq(0).all() and lse.eq(0).all() and lp.eq(-math.inf).all()
    gh, gW = rlk.linear_distill_bwd(h, W, torch.full_like(ids, -1), lg, lse, lp, g)
    assert gh.eq(0).all() and gW.eq(0).all()


@pytest.mark.parametrize("T", [20, 150])  # few rows and row tiles
@pytest.mark.parametrize("outside", [(500, -7), (2 ** 31 - 1, -2 ** 31), (2 ** 32 + 5, -2 ** 40)])
def test_undefined_rows_are_nan_and_only_they(T, outside):
    c = Case(T, 64, 500, seed=3)
    h, W = c.dev()
    y, g = i32_dev(c.y).long(), f32_dev(c.g)
    y[3], y[4] = outside
    logp, lse, ent, top, ids = rlk.linear_logp_top_fwd(h, W, y, 6)
    want = O.top_forward(c.h, c.W, np.where(np.isin(np.arange(T), (3, 4)), 0, c.y), 6)
    bad = torch.zeros(T, dtype=torch.bool, device=DEV)
    bad[3:5] = True
    assert logp[bad].isnan().all() and logp[~bad].isfinite().all()
    close("entropy", ent, want[2], ENT_TOL)
    assert np.array_equal(ids.cpu().numpy(), want[4])
    gh, gW = rlk.linear_logp_top_bwd(h, W, y, lse, ent, g, g)
    assert gh[bad].isnan().all() and gh[~bad].isfinite().all() and gW.isnan().all()
    n_ids, n_lg = c.teacher(4, empty=0.0)
    t_ids, lg = i32_dev(n_ids), f32_dev(n_lg)
    t_ids[3, 1] = min(outside[0], 2 ** 31 - 1)
    lg[4, 2] = float("nan") if T == 20 else float("inf")
    loss, lse, lp = rlk.linear_distill_fwd(h, W, t_ids, lg)
    assert loss[bad].isnan().all() and loss[~bad].isfinite().all()
    gh, _ = rlk.linear_distill_bwd(h, W, t_ids, lg, lse, lp, g, need_grad_W=False)
    assert gh[bad].isnan().all() and gh[~bad].isfinite().all()
    # a NaN in the weight: NaN statistics, and the token is no alternative
    W2 = W.clone()
    W2[7] = float("nan")
    logp, lse, ent, top, ids = rlk.linear_logp_top_fwd(h, W2, i32_dev(c.y), 128)
    assert logp.isnan().all() and lse.isnan().all() and ent.isnan().all() and not ids.eq(7).any() and ids.ge(0).all()


@pytest.mark.parametrize("T", [20, 150])
def test_rows_of_nan_and_targets_beyond_the_ignored_one(T):
    c = Case(T, 64, 500, seed=8)
    h, W = c.dev()
    y, g = i32_dev(c.y).long(), f32_dev(c.g)
    t_ids, lg = i32_dev(c.r.integers(0, 500, (T, 4))), f32_dev(c.r.standard_normal((T, 4)))
    want = rlk.linear_logp_top_fwd(h, W, y, 6)
    want_d = rlk.linear_distill_fwd(h, W, t_ids, lg)
    bad = torch.zeros(T, dtype=torch.bool, device=DEV)
    bad[3] = bad[T - 1] = True
    h2 = torch.where(bad[:, None], float("nan"), h)
    logp, lse, ent, top, ids = got = rlk.linear_logp_top_fwd(h2, W, y, 6)
    assert logp[bad].isnan().all() and ent[bad].isnan().all() and ids[bad].eq(-1).all()
    for a, b in zip(got, want):
        assert torch.equal(a[~bad], b[~bad])
    gh, gW = rlk.linear_logp_top_bwd(h2, W, y, lse, ent, g, g)
    assert gh[bad].isnan().all() and gh[~bad].isfinite().all() and gW.isnan().all()
    loss, lse, lp = got = rlk.linear_distill_fwd(h2, W, t_ids, lg)
    assert loss[bad].isnan().all()
    for a, b in zip(got, want_d):
        assert torch.equal(a[~bad], b[~bad])
    gh, gW = rlk.linear_distill_bwd(h2, W, t_ids, lg, lse, lp, g)
    assert gh[bad].isnan().all() and gh[~bad].isfinite().all() and gW.isnan().all()
    # targets at and past int32's ends, one of which is the ignored one
    for ignore, far in ((-2 ** 31, -2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31)):
        y2 = y.clone()
        y2[2], y2[5] = ignore, far
        logp, _, _, _, ids = rlk.linear_logp_top_fwd(h, W, y2, 6, ignore_index=ignore)
        assert logp[2] == 0 and ids[2].eq(-1).all()
        assert logp[5].isnan() and torch.equal(ids[5], want[4][5])


def test_lengths_and_strides():
    c = Case(33, 64, 900, 0.1, seed=6)
    h, W = c.dev()
    n_ids, n_lg = c.teacher(6)
    y = i32_dev(c.y)
    want = list(rlk.linear_logp_top_fwd(h, W, y, 7)) + list(rlk.linear_distill_fwd(h, W, i32_dev(n_ids), f32_dev(n_lg)))
    # the same values behind other strides, types and offsets
    h2 = torch.stack([h, h], dim=2)[:, :, 1]
    W2 = torch.cat([W, W], dim=1)[:, 64:]
    y2 = torch.cat([y[:1], y]).long()[1:]
    ids2 = i32_dev(n_ids).T.contiguous().T.long()
    lg2 = torch.cat([f32_dev(n_lg)] * 2, dim=1)[:, 6:]
    got = list(rlk.linear_logp_top_fwd(h2, W2, y2, 7)) + list(rlk.linear_distill_fwd(h2, W2, ids2, lg2))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    y3 = torch.cat([y[:1], y])[1:]  # int32 rows at a 4-byte offset
    assert torch.equal(rlk.linear_logp_top_fwd(h, W, y3, 7)[4], want[4])
    # logits in 16 bits are the values they hold; an id past int32 is outside every vocabulary
    b16 = f32_dev(n_lg).bfloat16()
    for a, b in zip(rlk.linear_distill_fwd(h, W, i32_dev(n_ids), b16), rlk.linear_distill_fwd(h, W, i32_dev(n_ids), b16.float())):
        assert torch.equal(a, b)
    far = torch.full((33, 1), 2 ** 33, device=DEV)
    assert rlk.linear_distill_fwd(h, W, far, torch.zeros((33, 1), device=DEV))[0].isnan().all()
    # no rows
    e = h[:0]
    out = rlk.linear_logp_top_fwd(e, W, y[:0], 3)
    assert [tuple(x.shape) for x in out] == [(0,), (0,), (0,), (0, 3), (0, 3)]
    for dt in (torch.float32, torch.bfloat16):
        gh, gW = rlk.linear_logp_top_bwd(e, W, y[:0], out[1], out[2], out[0], None, grad_W_dtype=dt)
        assert gh.shape == (0, 64) and gW.eq(0).all()
    d = rlk.linear_distill_fwd(e, W, ids2[:0], lg2[:0])
    gh, gW = rlk.linear_distill_bwd(e, W, ids2[:0], lg2[:0], d[1], d[2], d[0])
    assert gh.shape == (0, 64) and gW.eq(0).all()


def test_missing_gradients_and_outputs():
    c = Case(70, 128, 1500, 0.1, seed=8)
    h, W = c.dev()
    y, g, ge = i32_dev(c.y), f32_dev(c.g), f32_dev(c.ge)
    logp, lse, ent, _, _ = rlk.linear_logp_top_fwd(h, W, y, 0)
    zero = torch.zeros_like(g)
    for a, b in ((g, None), (None, ge)):
        got = rlk.linear_logp_top_bwd(h, W, y, lse, ent, a, b)
        want = rlk.linear_logp_top_bwd(h, W, y, lse, ent, zero if a is None else a, zero if b is None else b)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    full = rlk.linear_logp_top_bwd(h, W, y, lse, ent, g, ge)
    gh, none = rlk.linear_logp_top_bwd(h, W, y, lse, ent, g, ge, need_grad_W=False)
    assert none is None and torch.equal(gh, full[0])
    none, gW = rlk.linear_logp_top_bwd(h, W, y, lse, ent, g, ge, need_grad_h=False)
    assert none is None and torch.equal(gW, full[1])
    half = rlk.linear_logp_top_bwd(h, W, y, lse, ent, g, ge, grad_W_dtype=torch.bfloat16)
    assert torch.equal(half[1], full[1].bfloat16()) and torch.equal(half[0], full[0])  # rounded once


def test_autograd_and_a_run_of_both():
    """A teacher's alternatives train a student, with an entropy bonus: the
    operators together, as they are used."""
    t, s = Case(60, 128, 2000, 0.2, seed=11), Case(60, 64, 2000, 0.2, seed=12)
    th, tW = t.dev()
    h, W = s.dev()
    y = i32_dev(t.y)
    with torch.no_grad():
        _, _, top, ids = rlk.linear_logp_top(th, tW, y, 16)
    assert not top.requires_grad
    h.requires_grad_()
    W.requires_grad_()
    loss = rlk.linear_distill(h, W, ids, top, 1.5)
    logp, ent, _, best = rlk.linear_logp_top(h, W, y, 3)
    (loss.sum() - 0.1 * ent.sum() + 0.5 * logp.sum()).backward()
    assert h.grad.dtype == W.grad.dtype == torch.bfloat16
    n_ids, n_top = ids.cpu().numpy(), top.cpu().numpy()
    one = np.ones(60)
    d1, s1 = O.distill_dz(s.h, s.W, n_ids, n_top, one, 1.5)
    d2, s2 = O.top_dz(s.h, s.W, t.y, 0.5 * one, -0.1 * one)
    # each of the two gradients is rounded to bf16, and their sum once more
    for got, a, b, off in ((h.grad, d1 @ s.W, d2 @ s.W, lambda o: o @ np.abs(s.W)),
                           (W.grad, d1.T @ s.h, d2.T @ s.h, lambda o: o.T @ np.abs(s.h))):
        bound = 1.05 * off(5e-5 * (s1 + s2) + STEP * (np.abs(d1) + np.abs(d2)))
        bound += 1.05 * STEP * (np.abs(a) + np.abs(b) + np.abs(a + b))
        assert (np.abs(np64(got) - a - b) <= bound + 1e-30).all()
    # the entropy alone, and a second derivative refused
    h.grad = None
    ent = rlk.linear_logp_top(h, W, y)[1]
    gh, = torch.autograd.grad(ent.sum(), h, create_graph=True)
    with pytest.raises(RuntimeError):
        gh.sum().backward()


def test_differences():
    """The forward's own differences along a direction of h follow grad_h."""
    c = Case(24, 64, 800, seed=14, lean=4.0)
    h, W = c.dev()
    y = i32_dev(c.y)
    n_ids, n_lg = c.teacher(7)
    ids, lg = i32_dev(n_ids), f32_dev(n_lg)
    # steps of 1/8 stay on the grid; the losses' third derivative along the
    # direction v is bounded by 8 max|W v|^3 (a third cumulant and, for the
    # entropy, a fourth over the same range), times 1/6 step^2
    r = np.random.Generator(np.random.PCG64(5))
    v = np.zeros((24, 64))
    v[np.arange(24), r.integers(0, 64, 24)] = 1.0
    step = 0.125
    vd = torch.from_numpy(v).to(DEV)
    up, down = (h.double() + step * vd).bfloat16(), (h.double() - step * vd).bfloat16()
    reach = (np.abs(v @ c.W.T).max(axis=1)) ** 3 * 8 * (1 + np.log(800)) / 6 * step ** 2
    one = torch.ones(24, device=DEV)
    _, lse, ent, _, _ = rlk.linear_logp_top_fwd(h, W, y, 0)
    _, dl, dp = rlk.linear_distill_fwd(h, W, ids, lg)
    for f, gh, tol in ((lambda x: rlk.linear_logp_top_fwd(x, W, y, 0)[0], rlk.linear_logp_top_bwd(h, W, y, lse, ent, one)[0], LOGP_TOL),
                       (lambda x: rlk.linear_logp_top_fwd(x, W, y, 0)[2], rlk.linear_logp_top_bwd(h, W, y, lse, ent, None, one)[0], ENT_TOL),
                       (lambda x: rlk.linear_distill_fwd(x, W, ids, lg)[0], rlk.linear_distill_bwd(h, W, ids, lg, dl, dp, one)[0], LOSS_TOL)):
        diff = np64((f(up).double() - f(down).double()) / (2 * step))
        got = (np64(gh) * v).sum(axis=1)
        # grad_h's own error: half a bf16 step of dz times |W v|, summing to
        # at most 2 (1 + log V) max|W v|, and of itself
        own = STEP * (2 * (1 + np.log(800)) * np.abs(v @ c.W.T).max(axis=1) + np.abs(got))
        assert (np.abs(diff - got) <= reach + own + tol / step).all()


def test_streams_and_graphs():
    """On a side stream, and captured: two graphs of one workspace each, and
    replays between eager calls."""
    c = Case(90, 128, 3000, 0.2, seed=15)
    h, W = c.dev()
    y, g = i32_dev(c.y), f32_dev(c.g)
    n_ids, n_lg = c.teacher(12)
    ids, lg = i32_dev(n_ids), f32_dev(n_lg)
    T, H, V = 90, 128, 3000

    def all_of(w):
        out = list(rlk.linear_logp_top_fwd(h, W, y, 9, ws=w[0]))
        out += rlk.linear_logp_top_bwd(h, W, y, out[1], out[2], g, g, ws=w[1])
        d = list(rlk.linear_distill_fwd(h, W, ids, lg, 1.5, ws=w[2]))
        return out + d + list(rlk.linear_distill_bwd(h, W, ids, lg, d[1], d[2], g, 1.5, grad_W_dtype=torch.bfloat16, ws=w[3]))

    def spaces():
        return [torch.empty(rlk.vocab_workspace_bytes(op, T, H, V, k), dtype=torch.uint8, device=DEV)
                for op, k in ((0, 9), (1, 0), (2, 12), (3, 12))]

    want = [x.clone() for x in all_of([None] * 4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = all_of(spaces())
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    w = spaces()
    graphs = []
    for _ in range(2):  # both in one set of workspaces: they are replayed one after the other
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, all_of(w)))
    torch.cuda.synchronize()
    keep = [x.clone() for x in (h, y, ids)]
    for rep in range(3):
        for graph, out in graphs:
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), rep
            for x in w:
                x.fill_(0xFF)  # nothing in a workspace needs to keep its value
            all_of([None] * 4)
    # new values in the captured buffers, other rows inactive
    h.copy_(keep[0].flip(0))
    y.copy_(keep[1].flip(0))
    ids.copy_(keep[2].flip(0))
    lg.copy_(f32_dev(n_lg).flip(0))
    new = all_of([None] * 4)
    assert not torch.equal(new[0], want[0])
    for graph, out in graphs:
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, new))


def test_two_streams_at_once():
    """Calls on two streams, each with its own buffers, do not meet."""
    c = [Case(90, 128, 30_000, 0.1, seed=31), Case(300, 64, 30_000, 0.1, seed=32)]
    dev = []
    for x in c:
        n_ids, n_lg = x.teacher(16)
        dev.append((*x.dev(), i32_dev(x.y), f32_dev(x.g), i32_dev(n_ids), f32_dev(n_lg)))

    def all_of(h, W, y, g, ids, lg):
        out = list(rlk.linear_logp_top_fwd(h, W, y, 9))
        out += rlk.linear_logp_top_bwd(h, W, y, out[1], out[2], g, g)
        d = list(rlk.linear_distill_fwd(h, W, ids, lg))
        return out + d + list(rlk.linear_distill_bwd(h, W, ids, lg, d[1], d[2], g))

    want = [all_of(*x) for x in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for rep in range(3):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(all_of(*dev[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for out in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[k]))


def test_wrong_workspaces_are_refused():
    c = Case(10, 64, 100)
    h, W = c.dev()
    y = i32_dev(c.y)
    with pytest.raises(rlk.RlkError, match="workspace too small"):
        rlk.linear_logp_top_fwd(h, W, y, 4, ws=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="uint8"):
        rlk.linear_logp_top_fwd(h, W, y, 4, ws=torch.empty(1 << 20, device=DEV))
    with pytest.raises(rlk.RlkError, match="invalid argument"):
        rlk.linear_distill_fwd(h, W, i32_dev(np.zeros((10, 1))), torch.zeros((10, 1), device=DEV), 0.0)
    with pytest.raises(ValueError, match="must be on"):
        rlk.linear_distill_fwd(h, W, torch.zeros((10, 1), dtype=torch.int32), torch.zeros((10, 1)))


def test_rows_far_down_a_large_batch():
    """More rows than a launch dimension holds blocks of one row, several
    groups of splits: rows far down the batch equal the same rows alone."""
    T, H, V, K = 70_000, 64, 20_000, 128
    gen = torch.Generator(device=DEV).manual_seed(3)
    h = (torch.randn((T, H), device=DEV, generator=gen) * 16).round().clamp(-64, 64).div(16).bfloat16()
    W = (torch.randn((V, H), device=DEV, generator=gen) * 16).round().clamp(-64, 64).div(128).bfloat16()
    y = torch.randint(0, V, (T,), device=DEV, generator=gen, dtype=torch.int32)
    say(f"[large] {rlk.vocab_workspace_bytes(rlk.VOP_TOP_FWD, T, H, V, K)} bytes")
    out = rlk.linear_logp_top_fwd(h, W, y, K)
    d = rlk.linear_distill_fwd(h, W, out[4], out[3], 2.0)
    at = torch.tensor([0, 1, 34_567, T - 2, T - 1], device=DEV)
    one = rlk.linear_logp_top_fwd(h[at], W, y[at], K)
    for a, b in zip(one, out):
        assert torch.equal(a, b[at])
    for a, b in zip(rlk.linear_distill_fwd(h[at], W, one[4], one[3], 2.0), d):
        assert torch.equal(a, b[at])
    g = torch.ones(T, device=DEV)
    gh, _ = rlk.linear_distill_bwd(h, W, out[4], out[3], d[1], d[2], g, 2.0, need_grad_W=False)
    gh1, _ = rlk.linear_distill_bwd(h[at], W, one[4], one[3], d[1][at], d[2][at], g[at], 2.0, need_grad_W=False)
    assert torch.equal(gh[at], gh1)
