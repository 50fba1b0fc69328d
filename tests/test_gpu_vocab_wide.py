"""linear_logp_top and linear_distill over wide vocabularies: where the top
merge takes runs of several chunks as one (past 262144 tokens) and where a
row group's counters are the large ones (past 1048576), by row tiles, in one
group of splits and in several.  The same rows through the few-row kernels
give the same bits, and those rows are compared with the definitions in 64
bits (tolerances of test_gpu_vocab_ops.py).
"""
import math

import pytest
import torch

import selected_token_lm_amd as rlk
from tests.gpu_util import DEV, say
from tests.test_gpu_vocab_ops import ENT_TOL, LOGP_TOL, LOSS_TOL, STEP, close, np64

pytestmark = pytest.mark.gpu

H = 64


def draw(T, V, seed):
    """Rows on dyadic grids (every logit exact in fp32, many ties) that lean
    towards tokens of the first and the last splits."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    grid = lambda x, s: (x * s).round().clamp(-127, 127) / s  # noqa: E731
    W = grid(torch.randn((V, H), device=DEV, generator=gen) / 8, 128.0).bfloat16()
    lean = torch.randint(0, V // 40, (T,), device=DEV, generator=gen)
    lean = torch.where(torch.arange(T, device=DEV) % 2 == 0, lean, V - 1 - lean)
    h = grid(torch.randn((T, H), device=DEV, generator=gen) + 6 * W[lean].float(), 16.0).bfloat16()
    y = torch.where(torch.arange(T, device=DEV) % 3 == 0, -100, lean).int()
    return gen, h, W, lean, y


def log_p(h, W, tau=1.0):
    """log softmax(h W^T / tau) of a few rows in 64 bits and the lse."""
    z = torch.cat([h.double() @ w.double().T for w in W.split(1 << 20)], dim=1) / tau
    lse = torch.logsumexp(z, dim=1)
    return z - lse[:, None], lse


def check_grad_w(h, W, ids, dz_of, got):
    """Rows `ids` of grad_W against sum_t dz_t h_t in 64 bits; dz_of: dz [T, n]
    of these tokens and the sum of its terms' magnitudes."""
    dz, size = dz_of
    off = 5e-5 * size + STEP * dz.abs()
    want, bound = dz.T @ h.double(), 1.05 * off.T @ h.double().abs()
    if got.dtype == torch.bfloat16:
        bound = bound + STEP * want.abs()
    assert ((got[ids].double() - want).abs() <= bound + 1e-30).all()


# the budget that keeps the logits (top) or dz in groups of splits; 0: the default
@pytest.mark.parametrize("T,V,budget", [(150, 300_000, 0), (150, 300_000, 40), (130, 1_100_000, 0), (130, 8_000_000, 0)])
def test_top_of_a_wide_vocabulary(T, V, budget, monkeypatch):
    say(f"[wide top] T={T} V={V} budget {budget}")
    K = 128
    gen, h, W, lean, y = draw(T, V, 1)
    at = torch.tensor([0, 1, 2, 4, T - 2, T - 1], device=DEV)
    alone = rlk.linear_logp_top_fwd(h[at], W, y[at], K)  # few rows, all logits kept
    if budget:
        monkeypatch.setenv("RLK_DZ_BUDGET_MB", str(budget))
    out = rlk.linear_logp_top_fwd(h, W, y, K)
    for a, b in zip(alone, out):
        assert torch.equal(a, b[at])
    lp, lse = log_p(h[at], W)
    on = y[at] != -100
    best = torch.sort(lp, dim=1, descending=True, stable=True).indices[:, :K]
    assert torch.equal(alone[4][on].long(), best[on])
    close("logp", alone[0][on], np64(lp.gather(1, lean[at][:, None])[:, 0][on]), LOGP_TOL)
    close("lse", alone[1][on], np64(lse[on]), LOGP_TOL)
    close("entropy", alone[2][on], np64(-(lp.exp() * lp).sum(dim=1)[on]), ENT_TOL)
    close("top_logp", alone[3][on], np64(lp.gather(1, best)[on]), LOGP_TOL)
    g, ge = (torch.randn(T, device=DEV, generator=gen) for _ in range(2))
    gh, gW = rlk.linear_logp_top_bwd(h, W, y, out[1], out[2], g, ge, grad_W_dtype=torch.bfloat16)
    one, _ = rlk.linear_logp_top_bwd(h[at], W, y[at], alone[1], alone[2], g[at], ge[at], need_grad_W=False)
    assert torch.equal(gh[at], one)
    # rows of grad_W: the targets, the ends, and others
    ids = torch.cat([lean[:20], torch.tensor([0, V // 2, V - 1], device=DEV)]).unique()
    on = (y != -100)[:, None].double()
    p = h.double() @ W[ids].double().T - out[1].double()[:, None]
    a, b, ent = (x.double()[:, None] for x in (g, ge, out[2]))
    hot = (lean[:, None] == ids).double()
    size = on * (a.abs() * hot + p.exp() * (a.abs() + b.abs() * (ent + p.abs())))
    check_grad_w(h, W, ids, (on * (a * hot - p.exp() * (a + b * (ent + p))), size), gW)


@pytest.mark.parametrize("T,V,budget", [(150, 300_000, 40), (130, 1_048_576, 0), (130, 1_100_000, 0), (150, 1_100_000, 200),
                                        (130, 8_000_000, 0)])
def test_distill_over_a_wide_vocabulary(T, V, budget, monkeypatch):
    say(f"[wide distill] T={T} V={V} budget {budget}")
    K, tau = 100, 2.0
    gen, h, W, lean, y = draw(T, V, 2)
    # distinct ids: a few in the first splits, a few in the last, the rest anywhere
    ids = (torch.rand((T, K), device=DEV, generator=gen).double() ** torch.linspace(0.02, 8, K, device=DEV).double()
           * (V - K)).long().sort(dim=1).values + torch.arange(K, device=DEV)
    ids[:, 0], ids[:, K - 1] = 0, V - 1
    ids[y == -100] = -1
    lg = torch.randn((T, K), device=DEV, generator=gen) * 2
    ids = ids.int()
    at = torch.tensor([0, 1, 2, 4, T - 2, T - 1], device=DEV)
    alone = rlk.linear_distill_fwd(h[at], W, ids[at], lg[at], tau)
    if budget:
        monkeypatch.setenv("RLK_DZ_BUDGET_MB", str(budget))
    out = rlk.linear_distill_fwd(h, W, ids, lg, tau)
    for a, b in zip(alone, out):
        assert torch.equal(a, b[at])
    lp, lse = log_p(h[at], W, tau)
    on = y[at] != -100
    q = torch.log_softmax(lg[at].double() / tau, dim=1)
    lpk = lp.gather(1, ids[at].long().clamp_min(0))
    close("loss", alone[0][on], np64((q.exp() * (q - lpk)).sum(dim=1)[on]), LOSS_TOL)
    close("lse", alone[1][on], np64(lse[on]), LOGP_TOL)
    close("logp_ids", alone[2][on], np64(lpk[on]), LOGP_TOL)
    assert alone[2][~on].eq(-math.inf).all() and alone[0][~on].eq(0).all()
    g = torch.randn(T, device=DEV, generator=gen)
    gh, gW = rlk.linear_distill_bwd(h, W, ids, lg, out[1], out[2], g, tau, grad_W_dtype=torch.bfloat16)
    one, _ = rlk.linear_distill_bwd(h[at], W, ids[at], lg[at], alone[1], alone[2], g[at], tau, need_grad_W=False)
    assert torch.equal(gh[at], one)
    some = torch.cat([ids[1, ::7].long(), torch.tensor([0, V // 2, V - 1], device=DEV)]).unique()
    p = (h.double() @ W[some].double().T / tau - out[1].double()[:, None]).exp()
    full = torch.stack([((ids == v) * torch.softmax(lg.double() / tau, dim=1)).sum(dim=1) for v in some.tolist()], dim=1)
    c = torch.where(y != -100, g.double() / tau, 0.0)[:, None]
    check_grad_w(h, W, some, (c * (p - full), c.abs() * (p + full)), gW)
