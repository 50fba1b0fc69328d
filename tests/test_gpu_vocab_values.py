"""linear_logp_top and linear_distill on values at the edges: a teacher's
undefined logits.
"""
import numpy as np
import pytest
import torch

import selected_token_lm_amd as rlk
from tests.gpu_util import DEV, f32_dev, i32_dev
from tests.test_gpu_vocab_ops import Case

pytestmark = pytest.mark.gpu


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
