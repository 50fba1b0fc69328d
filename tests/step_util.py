"""Seeded inputs and error bounds for the tests of the operators before and
behind the LM head.

U is half a unit in the last place of fp32; a rounding to a type is off by at
most eps / 2 of the value.  Bounds are first order in U and carry one per
cent for the rest."""
import numpy as np
import torch

from tests.gpu_util import DEV

U = 2.0 ** -24
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rng(*seed):
    return np.random.Generator(np.random.PCG64(list(seed)))


def dev(a, dtype=torch.float32):
    """(the device tensor of `dtype`, its exact values in float64)."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dtype)
    return t.to(DEV), t.double().numpy()


def np64(t):
    return t.detach().double().cpu().numpy()


def same(a, b):
    """Equal bits."""
    assert a.shape == b.shape and a.dtype == b.dtype, (a.shape, b.shape, a.dtype, b.dtype)
    bits = [t.contiguous().reshape(-1, 1).view(torch.uint8) if t.numel() else None for t in (a, b)]
    return bits[0] is None or torch.equal(*bits)


def within(got, want, bound, dtype, what):
    """|got - want| <= bound, and the rounding to `dtype` (the smallest
    subnormals apart)."""
    got = np64(got)
    bound = 1.01 * bound + half_step(dtype) * (np.abs(want) + bound) + 1e-40
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), tuple(np.argwhere(bad)[0]), got[bad][0], want[bad][0],
                           np.broadcast_to(bound, bad.shape)[bad][0])


# Additions on the longest way into a row's sum: up to 16 elements of a thread
# (64 where a row is passed in pieces of 8192), 6 steps in a wave, up to 16
# waves, and a few operations around them.
ROW_CHAIN = 64 + 6 + 16 + 4


def norm_bounds(x, w, n, rstd, y):
    """(of y, of n): the mean is off by L U A, A = mean |x| (0 for rms_norm, which
    has none), so x - mean by that and U |x - mean|; rstd relative by L U (A
    rstd + 1); n by their sum and two roundings."""
    L = ROW_CHAIN
    A = np.abs(x).mean(axis=1, keepdims=True) * rstd[:, None]
    dn = L * U * (A + 1) * (np.abs(n) + 1) + 2 * U * np.abs(n)
    aw = 1.0 if w is None else np.abs(w)
    return aw * dn + U * (np.abs(n) * aw + 2 * np.abs(y)), dn


def norm_grad_bounds(x, w, g, n, rstd, gx, T, center):
    """(of grad_x, grad_w, grad_b), from the formulas: sums over a row have L
    roundings, sums over the rows those of a thread's rows (at least 64 blocks, or
    one a row), of up to 16 groups of rows in a block, 16 blocks and 32 groups."""
    L = ROW_CHAIN
    _, dn = norm_bounds(x, None, n, rstd, np.zeros_like(n))
    A = np.abs(x).mean(axis=1, keepdims=True) * rstd[:, None]
    rel = L * U * (A + 1)
    gw = np.abs(g if w is None else g * w)
    c1, c2 = (gw * np.abs(n)).mean(axis=1, keepdims=True), gw.mean(axis=1, keepdims=True) * center
    d1 = (gw * dn).mean(axis=1, keepdims=True) + (L + 2) * U * c1
    d2 = (L + 2) * U * c2
    r = rstd[:, None]
    bx = rel * np.abs(gx) + r * (4 * U * (gw + c2 + np.abs(n) * c1) + d2 + np.abs(n) * d1 + dn * c1)
    rows = -(-T // 64) + 16 + 16 + 32 + 4
    bw = (np.abs(g) * dn).sum(axis=0) + rows * U * np.abs(g * n).sum(axis=0)
    return bx, bw, rows * U * np.abs(g).sum(axis=0)
