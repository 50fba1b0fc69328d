"""layer_norm and rms_norm against the fp64 oracle: widths around every border
of the kernels, types, strides, few and many rows, values at the edges; and
their bits, which depend on the row alone."""
import numpy as np
import pytest
import torch

import selected_token_lm_amd as rlk
from oracle import step_ops as O
from tests.gpu_util import DEV
from tests.step_util import DTYPES, ROW_CHAIN, U, dev, norm_bounds, norm_grad_bounds, np64, rng, same, within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def make(T, H, seed=0, x=BF16, y=BF16, w=BF16, weight=True, bias=True):
    r = rng(seed, T, H)
    scale = np.exp(r.normal(size=(T, 1)))
    xd, xn = dev(scale * (r.normal(size=(T, H)) + r.normal(size=(T, 1))), x)
    wd, wn = dev(1 + 0.3 * r.normal(size=H), w) if weight else (None, None)
    bd, bn = dev(r.normal(size=H), w) if bias else (None, None)
    gd, gn = dev(r.normal(size=(T, H)), y)
    return (xd, wd, bd, gd), (xn, wn, bn, gn)


def run(center, x, w, b, g, eps, y_dtype, grad_dtype=F32):
    """[y, mean, rstd, grad_x, grad_w, grad_b] (None where rms_norm has none)."""
    if center:
        y, mean, rstd = rlk.layer_norm_fwd(x, w, b, eps, out_dtype=y_dtype)
        return [y, mean, rstd, *rlk.layer_norm_bwd(x, w, mean, rstd, g, grad_weight_dtype=grad_dtype)]
    y, rstd = rlk.rms_norm_fwd(x, w, eps, out_dtype=y_dtype)
    return [y, None, rstd, *rlk.rms_norm_bwd(x, w, rstd, g, grad_weight_dtype=grad_dtype), None]


def check(center, devs, hosts, eps, x, y, grad=F32):
    xd, wd, bd, gd = devs
    xn, wn, bn, gn = hosts
    if not center:
        bd = bn = None
    got = run(center, xd, wd, bd, gd, eps, y, grad)
    T = xn.shape[0]
    yn, n, mean, rstd = O.norm_forward(xn, wn, bn, eps, center)
    gx, gw, gb = O.norm_backward(xn, wn, gn, eps, center)
    by, _ = norm_bounds(xn, wn, n, rstd, yn)
    bx, bw, bb = norm_grad_bounds(xn, wn, gn, n, rstd, gx, T, center)
    within(got[0], yn, by, y, "y")
    within(got[3], gx, bx, x, "grad_x")
    within(got[4], gw, bw, grad, "grad_weight")
    if center:
        within(got[5], gb, bb, grad, "grad_bias")
    return got


WIDTHS = [1, 2, 7, 8, 9, 16, 63, 64, 127, 128, 129, 255, 256, 257, 505, 512, 513, 1000, 1024, 1025, 1999, 2048, 2050, 4095, 4096, 4097, 8191,
          8192, 8200, 16384, 16385, 65535, 65536]


@pytest.mark.parametrize("center", [False, True], ids=["rms", "layer"])
@pytest.mark.parametrize("H", WIDTHS)
def test_widths(H, center):
    devs, hosts = make(5, H, x=BF16, y=BF16)
    check(center, devs, hosts, 1e-5, BF16, BF16)
    devs, hosts = make(3, H, seed=1, x=F32, y=F32, w=F32)
    check(center, devs, hosts, 1e-5, F32, F32)


@pytest.mark.parametrize("center", [False, True], ids=["rms", "layer"])
@pytest.mark.parametrize("w", ["bf16", "f32"])
@pytest.mark.parametrize("y", ["bf16", "f32"])
@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("H", [320, 777, 3000, 9001, 20000])
def test_types(H, x, y, w, center):
    devs, hosts = make(9, H, seed=2, x=DTYPES[x], y=DTYPES[y], w=DTYPES[w])
    got = check(center, devs, hosts, 1e-6, DTYPES[x], DTYPES[y], DTYPES[w])
    assert got[0].dtype == DTYPES[y] and got[3].dtype == DTYPES[x] and got[4].dtype == DTYPES[w]


@pytest.mark.parametrize("center", [False, True], ids=["rms", "layer"])
@pytest.mark.parametrize("T,H", [(1, 4096), (2, 256), (63, 128), (257, 1024), (1777, 1999), (2049, 520), (5000, 64), (10001, 100), (4099, 250),
                                 (700, 8192), (300, 12000), (3, 1), (4096, 2048)])
def test_row_counts(T, H, center):
    devs, hosts = make(T, H, seed=3, x=F32)
    check(center, devs, hosts, 1e-5, F32, BF16)


@pytest.mark.parametrize("center", [False, True], ids=["rms", "layer"])
def test_without_weight_and_bias(center):
    for weight, bias in ((False, False), (False, True), (True, False)):
        devs, hosts = make(6, 300, seed=4, weight=weight, bias=bias)
        check(center, devs, hosts, 1e-5, BF16, BF16)


@pytest.mark.parametrize("center", [False, True], ids=["rms", "layer"])
@pytest.mark.parametrize("H", [20, 100, 200, 999, 2048, 4100, 9000, 17000])
def test_a_row_has_its_bits_in_every_batch_and_layout(H, center):
    """Alone, in a batch, with strided or unaligned rows, all rows the same."""
    (x, w, b, g), _ = make(37, H, seed=5)
    b = b if center else None
    want = run(center, x, w, b, g, 1e-5, BF16)
    again = run(center, x, w, b, g, 1e-5, BF16)
    assert all(p is q is None or same(p, q) for p, q in zip(want, again))
    for t in (0, 11, 36):
        one = run(center, x[t:t + 1], w, b, g[t:t + 1], 1e-5, BF16)
        for k in (0, 1, 2, 3):
            assert want[k] is None or same(one[k], want[k][t:t + 1]), (t, k)
    # rows at odd distances and from odd addresses
    wide = torch.full((37, H + 13), float("nan"), dtype=BF16, device=DEV)
    wide[:, 3:3 + H] = x
    wide_g = torch.full((37, 2 * H + 1), float("nan"), dtype=BF16, device=DEV)
    wide_g[:, 1:1 + H] = g
    for xs, gs in ((wide[:, 3:3 + H], wide_g[:, 1:1 + H]), (x.t().contiguous().t(), g)):
        got = run(center, xs, w, b, gs, 1e-5, BF16)
        assert all(p is q is None or same(p, q) for p, q in zip(want, got))
    got = run(center, x[5:6].expand(37, H), w, b, g[5:6].expand(37, H), 1e-5, BF16)
    for k in (0, 3):
        assert all(same(got[k][t], want[k][5]) for t in range(37))


@pytest.mark.parametrize("H", [64, 1000, 4096, 9000])
def test_what_is_asked_for_changes_no_bit(H):
    (x, w, b, g), _ = make(50, H, seed=6)
    y, mean, rstd = rlk.layer_norm_fwd(x, w, b)
    assert same(rlk.layer_norm(x, w, b), y) and same(rlk.rms_norm(x, w), rlk.rms_norm_fwd(x, w)[0])
    full = rlk.layer_norm_bwd(x, w, mean, rstd, g)
    for need in [(1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 1, 1), (1, 1, 0)]:
        got = rlk.layer_norm_bwd(x, w, mean, rstd, g, *map(bool, need))
        for a, c, n in zip(got, full, need):
            assert same(a, c) if n else a is None
    rstd = rlk.rms_norm_fwd(x, w)[1]
    full = rlk.rms_norm_bwd(x, w, rstd, g)
    assert same(rlk.rms_norm_bwd(x, w, rstd, g, need_grad_weight=False)[0], full[0])
    assert same(rlk.rms_norm_bwd(x, w, rstd, g, need_grad_x=False)[1], full[1])
    assert rlk.rms_norm_bwd(x, w, rstd, g, False, False) == (None, None)


@pytest.mark.parametrize("H", [8, 1999, 20000])
def test_no_rows(H):
    x, w = torch.empty((0, H), dtype=BF16, device=DEV), torch.ones(H, dtype=BF16, device=DEV)
    y, mean, rstd = rlk.layer_norm_fwd(x, w, w)
    assert y.shape == (0, H) and mean.shape == rstd.shape == (0,)
    gx, gw, gb = rlk.layer_norm_bwd(x, w, mean, rstd, x)
    assert gx.shape == (0, H) and not gw.any() and not gb.any()
    assert not rlk.rms_norm_bwd(x, w, rstd, x)[1].any()


@pytest.mark.parametrize("H", [60, 4096, 20000])
def test_values_at_the_edges(H):
    """Constant and zero rows, a NaN or an infinity that stays in its row, rows
    whose squares are near the end of the type."""
    r = rng(9, H)
    a = r.normal(size=(8, H)).astype(np.float32)
    a[0], a[1] = 5.0, 0.0
    a[2, 3], a[3, H - 1] = np.nan, np.inf
    a[4] *= 1e16
    a[5] *= 1e-18
    x = torch.from_numpy(a).to(DEV)
    w = torch.ones(H, device=DEV)
    y, mean, rstd = rlk.layer_norm_fwd(x, w, None, 1e-5)
    assert torch.count_nonzero(y[:2]) == 0 and mean[0] == 5.0
    assert torch.isnan(y[2:4]).all() and torch.isfinite(y[4:]).all()
    z, rs = rlk.rms_norm_fwd(x, w, 1e-5)
    assert torch.count_nonzero(z[1]) == 0 and torch.isnan(z[2]).all()
    # an infinite element: rstd is 0, so the row is 0 but for 0 * inf
    assert rs[3] == 0 and torch.isnan(z[3, H - 1]) and torch.count_nonzero(z[3, :H - 1]) == 0
    for row in (4, 5, 6):
        want = O.norm_forward(a[row:row + 1], None, None, 1e-5, True)
        n, _ = norm_bounds(a[row:row + 1].astype(np.float64), None, want[1], want[3], want[0])
        within(y[row:row + 1], want[0], n, F32, row)
    # eps 0: the formulas hold for rows that are not constant
    got = rlk.layer_norm_fwd(x[6:], w, None, 0.0)[0]
    want = O.norm_forward(a[6:], None, None, 0.0, True)
    within(got, want[0], norm_bounds(a[6:].astype(np.float64), None, want[1], want[3], want[0])[0], F32, "eps 0")
    # gradients: a NaN row leaves the others' grad_x alone and reaches every weight that sees it
    g = torch.ones_like(x)
    gx, gw, gb = rlk.layer_norm_bwd(x, w, mean, rstd, g)
    assert torch.isnan(gx[2:4]).all() and torch.isfinite(gx[4:]).all() and torch.isfinite(gx[:2]).all()
    assert torch.isnan(gw).all() and (gb == 8).all()


@pytest.mark.parametrize("H", [5, 200, 4096, 20000])
def test_squares_past_the_types_range(H):
    """rstd is 0 there, and y the bias."""
    x = torch.ones((3, H), device=DEV)
    x[1, ::2], x[1, 1::2] = 3e25, -3e25
    b = torch.arange(H, device=DEV).float()
    y, _, rstd = rlk.layer_norm_fwd(x, None, b)
    assert rstd[1] == 0 and torch.equal(y[1], b) and same(y[::2], rlk.layer_norm(x[::2], None, b))
    z, rstd = rlk.rms_norm_fwd(x)
    assert rstd[1] == 0 and not z[1].any() and same(z[::2], rlk.rms_norm(x[::2]))


def test_statistics_given_otherwise():
    """Strided and 64-bit statistics; wrong ones are refused."""
    (x, w, _, g), _ = make(9, 100, seed=8)
    _, mean, rstd = rlk.layer_norm_fwd(x, w)
    want = rlk.layer_norm_bwd(x, w, mean, rstd, g)
    wide = torch.stack([mean, rstd], dim=1)
    got = rlk.layer_norm_bwd(x, w, wide[:, 0], rstd.double(), g)
    assert all(same(a, c) for a, c in zip(got, want))
    for m, r, text in ((None, rstd, "mean is required"), (mean, None, "rstd is required"), (mean[:8], rstd, "T = 9"),
                       (mean, rstd[None], "T = 9"), (mean.cpu(), rstd, "must be on")):
        with pytest.raises(ValueError, match=text):
            rlk.layer_norm_bwd(x, w, m, r, g)


def test_many_rows():
    """More rows than a launch of the backward has blocks for, by far, and a
    forward of 2^20 rows."""
    T, H = 1 << 20, 24
    r = rng(12)
    x, xn = dev(r.normal(size=(T, H)), BF16)
    g, gn = dev(r.normal(size=(T, H)), BF16)
    y, mean, rstd = rlk.layer_norm_fwd(x)
    yn, n, _, rs = O.norm_forward(xn, None, None, 1e-5, True)
    within(y, yn, norm_bounds(xn, None, n, rs, yn)[0], BF16, "y")
    gx, gw, gb = rlk.layer_norm_bwd(x, None, mean, rstd, g)
    wx, ww, wb = O.norm_backward(xn, None, gn, 1e-5, True)
    bx, bw, bb = norm_grad_bounds(xn, None, gn, n, rs, wx, T, True)
    within(gx, wx, bx, BF16, "grad_x")
    within(gw, ww, bw, F32, "grad_weight")
    within(gb, wb, bb, F32, "grad_bias")


def test_offsets_past_32_bits():
    """A row stride that takes rows past 2^32 bytes and 2^31 elements."""
    H, ld = 256, 600_000_000
    flat = torch.empty(5 * ld, dtype=BF16, device=DEV)
    x = flat.as_strided((5, H), (ld, 1))
    small, _ = make(5, H, seed=13)
    x.copy_(small[0])
    w, g = small[1], small[3]
    assert same(rlk.rms_norm(x, w), rlk.rms_norm(small[0], w))
    rstd = rlk.rms_norm_fwd(x, w)[1]
    want = rlk.rms_norm_bwd(small[0], w, rstd, g)
    assert all(same(a, b) for a, b in zip(rlk.rms_norm_bwd(x, w, rstd, g), want))
    x.copy_(g)
    assert all(same(a, b) for a, b in zip(rlk.rms_norm_bwd(small[0], w, rstd, x), want))


@pytest.mark.parametrize("x,y", [(BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("H", [1, 20, 100, 250, 500, 999, 1999, 3001, 5003, 9001, 65535])
def test_a_large_constant_row_at_widths_that_fill_no_vector(H, x, y):
    """All exact: x = 2^100, whose sums, mean and differences (0) need no rounding;
    eps = 2^-80, so rstd = 2^40, and mean rstd is past the type's range.  n is 0
    and g's sum is 0, so grad_x = 2^40 g, grad_weight = 0 and grad_bias = g."""
    g = torch.zeros((3, H), device=DEV)
    g[:, 0:H - H % 2:2], g[:, 1:H:2] = 1.0, -1.0
    xd = torch.full((3, H), 2.0 ** 100, device=DEV)
    xd[1] = 1.0
    yd, mean, rstd = rlk.layer_norm_fwd(xd.to(x), None, None, 2.0 ** -80, out_dtype=y)
    assert not yd.any() and torch.equal(mean, xd[:, 0]) and (rstd == 2.0 ** 40).all()
    gx, gw, gb = rlk.layer_norm_bwd(xd.to(x), None, mean, rstd, g.to(y))
    assert torch.equal(gx.float(), 2.0 ** 40 * g) and not gw.any() and torch.equal(gb, 3 * g[0])


@pytest.mark.parametrize("x,y", [(BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("H", [2, 5, 200, 500, 999, 2048, 4096, 5003, 16384, 20000, 65535])
def test_sums_past_the_types_range(H, x, y):
    """Rows of one sign: the mean is in range though the sum is not.  Constant rows
    of a power of two are exact: mean is the value, y the bias, rstd 2^20 (eps
    2^-40).  Others have rstd 0, and y the bias."""
    a = torch.full((4, H), 2.0 ** 127, device=DEV)
    a[1] = -a[1]
    a[2] = 1e38 + 2e38 * torch.rand(H, device=DEV, generator=torch.Generator(DEV).manual_seed(H))
    a[3] = torch.arange(H, device=DEV) % 2
    a = a.to(x)
    b = (torch.arange(H, device=DEV) % 100).to(y)
    out, mean, rstd = rlk.layer_norm_fwd(a, None, b, 2.0 ** -40, out_dtype=y)
    assert torch.equal(mean[:2], a[:2, 0].float()) and (rstd[:2] == 2.0 ** 20).all() and rstd[2] == 0
    assert all(torch.equal(out[t], b) for t in range(3))
    assert same(out[3:], rlk.layer_norm(a[3:], None, b, 2.0 ** -40, out_dtype=y))
    # the sum's roundings as in norm_bounds, relative to a mean of one sign
    want = np64(a[2]).mean()
    assert abs(float(mean[2]) - want) <= 1.01 * (ROW_CHAIN + 2) * U * want
    g = torch.ones((4, H), device=DEV).to(y)
    gx, gw, gb = rlk.layer_norm_bwd(a, None, mean, rstd, g)
    assert torch.count_nonzero(gx[:3]) == 0 and (gb == 4).all() and torch.isfinite(gw).all()


@pytest.mark.parametrize("T,H", [(512, 1999), (1777, 1999), (1777, 2048), (5000, 1040)])
def test_sums_over_the_rows_are_a_tree(T, H):
    """512 blocks, a row each of the first 512: 2^24 and 511 ones (further rows are
    0), which lose what is added one at a time to the large one.  A tree adds in
    nine steps, so nine roundings of at most U (2^24 + 511)."""
    g = torch.zeros((T, H), device=DEV)
    g[:512] = 1.0
    total = 2.0 ** 24 + 511
    x, one, zero = torch.ones((T, H), device=DEV), torch.ones(T, device=DEV), torch.zeros(T, device=DEV)
    for large in (0, 37, 300, 511):
        g[:512] = 1.0
        g[large] = 2.0 ** 24
        _, gw, gb = rlk.layer_norm_bwd(x, None, zero, one, g)  # n = 1
        rw = rlk.rms_norm_bwd(x, None, one, g)[1]
        for t in (gw, gb, rw):
            assert (t.double() - total).abs().max() <= 9 * U * total, (large, float(t[0]) - total)


def rows_chain(T, H):
    """Roundings of a sum over the rows: those a thread takes, the groups of rows
    in a block one after the other, the blocks as a tree."""
    group = 16 if H <= 128 else 8 if H <= 256 else 4 if H <= 1024 else 1
    most = 64 if H > 8192 else 256 if H > 4096 or (H > 2048 and T <= 1536) else 512
    parts = min(most, -(-T // group))
    return -(-T // (parts * group)) + group + 9


SEVERAL = [(1000, 4096), (1536, 2050), (1537, 4096), (2049, 4096), (4096, 3000), (1777, 1999), (2500, 1040), (700, 6000),
           (300, 9001), (3000, 700), (9000, 200), (20000, 72)]


@pytest.mark.parametrize("center", [False, True], ids=["rms", "layer"])
@pytest.mark.parametrize("x,y", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("T,H", SEVERAL)
def test_blocks_that_take_several_rows(T, H, x, y, center):
    """More rows than blocks (and their groups of rows) at every width's kernel,
    on both sides of the rules for their number; the sums over the rows within
    the roundings that their split has."""
    devs, hosts = make(T, H, seed=20, x=x, y=y)
    got = check(center, devs, hosts, 1e-5, x, y)
    xn, wn, _, gn = hosts
    _, n, _, rstd = O.norm_forward(xn, wn, None, 1e-5, center)
    _, gw, gb = O.norm_backward(xn, wn, gn, 1e-5, center)
    _, dn = norm_bounds(xn, None, n, rstd, np.zeros_like(n))
    chain = rows_chain(T, H)
    # each term g n has the error of n and a rounding of the product
    within(got[4], gw, (np.abs(gn) * dn).sum(axis=0) + (chain + 1) * U * np.abs(gn * n).sum(axis=0), F32, "grad_weight")
    if center:
        within(got[5], gb, chain * U * np.abs(gn).sum(axis=0), F32, "grad_bias")


@pytest.mark.parametrize("x,y", [(BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("T,H", [*SEVERAL, (1 << 20, 24), (300_000, 130), (70_000, 520), (30_011, 1500), (16384, 2048), (6000, 4096),
                                 (5000, 8192), (2000, 20000), (1, 4096), (255, 3000)])
def test_sums_over_the_rows_count_every_row_once(T, H, x, y):
    """Whole numbers, |g n| <= 8 and |g| <= 1 with at most 2^20 rows: every sum, in
    any order, is exact in fp32, so that a lost or repeated row, group or part
    changes it."""
    gen = torch.Generator(DEV).manual_seed(T * 7 + H)
    xi = torch.randint(-8, 9, (T, H), device=DEV, generator=gen)
    gi = torch.randint(-1, 2, (T, H), device=DEV, generator=gen)
    one, zero = torch.ones(T, device=DEV), torch.zeros(T, device=DEV)
    xs, gs = xi.to(x), gi.to(y)
    want_w, want_b = (xi * gi).sum(dim=0), gi.sum(dim=0)
    for need in (True, False):
        _, gw, gb = rlk.layer_norm_bwd(xs, None, zero, one, gs, need_grad_x=need)  # n = x
        assert torch.equal(gw, want_w.float()) and torch.equal(gb, want_b.float())
        assert torch.equal(rlk.rms_norm_bwd(xs, None, one, gs, need_grad_x=need)[1], want_w.float())
