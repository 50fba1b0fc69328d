"""embed and its gradient against the fp64 oracle: repeated, ignored and bad
ids, long runs of one token, few and many tokens, types, strides; and bits."""
import numpy as np
import pytest
import torch

import selected_token_lm_amd as rlk
from oracle import step_ops as O
from tests.gpu_util import DEV
from tests.step_util import DTYPES, U, dev, np64, rng, same, within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def tokens(T, V, seed, mask=0.2, kind="text"):
    r = rng(seed, T, V)
    if kind == "text":  # a few frequent tokens, many rare ones
        ids = np.minimum(V - 1, np.floor(np.exp(r.uniform(0, np.log(V + 1), T))).astype(np.int64))
    elif kind == "one":
        ids = np.full(T, V // 2)
    elif kind == "two":
        ids = np.where(r.uniform(size=T) < 0.5, 0, V - 1)
    else:
        ids = r.permutation(max(T, V))[:T] % V
    return np.where(r.uniform(size=T) < mask, -100, ids).astype(np.int64)


def ids_dev(ids, dtype=torch.int64):
    return torch.from_numpy(np.asarray(ids)).to(dtype).to(DEV)


def grad_bound(ids, gn, V, scale, base=None):
    """Sums of up to 16 rows (15 roundings), of an eighth of these sums (n / 128 at
    the most), of 8 (7); the scale; the sum with what is there."""
    n = np.bincount(ids[(ids >= 0) & (ids < V)], minlength=V)[:, None]
    total = O.embed_backward(ids, np.abs(gn), V, abs(scale))
    chain = np.minimum(n, 15 + n / 128 + 7)
    b = (chain + 1) * U * total
    return b if base is None else b + U * (np.abs(base) + total)


@pytest.mark.parametrize("E,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("T,H", [(1, 4096), (48, 2048), (7, 1), (100, 77), (33, 1999), (3000, 320), (2100, 1028)])
def test_lookup(T, H, E, out):
    V, scale = 500, np.float32(np.sqrt(H))
    ids = tokens(T, V, 1)
    if T > 40:
        ids[[3, 17, 40]] = [V, -1, 2 ** 40]
    Ed, En = dev(rng(2, H).normal(size=(V, H)), DTYPES[E])
    got = rlk.embed(ids_dev(ids), Ed, float(scale), out_dtype=DTYPES[out])
    want = O.embed_forward(ids, En, float(scale))
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(np64(got)), nan)
    within(torch.nan_to_num(got), np.nan_to_num(want), U * np.abs(np.nan_to_num(want)), DTYPES[out], "out")
    assert not np64(got)[ids == -100].any()
    if T > 40:
        ids[40] = 2 ** 31 - 1
    assert same(rlk.embed(ids_dev(ids, torch.int32), Ed, float(scale), out_dtype=DTYPES[out]), got)
    # scale 1 copies
    ok = ids_dev(np.where((ids < 0) | (ids >= V), 0, ids))
    if E == out:
        assert same(rlk.embed(ok, Ed), Ed[ok])


CASES = [(1, 64, 10, "text"), (5, 8, 3, "text"), (64, 256, 4096, "text"), (63, 100, 50, "one"), (64, 100, 50, "one"),
         (65, 100, 50, "one"), (128, 40, 7, "two"), (129, 1000, 7, "two"), (1000, 77, 30, "text"),
         (300, 1999, 1000, "distinct"), (4096, 520, 5000, "text"), (5000, 48, 1, "one"), (2500, 513, 2, "two"),
         (16384, 64, 900, "text"), (16385, 64, 900, "text"), (16384, 24, 9, "one"), (40000, 72, 200000, "text"),
         (70000, 16, 300, "two"), (20000, 1030, 3, "text"), (33000, 8, 8000000, "distinct")]


@pytest.mark.parametrize("g,grad", [("bf16", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("T,H,V,kind", CASES)
def test_gradient(T, H, V, kind, g, grad):
    if V > 10 ** 6 and (g, grad) != ("bf16", "f32"):
        pytest.skip("one type of the widest table")
    scale = float(np.float32(1.7))
    ids = tokens(T, V, 3, kind=kind)
    if T > 60:
        ids[[5, 50]] = [V, -7]
    gd, gn = dev(rng(4, T, H).normal(size=(T, H)), DTYPES[g])
    gd[ids_dev((ids < 0) | (ids >= V), torch.bool)] = float("nan")  # rows that count nothing
    gn[(ids < 0) | (ids >= V)] = 0
    got = rlk.embed_bwd(ids_dev(ids), gd, V, scale, grad_E_dtype=DTYPES[grad])
    assert got.dtype == DTYPES[grad]
    if V > 10 ** 6:
        live = np.unique(ids[(ids >= 0) & (ids < V)])
        where = {v: k for k, v in enumerate(live)}
        short = np.array([where.get(i, -100) for i in ids])
        at = torch.from_numpy(live).to(DEV)
        within(got[at], O.embed_backward(short, gn, len(live), scale), grad_bound(short, gn, len(live), scale),
               DTYPES[grad], "grad_E")
        got[at] = 0
        assert torch.count_nonzero(got) == 0
        return
    within(got, O.embed_backward(ids, gn, V, scale), grad_bound(ids, gn, V, scale), DTYPES[grad], "grad_E")
    absent = np.setdiff1d(np.arange(V), ids)
    assert torch.count_nonzero(got[torch.from_numpy(absent).to(DEV)]) == 0
    assert same(rlk.embed_bwd(ids_dev(ids), gd, V, scale, grad_E_dtype=DTYPES[grad]), got)
    # added to a gradient that is there; rows of other tokens are left as they are
    base, bn = dev(rng(5, V, H).normal(size=(V, H)), DTYPES[grad])
    base[torch.from_numpy(absent).to(DEV)] = float("nan")
    bn[absent] = 0
    total = rlk.embed_bwd(ids_dev(ids, torch.int64), gd, V, scale, grad_E=base)
    assert total is base
    present = np.setdiff1d(np.arange(V), absent)
    at = torch.from_numpy(present).to(DEV)
    within(total[at], (bn + O.embed_backward(ids, gn, V, scale))[present],
           grad_bound(ids, gn, V, scale, bn)[present], DTYPES[grad], "added")
    assert torch.isnan(total[torch.from_numpy(absent).to(DEV)]).all()
    zero = torch.zeros((V, H), dtype=DTYPES[grad], device=DEV)
    assert torch.equal(rlk.embed_bwd(ids_dev(ids), gd, V, scale, grad_E=zero), got)


@pytest.mark.parametrize("H", [20, 640, 2048])
def test_a_tokens_row_depends_on_its_own_rows(H):
    """Its bits are those of a batch of its rows alone, wherever they stand, and
    of a batch so padded that the tokens are sorted another way."""
    V, T = 40, 9000
    ids = tokens(T, V, 6, mask=0.1)
    gd, _ = dev(rng(7, H).normal(size=(T, H)), BF16)
    got = rlk.embed_bwd(ids_dev(ids), gd, V, 0.5)
    for v in (0, 1, 5, 39):
        rows = torch.from_numpy(np.flatnonzero(ids == v)).to(DEV)
        one = rlk.embed_bwd(ids_dev(ids[ids == v]), gd[rows], V, 0.5)
        assert same(one[v], got[v]), v
        one[v] = 0
        assert torch.count_nonzero(one) == 0
    for pad in (16384 - T, 16385 - T, 30000):
        more = np.concatenate([np.full(pad // 2, -100), ids, np.full(pad - pad // 2, -100)])
        gm = torch.full((T + pad, H), float("nan"), dtype=BF16, device=DEV)
        gm[pad // 2:pad // 2 + T] = gd
        assert same(rlk.embed_bwd(ids_dev(more), gm, V, 0.5), got), pad
        assert same(rlk.embed_bwd(ids_dev(more, torch.int32), gm, V, 0.5), got), pad


@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("H", [5, 300, 1025])
@pytest.mark.parametrize("sizes", [
    [1] * 40, [2, 15, 1, 16, 17, 1], [31, 32, 33, 1, 47, 48, 49], [63, 64, 65], [16] * 30, [17] * 30,
    [1, 255, 256, 257, 1, 3], [1023, 1024, 1025, 2], [4097, 1, 16, 5000, 15], [16, 9000, 17, 8000],
], ids=lambda s: "-".join(map(str, s[:4])))
def test_tokens_of_every_number_of_rows(sizes, H, grad):
    """Around runs, their batches and their joins; sums of small whole numbers,
    exact in fp32."""
    r = rng(10, len(sizes), H, sizes[0])
    names = r.permutation(3 * len(sizes))[:len(sizes)]
    ids = r.permutation(np.concatenate([np.full(n, v) for n, v in zip(sizes, names)] + [np.full(11, -100)]))
    V = 3 * len(sizes)
    g = r.integers(-2, 3, (len(ids), H)).astype(np.float32)
    gd, gn = dev(g, BF16)
    want = torch.from_numpy(O.embed_backward(ids, gn, V, 0.5)).to(DTYPES[grad])
    assert torch.equal(rlk.embed_bwd(ids_dev(ids), gd, V, 0.5, grad_E_dtype=DTYPES[grad]).cpu(), want)
    base = torch.ones((V, H), dtype=DTYPES[grad], device=DEV)
    want = torch.from_numpy(O.embed_backward(ids, gn, V, 0.5) + 1).to(DTYPES[grad])
    assert torch.equal(rlk.embed_bwd(ids_dev(ids), gd, V, 0.5, grad_E=base).cpu(), want)


@pytest.mark.parametrize("T", [3, 40, 2000])
@pytest.mark.parametrize("H", [8191, 16384, 65535, 65536])
def test_wide_rows(H, T):
    V = 20
    ids = tokens(T, V, 11, mask=0.1)
    r = rng(12, H)
    Ed, En = dev(r.normal(size=(V, H)), BF16)
    assert same(rlk.embed(ids_dev(np.abs(ids) % V), Ed), Ed[ids_dev(np.abs(ids) % V)])
    g = r.integers(-3, 4, (T, 64)).astype(np.float32)
    gd = dev(g, BF16)[0].repeat(1, -(-H // 64))[:, :H]
    want = torch.from_numpy(O.embed_backward(ids, g, V, 1.0)).float().repeat(1, -(-H // 64))[:, :H]
    assert torch.equal(rlk.embed_bwd(ids_dev(ids), gd, V).cpu(), want)


@pytest.mark.parametrize("V", [1, 2, 1023, 1024, 1025, 2048, 131072, 131073, 8_000_000])
def test_vocabularies_around_powers_of_two(V):
    """Every token once (or the first and last 300, a thousand random ones), by
    both sorts."""
    r = rng(13, V)
    ids = r.permutation(np.unique(np.concatenate([np.arange(min(V, 300)), np.arange(max(0, V - 300), V),
                                                  r.integers(0, V, 1000)])))
    g = r.integers(-3, 4, (len(ids), 8)).astype(np.float32)
    gd = dev(g)[0]
    want = torch.zeros((V, 8))
    want[torch.from_numpy(ids)] = torch.from_numpy(g)
    got = rlk.embed_bwd(ids_dev(ids), gd, V)
    assert torch.equal(got.cpu(), want)
    more = 17000 - len(ids)
    nan = gd.new_full((more, 8), float("nan"))
    got2 = rlk.embed_bwd(ids_dev(np.concatenate([ids, np.full(more, -100)])), torch.cat([gd, nan]), V)
    assert same(got2, got)
    E = want.to(DEV)
    assert torch.equal(rlk.embed(ids_dev(ids), E), gd)


def test_strided_and_broadcast_gradients():
    V, T, H = 30, 400, 100
    ids = tokens(T, V, 8)
    gd, _ = dev(rng(9).normal(size=(T, H)), BF16)
    want = rlk.embed_bwd(ids_dev(ids), gd, V)
    wide = torch.full((T, 3 * H + 1), float("nan"), dtype=BF16, device=DEV)
    wide[:, H + 1:2 * H + 1] = gd
    assert same(rlk.embed_bwd(ids_dev(ids), wide[:, H + 1:2 * H + 1], V), want)
    assert same(rlk.embed_bwd(ids_dev(ids), gd.t().contiguous().t(), V), want)
    row = gd[:1].expand(T, H)
    assert same(rlk.embed_bwd(ids_dev(ids), row, V), rlk.embed_bwd(ids_dev(ids), row.contiguous(), V))
    assert same(rlk.embed_bwd(ids_dev(np.repeat(ids, 2))[::2], gd, V), want)


def test_no_tokens_and_no_live_tokens():
    for T in (0, 3, 100, 17000):
        ids = torch.full((T,), -100, device=DEV)
        g = torch.full((T, 24), float("nan"), device=DEV)
        assert not rlk.embed_bwd(ids, g, 50).any()
        base = torch.ones((50, 24), device=DEV)
        assert (rlk.embed_bwd(ids, g, 50, grad_E=base) == 1).all()
        assert not rlk.embed_fwd(ids, base).any() and rlk.embed_fwd(ids, base).shape == (T, 24)
    # an ignored id that is a token, and an id at int64's end
    ids = torch.tensor([0, 2, 0, -2 ** 63, 2 ** 63 - 1, 2], device=DEV)
    g = torch.ones((6, 8), device=DEV)
    got = rlk.embed_bwd(ids, g, 3, ignore_index=0)
    assert (got[2] == 2).all() and not got[:2].any()
    out = rlk.embed_fwd(ids, torch.ones((3, 8), device=DEV), ignore_index=0)
    assert not out[[0, 2]].any() and (out[[1, 5]] == 1).all() and torch.isnan(out[3:5]).all()


def test_nan_and_infinity_reach_their_token_alone():
    ids = torch.tensor([1, 2, 1, 3, 3], device=DEV)
    g = torch.ones((5, 40), dtype=BF16, device=DEV)
    g[2, 7], g[3, 0], g[4, 0] = float("nan"), float("inf"), float("-inf")
    got = rlk.embed_bwd(ids, g, 5)
    bad = torch.isnan(got)
    assert bad.sum() == 2 and bad[1, 7] and bad[3, 0]
    E = torch.zeros((5, 8), device=DEV)
    E[3, 1] = float("inf")
    out = rlk.embed_fwd(ids, E, 2.0)
    assert torch.isinf(out).sum() == 2 and torch.isinf(out[3:, 1]).all()


def test_a_table_past_32_bits():
    """V H past 2^32 elements: the last rows, their gradient and the rows between."""
    V, H = 8_000_000, 576
    assert V * H > 2 ** 32
    E = torch.zeros((V, H), dtype=BF16, device=DEV)
    E[V - 1], E[V - 2], E[7] = 3, 2, 1
    ids = torch.tensor([V - 1, 7, V - 2, V - 1], device=DEV)
    assert torch.equal(rlk.embed_fwd(ids, E, 2.0)[:, 5].float().cpu(), torch.tensor([6.0, 2, 4, 6]))
    del E
    g = torch.ones((4, H), dtype=BF16, device=DEV)
    got = rlk.embed_bwd(ids, g, V, grad_E_dtype=BF16)
    assert (got[V - 1] == 2).all() and (got[V - 2] == 1).all() and (got[7] == 1).all()
    got[[7, V - 2, V - 1]] = 0
    assert not got.view(torch.int32).any()


@pytest.mark.parametrize("T", [1 << 20, (1 << 23) - 5])
def test_many_tokens(T):
    """Up to the row limit: three digits of the sort, thousands of runs; the sums
    are exact in fp32 (small whole numbers)."""
    V, H = 3_000_000, 8
    gen = torch.Generator(device=DEV).manual_seed(T)
    ids = torch.randint(0, V, (T,), device=DEV, generator=gen)
    ids[torch.rand(T, device=DEV, generator=gen) < 0.3] = 12345
    g = torch.randint(-1, 2, (T, H), device=DEV, generator=gen).to(BF16)
    got = rlk.embed_bwd(ids, g, V)
    want = torch.zeros((V, H), device=DEV).index_add_(0, ids, g.float())
    assert torch.equal(got, want)
