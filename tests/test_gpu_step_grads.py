"""grad_norm and clip_grads against the fp64 oracle: many tensors, sizes around
a block's chunk, types, layouts, in place and into other tensors, values at
the edges."""
import math

import numpy as np
import pytest
import torch

import selected_token_lm_amd as rlk
from oracle import step_ops as O
from tests.gpu_util import DEV
from tests.step_util import DTYPES, U, dev, np64, rng, same, within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16

LISTS = {
    "one element": [(1,)],
    "chunk borders": [(16383,), (16384,), (16385,), (7,), (8,), (9,)],
    "empty ones": [(0,), (5, 0), (33,), (0, 3)],
    "a model": [(500, 64)] + [(64, 64), (64,)] * 30 + [(999, 77)],
    "launches of many": [(3,), (1000,)] * 150,
    "a large one": [(3000, 4111)],
}


def make(shapes, types, seed=0, scale=1.0):
    out = []
    for i, n in enumerate(shapes):
        t = DTYPES[types[i % len(types)]]
        d, h = dev(scale * 2.0 ** (i % 4) * rng(seed, i).normal(size=n), t)
        out.append((d, h))
    return [d for d, _ in out], [h for _, h in out]


def check_norm(got, hosts):
    """fp64 sums: far below the rounding to fp32."""
    want = O.grad_norm(hosts)
    assert got.shape == () and got.dtype == F32
    assert abs(float(got) - want) <= (U + 1e-11) * want, (float(got), want)
    return want


def check_clip(out, hosts, max_norm, dtypes):
    """max_norm is taken in fp32; c is rounded to it, the product once, the result
    to its type."""
    c = O.clip_factor(hosts, float(np.float32(max_norm)))
    for o, h, t in zip(out, hosts, dtypes):
        assert o.dtype == t
        within(o, c * h, (0 if c == 1 else 2 * U + 1e-11) * np.abs(c * h), t, "out")


@pytest.mark.parametrize("types", [("f32",), ("bf16",), ("f32", "bf16")], ids="-".join)
@pytest.mark.parametrize("name", LISTS)
def test_norm_and_clipping(name, types):
    ts, hosts = make(LISTS[name], types, seed=1)
    norm = rlk.grad_norm(ts)
    want = check_norm(norm, hosts)
    assert same(rlk.grad_norm(ts), norm)
    for most in (want / 3, want * 2, math.inf):
        copies = [t.clone() for t in ts]
        # into tensors of either type
        out = [torch.full(t.shape, float("nan"), dtype=(F32, BF16)[i % 2], device=DEV) for i, t in enumerate(ts)]
        got, o = rlk.clip_grads(ts, most, out=out)
        assert same(got, norm) and all(a is b for a, b in zip(o, out))
        check_clip(out, hosts, most, [t.dtype for t in out])
        assert all(same(a, b) for a, b in zip(ts, copies))
        # in place
        got, o = rlk.clip_grads(copies, most)
        assert same(got, norm) and all(a is b for a, b in zip(o, copies))
        check_clip(copies, hosts, most, [t.dtype for t in copies])
        if most > want:
            assert all(same(a, b) for a, b in zip(ts, copies))
        for a, b, t in zip(out, copies, ts):
            assert a.dtype != t.dtype or same(a, b)


def test_one_tensor_and_generators():
    assert float(rlk.grad_norm(torch.tensor(-3.0, device=DEV))) == 3.0
    t = torch.full((10,), 2.0, device=DEV)
    assert float(rlk.grad_norm(t)) == float(np.float32(math.sqrt(40)))
    assert float(rlk.grad_norm(iter([t, t]))) == float(np.float32(math.sqrt(80)))  # the same tensor twice counts twice
    norm, out = rlk.clip_grads((x for x in [t]), 1.0)
    assert out[0] is t and abs(float(rlk.grad_norm(t)) - 1) < 4 * U


def test_lists_of_nothing():
    for ts in ([torch.empty(0, device=DEV)], [torch.empty((0, 3), dtype=BF16, device=DEV)] * 200):
        assert float(rlk.grad_norm(ts)) == 0.0
        norm, out = rlk.clip_grads(ts, 0.0)
        assert float(norm) == 0.0 and all(a is b for a, b in zip(out, ts))
    with pytest.raises(ValueError, match="empty"):
        rlk.grad_norm([])


def test_layouts():
    """Transposed and unaligned tensors; a flat buffer's pieces as outputs."""
    r = rng(3)
    a, an = dev(r.normal(size=(31, 57)))
    flat = torch.zeros(4000, dtype=BF16, device=DEV)
    b = flat[1:1 + 777]
    b.copy_(torch.from_numpy(r.normal(size=777)))
    hosts = [an.T, np64(b)]
    want = check_norm(rlk.grad_norm([a.t(), b]), hosts)
    buf = torch.full((31 * 57 + 777 + 2,), 9.0, dtype=BF16, device=DEV)
    out = [buf[1:1 + 31 * 57].view(31, 57).t(), buf[1 + 31 * 57:-1]]
    rlk.clip_grads([a.t(), b], want / 2, out=out)
    check_clip(out, hosts, want / 2, [BF16, BF16])
    assert buf[0] == 9 and buf[-1] == 9
    rlk.clip_grads([b], O.grad_norm(hosts[1:]) / 2)
    assert flat[0] == 0 and not flat[778:].any()
    check_clip([b], hosts[1:], O.grad_norm(hosts[1:]) / 2, [BF16])
    with pytest.raises(ValueError, match="dense"):
        rlk.grad_norm([a[:, :5]])
    with pytest.raises(ValueError, match="layout"):
        rlk.clip_grads([a.t()], 1.0, out=[torch.empty((57, 31), device=DEV)])


def test_overlaps_are_refused():
    t = torch.ones(100, device=DEV)
    o = torch.zeros(200, device=DEV)
    for grads, out in (([t, t], None), ([t[:60], t[50:]], None), ([t], [t.view(BF16)[:100]]),
                       ([t[:50], o[:50]], [o[:50], o[100:150]]), ([t[:50], t[50:]], [o[:50], o[49:99]]),
                       ([o[:100]], [o[1:101]])):
        before = t.clone(), o.clone()
        with pytest.raises(rlk.RlkError, match="overlaps"):
            rlk.clip_grads(grads, 1.0, out=out)
        assert same(t, before[0]) and same(o, before[1])
    # the same gradient twice into two outputs, neighbours, empty tensors anywhere
    rlk.clip_grads([t, t], 1.0, out=[o[:100], o[100:]])
    assert torch.equal(o[:100], o[100:])
    rlk.clip_grads([t[:50], t[50:], t[10:10]], 1.0)


def test_values_at_the_edges():
    big = torch.full((1000,), 3e38, device=DEV)
    tiny = torch.full((1000,), 1e-42, device=DEV)
    # squares past the type's range on both sides, exact in 64 bits
    assert torch.isinf(rlk.grad_norm(big))  # past the type's range itself
    assert float(rlk.grad_norm(big[:1])) == float(big[0])
    v = float(tiny[0].double())
    assert abs(float(rlk.grad_norm(tiny)) - v * math.sqrt(1000)) <= 2.0 ** -149
    norm, out = rlk.clip_grads([big], 1.0, out=[torch.empty_like(big)])
    assert torch.isinf(norm)  # rounded: but c comes from the 64-bit norm
    # ... and is itself a subnormal of fp32, off by up to 2^-150
    off = 4 * U + 2.0 ** -150 * math.sqrt(1000) * 3e38
    assert abs(float(out[0][0]) * math.sqrt(1000) - 1) < off < 1e-5
    zero = torch.zeros(50, device=DEV)
    norm, _ = rlk.clip_grads([zero], 0.0)
    assert norm == 0 and not zero.any()
    one = torch.ones(50, dtype=BF16, device=DEV)
    norm, _ = rlk.clip_grads([one], 0.0)
    assert norm == np.float32(math.sqrt(50)) and not one.any()
    for bad in (float("nan"), float("inf"), float("-inf")):
        t, other = torch.ones(70000, device=DEV), torch.ones(10, dtype=BF16, device=DEV)
        t[40000] = bad
        norm = rlk.grad_norm([other, t])
        assert torch.isnan(norm) if bad != bad else norm == math.inf
        norm2, _ = rlk.clip_grads([other, t], 1.0)
        assert same(norm, norm2)
        if bad != bad:
            assert torch.isnan(t).all() and torch.isnan(other).all()
        else:
            assert torch.isnan(t[40000]) and torch.count_nonzero(t) == 1 and not other.any()


def test_a_tensor_past_32_bits():
    n = 2 ** 31 + 70001
    t = torch.zeros(n, dtype=BF16, device=DEV)
    t[0], t[n - 1], t[2 ** 31] = 3, 4, 12
    assert float(rlk.grad_norm(t)) == 13.0
    rlk.clip_grads([t], 6.5)
    assert t[0] == 1.5 and t[n - 1] == 2 and t[2 ** 31] == 6 and torch.count_nonzero(t.view(torch.int16)) == 3

