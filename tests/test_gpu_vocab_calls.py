"""linear_logp_top and linear_distill as programs call them: batches of which
few rows or none are active, a training step captured through autograd with
64-bit ids, a graph walked twice, two host threads at once.
"""
import threading

import numpy as np
import pytest
import torch

import selected_token_lm_amd as rlk
from tests.gpu_util import DEV, f32_dev, i32_dev
from tests.test_gpu_vocab_ops import Case

pytestmark = pytest.mark.gpu


def inputs(T, H, V, K, seed, mask=0.0):
    c = Case(T, H, V, mask, seed=seed)
    n_ids, n_lg = c.teacher(K)
    return (*c.dev(), i32_dev(c.y), i32_dev(n_ids), f32_dev(n_lg), f32_dev(c.g), f32_dev(c.ge))


def all_of(h, W, y, ids, lg, g, ge, K=9, tau=1.5):
    out = list(rlk.linear_logp_top_fwd(h, W, y, K))
    out += rlk.linear_logp_top_bwd(h, W, y, out[1], out[2], g, ge, grad_W_dtype=torch.bfloat16)
    d = list(rlk.linear_distill_fwd(h, W, ids, lg, tau))
    return out + d + list(rlk.linear_distill_bwd(h, W, ids, lg, d[1], d[2], g, tau))


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("T", [129, 300, 700])  # one row tile, two, three
@pytest.mark.parametrize("n", [0, 1, 63, 65, 128])
def test_few_active_rows_of_a_large_batch(T, n):
    """The active rows' results and grad_W are those of a batch of these rows
    alone, bit for bit; the others' are empty, whatever they hold."""
    h, W, y, ids, lg, g, ge = inputs(T, 192, 5000, 12, seed=n)
    on = torch.zeros(T, dtype=torch.bool, device=DEV)
    on[torch.from_numpy(np.random.Generator(np.random.PCG64(T + n)).permutation(T)[:n].copy()).to(DEV)] = True
    y[~on], ids[~on], h[~on], g[~on], ge[~on], lg[~on] = -100, -1, float("nan"), float("nan"), float("inf"), float("nan")
    got = all_of(h, W, y, ids, lg, g, ge)
    if n:
        want = all_of(*(x[on].contiguous() if x is not W else W for x in (h, W, y, ids, lg, g, ge)))
        for k, (a, b) in enumerate(zip(got, want)):
            assert same(a if k in (6, 11) else a[on], b), k
    else:
        assert torch.count_nonzero(got[6]) == 0 and torch.count_nonzero(got[11]) == 0
    for k, value in ((0, 0), (1, 0), (2, 0), (3, -np.inf), (4, -1), (5, 0), (7, 0), (8, 0), (9, -np.inf), (10, 0)):
        assert got[k][~on].eq(value).all(), k


@pytest.mark.parametrize("T", [60, 200])
def test_a_captured_training_step_with_64_bit_ids(T):
    """Both operators, forward and backward, through autograd in one graph;
    replayed between eager steps, and on new values."""
    h, W, y, ids, lg, g, ge = inputs(T, 128, 3000, 8, seed=T, mask=0.2)
    y, ids = y.long(), ids.long()
    h.requires_grad_()
    W.requires_grad_()

    def step():
        logp, ent, top, best = rlk.linear_logp_top(h, W, y, 5)
        loss = rlk.linear_distill(h, W, ids, lg, 1.5)
        total = (g * logp + ge * ent).sum() + (g * loss).sum()
        return [x.detach() for x in (logp, ent, top, best, loss)] + list(torch.autograd.grad(total, (h, W)))

    want = [x.clone() for x in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(out, want)), rep
        assert all(same(a, b) for a, b in zip(step(), want))
    with torch.no_grad():
        for x in (h, y, ids, lg, g):
            x.copy_(x.flip(0).clone())
    new = step()
    assert not same(new[0], want[0])
    graph.replay()
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(out, new))


def test_a_graph_walked_twice():
    h, W, y, ids, lg, g, ge = inputs(70, 64, 900, 6, seed=4)
    h.requires_grad_()
    W.requires_grad_()
    logp, ent, _, _ = rlk.linear_logp_top(h, W, y)
    for total in ((g * logp + ge * ent).sum(), (g * rlk.linear_distill(h, W, ids, lg)).sum()):
        a = torch.autograd.grad(total, (h, W), retain_graph=True)
        b = torch.autograd.grad(total, (h, W))
        assert all(same(x, y) for x, y in zip(a, b))


def test_two_host_threads():
    """Each on a stream of its own."""
    data = [inputs(T, 128, 9000, 10, seed=T) for T in (50, 260)]
    want = [all_of(*x) for x in data]
    torch.cuda.synchronize()
    got, streams = [[], []], [torch.cuda.Stream(), torch.cuda.Stream()]

    def work(k):
        with torch.cuda.stream(streams[k]):
            for _ in range(4):
                got[k].append(all_of(*data[k]))
            streams[k].synchronize()

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for k in range(2):
        assert len(got[k]) == 4
        for out in got[k]:
            assert all(same(a, b) for a, b in zip(out, want[k]))
