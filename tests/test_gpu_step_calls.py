"""The operators before and behind the LM head as a program calls them: through
autograd, in a training step with tied weights around linear_logp, captured
into a graph, on other streams, from two host threads."""
import threading

import numpy as np
import pytest
import torch

import oracle
import selected_token_lm_amd as rlk
import synth
from oracle import step_ops as O
from tests.gpu_util import DEV, GRAD_RTOL, LOGP_TOL, bf16_dev, f32_dev, i32_dev, rel_l2, to64
from tests.step_util import dev, np64, rng, same

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("center", [False, True], ids=["rms", "layer"])
@pytest.mark.parametrize("x_dtype,w_dtype", [(BF16, BF16), (F32, BF16), (BF16, F32)])
def test_norms_through_autograd(center, x_dtype, w_dtype):
    """The bits of the direct calls, gradients of the inputs' types, whatever is
    asked for; a broadcast upstream gradient."""
    T, H = 70, 200
    r = rng(1, T)
    x, w, b = dev(r.normal(size=(T, H)), x_dtype)[0], dev(r.normal(size=H), w_dtype)[0], dev(r.normal(size=H), w_dtype)[0]
    g = dev(r.normal(size=(T, H)), BF16)[0]
    if center:
        y0, mean, rstd = rlk.layer_norm_fwd(x, w, b, 1e-5, out_dtype=BF16)
        want = rlk.layer_norm_bwd(x, w, mean, rstd, g, grad_weight_dtype=w_dtype)
        leaves = [x, w, b]
        f = lambda x, w, b: rlk.layer_norm(x, w, b, 1e-5, out_dtype=BF16)  # noqa: E731
    else:
        y0, rstd = rlk.rms_norm_fwd(x, w, 1e-5, out_dtype=BF16)
        want = rlk.rms_norm_bwd(x, w, rstd, g, grad_weight_dtype=w_dtype)
        leaves = [x, w]
        f = lambda x, w: rlk.rms_norm(x, w, 1e-5, out_dtype=BF16)  # noqa: E731
    n = len(leaves)
    for ask in range(1, 2 ** n):
        args = [t.detach().clone().requires_grad_(bool(ask >> i & 1)) for i, t in enumerate(leaves)]
        y = f(*args)
        assert same(y.detach(), y0)
        y.backward(g, retain_graph=True)
        for i, t in enumerate(args):
            assert (t.grad is not None) == bool(ask >> i & 1)
            assert t.grad is None or same(t.grad, want[i])
        y.backward(g)  # a graph walked twice
        live = [t for t in args if t.requires_grad]
        assert all(torch.equal(t.grad, 2 * want[i]) for i, t in enumerate(args) if t.requires_grad)
        # an upstream gradient without memory of its own
        y = f(*args)
        got = torch.autograd.grad(y.sum(), live)
        ones = torch.ones_like(g)
        assert all(same(a, c) for a, c in zip(got, torch.autograd.grad(f(*args), live, ones)))
    with pytest.raises(RuntimeError, match="once_differentiable|differentiate twice"):
        (gx,) = torch.autograd.grad(f(*args).float().pow(2).sum(), [args[0]], create_graph=True)
        gx.sum().backward()
    with torch.no_grad():
        assert same(f(*args), y0) and not f(*args).requires_grad
    # no weight, no bias
    x1 = x.clone().requires_grad_()
    (rlk.layer_norm if center else rlk.rms_norm)(x1).sum().backward()
    assert x1.grad.dtype == x_dtype


def test_norms_gradients_against_differences():
    """The kernels' own forward differenced along random directions, in fp32."""
    T, H, eps = 5, 96, 1e-3
    r = rng(2)
    for center in (False, True):
        x, w, b, g, dx, dw, db = (dev(r.normal(size=s))[0] for s in ((T, H), (H,), (H,), (T, H), (T, H), (H,), (H,)))
        f = lambda s: ((rlk.layer_norm(x + s * dx, w + s * dw, b + s * db, eps) if center  # noqa: E731
                        else rlk.rms_norm(x + s * dx, w + s * dw, eps)).double() * g.double()).sum()
        if center:
            _, m, rs = rlk.layer_norm_fwd(x, w, b, eps)
            gx, gw, gb = rlk.layer_norm_bwd(x, w, m, rs, g)
        else:
            gx, gw = rlk.rms_norm_bwd(x, w, rlk.rms_norm_fwd(x, w, eps)[1], g)
            gb = torch.zeros_like(b)
        want = (gx.double() * dx).sum() + (gw.double() * dw).sum() + (gb.double() * db).sum()
        s = 2.0 ** -7
        # central differences of two widths: their error falls with the square of the width
        d1, d2 = (f(s) - f(-s)) / (2 * s), (f(s / 2) - f(-s / 2)) / s
        size = (gx.double() * dx).abs().sum() + (gw.double() * dw).abs().sum()
        assert (d2 - want).abs() <= (d1 - d2).abs() + 1e-4 * size, (center, d1, d2, want)


def test_embed_through_autograd():
    V, H, T = 300, 120, 500
    r = rng(3)
    E = dev(r.normal(size=(V, H)), BF16)[0].requires_grad_()
    ids = torch.from_numpy(r.integers(0, V, T)).to(DEV)
    ids[::7] = -100
    out = rlk.embed(ids, E, 3.0)
    assert same(out.detach(), rlk.embed_fwd(ids, E.detach(), 3.0))
    g = dev(r.normal(size=(T, H)), BF16)[0]
    out.backward(g)
    assert same(E.grad, rlk.embed_bwd(ids, g, V, 3.0, grad_E_dtype=BF16))
    out = rlk.embed(ids.int(), E, 3.0, out_dtype=F32)
    (grad,) = torch.autograd.grad(out.sum(), [E])
    n = torch.bincount(ids[ids >= 0], minlength=V).float()[:, None].expand(V, H)
    assert torch.equal(grad, (3 * n).to(BF16))
    with torch.no_grad():
        assert not rlk.embed(ids, E).requires_grad


def test_in_place_results_are_seen_by_autograd():
    """A tensor that a graph has saved cannot be changed behind its back."""
    t = torch.ones(10, device=DEV, requires_grad=True)
    m = torch.full((10,), 2.0, device=DEV)
    y = (t * m).sum()
    rlk.clip_grads([m], 1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    m = torch.zeros((4, 10), device=DEV)
    y = (t * m).sum()
    rlk.embed_bwd(torch.tensor([1], device=DEV), torch.ones((1, 10), device=DEV), 4, grad_E=m)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with pytest.raises(ValueError, match="p.grad"):
        rlk.clip_grads([t], 1.0)
    with pytest.raises(ValueError, match="E.grad"):
        rlk.embed_bwd(torch.tensor([1], device=DEV), torch.ones((1, 10), device=DEV), 1, grad_E=t.view(1, 10))
    with torch.inference_mode():
        n, out = rlk.clip_grads([torch.ones(16, device=DEV)], 2.0)
        assert n == 4 and (out[0] == 0.5).all()


# --- a training step with tied weights ------------------------------------------
class Step:
    """embed -> rms_norm -> linear_logp with the same table, its gradient: the
    head's part in fp32, the embedding's added to it, everything clipped."""

    def __init__(self, T=300, H=256, V=5000, seed=0):
        self.inp = synth.make_inputs(T, H, V, 0.15, name=f"step{seed}")
        r = rng(4, seed)
        self.ids_n = r.integers(0, V, T)
        self.ids_n[::11] = self.ids_n[0]
        self.E, self.y, self.g = bf16_dev(self.inp.W), i32_dev(self.inp.y), f32_dev(self.inp.g)
        self.ids = torch.from_numpy(self.ids_n).to(DEV)
        self.w, self.w_n = dev(1 + 0.1 * r.normal(size=H), BF16)
        self.scale = float(np.sqrt(H))
        self.V = V

    def run(self, most=0.5):
        x = rlk.embed_fwd(self.ids, self.E, self.scale)
        h, rstd = rlk.rms_norm_fwd(x, self.w)
        logp, lse = rlk.linear_logp_fwd(h, self.E, self.y)
        grad_h, grad_E = rlk.linear_logp_bwd(h, self.E, self.y, lse, self.g)
        grad_x, grad_w = rlk.rms_norm_bwd(x, self.w, rstd, grad_h)
        rlk.embed_bwd(self.ids, grad_x, self.V, self.scale, grad_E=grad_E)
        raw = [grad_E.clone(), grad_w.clone()]
        norm, (grad_E, grad_w) = rlk.clip_grads([grad_E, grad_w], most)
        return [logp, *raw, norm, grad_E, grad_w]

    def want(self):
        bits = lambda t: t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
        x = rlk.embed_fwd(self.ids, self.E, self.scale)
        h, _ = rlk.rms_norm_fwd(x, self.w)
        logp, _ = oracle.forward(bits(h), self.inp.W, self.inp.y)
        gh, gW = oracle.backward(bits(h), self.inp.W, self.inp.y, self.inp.g)
        gx, gw, _ = O.norm_backward(np64(x), self.w_n, gh, 1e-6, False)
        return logp, gW + O.embed_backward(self.ids_n, gx, self.V, self.scale), gw


def test_a_training_step_with_tied_weights():
    s = Step()
    logp, grad_E, grad_w, norm, c_E, c_w = s.run()
    w_logp, w_E, w_w = s.want()
    assert np.abs(np64(logp) - w_logp).max() <= LOGP_TOL
    assert rel_l2(to64(grad_E), w_E) <= GRAD_RTOL and rel_l2(to64(grad_w), w_w) <= GRAD_RTOL
    n = O.grad_norm([np64(grad_E), np64(grad_w)])
    assert abs(float(norm) - n) <= 2.0 ** -23 * n and n > 0.5
    assert rel_l2(to64(c_E), np64(grad_E) * 0.5 / n) < 1e-6 and rel_l2(to64(c_w), np64(grad_w) * 0.5 / n) < 1e-6
    assert all(same(a, b) for a, b in zip(s.run(), [logp, grad_E, grad_w, norm, c_E, c_w]))


def test_the_step_through_autograd():
    """The same step as a module would run it: the tied table's two gradients
    are summed by autograd, in the table's type."""
    s = Step()
    E, w = s.E.clone().requires_grad_(), s.w.clone().requires_grad_()
    h = rlk.rms_norm(rlk.embed(s.ids, E, s.scale), w)
    logp = rlk.linear_logp(h, E, s.y)
    (s.g * logp).sum().backward()
    _, w_E, w_w = s.want()
    assert E.grad.dtype == w.grad.dtype == BF16
    assert rel_l2(to64(E.grad), w_E) <= GRAD_RTOL and rel_l2(to64(w.grad), w_w) <= GRAD_RTOL
    before = [E.grad.clone(), w.grad.clone()]
    norm, _ = rlk.clip_grads([p.grad for p in (E, w)], 0.5)
    n = O.grad_norm([np64(t) for t in before])
    assert abs(float(norm) - n) <= 2.0 ** -23 * n
    assert rel_l2(to64(E.grad), np64(before[0]) * 0.5 / n) < 2.0 ** -8


def test_the_step_captured():
    """Replayed between eager steps, and on new values in the same tensors."""
    a, b = Step(seed=1), Step(seed=2)
    want = [a.run(), b.run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = a.run()
    for rep in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(p, q) for p, q in zip(out, want[0])), rep
        assert all(same(p, q) for p, q in zip(b.run(), want[1]))
    for name in ("E", "y", "g", "ids", "w"):
        getattr(a, name).copy_(getattr(b, name))
    assert not same(want[0][0], want[1][0])
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(p, q) for p, q in zip(out, want[1]))


def everything(T, H, V, seed):
    """Inputs and a call of every operator (T past one rank sort for some)."""
    r = rng(5, seed)
    x, w, g = dev(r.normal(size=(T, H)), BF16)[0], dev(r.normal(size=H), BF16)[0], dev(r.normal(size=(T, H)), BF16)[0]
    E = dev(r.normal(size=(V, H)), BF16)[0]
    ids = torch.from_numpy(np.minimum(r.integers(0, 4 * V, T), V - 1)).to(DEV)

    def call():
        y, mean, rstd = rlk.layer_norm_fwd(x, w, w)
        z, rs = rlk.rms_norm_fwd(x, w)
        e = rlk.embed_fwd(ids, E, 2.0)
        grads = [*rlk.layer_norm_bwd(x, w, mean, rstd, g), *rlk.rms_norm_bwd(x, w, rs, g),
                 rlk.embed_bwd(ids, g, V), rlk.embed_bwd(ids, g, V, grad_E=E.float())]
        norm, clipped = rlk.clip_grads([t.clone() for t in grads], 0.1)
        return [y, mean, rstd, z, rs, e, *grads, norm, *clipped]

    return call


@pytest.mark.parametrize("T,H,V", [(0, 40, 7), (1, 33, 5), (100, 200, 3), (17000, 24, 600)])
def test_captured(T, H, V):
    call = everything(T, H, V, T)
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(p, q) for p, q in zip(out, want))
        assert all(same(p, q) for p, q in zip(call(), want))


def test_two_graphs_share_one_workspace():
    """Each call is whole before the next begins, so graphs replayed one after
    the other may hold the same workspace."""
    sizes = [(300, 100, 40), (900, 512, 7)]
    data = []
    for T, H, V in sizes:
        r = rng(6, T)
        x, g = dev(r.normal(size=(T, H)), BF16)[0], dev(r.normal(size=(T, H)), BF16)[0]
        data.append((x, g, torch.from_numpy(r.integers(0, V, T)).to(DEV), V))
    n = max(max(rlk.step_workspace_bytes(rlk.SOP_NORM_BWD, T, H), rlk.step_workspace_bytes(rlk.SOP_EMBED_BWD, T, H, V))
            for T, H, V in sizes)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)

    def call(x, g, ids, V):
        _, mean, rstd = rlk.layer_norm_fwd(x)
        grads = [*rlk.layer_norm_bwd(x, None, mean, rstd, g, ws=ws), rlk.embed_bwd(ids, g, V, ws=ws)]
        return [*grads, rlk.grad_norm(grads, ws=ws)]

    want = [call(*d) for d in data]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for d in data:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call(*d))
        graphs.append(graph)
    for _ in range(3):
        for k in (0, 1):
            graphs[k].replay()
            torch.cuda.synchronize()
            ws.fill_(255)  # nothing of it is kept for the next call
            assert all(same(p, q) for p, q in zip(outs[k], want[k]))
    with pytest.raises(rlk.RlkError, match="need"):
        rlk.embed_bwd(data[0][2], data[0][1], 40, ws=ws[:64])
    with pytest.raises(ValueError, match="ws must be"):
        rlk.grad_norm([ws.float()], ws=ws[::2])


def test_two_host_threads_and_streams():
    calls = [everything(800, 320, 50, 1), everything(17500, 64, 90, 2)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    got, streams = [[], []], [torch.cuda.Stream(), torch.cuda.Stream()]

    def work(k):
        with torch.cuda.stream(streams[k]):
            for _ in range(4):
                got[k].append(calls[k]())
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


@pytest.mark.parametrize("T,H,V", [(5, 40, 7), (17, 100, 1), (1000, 512, 10), (4096, 2050, 30), (16384, 64, 9), (17000, 24, 600)])
def test_the_workspace_asked_for_is_enough(T, H, V):
    """Nothing behind it is written, and its contents before do not matter."""
    r = rng(7, T)
    x, g = dev(r.normal(size=(T, H)), BF16)[0], dev(r.normal(size=(T, H)), BF16)[0]
    ids = torch.from_numpy(r.integers(0, V, T)).to(DEV)
    _, mean, rstd = rlk.layer_norm_fwd(x)
    calls = [(rlk.SOP_NORM_BWD, T, H, 0, lambda ws: rlk.layer_norm_bwd(x, None, mean, rstd, g, ws=ws)),
             (rlk.SOP_EMBED_BWD, T, H, V, lambda ws: [rlk.embed_bwd(ids, g, V, ws=ws)]),
             (rlk.SOP_EMBED_BWD, T, H, V, lambda ws: [rlk.embed_bwd(ids, g, V, grad_E=torch.ones((V, H), device=DEV), ws=ws)]),
             (rlk.SOP_GRADS, 200, 0, 0, lambda ws: [rlk.grad_norm([x] * 200, ws=ws)]),
             (rlk.SOP_GRADS, 2, 0, 0, lambda ws: [rlk.clip_grads([x.clone(), g.clone()], 0.5, ws=ws)[0]])]
    for op, *sizes, call in calls:
        n = rlk.step_workspace_bytes(op, *sizes)
        want = call(None)
        for fill in (0, 255):
            buf = torch.full((n + 4096,), fill, dtype=torch.uint8, device=DEV)
            got = call(buf[:n])
            assert all(same(a, b) for a, b in zip(got, want)) and (buf[n:] == fill).all(), (op, sizes, fill)
