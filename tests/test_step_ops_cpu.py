"""The C ABI and the binding of the operators before and behind the LM head
(include/rlk/step_ops.h) without a GPU: exports, workspace sizes, and the
refusals that the host makes before anything touches a device."""
import ctypes
import os
import re

import pytest
import torch

import selected_token_lm_amd as rlk
from selected_token_lm_amd import step_ops as so

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL_ARG, BAD_SHAPE, BAD_ALIGN, _, WS_SMALL, HIP, DEVICE, BAD_ARG = range(9)
FAKE, ODD, OFF2, OFF8 = 0x100000, 0x100001, 0x100002, 0x100008  # never dereferenced
NAN, INF = float("nan"), float("inf")


def test_library_exports_the_header():
    text = open(os.path.join(ROOT, "include", "rlk", "step_ops.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(rlk_[a-z_0-9]+)\s*\(", text))
    assert names == set(so.SIGNATURES) and len(names) == 9
    L = ctypes.CDLL(rlk.library_path)
    assert all(hasattr(L, n) for n in names)
    assert set(dir(rlk)) >= {"layer_norm", "layer_norm_fwd", "layer_norm_bwd", "rms_norm", "rms_norm_fwd",
                             "rms_norm_bwd", "embed", "embed_fwd", "embed_bwd", "grad_norm", "clip_grads",
                             "step_workspace_bytes"}
    assert set(rlk.__all__) >= {"layer_norm", "rms_norm", "embed", "grad_norm", "clip_grads"}


def test_workspace_bytes():
    W = rlk.step_workspace_bytes
    norm, emb, grads = rlk.SOP_NORM_BWD, rlk.SOP_EMBED_BWD, rlk.SOP_GRADS
    for T, H in [(0, 1), (1, 1), (4096, 4096), (1 << 23, 65536)]:
        assert W(norm, T, H) > 0 and W(emb, T, H, 10) > 0
        # a part of the weight's and bias's gradients at the least
        assert W(norm, T, H) >= 8 * H
    for bad in [(-1, 8), ((1 << 23) + 1, 8), (4, 0), (4, 65537)]:
        assert W(norm, *bad) == 0 and W(emb, *bad, 10) == 0
    assert W(emb, 4, 8, 0) == 0 and W(emb, 4, 8, 8_000_001) == 0
    assert W(grads, 0) > 0 and W(grads, 1 << 20) > 0 and W(grads, -1) == 0 and W(grads, (1 << 20) + 1) == 0
    assert W(3, 4, 8, 10) == 0
    # sorted ids and rows, and parts of runs: two in 64 rows
    assert W(emb, 1000, 512, 10) >= 8 * 1000 + 2 * 16 * 512 * 4
    # the row limit with the widest rows stays below the memory's end
    assert W(emb, 1 << 23, 65536, 8_000_000) < 1 << 47


def ln_fwd(x=FAKE, xd=1, ldx=64, w=FAKE, b=FAKE, wd=1, T=8, H=64, eps=1e-5, y=FAKE, yd=1, mean=FAKE, rstd=FAKE):
    return rlk.lib().rlk_layer_norm_fwd(x, xd, ldx, w, b, wd, T, H, eps, y, yd, mean, rstd, None)


def rms_fwd(x=FAKE, xd=1, ldx=64, w=FAKE, wd=1, T=8, H=64, eps=1e-5, y=FAKE, yd=1, rstd=FAKE):
    return rlk.lib().rlk_rms_norm_fwd(x, xd, ldx, w, wd, T, H, eps, y, yd, rstd, None)


def ln_bwd(x=FAKE, xd=1, ldx=64, w=FAKE, wd=1, mean=FAKE, rstd=FAKE, g=FAKE, gd=1, ldg=64, T=8, H=64, gx=FAKE, gw=FAKE,
           gb=FAKE, dt=0, ws=FAKE, n=1 << 40):
    return rlk.lib().rlk_layer_norm_bwd(x, xd, ldx, w, wd, mean, rstd, g, gd, ldg, T, H, gx, gw, gb, dt, ws, n, None)


def rms_bwd(x=FAKE, xd=1, ldx=64, w=FAKE, wd=1, rstd=FAKE, g=FAKE, gd=1, ldg=64, T=8, H=64, gx=FAKE, gw=FAKE, dt=0,
            ws=FAKE, n=1 << 40):
    return rlk.lib().rlk_rms_norm_bwd(x, xd, ldx, w, wd, rstd, g, gd, ldg, T, H, gx, gw, dt, ws, n, None)


def refuses(f, status, **kw):
    assert f(**kw) == status, (f.__name__, kw)
    assert rlk.lib().rlk_last_error_message()


def test_norm_refusals():
    for f in (ln_fwd, rms_fwd):
        for a in ("x", "y"):
            refuses(f, NULL_ARG, **{a: None})
            refuses(f, BAD_ALIGN, **{a: ODD})
        refuses(f, BAD_ALIGN, w=ODD)
        refuses(f, BAD_ALIGN, rstd=OFF2)
        refuses(f, BAD_ALIGN, x=OFF2, xd=0)
        refuses(f, BAD_ALIGN, w=OFF2, wd=0)
        for eps in (-1e-9, NAN, INF):
            refuses(f, BAD_ARG, eps=eps)
        for a in ("xd", "yd", "wd"):
            refuses(f, BAD_ARG, **{a: 2})
        assert f(T=0, x=None, y=None) == OK and rlk.lib().rlk_last_error_message() == b""
    refuses(ln_fwd, BAD_ALIGN, b=ODD)
    refuses(ln_fwd, BAD_ALIGN, mean=OFF2)
    for f in (ln_bwd, rms_bwd):
        for a in ("x", "g", "rstd", "ws"):
            refuses(f, NULL_ARG, **{a: None})
        for a in ("x", "g", "w", "gx"):
            refuses(f, BAD_ALIGN, **{a: ODD})
        refuses(f, BAD_ALIGN, gw=OFF2)
        refuses(f, BAD_ALIGN, gw=ODD, dt=1)
        refuses(f, BAD_ALIGN, ws=OFF8)
        refuses(f, WS_SMALL, n=rlk.step_workspace_bytes(rlk.SOP_NORM_BWD, 8, 64) - 1)
        for a in ("xd", "gd", "wd", "dt"):
            refuses(f, BAD_ARG, **{a: -1})
        none = {"gw": None, **({"gb": None} if f is ln_bwd else {})}
        assert f(gx=None, ws=None, **none) == OK              # nothing wanted
        assert f(T=0, x=None, g=None, rstd=None, ws=None, **none) == OK
        refuses(f, NULL_ARG, T=0, ws=None)                     # zero sums are written
    refuses(ln_bwd, NULL_ARG, mean=None)
    refuses(ln_bwd, BAD_ALIGN, gb=OFF2)
    for f in (ln_fwd, rms_fwd, ln_bwd, rms_bwd):
        for bad in (dict(T=-1), dict(T=(1 << 23) + 1), dict(H=0), dict(H=65537), dict(ldx=-1), dict(ldx=1 << 41)):
            refuses(f, BAD_SHAPE, **bad)
    for f in (ln_bwd, rms_bwd):
        refuses(f, BAD_SHAPE, ldg=-1)


def emb_fwd(ids=FAKE, idb=8, E=FAKE, ed=1, T=8, H=64, V=100, ignore=-100, scale=1.0, out=FAKE, od=1):
    return rlk.lib().rlk_embed_fwd(ids, idb, E, ed, T, H, V, ignore, scale, out, od, None)


def emb_bwd(ids=FAKE, idb=8, g=FAKE, gd=1, ldg=64, T=8, H=64, V=100, ignore=-100, scale=1.0, gE=FAKE, dt=0, add=0,
            ws=FAKE, n=1 << 40):
    return rlk.lib().rlk_embed_bwd(ids, idb, g, gd, ldg, T, H, V, ignore, scale, gE, dt, add, ws, n, None)


def test_embed_refusals():
    for a in ("ids", "E", "out"):
        refuses(emb_fwd, NULL_ARG, **{a: None})
        refuses(emb_fwd, BAD_ALIGN, **{a: ODD})
    for a in ("ids", "g", "gE", "ws"):
        refuses(emb_bwd, NULL_ARG, **{a: None})
        refuses(emb_bwd, BAD_ALIGN, **{a: ODD})
    refuses(emb_bwd, BAD_ALIGN, ws=OFF8)
    refuses(emb_bwd, BAD_ALIGN, gE=OFF2)
    for f in (emb_fwd, emb_bwd):
        refuses(f, BAD_ALIGN, ids=0x100004)
        refuses(f, BAD_ALIGN, ids=OFF2, idb=4)
        refuses(f, BAD_ARG, idb=2)
        for scale in (NAN, INF, -INF):
            refuses(f, BAD_ARG, scale=scale)
        for bad in (dict(T=-1), dict(T=(1 << 23) + 1), dict(H=0), dict(H=65537), dict(V=0), dict(V=8_000_001)):
            refuses(f, BAD_SHAPE, **bad)
    refuses(emb_fwd, BAD_ARG, ed=2)
    refuses(emb_fwd, BAD_ARG, od=-1)
    for kw in (dict(gd=2), dict(dt=2), dict(add=2), dict(add=-1)):
        refuses(emb_bwd, BAD_ARG, **kw)
    refuses(emb_bwd, BAD_SHAPE, ldg=-1)
    refuses(emb_bwd, WS_SMALL, n=rlk.step_workspace_bytes(rlk.SOP_EMBED_BWD, 8, 64, 100) - 1)
    assert emb_fwd(T=0, ids=None, E=None, out=None) == OK
    assert emb_bwd(T=0, ids=None, g=None, ws=None, add=1) == OK
    refuses(emb_bwd, NULL_ARG, T=0, gE=None)


def lists(n, ptr=FAKE, size=4, code=0):
    step = 1 << 16
    return ((ctypes.c_void_p * n)(*(None if ptr is None else ptr + i * step for i in range(n))),
            (ctypes.c_int64 * n)(*([size] * n)), (ctypes.c_int32 * n)(*([code] * n)))


def norm_call(p, s, c, n, norm=FAKE, ws=FAKE, size=1 << 30):
    return rlk.lib().rlk_grad_norm(p, s, c, n, norm, ws, size, None)


def clip_call(p, s, c, n, most=1.0, out=None, oc=None, norm=FAKE, ws=FAKE, size=1 << 30):
    return rlk.lib().rlk_clip_grads(p, s, c, n, most, out, oc, norm, ws, size, None)


def test_gradient_list_refusals():
    p, s, c = lists(3)
    for f, more in ((norm_call, {}), (clip_call, dict(out=p, oc=c))):
        for kw in (dict(norm=None), dict(ws=None)):
            assert f(p, s, c, 3, **{**more, **kw}) == NULL_ARG
        assert f(p, s, c, 3, **{**more, "norm": OFF2}) == BAD_ALIGN
        assert f(p, s, c, 3, **{**more, "ws": OFF8}) == BAD_ALIGN
        assert f(p, s, c, 3, **{**more, "size": rlk.step_workspace_bytes(rlk.SOP_GRADS, 3) - 1}) == WS_SMALL
        assert f(None, s, c, 3, **more) == f(p, None, c, 3, **more) == f(p, s, None, 3, **more) == NULL_ARG
        assert f(p, s, c, -1, **more) == f(p, s, c, (1 << 20) + 1, **more) == BAD_SHAPE
        assert f(lists(3, None)[0], s, c, 3, **more) == NULL_ARG
        assert f(lists(3, OFF2)[0], s, c, 3, **more) == BAD_ALIGN
        assert f(p, lists(3, size=-1)[1], c, 3, **more) == BAD_SHAPE
        assert f(p, lists(3, size=(1 << 36) + 1)[1], c, 3, **more) == BAD_SHAPE
        assert f(p, s, lists(3, code=2)[2], 3, **more) == BAD_ARG
    for most in (-1e-9, NAN, -INF):
        assert clip_call(p, s, c, 3, most, p, c) == BAD_ARG
    assert clip_call(p, s, c, 3, 1.0, None, c) == clip_call(p, s, c, 3, 1.0, p, None) == NULL_ARG
    assert clip_call(p, s, c, 3, 1.0, lists(3, None)[0], c) == NULL_ARG
    assert clip_call(p, s, c, 3, 1.0, lists(3, OFF2)[0], c) == BAD_ALIGN
    assert clip_call(p, s, c, 3, 1.0, p, lists(3, code=7)[2]) == BAD_ARG


def test_overlapping_outputs_are_refused():
    """Outputs against outputs and against gradients that are not their own."""
    n = 2

    def call(g, o, size=16, gc=0, oc=0):
        arr = lambda v: (ctypes.c_void_p * n)(*v)  # noqa: E731
        s, a, b = (ctypes.c_int64 * n)(size, size), (ctypes.c_int32 * n)(gc, gc), (ctypes.c_int32 * n)(oc, oc)
        return clip_call(arr(g), s, a, n, 1.0, arr(o), b)

    A, B, C, D = (FAKE + 64 * i for i in range(4))
    ok = (HIP, DEVICE)  # past the checks of the arguments: no GPU here
    if torch.cuda.is_available():
        pytest.skip("the calls that pass would run on the fake addresses")
    assert call((A, B), (A, B)) in ok and call((A, B), (C, D)) in ok and call((A, A), (C, D)) in ok
    assert call((A, B), (A, C)) in ok and call((A, B), (C, B)) in ok
    for g, o in (((A, A), (A, A)), ((A, B), (B, A)), ((A, B), (B, C)), ((A, B), (C, C)), ((A, B), (C, C + 60)),
                 ((A, B), (A + 4, C)), ((A, B), (B + 60, D)), ((A, B), (C + 60, C))):
        assert call(g, o) == BAD_ARG, (g, o)
    # the same address as another type is not its own
    assert call((A, C), (A, C), oc=1) == BAD_ARG
    assert call((A, B), (A, A), size=0) in ok


T, H, V = 6, 32, 50


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_binding_refuses_shapes_and_types():
    for f in (rlk.layer_norm, rlk.rms_norm):
        with pytest.raises(ValueError, match=r"x must be \[T, H\]"):
            f(bf(2, 3, 4), bf(4))
        with pytest.raises(TypeError, match="x must be float32 or bfloat16"):
            f(bf(T, H).half(), bf(H))
        with pytest.raises(ValueError, match="1 to 65536"):
            f(bf(T, 0), bf(0))
        with pytest.raises(ValueError, match="x must be on a GPU"):
            f(bf(T, H), bf(H))
        for eps in (-1.0, NAN, INF):
            with pytest.raises(ValueError, match="eps"):
                f(bf(T, H), bf(H), eps=eps)
    with pytest.raises(ValueError, match=r"weight must be \[H\]"):
        so._vectors(H, torch.device("cpu"), weight=bf(H + 1))
    with pytest.raises(TypeError, match="one dtype"):
        so._vectors(H, torch.device("cpu"), weight=bf(H), bias=bf(H).float())
    with pytest.raises(ValueError, match="weight must be on"):
        so._vectors(H, torch.device("cpu"), weight=bf(H))
    with pytest.raises(ValueError, match="g must be"):
        so._matrix("g", bf(T, H + 1), (T, H), torch.device("cpu"))
    with pytest.raises(TypeError, match="out_dtype"):
        so._dtype("out_dtype", torch.float16)


def test_binding_refuses_embeddings():
    i64 = torch.zeros(T, dtype=torch.int64)
    with pytest.raises(ValueError, match=r"E must be \[V, H\]"):
        rlk.embed(i64, bf(V))
    with pytest.raises(TypeError, match="E must be"):
        rlk.embed(i64, bf(V, H).double())
    with pytest.raises(ValueError, match="E must be a device tensor"):
        rlk.embed(i64, bf(V, H))
    with pytest.raises(ValueError, match="g must be on a GPU"):
        rlk.embed_bwd(i64, bf(T, H), V)
    with pytest.raises(ValueError, match=r"ids must be \[T\]"):
        so._ids(i64.view(2, 3), torch.device("cpu"))
    with pytest.raises(TypeError, match="int32 or int64"):
        so._ids(i64.float(), torch.device("cpu"))
    with pytest.raises(ValueError, match="ids must be on"):
        so._ids(i64, torch.device("cpu"))
    for scale in (NAN, INF, -INF, 1e39):
        with pytest.raises(ValueError, match="scale"):
            so._scale(scale)
    for i in (2 ** 63, -2 ** 63 - 1):
        with pytest.raises(ValueError, match="int64"):
            so._ignore(i)


def test_binding_refuses_gradient_lists():
    for f in (rlk.grad_norm, lambda g: rlk.clip_grads(g, 1.0)):
        with pytest.raises(ValueError, match="empty"):
            f([])
        with pytest.raises(TypeError, match=r"grads\[0\]"):
            f([bf(3).half(), bf(3)])
        with pytest.raises(ValueError, match="one GPU"):
            f([bf(3)])
    for most in (-1.0, NAN, -INF):
        with pytest.raises(ValueError, match="max_norm"):
            rlk.clip_grads([bf(3)], most)


def stand_ins(monkeypatch):
    """The kernels' forwards on the CPU, without a graph, as the kernels have none."""
    def norm(center, x, weight, bias, eps, out_dtype, stats):
        rows = x.detach()[:, 0].clone()
        return x.detach().clone(), rows if center else None, rows

    monkeypatch.setattr(so, "_norm_fwd", norm)
    monkeypatch.setattr(so, "embed_fwd", lambda ids, E, *rest: E.detach()[ids])


@pytest.mark.parametrize("grad", [True, False])
def test_a_tangent_is_refused_not_dropped(monkeypatch, grad):
    """Forward-mode derivatives are not implemented: an input with a tangent
    raises, with and without no_grad; other inputs inside a dual level do not."""
    from torch.autograd import forward_ad as fw
    stand_ins(monkeypatch)
    x, v, E, ids = torch.randn(T, H), torch.randn(H), torch.randn(V, H), torch.arange(T)
    with fw.dual_level(), torch.set_grad_enabled(grad):
        dual = lambda t: fw.make_dual(t, torch.ones_like(t))  # noqa: E731
        for call in (lambda: rlk.rms_norm(dual(x)), lambda: rlk.rms_norm(x, dual(v)), lambda: rlk.layer_norm(dual(x), v, v),
                     lambda: rlk.layer_norm(x, dual(v), v), lambda: rlk.layer_norm(x, v, dual(v)),
                     lambda: rlk.embed(ids, dual(E))):
            with pytest.raises(NotImplementedError, match="jvp"):
                call()
        assert torch.equal(rlk.rms_norm(x, v), x) and torch.equal(rlk.layer_norm(x, v, v), x)
        assert torch.equal(rlk.embed(ids, E), E[ids])
    assert rlk.rms_norm(x.requires_grad_(), v).requires_grad == torch.is_grad_enabled()


def test_tangents_of_gradients_are_refused(monkeypatch):
    """A norm or a changed gradient would lack them."""
    from torch.autograd import forward_ad as fw
    monkeypatch.setattr(so, "_tensors", lambda what, ts: (ts[0].device, None, None, True))
    with fw.dual_level():
        t = torch.ones(3)
        d = fw.make_dual(torch.ones(3), t)
        for call in (lambda: rlk.grad_norm([t, d]), lambda: rlk.clip_grads([t, d], 1.0),
                     lambda: rlk.clip_grads([t, t], 1.0, out=[torch.ones(3), d])):
            with pytest.raises(ValueError, match="must carry no forward-mode tangent"):
                call()
        monkeypatch.setattr(so, "_matrix", lambda name, g: (g, 0, g.stride(0)))
        monkeypatch.setattr(so, "_ids", lambda ids, device: (ids, 8))
        monkeypatch.setattr(so, "_table", lambda name, E: 0)
        E = fw.make_dual(torch.zeros(V, H), torch.ones(V, H))
        with pytest.raises(ValueError, match="grad_E must carry no forward-mode tangent"):
            rlk.embed_bwd(torch.arange(T), torch.ones(T, H), V, grad_E=E)


def test_missing_gradients_are_named():
    """A frozen parameter's None, first or later, and what is no tensor."""
    t = torch.ones(3)
    for f in (rlk.grad_norm, lambda g: rlk.clip_grads(g, 1.0), lambda g: rlk.clip_grads([t] * len(g), 1.0, out=g)):
        for i in (0, 1):
            grads = [t, t]
            grads[i] = None
            with pytest.raises(TypeError, match=rf"(grads|out)\[{i}\] is None: leave out parameters without a gradient"):
                f(grads)
        with pytest.raises(TypeError, match=r"\[1\] must be a tensor, got <class 'float'>"):
            f([t, 3.5])


@pytest.mark.parametrize("T,H,V", [(17, 512, 10), (1000, 512, 10), (16384, 2048, 151936), (16385, 1, 3), (100_000, 33, 600),
                                   (1 << 23, 65536, 8_000_000)])
def test_workspace_holds_every_part(T, H, V):
    """The embedding's gradient: a key and a row a token (twice where a radix sort
    has more than one digit of nine bits), two sums of H for every run of 16 rows.
    The norms': two rows of sums a block."""
    digits = 1 if T <= 16384 else -(-V.bit_length() // 9)
    need = 8 * T * min(2, digits) + 2 * -(-T // 16) * H * 4
    assert need <= rlk.step_workspace_bytes(rlk.SOP_EMBED_BWD, T, H, V) <= need + 4 * 512 * (T // 4096 + 2) + 8 * 256
    group = 16 if H <= 128 else 8 if H <= 256 else 4 if H <= 1024 else 1
    blocks = min(64 if H > 8192 else 256, -(-T // group))
    assert rlk.step_workspace_bytes(rlk.SOP_NORM_BWD, T, H) >= 2 * 4 * blocks * H
