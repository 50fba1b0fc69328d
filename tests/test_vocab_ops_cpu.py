"""The C ABI and the binding of the operators on the whole distribution
(include/rlk/vocab_ops.h) without a GPU: exports, workspace sizes, and the
refusals that the host makes before anything touches a device."""
import ctypes
import os
import re

import pytest
import torch

import selected_token_lm_amd as rlk
from selected_token_lm_amd import vocab_ops as vo

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL_ARG, BAD_SHAPE, BAD_ALIGN, _, WS_SMALL, HIP, DEVICE, BAD_ARG = range(9)
FAKE, OFF8, OFF2 = 0x100000, 0x100008, 0x100002  # never dereferenced


def test_library_exports_the_header():
    text = open(os.path.join(ROOT, "include", "rlk", "vocab_ops.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(rlk_[a-z_0-9]+)\s*\(", text))
    assert names == set(vo.SIGNATURES) and len(names) == 5
    L = ctypes.CDLL(rlk.library_path)
    assert all(hasattr(L, n) for n in names)
    assert set(dir(rlk)) >= {"linear_logp_top", "linear_logp_top_fwd", "linear_logp_top_bwd", "linear_distill",
                             "linear_distill_fwd", "linear_distill_bwd", "vocab_workspace_bytes"}


def test_workspace_bytes(monkeypatch):
    W = rlk.vocab_workspace_bytes
    for op in range(4):
        assert W(op, 0, 64, 10, 1) > 0
        for bad in [(-1, 64, 10, 1), (4, 63, 10, 1), (4, 64, 0, 1), (4, 64, 8_000_001, 1), (4, 64, 10, 129),
                    (4, 64, 10, -1), ((1 << 23) + 1, 64, 10, 1)]:
            assert W(op, *bad) == 0, (op, bad)
    assert W(4, 4, 64, 10, 1) == 0
    assert W(rlk.VOP_TOP_FWD, 4, 64, 10, 0) > 0 and W(rlk.VOP_DISTILL_FWD, 4, 64, 10, 0) == 0
    # no logits are kept when no alternative is asked for
    assert W(rlk.VOP_TOP_FWD, 4096, 4096, 151936, 0) < W(rlk.VOP_TOP_FWD, 4096, 4096, 151936, 1) - (2 << 30)
    # the forward's logits stay within the budget: a quarter of the splits in 1 GiB
    per_split = 4 * 4096 * 38 * 128
    full = W(rlk.VOP_TOP_FWD, 4096, 4096, 151936, 8)
    monkeypatch.setenv("RLK_DZ_BUDGET_MB", "1024")
    part = W(rlk.VOP_TOP_FWD, 4096, 4096, 151936, 8)
    assert full - part == (32 - 8) * per_split - 8 * 4096 * 8  # ... and the running bests
    monkeypatch.setenv("RLK_DZ_BUDGET_MB", "1")
    assert W(rlk.VOP_TOP_FWD, 4096, 4096, 151936, 8) == part - 7 * per_split


def top_fwd(h=FAKE, W=FAKE, y=FAKE, T=64, H=256, V=4096, K=8, logp=FAKE, lse=FAKE, ent=FAKE, tl=FAKE, ti=FAKE,
            ws=FAKE, n=1 << 40):
    return rlk.lib().rlk_linear_logp_top_fwd(h, W, y, T, H, V, -100, K, logp, lse, ent, tl, ti, ws, n, None)


def test_top_forward_refusals():
    for a in ("h", "W", "y", "logp", "ent", "tl", "ti", "ws"):
        assert top_fwd(**{a: None}) == NULL_ARG, a
    for a in ("h", "W", "ws"):
        assert top_fwd(**{a: OFF8}) == BAD_ALIGN, a
    for a in ("y", "logp", "lse", "ent", "tl", "ti"):
        assert top_fwd(**{a: OFF2}) == BAD_ALIGN, a
    for bad in (dict(T=-1), dict(H=96), dict(V=0), dict(V=9_000_000), dict(K=129), dict(K=-1), dict(T=(1 << 23) + 1)):
        assert top_fwd(**bad) == BAD_SHAPE, bad
    need = rlk.vocab_workspace_bytes(rlk.VOP_TOP_FWD, 64, 256, 4096, 8)
    assert top_fwd(n=need - 1) == WS_SMALL
    assert b"need" in rlk.lib().rlk_last_error_message()
    assert top_fwd(T=0, h=None, y=None, logp=None, ent=None, ws=None, n=0) == OK
    assert rlk.lib().rlk_last_error_message() == b""
    # more tiles than a launch holds: 32768 row tiles x 32 x 977 column tiles
    assert top_fwd(T=1 << 23, H=64, V=8_000_000, K=0) == WS_SMALL
    assert top_fwd(T=1 << 23, H=64, V=8_000_000, K=0, n=1 << 60) in (BAD_SHAPE, HIP, DEVICE)


def top_bwd(h=FAKE, W=FAKE, y=FAKE, lse=FAKE, ent=FAKE, g=FAKE, ge=FAKE, T=64, H=256, V=4096, gh=FAKE, gW=FAKE, dt=0,
            ws=FAKE, n=1 << 40):
    return rlk.lib().rlk_linear_logp_top_bwd(h, W, y, lse, ent, g, ge, T, H, V, -100, gh, gW, dt, ws, n, None)


def test_top_backward_refusals():
    for a in ("h", "W", "y", "lse", "ent", "ws"):
        assert top_bwd(**{a: None}) == NULL_ARG, a
    for a in ("h", "W", "ws", "gh", "gW"):
        assert top_bwd(**{a: OFF8}) == BAD_ALIGN, a
    for a in ("y", "lse", "ent", "g", "ge"):
        assert top_bwd(**{a: OFF2}) == BAD_ALIGN, a
    assert top_bwd(dt=2) == BAD_ARG
    assert top_bwd(H=100) == BAD_SHAPE
    assert top_bwd(n=rlk.vocab_workspace_bytes(rlk.VOP_TOP_BWD, 64, 256, 4096, 0) - 1) == WS_SMALL
    assert top_bwd(gh=None, gW=None) == OK       # nothing wanted
    assert top_bwd(T=0, gW=None, h=None, ws=None) == OK


def dis_fwd(h=FAKE, W=FAKE, ids=FAKE, lg=FAKE, T=64, H=256, V=4096, K=8, tau=1.0, loss=FAKE, lse=FAKE, lp=FAKE,
            ws=FAKE, n=1 << 40):
    return rlk.lib().rlk_linear_distill_fwd(h, W, ids, lg, T, H, V, K, tau, loss, lse, lp, ws, n, None)


def dis_bwd(h=FAKE, W=FAKE, ids=FAKE, lg=FAKE, lse=FAKE, lp=FAKE, g=FAKE, T=64, H=256, V=4096, K=8, tau=1.0, gh=FAKE,
            gW=FAKE, dt=1, ws=FAKE, n=1 << 40):
    return rlk.lib().rlk_linear_distill_bwd(h, W, ids, lg, lse, lp, g, T, H, V, K, tau, gh, gW, dt, ws, n, None)


def test_distill_refusals():
    for a in ("h", "W", "ids", "lg", "loss", "lse", "lp", "ws"):
        assert dis_fwd(**{a: None}) == NULL_ARG, a
    for a in ("h", "W", "ids", "lg", "lse", "lp", "g", "ws"):
        assert dis_bwd(**{a: None}) == NULL_ARG, a
    for f in (dis_fwd, dis_bwd):
        for a in ("h", "W", "ws"):
            assert f(**{a: OFF8}) == BAD_ALIGN, a
        for a in ("ids", "lg", "lse", "lp"):
            assert f(**{a: OFF2}) == BAD_ALIGN, a
        for bad in (dict(T=-1), dict(H=32), dict(V=0), dict(K=0), dict(K=129)):
            assert f(**bad) == BAD_SHAPE, bad
        for tau in (0.0, -1.0, float("nan"), float("inf"), 1e-45, 1e39):
            assert f(tau=tau) == BAD_ARG, tau
        assert f(n=1000) == WS_SMALL
    assert dis_bwd(g=OFF2) == BAD_ALIGN
    assert dis_bwd(gW=OFF8) == BAD_ALIGN
    assert dis_bwd(dt=-1) == BAD_ARG
    assert dis_bwd(gh=None, gW=None) == OK
    assert dis_fwd(T=0, h=None, ids=None, ws=None) == OK
    assert dis_bwd(T=0, gW=None, h=None, ws=None) == OK


T, H, V, K = 8, 64, 100, 5


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def f32(*shape):
    return torch.zeros(shape)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


@pytest.fixture
def host_as_device(monkeypatch):
    """CPU tensors get past the checks of h and W; those of the other
    arguments must still fire first."""
    monkeypatch.setattr(vo, "_prep", lambda h, W, y: (h, W, y))
    monkeypatch.setattr(vo, "_head", lambda h, W: (h, W))


@pytest.mark.parametrize("bad", [-1, 129, 2.0, True, None, torch.ones(2, dtype=torch.int64)[0] * 1.5])
def test_binding_refuses_top_k(bad):
    with pytest.raises(ValueError, match="top_k"):
        rlk.linear_logp_top_fwd(bf(T, H), bf(V, H), i32(T), bad)


def test_binding_refuses_shapes_and_types(host_as_device):
    for name in ("lse", "entropy", "g", "g_entropy"):
        kw = dict(lse=f32(T), entropy=f32(T), g=f32(T), g_entropy=f32(T))
        kw[name] = f32(T + 1)
        with pytest.raises(ValueError, match=f"{name} must be 1-D of length T = {T}"):
            rlk.linear_logp_top_bwd(bf(T, H), bf(V, H), i32(T), **kw)
    with pytest.raises(ValueError, match="lse is required"):
        rlk.linear_logp_top_bwd(bf(T, H), bf(V, H), i32(T), None, f32(T), None)
    d = lambda ids, lg: rlk.linear_distill_fwd(bf(T, H), bf(V, H), ids, lg)  # noqa: E731
    for ids, lg, err, text in [(i32(T - 1, K), f32(T - 1, K), ValueError, "ids must be"),
                               (i32(T), f32(T), ValueError, "ids must be"),
                               (i32(T, 0), f32(T, 0), ValueError, "ids must be"),
                               (i32(T, 129), f32(T, 129), ValueError, "ids must be"),
                               (i32(T, K), f32(T, K - 1), ValueError, "logits must be"),
                               (f32(T, K), f32(T, K), TypeError, "int32 or int64"),
                               (i32(T, K), f32(T, K).double(), TypeError, "logits must be"),
                               (i32(T, K), f32(T, K), ValueError, "must be on")]:
        with pytest.raises(err, match=text):
            d(ids, lg)


def test_binding_refuses_the_rest():
    for f in (lambda i: rlk.linear_logp_top_fwd(bf(T, H), bf(V, H), i32(T), 1, ignore_index=i),
              lambda i: rlk.linear_logp_top_bwd(bf(T, H), bf(V, H), i32(T), f32(T), f32(T), f32(T), ignore_index=i)):
        for bad in (2 ** 31, -2 ** 31 - 1, 2 ** 40):
            with pytest.raises(ValueError, match="int32"):
                f(bad)
    with pytest.raises(ValueError, match="device tensors"):
        rlk.linear_logp_top(bf(T, H), bf(V, H), i32(T), 4)
    with pytest.raises(ValueError, match="device tensors"):
        rlk.linear_distill(bf(T, H), bf(V, H), i32(T, K), f32(T, K))
    with pytest.raises(ValueError, match="no gradient"):
        rlk.linear_distill(bf(T, H), bf(V, H), i32(T, K), f32(T, K).requires_grad_())
    with pytest.raises(TypeError, match="bfloat16"):
        rlk.linear_distill(f32(T, H), bf(V, H), i32(T, K), f32(T, K))
    with pytest.raises(TypeError, match="grad_W_dtype"):
        vo._grads(bf(T, H), bf(V, H), True, True, torch.float16)
    with pytest.raises(ValueError, match="must be float32"):
        vo._slot_values(T, K, torch.device("cpu"), logp_ids=f32(T, K + 1))


@pytest.mark.parametrize("H,V,parts", [(512, 32768, (4, 8)), (512, 65536, (8, 16)), (64, 131072, (16, 32)),
                                       (512, 131072, (16, 32)), (1024, 65536, (8, 16)), (1024, 131072, (16, 16)),
                                       (2048, 32768, (4, 8)), (2048, 65536, (8, 8)), (4096, 131072, (4, 4)),
                                       (512, 151936, (32, 32))])
def test_parts_of_grad_h_by_width_and_vocabulary(H, V, parts):
    """The backward's workspace holds grad_h's fp32 parts: their number (it
    fixes grad_h's bits) on both sides of a vocabulary, all else being equal."""
    T = 256
    below, at = (rlk.vocab_workspace_bytes(rlk.VOP_TOP_BWD, T, H, v, 0) for v in (V - 1, V))
    assert -(-(V - 1) // 32) == -(-V // 32)  # one split width
    assert at - below == 4 * T * H * (parts[1] - parts[0])
    wide = rlk.vocab_workspace_bytes(rlk.VOP_TOP_BWD, 2 * T, H, V, 0)
    # twice the rows: twice the parts, beside the rows' indices (4 bytes) and
    # coefficients (20), h and the dz of 32 splits
    S_pad = (V // 32 + 63) // 64 * 64
    assert wide - at == T * (4 + 20) + 2 * T * H + 2 * T * 32 * S_pad + 4 * T * H * parts[1]
