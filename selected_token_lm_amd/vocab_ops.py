"""Operators on the whole next-token distribution of an LM head (the C ABI of
``include/rlk/vocab_ops.h``), re-exported by the package:

    logp, entropy, top_logp, top_ids = linear_logp_top(h, W, y, top_k)     # autograd-aware
    logp, lse, entropy, top_logp, top_ids = linear_logp_top_fwd(h, W, y, top_k)
    grad_h, grad_W = linear_logp_top_bwd(h, W, y, lse, entropy, g, g_entropy)

    loss = linear_distill(h, W, ids, logits, temperature)                  # autograd-aware
    loss, lse, logp_ids = linear_distill_fwd(h, W, ids, logits, temperature)
    grad_h, grad_W = linear_distill_bwd(h, W, ids, logits, lse, logp_ids, g, temperature)

As in the rest of the package only argument marshalling lives here.  A
teacher's ``top_ids`` and ``top_logp`` are a student's ``ids`` and ``logits``
as they are: inactive rows hold ids of -1 and log-probabilities of -inf,
which mark empty slots.
"""
from __future__ import annotations

import contextlib
import ctypes
import operator

import torch
from torch.autograd.function import once_differentiable

from . import IGNORE_INDEX, _c_void_p, _check, _given_workspace, _i32, _i64, _prep, _ptr, _rows, _size, _stream, lib

MAX_K = 128
VOP_TOP_FWD, VOP_TOP_BWD, VOP_DISTILL_FWD, VOP_DISTILL_BWD = 0, 1, 2, 3
_GRAD_W_DTYPES = {torch.float32: 0, torch.bfloat16: 1}

_f32 = ctypes.c_float
_p = _c_void_p
SIGNATURES = {
    "rlk_vocab_workspace_bytes": (_size, [_i32, _i64, _i64, _i64, _i64]),
    "rlk_linear_logp_top_fwd": (_i32, [_p, _p, _p, _i64, _i64, _i64, _i32, _i64, _p, _p, _p, _p, _p, _p, _size, _p]),
    "rlk_linear_logp_top_bwd": (_i32, [_p, _p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _i32, _p, _p, _i32, _p, _size, _p]),
    "rlk_linear_distill_fwd": (_i32, [_p, _p, _p, _p, _i64, _i64, _i64, _i64, _f32, _p, _p, _p, _p, _size, _p]),
    "rlk_linear_distill_bwd": (_i32, [_p, _p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _i64, _f32, _p, _p, _i32, _p, _size,
                                      _p]),
}


def vocab_workspace_bytes(op: int, T: int, H: int, V: int, K: int) -> int:
    """Workspace bytes of one of the operators (VOP_*); 0 for invalid sizes."""
    return int(lib().rlk_vocab_workspace_bytes(op, T, H, V, K))


_SAME = contextlib.nullcontext()


def _on(device):
    """`device` as the current one (the library works on the current device's
    stream); free where it already is."""
    return _SAME if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _ws(ws, op, T, H, V, K, device):
    if ws is not None:
        return _given_workspace(ws, device)
    n = vocab_workspace_bytes(op, T, H, V, K)
    if n == 0:
        raise ValueError(f"invalid shape T={T} H={H} V={V} K={K}")
    return torch.empty(n, dtype=torch.uint8, device=device), n


def _top_k(k):
    try:
        n = -1 if isinstance(k, bool) else operator.index(k)
    except TypeError:
        n = -1
    if not 0 <= n <= MAX_K:
        raise ValueError(f"top_k must be an integer in [0, {MAX_K}], got {k!r}")
    return n


def _targets(h, W, y, ignore_index):
    """_prep, with 64-bit targets and ignore_index kept inside 32 bits: a
    target past int32 stays outside every vocabulary, and apart from an
    ignore_index at int32's end."""
    lo, hi = -2 ** 31, 2 ** 31 - 1
    if not lo <= ignore_index <= hi:
        raise ValueError(f"ignore_index must fit an int32, got {ignore_index}")
    if y.dtype == torch.int64:
        inside = y.clamp(lo + (ignore_index == lo), hi - (ignore_index == hi))
        y = torch.where(y == ignore_index, y, inside) if ignore_index in (lo, hi) else inside
    return _prep(h, W, y)


def _slots(T, device, ids, logits):
    """The teacher's [T, K] ids (int32) and logits (fp32): shapes and types
    first, then the device, as in _prep."""
    if ids.dim() != 2 or ids.shape[0] != T or not 1 <= ids.shape[1] <= MAX_K:
        raise ValueError(f"ids must be [T, K] = [{T}, 1 .. {MAX_K}], got {list(ids.shape)}")
    if logits.shape != ids.shape:
        raise ValueError(f"logits must be {list(ids.shape)} as ids, got {list(logits.shape)}")
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("ids must hold int32 or int64 token ids")
    if logits.dtype not in (torch.float32, torch.bfloat16, torch.float16):
        raise TypeError("logits must be float32, bfloat16 or float16")
    if not ids.is_cuda or not logits.is_cuda or ids.device != device or logits.device != device:
        raise ValueError(f"ids and logits must be on {device}")
    if ids.dtype == torch.int64:
        # an id past int32 stays an id outside every vocabulary
        ids = ids.clamp(-1, 2 ** 31 - 1)
    return ids.to(torch.int32).contiguous(), logits.to(torch.float32).contiguous()


def _slot_values(T, K, device, **named):
    for name, t in named.items():
        if t.dim() != 2 or tuple(t.shape) != (T, K) or t.dtype != torch.float32:
            raise ValueError(f"{name} must be float32 [T, K] = [{T}, {K}], got {t.dtype} {list(t.shape)}")
    for name, t in named.items():
        if not t.is_cuda or t.device != device:
            raise ValueError(f"{name} must be on {device}")
    return [t.contiguous() for t in named.values()]


def _head(h, W):
    """The checks of _prep for h and W alone."""
    if h.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
        raise TypeError("h and W must be bfloat16")
    if h.dim() != 2 or W.dim() != 2 or h.shape[1] != W.shape[1]:
        raise ValueError("h must be [T, H] and W [V, H]")
    if not (h.is_cuda and W.is_cuda):
        raise ValueError("h and W must be device tensors")
    if W.device != h.device:
        raise ValueError("h and W must be on one device")
    return h.contiguous(), W.contiguous()


def _grads(h, W, need_grad_h, need_grad_W, grad_W_dtype):
    if grad_W_dtype not in _GRAD_W_DTYPES:
        raise TypeError("grad_W_dtype must be float32 or bfloat16")
    grad_h = torch.empty(h.shape, dtype=torch.bfloat16, device=h.device) if need_grad_h else None
    grad_W = torch.empty(W.shape, dtype=grad_W_dtype, device=h.device) if need_grad_W else None
    return grad_h, grad_W, _GRAD_W_DTYPES[grad_W_dtype]


def linear_logp_top_fwd(h, W, y, top_k: int, ignore_index: int = IGNORE_INDEX, ws=None):
    """(logp, lse, entropy) fp32 [T] and (top_logp fp32, top_ids int32) [T, top_k].

    logp and lse are linear_logp_fwd's, bit for bit.  entropy is that of the
    whole distribution in nats.  The alternatives are the top_k (0 .. 128)
    most likely tokens, best first, ties to the lowest id; slots past the
    vocabulary hold id -1 and -inf, and so do inactive rows (y ==
    ignore_index), whose logp, lse and entropy are 0.
    """
    top_k = _top_k(top_k)
    h, W, y = _targets(h, W, y, ignore_index)
    T, H = h.shape
    V = W.shape[0]
    with _on(h.device):
        logp, lse, entropy = (torch.empty(T, dtype=torch.float32, device=h.device) for _ in range(3))
        top_logp = torch.empty((T, top_k), dtype=torch.float32, device=h.device)
        top_ids = torch.empty((T, top_k), dtype=torch.int32, device=h.device)
        ws, n = _ws(ws, VOP_TOP_FWD, T, H, V, top_k, h.device)
        _check(lib().rlk_linear_logp_top_fwd(_ptr(h), _ptr(W), _ptr(y), T, H, V, ignore_index, top_k, _ptr(logp),
                                             _ptr(lse), _ptr(entropy), _ptr(top_logp), _ptr(top_ids), _ptr(ws), n,
                                             _stream()),
               "rlk_linear_logp_top_fwd")
    return logp, lse, entropy, top_logp, top_ids


def linear_logp_top_bwd(h, W, y, lse, entropy, g, g_entropy=None, ignore_index: int = IGNORE_INDEX,
                        need_grad_h: bool = True, need_grad_W: bool = True, grad_W_dtype=torch.float32, ws=None):
    """(grad_h bf16 [T,H] or None, grad_W [V,H] of grad_W_dtype or None) of
    sum_t g_t logp_t + g_entropy_t entropy_t; g or g_entropy may be None (zero)."""
    h, W, y = _targets(h, W, y, ignore_index)
    T, H = h.shape
    V = W.shape[0]
    named = dict(lse=lse, entropy=entropy, g=g, g_entropy=g_entropy)
    named = {k: v for k, v in named.items() if v is not None or k in ("lse", "entropy")}
    rows = dict(zip(named, _rows(T, h.device, **named)))
    with _on(h.device):
        grad_h, grad_W, code = _grads(h, W, need_grad_h, need_grad_W, grad_W_dtype)
        ws, n = _ws(ws, VOP_TOP_BWD, T, H, V, 0, h.device)
        _check(lib().rlk_linear_logp_top_bwd(_ptr(h), _ptr(W), _ptr(y), _ptr(rows["lse"]), _ptr(rows["entropy"]),
                                             _ptr(rows.get("g")), _ptr(rows.get("g_entropy")), T, H, V, ignore_index,
                                             _ptr(grad_h), _ptr(grad_W), code, _ptr(ws), n, _stream()),
               "rlk_linear_logp_top_bwd")
    return grad_h, grad_W


def linear_distill_fwd(h, W, ids, logits, temperature: float = 1.0, ws=None):
    """(loss, lse) fp32 [T] and logp_ids fp32 [T, K]: KL(q || p) of every row,
    q = softmax of the teacher's kept logits / temperature over their ids,
    p = softmax of h W^T / temperature over the vocabulary; lse and logp_ids
    (the student's log p at the ids) are the state the backward needs.  An id
    below 0 or a logit of -inf marks an empty slot; rows without a kept slot
    have loss 0 and no gradient.  The ids of a row are meant to be distinct:
    where one is repeated its slots keep their own log q, so the loss is below
    KL(q || p) by a constant of the teacher (the gradient has their sum)."""
    h, W = _head(h, W)
    T, H = h.shape
    V = W.shape[0]
    ids, logits = _slots(T, h.device, ids, logits)
    K = ids.shape[1]
    with _on(h.device):
        loss, lse = (torch.empty(T, dtype=torch.float32, device=h.device) for _ in range(2))
        logp_ids = torch.empty((T, K), dtype=torch.float32, device=h.device)
        ws, n = _ws(ws, VOP_DISTILL_FWD, T, H, V, K, h.device)
        _check(lib().rlk_linear_distill_fwd(_ptr(h), _ptr(W), _ptr(ids), _ptr(logits), T, H, V, K, temperature,
                                            _ptr(loss), _ptr(lse), _ptr(logp_ids), _ptr(ws), n, _stream()),
               "rlk_linear_distill_fwd")
    return loss, lse, logp_ids


def linear_distill_bwd(h, W, ids, logits, lse, logp_ids, g, temperature: float = 1.0, need_grad_h: bool = True,
                       need_grad_W: bool = True, grad_W_dtype=torch.float32, ws=None):
    """(grad_h bf16 [T,H] or None, grad_W [V,H] of grad_W_dtype or None) of sum_t g_t loss_t."""
    h, W = _head(h, W)
    T, H = h.shape
    V = W.shape[0]
    ids, logits = _slots(T, h.device, ids, logits)
    K = ids.shape[1]
    lse, g = _rows(T, h.device, lse=lse, g=g)
    logp_ids, = _slot_values(T, K, h.device, logp_ids=logp_ids)
    with _on(h.device):
        grad_h, grad_W, code = _grads(h, W, need_grad_h, need_grad_W, grad_W_dtype)
        ws, n = _ws(ws, VOP_DISTILL_BWD, T, H, V, K, h.device)
        _check(lib().rlk_linear_distill_bwd(_ptr(h), _ptr(W), _ptr(ids), _ptr(logits), _ptr(lse), _ptr(logp_ids),
                                            _ptr(g), T, H, V, K, temperature, _ptr(grad_h), _ptr(grad_W), code,
                                            _ptr(ws), n, _stream()),
               "rlk_linear_distill_bwd")
    return grad_h, grad_W


class _LinearLogpTop(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, W, y, top_k, ignore_index):
        logp, lse, entropy, top_logp, top_ids = linear_logp_top_fwd(h, W, y, top_k, ignore_index)
        ctx.save_for_backward(h, W, y, lse, entropy)
        ctx.ignore_index = ignore_index
        ctx.mark_non_differentiable(top_logp, top_ids)
        ctx.set_materialize_grads(False)
        return logp, entropy, top_logp, top_ids

    @staticmethod
    @once_differentiable
    def backward(ctx, g, g_entropy, _g_top, _g_ids):
        h, W, y, lse, entropy = ctx.saved_tensors
        if g is None and g_entropy is None:
            return None, None, None, None, None
        gh, gW = linear_logp_top_bwd(h, W, y, lse, entropy, g, g_entropy, ctx.ignore_index,
                                     need_grad_h=ctx.needs_input_grad[0], need_grad_W=ctx.needs_input_grad[1],
                                     grad_W_dtype=W.dtype)
        return gh, gW, None, None, None


def linear_logp_top(h, W, y, top_k: int = 0, ignore_index: int = IGNORE_INDEX):
    """(logp, entropy, top_logp, top_ids) of linear_logp_top_fwd, autograd-aware
    through logp and entropy (the alternatives carry no gradient)."""
    return _LinearLogpTop.apply(h, W, y, top_k, ignore_index)


class _LinearDistill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, W, ids, logits, temperature):
        loss, lse, logp_ids = linear_distill_fwd(h, W, ids, logits, temperature)
        ctx.save_for_backward(h, W, ids, logits, lse, logp_ids)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        h, W, ids, logits, lse, logp_ids = ctx.saved_tensors
        gh, gW = linear_distill_bwd(h, W, ids, logits, lse, logp_ids, g, ctx.temperature,
                                    need_grad_h=ctx.needs_input_grad[0], need_grad_W=ctx.needs_input_grad[1],
                                    grad_W_dtype=W.dtype)
        return gh, gW, None, None, None


def linear_distill(h, W, ids, logits, temperature: float = 1.0):
    """KL(q || p) per row (linear_distill_fwd), autograd-aware in h and W.  The
    teacher's logits carry no gradient: a tensor that asks for one is refused."""
    if logits.requires_grad and torch.is_grad_enabled():
        raise ValueError("logits carry no gradient: pass logits.detach()")
    return _LinearDistill.apply(h, W, ids, logits, temperature)
