"""Operators that stand before and behind the LM head in a training step (the
C ABI of ``include/rlk/step_ops.h``), re-exported by the package:

    y = layer_norm(x, weight, bias, eps)                    # autograd-aware
    y, mean, rstd = layer_norm_fwd(x, weight, bias, eps)
    grad_x, grad_weight, grad_bias = layer_norm_bwd(x, weight, mean, rstd, g)
    y = rms_norm(x, weight, eps)                            # autograd-aware
    y, rstd = rms_norm_fwd(x, weight, eps)
    grad_x, grad_weight = rms_norm_bwd(x, weight, rstd, g)

    out = embed(ids, E, scale)                              # autograd-aware
    out = embed_fwd(ids, E, scale)
    grad_E = embed_bwd(ids, g, V, scale)                    # dense
    embed_bwd(ids, g, V, scale, grad_E=grad_W)              # added to the head's gradient (tied weights)

    norm = grad_norm(grads)
    norm, grads = clip_grads(grads, max_norm)               # in place, or into out=

As in the rest of the package only argument marshalling lives here.  Tensors
are bfloat16 or float32, in any mixture; rows may be strided.  Autograd is
followed backwards; an input with a forward-mode tangent raises.
"""
from __future__ import annotations

import ctypes
from array import array

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import IGNORE_INDEX, _c_void_p, _check, _given_workspace, _i32, _i64, _ptr, _rows, _size, lib
from .vocab_ops import _on

SOP_NORM_BWD, SOP_EMBED_BWD, SOP_GRADS = 0, 1, 2
MAX_ROWS, MAX_WIDTH = 1 << 23, 1 << 16
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}

_f32 = ctypes.c_float
_p = _c_void_p
SIGNATURES = {
    "rlk_step_workspace_bytes": (_size, [_i32, _i64, _i64, _i64]),
    "rlk_layer_norm_fwd": (_i32, [_p, _i32, _i64, _p, _p, _i32, _i64, _i64, _f32, _p, _i32, _p, _p, _p]),
    "rlk_layer_norm_bwd": (_i32, [_p, _i32, _i64, _p, _i32, _p, _p, _p, _i32, _i64, _i64, _i64, _p, _p, _p, _i32, _p,
                                  _size, _p]),
    "rlk_rms_norm_fwd": (_i32, [_p, _i32, _i64, _p, _i32, _i64, _i64, _f32, _p, _i32, _p, _p]),
    "rlk_rms_norm_bwd": (_i32, [_p, _i32, _i64, _p, _i32, _p, _p, _i32, _i64, _i64, _i64, _p, _p, _i32, _p, _size, _p]),
    "rlk_embed_fwd": (_i32, [_p, _i32, _p, _i32, _i64, _i64, _i64, _i64, _f32, _p, _i32, _p]),
    "rlk_embed_bwd": (_i32, [_p, _i32, _p, _i32, _i64, _i64, _i64, _i64, _i64, _f32, _p, _i32, _i32, _p, _size, _p]),
    "rlk_grad_norm": (_i32, [_p, _p, _p, _i32, _p, _p, _size, _p]),
    "rlk_clip_grads": (_i32, [_p, _p, _p, _i32, _f32, _p, _p, _p, _p, _size, _p]),
}


def step_workspace_bytes(op: int, T: int, H: int = 0, V: int = 0) -> int:
    """Workspace bytes of a norm's backward (SOP_NORM_BWD), of embed_bwd
    (SOP_EMBED_BWD), or of grad_norm and clip_grads for T tensors (SOP_GRADS);
    0 for invalid sizes."""
    return int(lib().rlk_step_workspace_bytes(op, T, H, V))


def _ws(ws, op, T, H, V, device):
    if ws is not None:
        return _given_workspace(ws, device)
    n = step_workspace_bytes(op, T, H, V)
    if n == 0:
        raise ValueError(f"invalid shape T={T} H={H} V={V}")
    return torch.empty(n, dtype=torch.uint8, device=device), n


def _stream(device):
    """The device's current stream, without the object around it (2.6 us)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _dtype(name, dtype):
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {dtype}")
    return code


def _matrix(name, t, shape=None, device=None):
    """(t, its dtype's code, its row stride): [T, H] rows whose elements lie
    next to each other (copied where they do not)."""
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be {'[T, H]' if shape is None else list(shape)}, got {list(t.shape)}")
    code = _dtype(name, t.dtype)
    if shape is None and not (1 <= t.shape[1] <= MAX_WIDTH and t.shape[0] <= MAX_ROWS):
        raise ValueError(f"{name} must have at most 2^23 rows of 1 to {MAX_WIDTH} elements, got {list(t.shape)}")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be on {'a GPU' if device is None else device}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        t = t.contiguous()
    return t, code, t.stride(0)


def _vectors(H, device, **named):
    """(the tensors, contiguous, and the code of the dtype they share)."""
    code, out = None, []
    for name, t in named.items():
        if t is None:
            out.append(None)
            continue
        if t.dim() != 1 or t.shape[0] != H:
            raise ValueError(f"{name} must be [H] = [{H}], got {list(t.shape)}")
        c = _dtype(name, t.dtype)
        if code is not None and c != code:
            raise TypeError(f"{' and '.join(named)} must have one dtype")
        code = c
        out.append(t if t.is_contiguous() else t.contiguous())
    for name, t in named.items():
        if t is not None and (t.device != device or not t.is_cuda):
            raise ValueError(f"{name} must be on {device}")
    return out, code or 0


def _tangent(t):
    return t is not None and forward_ad.unpack_dual(t).tangent is not None


def _followed(*tensors):
    """Whether autograd follows one of them: backwards, or forwards with a
    tangent, which no_grad leaves on (the autograd functions refuse it)."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        return True
    # no tangents outside of dual levels; asking each tensor takes 0.8 us
    return forward_ad._current_level >= 0 and any(_tangent(t) for t in tensors)


def _no_tangents(what, tensors):
    """Refuses tangents that a result would lack, or that a change in place
    would leave behind."""
    if forward_ad._current_level >= 0 and any(_tangent(t) for t in tensors):
        raise ValueError(f"{what} must carry no forward-mode tangent")


def _eps(eps):
    eps = float(eps)
    if not 0.0 <= eps <= 3.4028234663852886e38:
        raise ValueError(f"eps must be finite and not negative, got {eps}")
    return eps


def _norm_fwd(center, x, weight, bias, eps, out_dtype, stats):
    """(y, mean or None, rstd or None); no statistics are kept unless asked for."""
    eps = _eps(eps)
    x, xd, ld = _matrix("x", x)
    T, H = x.shape
    dev = x.device
    (weight, bias), wd = _vectors(H, dev, weight=weight, bias=bias)
    out_dtype = x.dtype if out_dtype is None else out_dtype
    yd = _dtype("out_dtype", out_dtype)
    with _on(dev):
        y = torch.empty_like(x) if out_dtype is x.dtype and x.is_contiguous() else x.new_empty((T, H), dtype=out_dtype)
        mean = x.new_empty(T, dtype=torch.float32) if stats and center else None
        rstd = x.new_empty(T, dtype=torch.float32) if stats else None
        if center:
            _check(lib().rlk_layer_norm_fwd(_ptr(x), xd, ld, _ptr(weight), _ptr(bias), wd, T, H, eps, _ptr(y), yd,
                                            _ptr(mean), _ptr(rstd), _stream(dev)),
                   "rlk_layer_norm_fwd")
        else:
            _check(lib().rlk_rms_norm_fwd(_ptr(x), xd, ld, _ptr(weight), wd, T, H, eps, _ptr(y), yd, _ptr(rstd),
                                          _stream(dev)),
                   "rlk_rms_norm_fwd")
    return y, mean, rstd


def _stat(name, t, T, device):
    """A row statistic as _rows has it, at no cost where it is one already."""
    if t is not None and t.dtype is torch.float32 and t.shape == (T,) and t.device == device and t.is_contiguous():
        return t
    return _rows(T, device, **{name: t})[0]


def _norm_bwd(center, x, weight, mean, rstd, g, need_x, need_w, need_b, grad_dtype, ws):
    x, xd, ldx = _matrix("x", x)
    T, H = x.shape
    dev = x.device
    g, gd, ldg = _matrix("g", g, x.shape, dev)
    (weight,), wd = _vectors(H, dev, weight=weight)
    mean = _stat("mean", mean, T, dev) if center else None
    rstd = _stat("rstd", rstd, T, dev)
    code = _dtype("grad_weight_dtype", grad_dtype)
    with _on(dev):
        grad_x = None
        if need_x:
            grad_x = torch.empty_like(x) if x.is_contiguous() else x.new_empty((T, H))
        grad_w = x.new_empty(H, dtype=grad_dtype) if need_w else None
        grad_b = x.new_empty(H, dtype=grad_dtype) if need_b else None
        n = 0
        if need_w or need_b:
            ws, n = _ws(ws, SOP_NORM_BWD, T, H, 0, dev)
        if center:
            _check(lib().rlk_layer_norm_bwd(_ptr(x), xd, ldx, _ptr(weight), wd, _ptr(mean), _ptr(rstd), _ptr(g), gd,
                                            ldg, T, H, _ptr(grad_x), _ptr(grad_w), _ptr(grad_b), code, _ptr(ws), n,
                                            _stream(dev)),
                   "rlk_layer_norm_bwd")
        else:
            _check(lib().rlk_rms_norm_bwd(_ptr(x), xd, ldx, _ptr(weight), wd, _ptr(rstd), _ptr(g), gd, ldg, T, H,
                                          _ptr(grad_x), _ptr(grad_w), code, _ptr(ws), n, _stream(dev)),
                   "rlk_rms_norm_bwd")
    return grad_x, grad_w, grad_b


def layer_norm_fwd(x, weight=None, bias=None, eps: float = 1e-5, out_dtype=None):
    """(y [T, H] of out_dtype (x's by default), mean, rstd fp32 [T]):
    y = (x - mean) rstd weight + bias, rstd = 1 / sqrt(variance + eps).
    Computed in fp32, y rounded once; a row's results depend on that row alone."""
    return _norm_fwd(True, x, weight, bias, eps, out_dtype, True)


def layer_norm_bwd(x, weight, mean, rstd, g, need_grad_x: bool = True, need_grad_weight: bool = True,
                   need_grad_bias: bool = True, grad_weight_dtype=torch.float32, ws=None):
    """(grad_x [T, H] of x's dtype, grad_weight, grad_bias [H] of
    grad_weight_dtype) of sum(g * y), None where not needed.  weight may be
    None (ones)."""
    return _norm_bwd(True, x, weight, mean, rstd, g, need_grad_x, need_grad_weight, need_grad_bias, grad_weight_dtype,
                     ws)


def rms_norm_fwd(x, weight=None, eps: float = 1e-6, out_dtype=None):
    """(y [T, H] of out_dtype (x's by default), rstd fp32 [T]): y = x rstd weight,
    rstd = 1 / sqrt(mean of x^2 + eps)."""
    y, _, rstd = _norm_fwd(False, x, weight, None, eps, out_dtype, True)
    return y, rstd


def rms_norm_bwd(x, weight, rstd, g, need_grad_x: bool = True, need_grad_weight: bool = True,
                 grad_weight_dtype=torch.float32, ws=None):
    """(grad_x [T, H] of x's dtype, grad_weight [H] of grad_weight_dtype) of
    sum(g * y), None where not needed."""
    return _norm_bwd(False, x, weight, None, rstd, g, need_grad_x, need_grad_weight, False, grad_weight_dtype, ws)[:2]


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, center, x, weight, bias, eps, out_dtype):
        y, mean, rstd = _norm_fwd(center, x, weight, bias, eps, out_dtype, True)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.center = center
        ctx.vector_dtype = next((t.dtype for t in (weight, bias) if t is not None), torch.float32)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        grads = _norm_bwd(ctx.center, x, weight, mean, rstd, g, need[1], need[2], need[3], ctx.vector_dtype, None)
        return None, *grads, None, None


def _norm(center, x, weight, bias, eps, out_dtype):
    if not _followed(x, weight, bias):
        return _norm_fwd(center, x, weight, bias, eps, out_dtype, False)[0]
    return _Norm.apply(center, x, weight, bias, eps, out_dtype)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, out_dtype=None):
    """y of layer_norm_fwd, autograd-aware in x, weight and bias."""
    return _norm(True, x, weight, bias, eps, out_dtype)


def rms_norm(x, weight=None, eps: float = 1e-6, out_dtype=None):
    """y of rms_norm_fwd, autograd-aware in x and weight."""
    return _norm(False, x, weight, None, eps, out_dtype)


def _ids(ids, device):
    if ids.dim() != 1:
        raise ValueError(f"ids must be [T], got {list(ids.shape)}")
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("ids must hold int32 or int64 token ids")
    if ids.shape[0] > MAX_ROWS:
        raise ValueError(f"at most 2^23 ids, got {ids.shape[0]}")
    if not ids.is_cuda or ids.device != device:
        raise ValueError(f"ids must be on {device}")
    return ids.contiguous(), 8 if ids.dtype == torch.int64 else 4


def _table(name, E):
    if E.dim() != 2 or not 1 <= E.shape[1] <= MAX_WIDTH or E.shape[0] < 1:
        raise ValueError(f"{name} must be [V, H], H at most {MAX_WIDTH}, got {list(E.shape)}")
    code = _dtype(name, E.dtype)
    if not E.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return code


def _scale(scale):
    scale = float(scale)
    if not abs(scale) <= 3.4028234663852886e38:
        raise ValueError(f"scale must be finite, got {scale}")
    return scale


def _ignore(ignore_index):
    if not -2 ** 63 <= ignore_index < 2 ** 63:
        raise ValueError(f"ignore_index must fit an int64, got {ignore_index}")
    return ignore_index


def embed_fwd(ids, E, scale: float = 1.0, ignore_index: int = IGNORE_INDEX, out_dtype=None):
    """scale * E[ids], [T, H] of out_dtype (E's by default), rounded once.  Rows
    of ignore_index are zero; an id outside [0, V) makes its row NaN."""
    ed = _table("E", E)
    ids, width = _ids(ids, E.device)
    E = E.contiguous()
    T, (V, H) = ids.shape[0], E.shape
    out_dtype = E.dtype if out_dtype is None else out_dtype
    od = _dtype("out_dtype", out_dtype)
    scale, ignore_index = _scale(scale), _ignore(ignore_index)
    dev = E.device
    with _on(dev):
        out = torch.empty((T, H), dtype=out_dtype, device=dev)
        _check(lib().rlk_embed_fwd(_ptr(ids), width, _ptr(E), ed, T, H, V, ignore_index, scale, _ptr(out), od,
                                   _stream(dev)),
               "rlk_embed_fwd")
    return out


def embed_bwd(ids, g, V: int, scale: float = 1.0, ignore_index: int = IGNORE_INDEX, grad_E_dtype=torch.float32,
              grad_E=None, ws=None):
    """The table's gradient: row v is scale times the sum of g's rows whose id
    is v, in their order.  Without grad_E: a new [V, H] of grad_E_dtype, zero for
    tokens that do not occur.  With it (contiguous [V, H]): the sums are added to
    it in place, rows of other tokens are not touched, and it is returned.  Ids
    of ignore_index or outside [0, V) count nothing."""
    g, gd, ldg = _matrix("g", g)
    T, H = g.shape
    dev = g.device
    ids, width = _ids(ids, dev)
    if ids.shape[0] != T:
        raise ValueError(f"ids must be [T] = [{T}], got {list(ids.shape)}")
    scale, ignore_index = _scale(scale), _ignore(ignore_index)
    add = grad_E is not None
    if add:
        od = _table("grad_E", grad_E)
        if grad_E.shape != (V, H) or not grad_E.is_contiguous() or grad_E.device != dev:
            raise ValueError(f"grad_E must be a contiguous [{V}, {H}] tensor on {dev}, got {list(grad_E.shape)}")
        if grad_E.requires_grad and torch.is_grad_enabled():
            raise ValueError("grad_E requires a gradient itself: pass E.grad, not E")
        _no_tangents("grad_E", [grad_E])
    else:
        od = _dtype("grad_E_dtype", grad_E_dtype)
    with _on(dev):
        ws, n = _ws(ws, SOP_EMBED_BWD, T, H, V, dev)
        if not add:
            grad_E = torch.empty((V, H), dtype=grad_E_dtype, device=dev)
        _check(lib().rlk_embed_bwd(_ptr(ids), width, _ptr(g), gd, ldg, T, H, V, ignore_index, scale, _ptr(grad_E), od,
                                   int(add), _ptr(ws), n, _stream(dev)),
               "rlk_embed_bwd")
    if add:
        _written([grad_E])
    return grad_E


class _Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, E, scale, ignore_index, out_dtype):
        ctx.save_for_backward(ids)
        ctx.rest = E.shape[0], scale, ignore_index, E.dtype
        return embed_fwd(ids, E, scale, ignore_index, out_dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        V, scale, ignore_index, dtype = ctx.rest
        return None, embed_bwd(ctx.saved_tensors[0], g, V, scale, ignore_index, grad_E_dtype=dtype), None, None, None


def embed(ids, E, scale: float = 1.0, ignore_index: int = IGNORE_INDEX, out_dtype=None):
    """embed_fwd, autograd-aware in E (a dense gradient of E's dtype)."""
    if not _followed(E):
        return embed_fwd(ids, E, scale, ignore_index, out_dtype)
    return _Embed.apply(ids, E, scale, ignore_index, out_dtype)


def _tensors(what, tensors):
    """The device and the host arrays of a list of dense tensors: pointers and
    dtypes; and whether all are contiguous.  A sum of squares and a scaling go
    by memory, so any dense layout serves."""
    n, device = len(tensors), tensors[0].device
    dtypes = [t.dtype for t in tensors]
    if dtypes.count(dtypes[0]) == n and dtypes[0] in _DTYPES:
        codes = array("i", [_DTYPES[dtypes[0]]]) * n
    else:
        codes = array("i", [_DTYPES.get(d, -1) for d in dtypes])
        if -1 in codes:
            i = codes.index(-1)
            raise TypeError(f"{what}[{i}] must be float32 or bfloat16, got {dtypes[i]}")
    if not tensors[0].is_cuda or [t.get_device() for t in tensors].count(device.index) != n:
        raise ValueError(f"all of {what} must be on one GPU")
    contiguous = [t.is_contiguous() for t in tensors]
    plain = all(contiguous)
    for i, c in enumerate(() if plain else contiguous):
        if not c and not torch.ops.aten.is_non_overlapping_and_dense(tensors[i]):
            raise ValueError(f"{what}[{i}] must be dense in memory, got strides {list(tensors[i].stride())}")
    return device, array("Q", [t.data_ptr() for t in tensors]), codes, plain


def _sizes(tensors):
    return array("q", [t.numel() for t in tensors])


def _at(values):
    """The address of an array's values (the library reads them before it returns)."""
    return values.buffer_info()[0]


def _written(tensors):
    """Tells autograd that these tensors were changed in place."""
    try:
        torch.autograd.graph.increment_version(tensors)
    except RuntimeError:  # inference tensors have no version
        torch.autograd.graph.increment_version([t for t in tensors if not t.is_inference()])


def _list(what, tensors):
    tensors = [tensors] if isinstance(tensors, torch.Tensor) else list(tensors)
    if set(map(type, tensors)) - {torch.Tensor}:
        for i, t in enumerate(tensors):
            if t is None:
                raise TypeError(f"{what}[{i}] is None: leave out parameters without a gradient")
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{what}[{i}] must be a tensor, got {type(t)}")
    return tensors


def grad_norm(grads, ws=None):
    """The norm of all elements of a list of tensors, fp32 [] on their device:
    squares are summed in fp64 and the root rounded once.  A value: autograd
    does not follow it."""
    grads = _list("grads", grads)
    if not grads:
        raise ValueError("grads is empty")
    _no_tangents("grads", grads)
    dev, ptrs, codes, _ = _tensors("grads", grads)
    n, sizes = len(grads), _sizes(grads)
    with _on(dev):
        ws, size = _ws(ws, SOP_GRADS, n, 0, 0, dev)
        norm = torch.empty((), dtype=torch.float32, device=dev)
        _check(lib().rlk_grad_norm(_at(ptrs), _at(sizes), _at(codes), n, _ptr(norm), _ptr(ws), size, _stream(dev)),
               "rlk_grad_norm")
    return norm


def clip_grads(grads, max_norm: float, out=None, ws=None):
    """(norm, out): the norm of all gradients (as grad_norm) and c grads, c =
    max_norm / norm where the norm is above max_norm, else 1.  In place, or
    into the list `out` of tensors of the same shapes and layouts (float32 or
    bfloat16 each).  Nothing waits for the GPU, and autograd does not follow.
    With a NaN norm every gradient becomes NaN."""
    grads = _list("grads", grads)
    if not grads:
        raise ValueError("grads is empty")
    _no_tangents("grads", grads)
    out = None if out is None else _list("out", out)
    max_norm = float(max_norm)
    if not max_norm >= 0.0:
        raise ValueError(f"max_norm must not be negative, got {max_norm}")
    dev, ptrs, codes, plain = _tensors("grads", grads)
    n, sizes = len(grads), _sizes(grads)
    if out is None:
        out, optrs, ocodes = grads, ptrs, codes
    else:
        if len(out) != n:
            raise ValueError(f"out must have {n} tensors, got {len(out)}")
        _no_tangents("out", out)
        odev, optrs, ocodes, oplain = _tensors("out", out)
        if odev != dev:
            raise ValueError(f"out must be on {dev}")
        same = [t.shape for t in grads] == [o.shape for o in out]
        for i, (t, o) in enumerate(() if same and plain and oplain else zip(grads, out)):
            if o.shape != t.shape or (o.stride() != t.stride() and not (o.is_contiguous() and t.is_contiguous())):
                raise ValueError(f"out[{i}] must have the shape and layout of grads[{i}]")
    if torch.is_grad_enabled() and any([t.requires_grad for t in out]):
        raise ValueError("gradients to be scaled require a gradient themselves: pass p.grad, not p")
    with _on(dev):
        ws, size = _ws(ws, SOP_GRADS, n, 0, 0, dev)
        norm = torch.empty((), dtype=torch.float32, device=dev)
        _check(lib().rlk_clip_grads(_at(ptrs), _at(sizes), _at(codes), n, max_norm, _at(optrs), _at(ocodes),
                                    _ptr(norm), _ptr(ws), size, _stream(dev)),
               "rlk_clip_grads")
    _written(out)
    return norm, out
