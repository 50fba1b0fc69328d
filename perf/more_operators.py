"""Measured cases of the operators that stand before and behind the LM head in a training step.

``rms_norm`` and ``layer_norm``: the norm that makes the hidden states, forward and backward, with the weight's (and
bias's) gradient summed over the rows.

``embed``: the lookup of token embeddings with a scale, and its gradient: dense, or added to a gradient that is there
(the LM head's, where the two weights are tied).

``grad_norm`` and ``clip_grads``: the norm of all gradients of a step, and their scaling to a largest norm.

``own`` false computes them in elementary torch operations in 32 bits; ``own`` true calls the framework.
"""
import math

import torch

own = False  # set by whoever measures

_V = 151936  # vocabulary of the LM-head workloads of this repository
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}


def _norm(name, op, T, H, x="bf16", y="bf16", w="bf16", train=True):
    return {"name": name, "op": op, "T": T, "H": H, "x_type": x, "y_type": y, "w_type": w, "train": train}


def _embed(name, T, H, V, mask=0.0, grad="bf16", tied=False, train=True):
    return {"name": name, "op": "embed", "T": T, "H": H, "V": V, "mask": mask, "grad": grad, "tied": tied,
            "train": train}


def _grads(name, op, rows, H, mats, vecs, type="f32", out="f32", most=1.0):
    return {"name": name, "op": op, "rows": rows, "H": H, "mats": mats, "vecs": vecs, "type": type, "out_type": out,
            "most": most}


def listed():
    return [
        # one sequence's next token in serving: latency counts
        _norm("rms decode 1", "rms", 1, 4096, train=False),
        # a training batch of the Qwen3-8B shape
        _norm("rms train 4096", "rms", 4096, 4096),
        # a ragged batch of an odd width, kept in 32 bits
        _norm("layer train odd", "layer", 1777, 1999, x="f32", y="f32", w="f32"),
        # a long packed batch: the residual stream in 32 bits, the head's input in bf16
        _norm("layer train 16384", "layer", 16384, 2048, x="f32", w="f32"),
        # a decoding batch
        _embed("embed decode 48", 48, 2048, _V, train=False),
        # a toy model's step
        _embed("embed train tiny", 64, 256, 4096, grad="f32"),
        # a training batch with padding: the table's whole gradient is written
        _embed("embed train 4096", 4096, 4096, _V, mask=0.15),
        # tied weights, a long packed batch: added to the head's gradient
        _embed("embed tied 16384", 16384, 2048, _V, mask=0.15, grad="f32", tied=True),
        # a toy model's gradients, watched in training
        _grads("norm tiny", "norm", 4096, 256, 16, 9),
        # the head's gradient as its backward leaves it
        _grads("norm head", "norm", _V, 4096, 0, 2),
        # a toy model's step, gradients below the limit
        _grads("clip tiny", "clip", 4096, 256, 16, 9, most=10.0),
        # a step's gradients in 32 bits, clipped into those of the weights' type
        _grads("clip step", "clip", _V, 2048, 24, 49, out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rms", "layer", "embed", "norm", "clip"])
    kind = lambda: rng.choice(["bf16", "f32"])  # noqa: E731
    if op in ("rms", "layer"):
        T, H = _log_int(rng, 1, 16384), _log_int(rng, 64, 8192)
        H = min(H, 2 ** 25 // T)
        return {"op": op, "T": T, "H": H, "x_type": kind(), "y_type": kind(), "w_type": kind(), "train": rng.random() < 0.7}
    if op == "embed":
        H = rng.choice([64 * _log_int(rng, 2, 32), _log_int(rng, 100, 2048)])
        return {"op": op, "T": _log_int(rng, 1, 16384), "H": H, "V": _log_int(rng, 1000, _V),
                "mask": rng.choice([0.0, 0.15, 0.5]), "grad": kind(), "tied": rng.random() < 0.4,
                "train": rng.random() < 0.7}
    return {"op": op, "rows": _log_int(rng, 500, _V), "H": _log_int(rng, 64, 2048), "mats": rng.randint(0, 24),
            "vecs": rng.randint(1, 200), "type": kind(), "out_type": kind(), "most": rng.choice([0.1, 1.0, 10.0])}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = {"device": "cuda", "generator": gen}
    s = dict(case)
    if case["op"] in ("rms", "layer"):
        # a residual stream: rows of various sizes and means, a few columns much larger than the others
        T, H = case["T"], case["H"]
        spread = torch.exp(0.7 * torch.randn(T, 1, **dev))
        x = spread * (torch.randn(T, H, **dev) + 0.5 * torch.randn(T, 1, **dev))
        x *= torch.where(torch.rand(H, **dev) < 0.005, 20.0, 1.0)
        s["x"], s["eps"] = x.to(_TYPES[case["x_type"]]), 1e-6
        s["weight"] = (1.0 + 0.2 * torch.randn(H, **dev)).to(_TYPES[case["w_type"]])
        s["bias"] = (0.1 * torch.randn(H, **dev)).to(_TYPES[case["w_type"]]) if case["op"] == "layer" else None
        if case["train"]:
            s["g"] = torch.randn(T, H, **dev).to(_TYPES[case["y_type"]])
    elif case["op"] == "embed":
        # text: the few frequent tokens are a large part of it, most tokens occur once or never
        T, H, V = case["T"], case["H"], case["V"]
        rank = torch.floor(torch.exp(torch.rand(T, **dev).double() * math.log(V))).long().clamp(1, V) - 1
        ids = (rank * 40503 + 12345) % V
        s["ids"] = torch.where(torch.rand(T, **dev) < case["mask"], -100, ids)
        s["E"] = torch.randn(V, H, **dev).to(torch.bfloat16)
        s["scale"] = math.sqrt(H)
        if case["train"]:
            s["g"] = torch.randn(T, H, **dev).to(torch.bfloat16)
            if case["tied"]:
                s["grad_E"] = torch.randn(V, H, **dev).to(_TYPES[case["grad"]])
    else:
        # matrices whose gradients differ in size, and vectors
        H = case["H"]
        shapes = [(case["rows"], H)] + [(H, H)] * case["mats"] + [(H,)] * case["vecs"]
        s["grads"] = [(1e-3 * 2.0 ** (i % 5) * torch.randn(*n, **dev)).to(_TYPES[case["type"]])
                      for i, n in enumerate(shapes)]
        if case["op"] == "clip":
            # one buffer, as an optimizer or a reduction over ranks keeps it
            sizes = [math.prod(n) for n in shapes]
            s["flat"] = torch.empty(sum(sizes), dtype=_TYPES[case["out_type"]], device="cuda")
            s["out"] = [v.view(n) for v, n in zip(s["flat"].split(sizes), shapes)]
    return s


def _own(s):
    import selected_token_lm_amd as rlk

    if s["op"] == "rms":
        if not s["train"]:
            return {"y": rlk.rms_norm(s["x"], s["weight"], s["eps"], out_dtype=_TYPES[s["y_type"]])}
        y, rstd = rlk.rms_norm_fwd(s["x"], s["weight"], s["eps"], out_dtype=_TYPES[s["y_type"]])
        gx, gw = rlk.rms_norm_bwd(s["x"], s["weight"], rstd, s["g"], grad_weight_dtype=_TYPES[s["w_type"]])
        return {"y": y, "grad_x": gx, "grad_weight": gw}
    if s["op"] == "layer":
        if not s["train"]:
            return {"y": rlk.layer_norm(s["x"], s["weight"], s["bias"], s["eps"], out_dtype=_TYPES[s["y_type"]])}
        y, mean, rstd = rlk.layer_norm_fwd(s["x"], s["weight"], s["bias"], s["eps"], out_dtype=_TYPES[s["y_type"]])
        gx, gw, gb = rlk.layer_norm_bwd(s["x"], s["weight"], mean, rstd, s["g"], grad_weight_dtype=_TYPES[s["w_type"]])
        return {"y": y, "grad_x": gx, "grad_weight": gw, "grad_bias": gb}
    if s["op"] == "embed":
        out = {"out": rlk.embed_fwd(s["ids"], s["E"], s["scale"])}
        if s["train"]:
            out["grad_E"] = rlk.embed_bwd(s["ids"], s["g"], s["V"], s["scale"], grad_E_dtype=_TYPES[s["grad"]],
                                          grad_E=s.get("grad_E"))
        return out
    if s["op"] == "norm":
        return {"norm": rlk.grad_norm(s["grads"])}
    norm, _ = rlk.clip_grads(s["grads"], s["most"], out=s["out"])
    return {"norm": norm, "out": s["flat"]}


def _plain_norm(s):
    x, w = s["x"].float(), s["weight"].float()
    mean = x.mean(dim=1, keepdim=True) if s["op"] == "layer" else 0.0
    centred = x - mean
    rstd = torch.rsqrt((centred * centred).mean(dim=1, keepdim=True) + s["eps"])
    n = centred * rstd
    y = n * w
    if s["op"] == "layer":
        y = y + s["bias"].float()
    out = {"y": y.to(_TYPES[s["y_type"]])}
    if s["train"]:
        g = s["g"].float()
        gw = g * w
        grad = gw - n * (gw * n).mean(dim=1, keepdim=True)
        if s["op"] == "layer":
            grad = grad - gw.mean(dim=1, keepdim=True)
        out["grad_x"] = (rstd * grad).to(_TYPES[s["x_type"]])
        out["grad_weight"] = (g * n).sum(dim=0).to(_TYPES[s["w_type"]])
        if s["op"] == "layer":
            out["grad_bias"] = g.sum(dim=0).to(_TYPES[s["w_type"]])
    return out


def _plain_embed(s):
    on = (s["ids"] != -100)[:, None]
    at = torch.where(on[:, 0], s["ids"], 0)
    out = {"out": torch.where(on, s["E"][at].float() * s["scale"], 0.0).to(torch.bfloat16)}
    if s["train"]:
        g = torch.where(on, s["g"].float() * s["scale"], 0.0)
        if s["tied"] and s["grad"] == "f32":
            out["grad_E"] = s["grad_E"].index_add_(0, at, g)
        elif s["tied"]:
            # what is added up in 32 bits and rounded once, into the gradient that is there
            out["grad_E"] = s["grad_E"].copy_(s["grad_E"].float().index_add_(0, at, g))
        else:
            grad = torch.zeros(s["V"], s["H"], device=g.device).index_add_(0, at, g)
            out["grad_E"] = grad.to(_TYPES[s["grad"]])
    return out


def _plain_grads(s):
    squares = [(t.float() * t.float()).sum() for t in s["grads"]]
    norm = torch.sqrt(torch.stack(squares).sum())
    if s["op"] == "norm":
        return {"norm": norm}
    c = torch.where(norm > s["most"], s["most"] / norm, 1.0)
    for t, o in zip(s["grads"], s["out"]):
        o.copy_(t.float() * c)
    return {"norm": norm, "out": s["flat"]}


def run(state):
    if own:
        return _own(state)
    if state["op"] in ("rms", "layer"):
        return _plain_norm(state)
    return _plain_embed(state) if state["op"] == "embed" else _plain_grads(state)


def work(case):
    if case["op"] in ("rms", "layer"):
        T, H, xb, yb, wb = case["T"], case["H"], _BYTES[case["x_type"]], _BYTES[case["y_type"]], _BYTES[case["w_type"]]
        vectors = 2 if case["op"] == "layer" else 1
        n, ops = T * H * (xb + yb) + vectors * H * wb, (8 if case["op"] == "layer" else 5)
        if case["train"]:  # x and g read, grad_x written; the weight read again, its gradient written
            n += T * H * (2 * xb + yb) + H * wb + vectors * H * wb
            ops += 16 if case["op"] == "layer" else 12
        return {"bytes": float(n), "flops": float(ops) * T * H}
    if case["op"] == "embed":
        T, H, V, on = case["T"], case["H"], case["V"], max(1.0, case["T"] * (1.0 - case["mask"]))
        # distinct tokens of n draws whose probability falls as one over the rank
        distinct = sum(k * (1.0 - (1.0 - math.log1p(1.0 / r) / math.log(V)) ** on)
                       for r, k in ((1.41 * 2 ** i, min(2 ** i, V - 2 ** i + 1)) for i in range(V.bit_length())))
        distinct = min(distinct, on)
        n = 8.0 * T + distinct * H * 2 + T * H * 2
        if case["train"]:
            n += on * H * 2 + _BYTES[case["grad"]] * H * (2 * distinct if case["tied"] else V)
        return {"bytes": n, "flops": (2.0 if case["train"] else 1.0) * on * H}
    n = case["rows"] * case["H"] + case["mats"] * case["H"] ** 2 + case["vecs"] * case["H"]
    if case["op"] == "norm":
        return {"bytes": float(n * _BYTES[case["type"]] + 4), "flops": 2.0 * n}
    # the gradients are read again once their norm is known
    return {"bytes": float(n * (2 * _BYTES[case["type"]] + _BYTES[case["out_type"]]) + 4), "flops": 3.0 * n}


def exact(case, seed):
    """The definitions in 64 bits; gradients of the norms by differentiation, of the embedding as a sum over tokens."""
    s = prepare(case, seed)
    if case["op"] in ("rms", "layer"):
        leaves = [s["x"].double().requires_grad_(), s["weight"].double().requires_grad_()]
        if case["op"] == "layer":
            leaves.append(s["bias"].double().requires_grad_())
            var, mean = torch.var_mean(leaves[0], dim=1, keepdim=True, correction=0)
            y = (leaves[0] - mean) / torch.sqrt(var + s["eps"]) * leaves[1] + leaves[2]
        else:
            y = leaves[0] / torch.sqrt(leaves[0].pow(2).mean(dim=1, keepdim=True) + s["eps"]) * leaves[1]
        out = {"y": y.detach()}
        if case["train"]:
            names = ("grad_x", "grad_weight", "grad_bias")
            out.update(zip(names, torch.autograd.grad(y, leaves, s["g"].double())))
        return out
    if case["op"] == "embed":
        live = torch.nonzero(s["ids"] >= 0)[:, 0]
        at = s["ids"][live]
        out = torch.zeros(case["T"], case["H"], dtype=torch.float64, device="cuda")
        out[live] = s["E"][at].double() * s["scale"]
        res = {"out": out}
        if case["train"]:
            base = s["grad_E"].double() if case["tied"] else torch.zeros(case["V"], case["H"], dtype=torch.float64, device="cuda")
            token, which = torch.unique(at, return_inverse=True)
            sums = torch.zeros(len(token), case["H"], dtype=torch.float64, device="cuda")
            sums.index_put_((which,), s["g"][live].double(), accumulate=True)
            base[token] += s["scale"] * sums
            res["grad_E"] = base
        return res
    total = sum(float(torch.linalg.vector_norm(t, dtype=torch.float64)) ** 2 for t in s["grads"])
    norm = torch.tensor(math.sqrt(total), dtype=torch.float64, device="cuda")
    if case["op"] == "norm":
        return {"norm": norm}
    c = min(1.0, case["most"] / math.sqrt(total))
    return {"norm": norm, "out": torch.cat([t.flatten().double() * c for t in s["grads"]])}
