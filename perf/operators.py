"""Measured cases of the LM-head operators that go beyond the selected log-probability.

``linear_logp_top``: from bf16 hidden states h [T, H], the LM-head weight W [V, H] and the given tokens
y [T], the given tokens' log-probabilities, the entropy of the whole distribution and the K most likely
alternatives of every row; its backward takes a gradient of the log-probability and one of the entropy.

``linear_distill``: the cross-entropy-like divergence KL(q || p) of a student head's softmax p from a
teacher's distribution q over its K kept tokens (softmax of the kept logits), with its gradient.

``own`` false computes them in elementary torch operations in 32 bits; ``own`` true calls the framework.
"""
import math

import torch

own = False  # set by whoever measures

_V = 151936  # vocabulary of the LM-head workloads of this repository


def _top(name, T, H, V, K, mask=0.0, train=False):
    return {"name": name, "op": "top", "T": T, "H": H, "V": V, "K": K, "mask": mask, "train": train, "tau": 1.0}


def _distill(name, T, H, V, K, mask=0.0, train=True, tau=1.0):
    return {"name": name, "op": "distill", "T": T, "H": H, "V": V, "K": K, "mask": mask, "train": train, "tau": tau}


def listed():
    return [
        # one sequence's next token in serving: the head is read once, latency counts
        _top("top decode 1", 1, 4096, _V, 20),
        # a decoding batch that asks for a few alternatives
        _top("top decode 48", 48, 2048, _V, 8),
        # the log-probabilities of a prompt, with many alternatives
        _top("top prompt 1000", 1000, 4096, _V, 64),
        # a rollout batch scored again by the trainer: padding ignored
        _top("top score 4096", 4096, 4096, _V, 20, mask=0.15),
        # policy gradient with an entropy bonus, a toy head
        _top("top train tiny", 64, 256, 4096, 5, train=True),
        # policy gradient with an entropy bonus on a ragged batch
        _top("top train 1777", 1777, 2048, _V, 1, mask=0.15, train=True),
        # distillation of a toy head
        _distill("distill tiny", 64, 256, 4096, 8),
        # a student's loss on held-out text, softened, on half the vocabulary
        _distill("distill eval 300", 300, 2048, _V // 2, 128, train=False, tau=2.0),
        # one micro-batch of long-context training
        _distill("distill train 257", 257, 4096, _V, 64),
        # an odd vocabulary, softened
        _distill("distill train odd", 1000, 1984, 49999, 100, mask=0.3, tau=1.5),
        # a training batch with padding
        _distill("distill train 4096", 4096, 4096, _V, 64, mask=0.15),
        # the largest: a long packed batch
        _distill("distill train 16384", 16384, 2048, _V, 32, mask=0.15),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["top", "distill"])
    train = rng.random() < 0.5
    T = _log_int(rng, 1, 8192)
    H = 64 * _log_int(rng, 4, 64)
    V = _log_int(rng, 2000, _V)
    K = _log_int(rng, 1, 128)
    mask = rng.choice([0.0, 0.0, 0.15, 0.5])
    tau = 1.0 if op == "top" else rng.choice([1.0, 1.0, 0.7, 2.0, 4.0])
    return {"op": op, "T": T, "H": H, "V": V, "K": K, "mask": mask, "train": train, "tau": tau}


def _grid(x, steps):
    """x on the grid of 1 / steps, at most 127 steps from zero (seven bits and a sign: exact in bf16)."""
    return torch.clamp(torch.round(x * steps), -127, 127) / steps


def _inputs(case, seed):
    """Hidden states and weights of the workloads' spread (h about N(0, 1), W about N(0, 1/sqrt(H))), on dyadic grids
    (h in 1/16, W in 1/16 of its spread): every logit is then exact in 32 bits in whatever order its products are
    summed, so the order of the alternatives is a fact of the inputs, ties and all.  A row leans towards one token by
    0 to 16, so that unsure and confident rows both occur."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T, H, V, K = case["T"], case["H"], case["V"], case["K"]
    dev = {"device": "cuda", "generator": gen}
    steps = 2.0 ** round(math.log2(16.0 * math.sqrt(H)))
    W = _grid(torch.randn(V, H, **dev) / math.sqrt(H), steps).to(torch.bfloat16)
    lean = torch.randint(0, V, (T,), **dev)
    x = torch.randn(T, H, **dev) + 16.0 * torch.rand(T, 1, **dev) * W[lean].float()
    h = _grid(x, 16.0).to(torch.bfloat16)
    off = torch.rand(T, **dev) < case["mask"]
    return gen, h, W, lean, off


def _teacher(case, gen, lean, off):
    """A teacher's K best tokens of every row, best first: distinct ids, the leaning token first, more of them among
    the low ids; log-probabilities that fall off; some rows hold fewer than K, rows off hold none."""
    T, V, K = case["T"], case["V"], case["K"]
    dev = {"device": "cuda", "generator": gen}
    ids = torch.sort((torch.rand(T, K, **dev).double() ** 3 * (V - K)).long(), dim=1).values + torch.arange(K, device="cuda")
    ids = torch.gather(ids, 1, torch.argsort(torch.rand(T, K, **dev), dim=1))
    has = (ids == lean[:, None]).any(dim=1)
    ids[:, 0] = torch.where(has, ids[:, 0], lean)
    falls = -torch.log(torch.rand(T, K, **dev).clamp_min(1e-6)) * 2.0 / torch.arange(1, K + 1, device="cuda")
    logits = -torch.cumsum(falls, dim=1)
    kept = torch.where(torch.rand(T, **dev) < 0.1, torch.randint(1, K + 1, (T,), **dev), K)
    empty = (torch.arange(K, device="cuda")[None, :] >= kept[:, None]) | off[:, None]
    ids = torch.where(empty, -1, ids)
    return ids.to(torch.int32), logits.masked_fill(empty, -math.inf)


def prepare(case, seed):
    gen, h, W, lean, off = _inputs(case, seed)
    s = dict(case, h=h, W=W)
    dev = {"device": "cuda", "generator": gen}
    if case["op"] == "top":
        other = torch.randint(0, case["V"], (case["T"],), **dev)
        y = torch.where(torch.rand(case["T"], **dev) < 0.5, lean, other)
        s["y"] = torch.where(off, -100, y).to(torch.int32)
        s["g_entropy"] = 0.1 * torch.randn(case["T"], **dev)
    else:
        s["ids"], s["logits"] = _teacher(case, gen, lean, off)
    s["g"] = torch.randn(case["T"], **dev)
    return s


def _own(s):
    import selected_token_lm_amd as rlk

    kw = {"grad_W_dtype": torch.bfloat16}
    if s["op"] == "top":
        logp, lse, entropy, top_logp, top_ids = rlk.linear_logp_top_fwd(s["h"], s["W"], s["y"], s["K"])
        out = {"logp": logp, "entropy": entropy, "top_logp": top_logp, "top_ids": top_ids}
        if s["train"]:
            out["grad_h"], out["grad_W"] = rlk.linear_logp_top_bwd(s["h"], s["W"], s["y"], lse, entropy, s["g"], s["g_entropy"], **kw)
    else:
        loss, lse, logp_ids = rlk.linear_distill_fwd(s["h"], s["W"], s["ids"], s["logits"], temperature=s["tau"])
        out = {"loss": loss, "logp_ids": logp_ids}
        if s["train"]:
            out["grad_h"], out["grad_W"] = rlk.linear_distill_bwd(s["h"], s["W"], s["ids"], s["logits"], lse, logp_ids, s["g"], temperature=s["tau"], **kw)
    return out


def _best(z, K):
    """The K largest of every row, ties to the lowest index."""
    bits = (z + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits) * 2 ** 32 + torch.arange(z.shape[1] - 1, -1, -1, device=z.device)
    return z.shape[1] - 1 - (torch.topk(key, K, dim=1).values & 0xFFFFFFFF)


def _plain_top(s):
    h, W, y = s["h"].float(), s["W"].float(), s["y"].long()
    on = y != -100
    z = h @ W.T
    m = z.max(dim=1, keepdim=True).values
    e = torch.exp(z - m)
    total = e.sum(dim=1, keepdim=True)
    lp = z - m - torch.log(total)
    p = e / total
    at = torch.where(on, y, 0)[:, None]
    entropy = -(p * lp).sum(dim=1)
    ids = _best(z, s["K"])
    out = {"logp": torch.where(on, torch.gather(lp, 1, at)[:, 0], 0.0), "entropy": torch.where(on, entropy, 0.0),
           "top_logp": torch.where(on[:, None], torch.gather(lp, 1, ids), -math.inf),
           "top_ids": torch.where(on[:, None], ids, -1).to(torch.int32)}
    if s["train"]:
        g, ge = (torch.where(on, s[n], 0.0)[:, None] for n in ("g", "g_entropy"))
        dz = -p * (g + ge * (lp + entropy[:, None]))
        dz.scatter_add_(1, at, g)
        out["grad_h"], out["grad_W"] = (dz @ W).to(torch.bfloat16), (dz.T @ h).to(torch.bfloat16)
    return out


def _plain_distill(s):
    h, W, ids = s["h"].float(), s["W"].float(), s["ids"].long()
    kept = (ids >= 0) & (s["logits"] > -math.inf)
    on = kept.any(dim=1)
    top = torch.where(kept, s["logits"] / s["tau"], -math.inf)
    top = torch.where(on[:, None], top - top.max(dim=1, keepdim=True).values, 0.0)
    q = torch.where(kept, torch.exp(top), 0.0)
    total = torch.where(on, q.sum(dim=1), 1.0)[:, None]
    log_q = torch.where(kept, top - torch.log(total), 0.0)
    q = q / total
    z = (h @ W.T) / s["tau"]
    m = z.max(dim=1, keepdim=True).values
    e = torch.exp(z - m)
    lse_m = torch.log(e.sum(dim=1, keepdim=True))
    at = torch.where(ids >= 0, ids, 0)
    lp = torch.where(kept, torch.gather(z, 1, at) - m - lse_m, 0.0)
    out = {"loss": (q * (log_q - lp)).sum(dim=1), "logp_ids": torch.where(kept, lp, -math.inf)}
    if s["train"]:
        g = torch.where(on, s["g"] / s["tau"], 0.0)[:, None]
        dz = e * (torch.exp(-lse_m) * g)
        dz.scatter_add_(1, at, -g * q)
        out["grad_h"], out["grad_W"] = (dz @ W).to(torch.bfloat16), (dz.T @ h).to(torch.bfloat16)
    return out


def run(state):
    if own:
        return _own(state)
    return _plain_top(state) if state["op"] == "top" else _plain_distill(state)


def work(case):
    T, H, V, K = case["T"], case["H"], case["V"], case["K"]
    on = max(1.0, T * (1.0 - case["mask"]))
    n = 2.0 * V * H + 2.0 * T * H + (T * (4 + 8) + T * K * 8 if case["op"] == "top" else T * 4 + T * K * 12)
    if case["train"]:  # the two gradients, and the upstream ones
        n += 2.0 * V * H + 2.0 * T * H + T * (8 if case["op"] == "top" else 4)
    return {"bytes": n, "flops": 2.0 * on * H * V * (3 if case["train"] else 1)}


def exact(case, seed):
    """The definitions in 64 bits, a block of rows at a time: log p = log softmax(h W^T / tau), the gradients by
    the chain rule dL/dz_v = sum_u dL/dlog p_u ([u = v] - p_v)."""
    s = prepare(case, seed)
    T, H, V, K, tau = (case[n] for n in ("T", "H", "V", "K", "tau"))
    h, W = s["h"].double(), s["W"].double()
    out, grad_h = [], torch.zeros_like(h)
    grad_W = torch.zeros_like(W) if case["train"] else None
    for a in range(0, T, 2048):
        rows = slice(a, min(T, a + 2048))
        logp = torch.log_softmax(h[rows] @ W.T / tau, dim=1)
        if case["op"] == "top":
            y = s["y"][rows].long()
            live = (y != -100).double()
            ent = -(logp.exp() * logp).sum(dim=1)
            order = torch.sort(logp, dim=1, descending=True, stable=True).indices[:, :K]
            sel = logp.gather(1, y.clamp_min(0)[:, None])[:, 0]
            none = live == 0
            out.append((sel * live, ent * live, logp.gather(1, order).masked_fill(none[:, None], -math.inf), order.int().masked_fill(none[:, None], -1)))
            if case["train"]:
                # d entropy / d log p_v = -p_v (log p_v + 1), d logp / d log p_v = [v = y]
                up = -(s["g_entropy"][rows].double() * live)[:, None] * logp.exp() * (logp + 1)
                up.scatter_add_(1, y.clamp_min(0)[:, None], (s["g"][rows].double() * live)[:, None])
        else:
            ids, t = s["ids"][rows].long(), s["logits"][rows].double() / tau
            t = t.masked_fill(ids < 0, -math.inf)
            live = torch.isfinite(t).any(dim=1)
            q = torch.nan_to_num(torch.softmax(t, dim=1))
            lp = logp.gather(1, ids.clamp_min(0))
            out.append(((torch.xlogy(q, q) - q * lp).sum(dim=1), lp.masked_fill(~torch.isfinite(t), -math.inf)))
            if case["train"]:
                up = torch.zeros_like(logp).scatter_add_(1, ids.clamp_min(0), -q * (s["g"][rows].double() * live)[:, None])
        if case["train"]:
            dz = (up - logp.exp_() * up.sum(dim=1, keepdim=True)) / tau
            grad_h[rows] = dz @ W
            grad_W.addmm_(dz.T, h[rows])
    names = ("logp", "entropy", "top_logp", "top_ids") if case["op"] == "top" else ("loss", "logp_ids")
    out = {n: torch.cat(v) for n, v in zip(names, zip(*out))}
    return dict(out, grad_h=grad_h, grad_W=grad_W) if case["train"] else out
