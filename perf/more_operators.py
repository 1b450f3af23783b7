"""What the operators for fine-tuning a draft on its target are measured on.

Four operators, each in its plain form (elementary torch operations in 32
bits, 64 where noted, rounded once at the end) and as this package's calls:

  top      top_logits: the largest logits of each row with their tokens, and
           the row's log-sum-exp: what is kept of a target's logits
  distill  distill_loss: divergence of a draft from its target's top logits,
           with the gradient of the draft's logits
  layer    layer_norm: layer norm with the residual's addition
  back     layer_norm_backward, rms_norm_backward: gradients of the norms'
           inputs and of their weights

``listed()`` names the cases that are timed; ``draw`` gives more of the same
ranges.
"""
from __future__ import annotations

import math

import torch

own = False

E4M3_MAX = 448.0
FLT_MIN = 2.0 ** -126
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}


# ---------------------------------------------------------------- the cases

def _top(name, rows, V, k, dtype, T=1.0):
    return {"name": name, "op": "top", "rows": rows, "V": V, "k": k, "dtype": dtype, "T": T}


def _distill(name, rows, V, k, dtype, T, rest, loss=True, grad=True, pad=False, short=False):
    """rest: the teacher's log-sum-exp is given, and what its list leaves is one more outcome; pad: an eighth of the
    rows has weight 0; short: lists of k / 2 to k entries."""
    return {"name": name, "op": "distill", "rows": rows, "V": V, "k": k, "dtype": dtype, "T": T, "rest": rest,
            "loss": loss, "grad": grad, "pad": pad, "short": short}


def _layer(name, rows, d, dtype, residual, out, affine=True):
    return {"name": name, "op": "layer", "rows": rows, "d": d, "dtype": dtype, "residual": residual, "out": out,
            "affine": affine}


def _back(name, norm, rows, d, dtype, residual, params=True):
    """residual: a gradient arrives at the norm's input from the residual stream too; params: the weights' gradients
    are wanted (not where the norms are frozen)."""
    return {"name": name, "op": "back", "norm": norm, "rows": rows, "d": d, "dtype": dtype, "residual": residual,
            "params": params}


def listed():
    return [
        # the positions of one sequence's round, with the log-probabilities a user asked for: latency
        _top("top-7x128256-k20-bf16", 7, 128256, 20, "bf16"),
        # the target rows of the headline round, kept for the draft's training
        _top("top-448x128256-k64-bf16", 448, 128256, 64, "bf16"),
        # the target rows of the widest round, long lists
        _top("top-2304x152064-k256-f32", 2304, 152064, 256, "f32", 2.0),
        # a short sequence and a small vocabulary: latency
        _distill("distill-16x32000-k8-f32", 16, 32000, 8, "f32", 2.0, False),
        # a training step on the headline round's rows
        _distill("distill-448x128256-k64-bf16", 448, 128256, 64, "bf16", 1.0, True, pad=True),
        # evaluation: the loss alone, rows that start at any 2 bytes, lists of unlike length
        _distill("distill-777x24979-k33-bf16-eval", 777, 24979, 33, "bf16", 1.5, True, grad=False, short=True),
        # a training step on the widest round's rows
        _distill("distill-2304x152064-k256-f32", 2304, 152064, 256, "f32", 1.0, True),
        # one decoded token: latency
        _layer("layer-1x4096-bf16", 1, 4096, "bf16", False, "bf16"),
        # a long prompt's rows
        _layer("layer-16384x8192-bf16", 16384, 8192, "bf16", True, "bf16"),
        # the draft's last norm in a training step on the headline round's rows
        _back("layer-backward-448x4096-bf16", "layer", 448, 4096, "bf16", False),
        # a long sequence, with the residual stream's gradient
        _back("layer-backward-16384x8192-bf16", "layer", 16384, 8192, "bf16", True),
        # odd sizes in float32
        _back("rms-backward-1557x5001-f32", "rms", 1557, 5001, "f32", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["top", "distill", "distill", "layer", "back"])
    if op in ("top", "distill"):
        V = _log(rng, 1000, 152064)
        if rng.random() < 0.5:
            V = max(1000, V // 64 * 64)
        k = _log(rng, 1, 256)
        rows = _log(rng, 1, min(16384, 2304 * 152064 // (2 * V)))
        dtype, T = rng.choice(["bf16", "f32"]), rng.choice([0.7, 1.0, 2.0])
        if op == "top":
            c = _top("", rows, V, k, dtype, T)
        else:
            loss, grad = rng.choice([(True, True), (True, True), (True, False), (False, True)])
            c = _distill("", rows, V, k, dtype, T, rng.random() < 0.6, loss, grad, rng.random() < 0.3, rng.random() < 0.3)
    else:
        d = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            d = max(64, d // 64 * 64)
        rows = _log(rng, 1, min(16384, 16384 * 8192 // (2 * d)))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if op == "layer":
            c = _layer("", rows, d, dtype, rng.random() < 0.7, rng.choice(["bf16", "f32", "e4m3"]), rng.random() < 0.8)
        else:
            c = _back("", rng.choice(["layer", "rms"]), rows, d, dtype, rng.random() < 0.5, rng.random() < 0.8)
    del c["name"]
    return c


def _live(c):
    return c["rows"] - c["rows"] // 8 if c["pad"] else c["rows"]


def work(c):
    b = BYTES[c["dtype"]]
    if c["op"] == "top":
        n = c["rows"] * c["V"]
        return {"bytes": n * b + c["rows"] * (8 * c["k"] + 4), "flops": 4 * n}
    if c["op"] == "distill":
        n = _live(c) * c["V"]
        by = n * b + _live(c) * 8 * c["k"] + c["rows"] * (8 if c["rest"] else 4)
        by += (4 * c["rows"] if c["loss"] else 0) + (c["rows"] * c["V"] * b if c["grad"] else 0)
        return {"bytes": by, "flops": (8 if c["grad"] else 4) * n}
    n = c["rows"] * c["d"]
    if c["op"] == "layer":
        by = n * (b + BYTES[c["out"]] + (2 * b if c["residual"] else 0)) + (2 * c["d"] * b if c["affine"] else 0)
        by += 4 * c["rows"] if c["out"] == "e4m3" else 0
        return {"bytes": by, "flops": 8 * n}
    by = n * b * (4 if c["residual"] else 3) + c["d"] * b
    if c["params"]:
        by += c["d"] * (8 if c["norm"] == "layer" else 4)
    return {"bytes": by, "flops": 16 * n}


# --------------------------------------------------------------- the inputs

def _rows_of_logits(g, rows, V):
    """Long-tailed rows: the logarithm of a token's frequency, common to all rows, and the context's share."""
    rank = torch.randperm(V, device="cuda", generator=g).float().add_(1)
    return torch.randn((rows, V), device="cuda", generator=g).mul_(1.5).sub_(3 * rank.log10())


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"c": c}
    t = DTYPES[c["dtype"]]
    rows = c["rows"]
    if c["op"] == "top":
        s["logits"] = _rows_of_logits(g, rows, c["V"]).to(t)
        return s
    if c["op"] == "distill":
        V, k, T = c["V"], c["k"], c["T"]
        teacher = _rows_of_logits(g, rows, V)
        top, index = teacher.topk(k, 1)
        s["top_index"], s["top_values"], s["top_lse"] = index.to(torch.int32), top, None
        if c["rest"]:
            s["top_lse"] = torch.empty((rows,), device="cuda")
            for r in range(0, rows, 256):
                s["top_lse"][r:r + 256] = (teacher[r:r + 256] / T).logsumexp(1)
        if c["short"]:
            n = torch.randint((k + 1) // 2, k + 1, (rows, 1), device="cuda", generator=g)
            absent = torch.arange(k, device="cuda")[None, :] >= n
            s["top_index"].masked_fill_(absent, -1)
            s["top_values"].masked_fill_(absent, -math.inf)
        # a draft that has learnt most of it: the teacher's logits, perturbed
        s["logits"] = teacher.add_(torch.randn((rows, V), device="cuda", generator=g).mul_(0.7)).to(t)
        s["weight"] = torch.full((rows,), 1.0 / _live(c), device="cuda")
        if c["pad"]:
            s["weight"][torch.randperm(rows, device="cuda", generator=g)[:rows - _live(c)]] = 0.0
        return s
    d = c["d"]
    # hidden states of unlike magnitude and away from zero: a spread of a factor of ten between rows
    size = torch.rand((rows, 1), device="cuda", generator=g).mul_(2.3).exp_()

    def hidden():
        return torch.randn((rows, d), device="cuda", generator=g).add_(0.3).mul_(size).to(t)

    s["x"] = hidden()
    s["weight"] = (1.0 + 0.2 * torch.randn((d,), device="cuda", generator=g)).to(t)
    s["eps"] = 1e-5
    if c["op"] == "layer":
        s["bias"] = (0.2 * torch.randn((d,), device="cuda", generator=g)).to(t)
        if not c["affine"]:
            s["weight"] = s["bias"] = None
        s["residual"] = hidden() if c["residual"] else None
    else:
        s["grad"] = torch.randn((rows, d), device="cuda", generator=g).mul_(0.01).to(t)
        s["grad_residual"] = None
        if c["residual"]:
            s["grad_residual"] = torch.randn((rows, d), device="cuda", generator=g).mul_(0.01).to(t)
    return s


# ----------------------------------------------------- the operators, plain

def _plain_top(s):
    c = s["c"]
    x = s["logits"].float()
    # order: the value, then the lower token first, as one whole number
    bits = (x + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * 2 ** 32
    key += torch.arange(c["V"] - 1, -1, -1, device="cuda")
    index = c["V"] - 1 - (key.topk(c["k"], 1).values & 0xFFFFFFFF)
    m = x.amax(1, keepdim=True)
    lse = (m / c["T"]).squeeze(1) + ((x - m) / c["T"]).exp().sum(1).log()
    return {"values": x.gather(1, index), "index": index.to(torch.int32), "lse": lse}


def _plain_distill(s):
    c = s["c"]
    V, T = c["V"], c["T"]
    here = s["top_index"] >= 0
    index = s["top_index"].long().clamp_min(0)
    # the lists are short, and what they leave is a difference of numbers close to each other: 64 bits
    t = (s["top_values"].double() / T).masked_fill(~here, -math.inf)
    if c["rest"]:
        p = (t - s["top_lse"].double()[:, None]).exp()
        r = (1 - p.sum(1)).clamp_min(0)
    else:
        p = (t - t.amax(1, keepdim=True)).exp()
        p = p / p.sum(1, keepdim=True)
        r = torch.zeros_like(p[:, 0])
    x = s["logits"].float()
    taken = torch.zeros((c["rows"], V + 1), device="cuda", dtype=torch.bool)
    taken.scatter_(1, torch.where(here, index, V), True)
    top = x.gather(1, index).double().div(T).masked_fill(~here, -math.inf)
    x = x.masked_fill(taken[:, :V], -math.inf)
    m = x.amax(1, keepdim=True)
    e = ((x - m) / T).exp()
    total = e.sum(1)
    rest = m.squeeze(1).double() / T + total.double().log()
    lse = torch.logaddexp(rest, top.logsumexp(1))
    out = {}
    if c["loss"]:
        loss = torch.where(p > 0, p * (p.log() - (top - lse[:, None])), 0.0).sum(1)
        loss += torch.where(r > 0, r * (r.log() - (rest - lse)), 0.0)
        out["loss"] = (s["weight"] * loss).float()
    if c["grad"]:
        scale = s["weight"].double() / T
        g = e * (scale * ((rest - lse).exp() - r) / total.double()).float()[:, None]
        at = scale[:, None] * ((top - lse[:, None]).exp() - p)
        g.scatter_add_(1, index, torch.where(here, at, 0.0).float())
        out["grad"] = g.to(s["logits"].dtype)
    return out


def _plain_layer(s):
    c = s["c"]
    h = s["x"].float()
    r = None
    if c["residual"]:
        h = h + s["residual"].float()
        r = h.to(s["x"].dtype)
    h = h - h.mean(1, keepdim=True)
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + s["eps"])
    if c["affine"]:
        y = y * s["weight"].float() + s["bias"].float()
    if c["out"] != "e4m3":
        return {"out": y.to(DTYPES[c["out"]]), "residual": r}
    scale = (y.abs().amax(1) / E4M3_MAX).clamp_min(FLT_MIN)
    q = (y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return {"out": q, "scale": scale, "residual": r}


def _plain_back(s):
    c = s["c"]
    h, dy = s["x"].float(), s["grad"].float()
    if c["norm"] == "layer":
        h = h - h.mean(1, keepdim=True)
    rs = torch.rsqrt(h.square().mean(1, keepdim=True) + s["eps"])
    xh = h * rs
    g = dy * s["weight"].float()
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if c["norm"] == "layer":
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * rs
    if c["residual"]:
        dx = dx + s["grad_residual"].float()
    out = {"grad_x": dx.to(s["x"].dtype)}
    if c["params"]:
        out["grad_weight"] = (dy * xh).sum(0)
        if c["norm"] == "layer":
            out["grad_bias"] = dy.sum(0)
    return out


def run(s):
    c = s["c"]
    if not own:
        return {"top": _plain_top, "distill": _plain_distill, "layer": _plain_layer, "back": _plain_back}[c["op"]](s)
    import rejection_sampling_verify_09_amd as sv

    if c["op"] == "top":
        values, index, lse = sv.top_logits(s["logits"], c["k"], temperature=c["T"])
        return {"values": values, "index": index, "lse": lse}
    if c["op"] == "distill":
        loss, grad = sv.distill_loss(s["logits"], s["top_index"], s["top_values"], top_lse=s["top_lse"],
                                     temperature=c["T"], weight=s["weight"], with_loss=c["loss"], with_grad=c["grad"])
        return {k: v for k, v in (("loss", loss), ("grad", grad)) if v is not None}
    if c["op"] == "layer":
        y, scale, r = sv.layer_norm(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=s["eps"],
                                    out_dtype=DTYPES[c["out"]])
        if c["out"] == "e4m3":
            return {"out": y, "scale": scale, "residual": r}
        return {"out": y, "residual": r}
    if c["norm"] == "layer":
        dx, dw, db = sv.layer_norm_backward(s["grad"], s["x"], s["weight"], grad_residual=s["grad_residual"],
                                            eps=s["eps"], with_weight=c["params"], with_bias=c["params"])
        return {"grad_x": dx, "grad_weight": dw, "grad_bias": db} if c["params"] else {"grad_x": dx}
    dx, dw = sv.rms_norm_backward(s["grad"], s["x"], s["weight"], grad_residual=s["grad_residual"], eps=s["eps"],
                                  with_weight=c["params"])
    return {"grad_x": dx, "grad_weight": dw} if c["params"] else {"grad_x": dx}


# --------------------------------------------- the definitions, in 64 bits

def _exact_top(c, s):
    values, index, lse = [], [], []
    for x in s["logits"].split(64):
        x = x.double()
        v, i = x.sort(dim=1, descending=True, stable=True)
        values.append(v[:, :c["k"]].clone())
        index.append(i[:, :c["k"]].to(torch.int32))
        lse.append(torch.logsumexp(x / c["T"], 1))
    return {"values": torch.cat(values), "index": torch.cat(index), "lse": torch.cat(lse)}


def _exact_distill(c, s):
    """Row by row a divergence between two distributions over the list and the rest; its gradient by differentiation."""
    losses, grads = [], []
    for r in range(0, c["rows"], 64):
        at = slice(r, r + 64)
        x = s["logits"][at].double().requires_grad_(c["grad"])
        i, t = s["top_index"][at].long(), s["top_values"][at].double() / c["T"]
        here = i >= 0
        t = torch.where(here, t, -math.inf)
        if c["rest"]:
            logp = t - s["top_lse"][at].double()[:, None]
            left = 1 - logp.exp().sum(1)
        else:
            logp = torch.log_softmax(t, 1)
            left = torch.zeros_like(t[:, 0])
        left = left.clamp_min(0)
        logq = torch.log_softmax(x / c["T"], 1)
        outside = torch.ones_like(x, dtype=torch.bool)
        n = here.nonzero()
        outside[n[:, 0], i[n[:, 0], n[:, 1]]] = False
        p = torch.where(here, logp.exp(), 0.0)
        cross = (p * torch.where(here, logq.gather(1, i.clamp_min(0)), 0.0)).sum(1)
        log_rest = torch.logsumexp(logq.masked_fill(~outside, -math.inf), 1)
        loss = torch.special.xlogy(p, p).sum(1) + torch.special.xlogy(left, left) - cross - left * log_rest
        loss = loss * s["weight"][at].double()
        if c["grad"]:
            grads.append(torch.autograd.grad(loss.sum(), x)[0])
        losses.append(loss.detach())
    out = {}
    if c["loss"]:
        out["loss"] = torch.cat(losses)
    if c["grad"]:
        out["grad"] = torch.cat(grads)
    return out


def _norm64(h, eps, center):
    if center:
        h = h - h.sum(1, keepdim=True) / h.shape[1]
    return h / (torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / h.shape[1] + eps) ** 0.5


def _exact_layer(c, s):
    h = s["x"].double() + (s["residual"].double() if c["residual"] else 0.0)
    y = _norm64(h, s["eps"], True)
    if c["affine"]:
        y = y * s["weight"].double() + s["bias"].double()
    r = {"out": y, "residual": h if c["residual"] else None}
    if c["out"] == "e4m3":
        scale = torch.maximum(y.abs().max(1).values / E4M3_MAX, torch.full_like(y[:, 0], FLT_MIN))
        v = y / scale[:, None]
        # steps of e4m3: 2^-3 of the power of two below, at least 2^-9
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
        r["out"] = (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
        r["scale"] = scale
    return r


def _exact_back(c, s):
    """By differentiation of the norm itself, a part of the rows at a time."""
    w = s["weight"].double().requires_grad_()
    b = torch.zeros_like(w).requires_grad_()
    dx, dw, db = [], 0.0, 0.0
    for at in torch.arange(c["rows"], device="cuda").split(2048):
        h = s["x"][at].double().requires_grad_()
        y = _norm64(h, s["eps"], c["norm"] == "layer") * w + b
        gh, gw, gb = torch.autograd.grad(y, (h, w, b), s["grad"][at].double())
        dx.append(gh + s["grad_residual"][at].double() if c["residual"] else gh)
        dw, db = dw + gw, db + gb
    out = {"grad_x": torch.cat(dx)}
    if c["params"]:
        out["grad_weight"] = dw
        if c["norm"] == "layer":
            out["grad_bias"] = db
    return out


def exact(c, seed):
    s = prepare(c, seed)
    return {"top": _exact_top, "distill": _exact_distill, "layer": _exact_layer, "back": _exact_back}[c["op"]](c, s)
