"""What the operators between a model's last layer and the verification are measured on.

Three operators, each in its plain form (elementary torch operations in 32
bits, rounded once at the end) and as this package's calls:

  norm    rms_norm: root-mean-square norm with the residual's addition; output
          in bfloat16, float32 or 8 bits (e4m3) with one scale a row
  linear  linear: matrix product with bias, activation and residual in its
          epilogue, bfloat16 or e4m3 operands (draft heads, projections)
  adjust  adjust_logits: penalties for repeated tokens, biases and grammar
          masks on the logits of every position of a verification round

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

def _norm(name, rows, d, dtype, residual, out):
    return {"name": name, "op": "norm", "rows": rows, "d": d, "dtype": dtype, "residual": residual, "out": out}


def _linear(name, M, N, K, dtype, out, act, bias, res_cols):
    """res_cols: columns of the residual (0: none); output column n adds its column n mod res_cols."""
    return {"name": name, "op": "linear", "M": M, "N": N, "K": K, "dtype": dtype, "out": out, "act": act,
            "bias": bias, "res_cols": res_cols}


def _adjust(name, B, K, V, dtype, form, hist, penalties, nbias, mask, inplace=False):
    """form: the rows each sequence has: "target" (K + 1, row i after i drafts), "draft" (K of them), "step" (one
    row, after K drafts), "ragged" (target rows, 0..K drafts a sequence).  hist: longest history; nbias: biased
    tokens a sequence; mask: whether rows carry grammar masks."""
    return {"name": name, "op": "adjust", "B": B, "K": K, "V": V, "dtype": dtype, "form": form, "hist": hist,
            "penalties": penalties, "nbias": nbias, "mask": mask, "inplace": inplace}


def listed():
    return [
        # the last norm of one decoded token: latency
        _norm("norm-1x4096-bf16", 1, 4096, "bf16", False, "bf16"),
        # the target's positions of the headline round (64 sequences, 7 positions), residual added, ready for an
        # 8-bit projection
        _norm("norm-448x4096-e4m3", 448, 4096, "bf16", True, "e4m3"),
        # a long prompt's rows
        _norm("norm-16384x8192-bf16", 16384, 8192, "bf16", True, "bf16"),
        # one draft head's residual block for one sequence: x + silu(x W^T + b)
        _linear("linear-1x4096x4096-silu", 1, 4096, 4096, "bf16", "bf16", "silu", True, 4096),
        # six draft heads of 64 sequences in one product: the heads' weights stacked, the residual shared by all
        _linear("linear-64x24576x4096-heads", 64, 24576, 4096, "bf16", "bf16", "silu", True, 4096),
        # odd sizes: rows and columns that end inside a tile
        _linear("linear-333x5001x2112-gelu", 333, 5001, 2112, "bf16", "f32", "gelu", True, 0),
        # the 8-bit output projection of one sequence's positions, float32 logits
        _linear("linear-7x128256x4096-e4m3", 7, 128256, 4096, "e4m3", "f32", "none", False, 0),
        # the 8-bit output projection of the headline round, whose logits are bfloat16
        _linear("linear-448x128256x4096-e4m3", 448, 128256, 4096, "e4m3", "bf16", "none", False, 0),
        # one decoded token of one sequence: latency
        _adjust("adjust-b1-v32000-step", 1, 0, 32000, "f32", "step", 512, True, 4, False),
        # the headline round's target rows: penalties over histories, the drafts before each position counted
        _adjust("adjust-b64-k6-v128256", 64, 6, 128256, "bf16", "target", 4096, True, 32, False),
        # the widest round: long histories, biases and a grammar mask on every row
        _adjust("adjust-b256-k8-v152064", 256, 8, 152064, "f32", "target", 8192, True, 300, True),
        # structured output: grammar masks alone, applied in place
        _adjust("adjust-b32-k6-v128256-mask", 32, 6, 128256, "bf16", "target", 0, False, 0, True, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "adjust", "adjust"])
    if op == "norm":
        d = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            d = max(64, d // 64 * 64)
        rows = _log(rng, 1, min(16384, 16384 * 8192 // (2 * d)))
        c = _norm("", rows, d, rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.7, rng.choice(["bf16", "f32", "e4m3"]))
    elif op == "linear":
        K = 64 * _log(rng, 1, 128)
        M = _log(rng, 1, 1024)
        heads = rng.choice([1, 1, 3, 6])
        N = _log(rng, 1, min(131072, 448 * 128256 * 4096 // (M * K)) // heads) * heads
        dtype = rng.choice(["bf16", "e4m3"])
        c = _linear("", M, N, K, dtype, rng.choice(["bf16", "f32"]),
                    rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]), rng.random() < 0.5,
                    rng.choice([0, N // heads]))
    else:
        form = rng.choice(["target", "draft", "step", "ragged"])
        K = rng.randint(1, 16)
        V = _log(rng, 1000, 152064)
        rows = 256 * 9 * 152064 // V
        B = _log(rng, 1, max(1, min(256, rows // (K + 1))))
        penalties, mask = rng.random() < 0.8, rng.random() < 0.5
        nbias = rng.choice([0, 1, 17, 300])
        c = _adjust("", B, K, V, rng.choice(["bf16", "f32"]), form, _log(rng, 1, 8192), penalties, nbias,
                    mask or not (penalties or nbias))
    del c["name"]
    return c


def work(c):
    if c["op"] == "norm":
        n = c["rows"] * c["d"]
        b = BYTES[c["dtype"]]
        by = n * (b + BYTES[c["out"]] + (2 * b if c["residual"] else 0)) + c["d"] * b
        by += 4 * c["rows"] if c["out"] == "e4m3" else 0
        return {"bytes": by, "flops": 6 * n}
    if c["op"] == "linear":
        M, N, K, b, o = c["M"], c["N"], c["K"], BYTES[c["dtype"]], BYTES[c["out"]]
        by = (M + N) * K * b + M * N * o + (N * o if c["bias"] else 0) + M * c["res_cols"] * o
        by += 4 * (M + N) if c["dtype"] == "e4m3" else 0
        return {"bytes": by, "flops": 2 * M * N * K}
    B, V, b = c["B"], c["V"], BYTES[c["dtype"]]
    ragged = B + sum(b % (c["K"] + 1) for b in range(B))
    rows = {"target": B * (c["K"] + 1), "draft": B * c["K"], "step": B, "ragged": ragged}[c["form"]]
    by = B * (c["hist"] * 3) + B * c["nbias"] * 8  # histories of 4-byte tokens, 3/4 full on the mean
    by += rows * V / 8 if c["mask"] else 0
    # in place: about half of the masked rows' logits are overwritten and none is read; otherwise every logit is
    # read once and written once
    by += rows * V * b * (0.5 if c["inplace"] else 2)
    return {"bytes": int(by), "flops": int(4 * rows * V)}


# --------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def prepare(c, seed):
    g = _gen(seed)
    s = {"c": c}
    if c["op"] == "norm":
        shape = (c["rows"], c["d"])
        t = DTYPES[c["dtype"]]
        # hidden states of unlike magnitude: a spread of a factor of ten between rows
        size = torch.rand((c["rows"], 1), device="cuda", generator=g).mul_(2.3).exp_()
        s["x"] = torch.randn(shape, device="cuda", generator=g).mul_(size).to(t)
        s["residual"] = torch.randn(shape, device="cuda", generator=g).mul_(size).to(t) if c["residual"] else None
        s["weight"] = (1.0 + 0.2 * torch.randn((c["d"],), device="cuda", generator=g)).to(t)
        s["eps"] = 1e-5
    elif c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        x = torch.randn((M, K), device="cuda", generator=g)
        s["x_scale"] = s["weight_scale"] = None
        w = torch.empty((N, K), device="cuda", dtype=DTYPES[c["dtype"]])
        f = torch.randn((N, K), device="cuda", generator=g).mul_(K ** -0.5)
        if c["dtype"] == "e4m3":
            ws = f.abs().amax(1).div_(E4M3_MAX).clamp_min_(FLT_MIN)
            w.copy_(f.div_(ws[:, None]))
            xs = x.abs().amax(1).div_(E4M3_MAX).clamp_min_(FLT_MIN)
            x = x.div_(xs[:, None])
            s["x_scale"], s["weight_scale"] = xs, ws
        else:
            w.copy_(f)
        del f
        s["x"], s["weight"] = x.to(DTYPES[c["dtype"]]), w
        o = DTYPES[c["out"]]
        s["bias"] = torch.randn((N,), device="cuda", generator=g).to(o) if c["bias"] else None
        s["residual"] = torch.randn((M, c["res_cols"]), device="cuda", generator=g).to(o) if c["res_cols"] else None
    else:
        B, K, V = c["B"], c["K"], c["V"]
        s["cu"] = None
        # the row's sequence, and the drafts that stand before its position
        if c["form"] == "ragged":
            k = torch.randperm(B, device="cuda", generator=g) % (K + 1)
            cu = torch.zeros((B + 1,), device="cuda", dtype=torch.int64)
            cu[1:] = k.cumsum(0)
            s["cu"], s["max_k"] = cu.to(torch.int32), K
            rows = int(cu[-1]) + B
            s["first"], s["drafts"] = 0, rows - B
            shape = (rows, V)
        else:
            R = {"target": K + 1, "draft": K, "step": 1}[c["form"]]
            s["first"] = K if c["form"] == "step" else 0
            rows = B * R
            shape = (B, R, V)
        s["logits"] = torch.empty(shape, device="cuda", dtype=DTYPES[c["dtype"]])
        s["logits"].copy_(torch.randn(shape, device="cuda", generator=g).mul_(2.0))
        s["out"] = s["logits"] if c["inplace"] else torch.empty_like(s["logits"])

        def tokens(*n):
            """Token ids with the long-tailed frequencies of text."""
            r = (torch.rand(n, device="cuda", generator=g, dtype=torch.float64) * math.log(V)).exp_().long() - 1
            return (r * 7919 % V).to(torch.int32)

        s["draft_tokens"] = tokens(*((s["drafts"],) if s["cu"] is not None else (B, K)))
        s["history"] = s["history_len"] = s["prompt_len"] = None
        s["repetition"] = s["frequency"] = s["presence"] = None
        if c["penalties"]:
            s["history"] = tokens(B, c["hist"])
            n = torch.randint(c["hist"] // 2, c["hist"] + 1, (B,), device="cuda", generator=g)
            s["history_len"] = n.to(torch.int32)
            s["prompt_len"] = (n * torch.rand((B,), device="cuda", generator=g)).to(torch.int32)
            s["repetition"] = 1.0 + 0.3 * torch.rand((B,), device="cuda", generator=g)
            s["frequency"] = 0.5 * torch.rand((B,), device="cuda", generator=g)
            s["presence"] = 0.5 * torch.rand((B,), device="cuda", generator=g)
        s["bias"] = None
        if c["nbias"]:
            cu_bias = torch.arange(0, (B + 1) * c["nbias"], c["nbias"], device="cuda", dtype=torch.int32)
            s["bias"] = (cu_bias, torch.randint(0, V, (B * c["nbias"],), device="cuda", generator=g, dtype=torch.int32),
                         torch.randn((B * c["nbias"],), device="cuda", generator=g))
        s["mask"] = None
        if c["mask"]:
            # the states of a grammar: a few tokens allowed, half of them, all but a few
            words = (V + 31) // 32
            share = torch.tensor([0.002, 0.5, 0.998], device="cuda")[torch.randint(0, 3, (rows,), device="cuda", generator=g)]
            mask = torch.zeros((rows, words), device="cuda", dtype=torch.int32)
            for bit in range(32):
                on = torch.rand((rows, words), device="cuda", generator=g) < share[:, None]
                mask |= on.to(torch.int32) << bit
            s["mask"] = mask
    return s


# ----------------------------------------------------- the operators, plain

def _act(y, act):
    if act == "relu":
        return y.clamp_min(0)
    if act == "silu":
        return y / (1 + torch.exp(-y))
    if act == "gelu":
        return y * 0.5 * (1 + torch.erf(y * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return y * 0.5 * (1 + torch.tanh((2 / math.pi) ** 0.5 * (y + 0.044715 * y * y * y)))
    return y


def _plain_norm(s):
    c = s["c"]
    h = s["x"].float()
    r = None
    if c["residual"]:
        h = h + s["residual"].float()
        r = h.to(s["x"].dtype)
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + s["eps"]) * s["weight"].float()
    if c["out"] != "e4m3":
        return {"out": y.to(DTYPES[c["out"]]), "residual": r}
    scale = (y.abs().amax(1) / E4M3_MAX).clamp_min(FLT_MIN)
    q = (y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return {"out": q, "scale": scale, "residual": r}


def _plain_linear(s):
    c = s["c"]
    y = s["x"].float() @ s["weight"].float().t()
    if c["dtype"] == "e4m3":
        y = y * s["x_scale"][:, None] * s["weight_scale"][None, :]
    if c["bias"]:
        y = y + s["bias"].float()
    y = _act(y, c["act"])
    if c["res_cols"]:
        y = (y.view(c["M"], -1, c["res_cols"]) + s["residual"].float()[:, None, :]).view(c["M"], c["N"])
    return y.to(DTYPES[c["out"]])


def _rows_of(s):
    """Of each row: its sequence, the index of its sequence's first draft, and how many drafts stand before it."""
    c = s["c"]
    B, n = c["B"], s["logits"].numel() // c["V"]
    at = torch.arange(n, device="cuda")
    if s["cu"] is not None:
        cu = s["cu"].long()
        seq = torch.searchsorted(cu[1:] + torch.arange(1, B + 1, device="cuda"), at, right=True)
        return seq, cu[seq], at - cu[seq] - seq
    R = n // B
    return at // R, at // R * c["K"], s["first"] + at % R


def _plain_adjust(s):
    c = s["c"]
    V, B = c["V"], c["B"]
    logits = s["logits"].view(-1, V)
    rows = logits.shape[0]
    if c["penalties"] or c["nbias"]:
        seq, first, seen = _rows_of(s)
        y = logits.float()
        if c["penalties"]:
            at = torch.arange(c["hist"], device="cuda")[None, :]
            live = at < s["history_len"][:, None]
            old = at < s["prompt_len"][:, None]
            hist = s["history"].long()
            prompt = torch.zeros((B, V), device="cuda").scatter_add_(1, hist, (live & old).float())
            count = torch.zeros((B, V), device="cuda").scatter_add_(1, hist, (live & ~old).float())[seq]
            if s["draft_tokens"].numel():
                k = torch.arange(max(c["K"], 1), device="cuda")[None, :]
                x = s["draft_tokens"].reshape(-1).long()
                x = x[(first[:, None] + k).clamp_max(x.numel() - 1)]
                count.scatter_add_(1, x, (k < seen[:, None]).float())
            rep = torch.where((prompt[seq] > 0) | (count > 0), s["repetition"][seq][:, None], 1.0)
            y = torch.where(y > 0, y / rep, y * rep)
            y = y - s["frequency"][seq][:, None] * count - s["presence"][seq][:, None] * (count > 0)
        if c["nbias"]:
            cu, tok, val = s["bias"]
            b = torch.arange(B, device="cuda").repeat_interleave(c["nbias"])
            bias = torch.zeros((B, V), device="cuda", dtype=torch.float64).index_put_((b, tok.long()), val.double(), accumulate=True)
            y = y + bias.float()[seq]
        y = y.to(logits.dtype)
    elif c["inplace"]:
        y = logits
    else:
        y = logits.clone()
    if c["mask"]:
        bits = (s["mask"][:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        y.masked_fill_(bits.view(rows, -1)[:, :V] == 0, -math.inf)
    return y.view(s["logits"].shape)


def run(s):
    c = s["c"]
    if own:
        from rejection_sampling_verify_09_amd import adjust_logits, linear, rms_norm

        if c["op"] == "norm":
            y, scale, r = rms_norm(s["x"], s["weight"], residual=s["residual"], eps=s["eps"], out_dtype=DTYPES[c["out"]])
            if c["out"] == "e4m3":
                return {"out": y, "scale": scale, "residual": r}
            return {"out": y, "residual": r}
        if c["op"] == "linear":
            return linear(s["x"], s["weight"], bias=s["bias"], residual=s["residual"], activation=c["act"],
                          x_scale=s["x_scale"], weight_scale=s["weight_scale"], out_dtype=DTYPES[c["out"]])
        ragged = {} if s["cu"] is None else {"cu_num_draft": s["cu"], "max_k": s["max_k"]}
        return adjust_logits(s["logits"], history=s["history"], history_len=s["history_len"],
                             prompt_len=s["prompt_len"], draft_tokens=s["draft_tokens"], drafts_seen=s["first"],
                             repetition_penalty=s["repetition"], frequency_penalty=s["frequency"],
                             presence_penalty=s["presence"], bias=s["bias"], mask=s["mask"], out=s["out"], **ragged)
    return {"norm": _plain_norm, "linear": _plain_linear, "adjust": _plain_adjust}[c["op"]](s)


# --------------------------------------------- the definitions, in 64 bits

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "norm":
        h = s["x"].double() + (s["residual"].double() if c["residual"] else 0.0)
        rms = (torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / c["d"] + s["eps"]) ** 0.5
        y = h / rms * s["weight"].double()
        r = {"out": y, "residual": h if c["residual"] else None}
        if c["out"] == "e4m3":
            scale = torch.maximum(y.abs().max(1).values / E4M3_MAX, torch.full_like(y[:, 0], FLT_MIN))
            v = y / scale[:, None]
            # steps of e4m3: 2^-3 of the power of two below, at least 2^-9
            step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
            r["out"] = (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
            r["scale"] = scale
        return r
    if c["op"] == "linear":
        x, w = s["x"].to(torch.float64), s["weight"]
        y = torch.empty((c["M"], c["N"]), device="cuda", dtype=torch.float64)
        for n in range(0, c["N"], 16384):
            y[:, n:n + 16384] = x @ w[n:n + 16384].to(torch.float64).t()
        if c["dtype"] == "e4m3":
            y *= torch.outer(s["x_scale"].double(), s["weight_scale"].double())
        if c["bias"]:
            y += s["bias"].double()
        if c["act"] == "relu":
            y = torch.where(y > 0, y, torch.zeros_like(y))
        elif c["act"] == "silu":
            y = y * torch.sigmoid(y)
        elif c["act"] == "gelu":
            y = y * torch.special.ndtr(y)
        elif c["act"] == "gelu_tanh":
            y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
        if c["res_cols"]:
            y += s["residual"].double().repeat(1, c["N"] // c["res_cols"])
        return y
    # row by row: the tokens each position has seen, counted
    B, V = c["B"], c["V"]
    out = s["logits"].view(-1, V).double()
    cu = s["cu"].tolist() if s["cu"] is not None else None
    drafts = s["draft_tokens"].reshape(-1).long()
    row = 0
    R = out.shape[0] // B
    for b in range(B):
        rows = cu[b + 1] - cu[b] + 1 if cu else R
        x = drafts[cu[b]:cu[b + 1]] if cu else drafts[b * c["K"]:(b + 1) * c["K"]]
        add = None
        if c["nbias"]:
            at = slice(b * c["nbias"], (b + 1) * c["nbias"])
            add = torch.zeros(V, device="cuda", dtype=torch.float64)
            add.index_add_(0, s["bias"][1][at].long(), s["bias"][2][at].double())
        if c["penalties"]:
            n, p = int(s["history_len"][b]), int(s["prompt_len"][b])
            seen = s["history"][b, :n].long()
            rep, freq, pres = (float(s[k][b]) for k in ("repetition", "frequency", "presence"))
            prompt = torch.bincount(seen[:p], minlength=V) > 0
        for i in range(rows):
            y = out[row]
            if c["penalties"]:
                said = torch.bincount(torch.cat([seen[p:], x[:s["first"] + i]]), minlength=V)
                hit = prompt | (said > 0)
                y = torch.where(hit, torch.where(y > 0, y / rep, y * rep), y) - freq * said - pres * (said > 0).double()
            if add is not None:
                y = y + add
            out[row] = y
            row += 1
    if c["mask"]:
        off = [(s["mask"] & (1 << i if i < 31 else -(1 << 31))) == 0 for i in range(32)]
        out.masked_fill_(torch.stack(off, 2).view(out.shape[0], -1)[:, :V], -math.inf)
    return out.view(s["logits"].shape)
