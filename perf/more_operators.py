"""Cases that time the operators of expert blocks in 8 and 16 bits: the layer norm
before a block and its gradients, the quantisation of rows to 8 bits, the 8-bit
products grouped by expert, and the whole layer of 16-bit experts for a few tokens.

`run` computes one pass of one operator: with elementary torch operations in
32 bits (64 for values next to a rounding border) where `own` is false, through the
framework's entry points where it is true.  `exact` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-5


# --------------------------------------------------------------------- cases
def _norm(name, direction, rows, d, dtype, ptype, residual):
    return {"name": name, "op": "norm", "dir": direction, "rows": rows, "d": d, "dtype": dtype, "ptype": ptype,
            "residual": residual}


def _quant(name, tokens, k, d, dtype):
    return {"name": name, "op": "quant", "tokens": tokens, "k": k, "d": d, "dtype": dtype}


def _product(name, tokens, k, experts, n, kk, dtype, route):
    return {"name": name, "op": "product", "tokens": tokens, "k": k, "experts": experts, "n": n, "kdim": kk,
            "dtype": dtype, "route": route}


def _layer(name, tokens, k, experts, d, f, dtype):
    return {"name": name, "op": "layer", "tokens": tokens, "k": k, "experts": experts, "d": d, "f": f, "dtype": dtype}


def listed():
    return [
        # the norm before a block for three concurrent requests, residual added: a decode step, where latency counts
        _norm("layer norm 3 rows", "fwd", 3, 2048, "bf16", "bf16", True),
        # the same over a prompt of the large layer
        _norm("layer norm 4096", "fwd", 4096, 7168, "bf16", "bf16", True),
        # its gradients in training, parameters kept in 32 bits, the stream's gradient added
        _norm("layer norm grad 4096", "bwd", 4096, 2048, "bf16", "f32", True),
        # the rows between the two products of one token's 8 experts, in place
        _quant("quantize 1 token", 8, 1, 768, "f16"),
        # a prompt's rows, gathered in the experts' order on the way
        _quant("quantize 4096", 4096, 8, 2048, "bf16"),
        # 8-bit gate_up of one token's 8 experts: bound by reading 8 experts' weights
        _product("experts i8 1 token", 1, 8, 128, 1536, 2048, "bf16", "normal"),
        # 8-bit down projection of the large layer at 512 tokens: 3.8 GB of weights, about 16 rows an expert
        _product("experts i8 large 512", 512, 8, 256, 7168, 2048, "bf16", "normal"),
        # 8-bit gate_up of a long prompt with Zipf-skewed experts: segments from empty to thousands of rows
        _product("experts i8 4096 skewed", 4096, 8, 128, 1536, 2048, "bf16", "zipf"),
        # a small batch with odd segments and widths that fill no tile
        _product("experts i8 ragged", 619, 2, 8, 520, 272, "f16", "biased"),
        # a whole layer for one token: single-stream decoding
        _layer("layer 1 token", 1, 8, 128, 2048, 768, "bf16"),
        # 8 concurrent requests at the large layer: about 57 of 256 experts of 88 MB
        _layer("layer large 8 tokens", 8, 8, 256, 7168, 2048, "bf16"),
        # a small model's batch: odd numbers of tokens, experts and choices, most experts with several rows
        _layer("layer 27 tokens", 27, 3, 17, 576, 320, "f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, unit=8):
    return max(lo, _log(rng, lo, hi) // unit * unit)


def draw(rng):
    op = rng.choice(["norm", "quant", "product", "product", "layer", "layer"])
    if op == "norm":
        t = rng.choice(["bf16", "f16", "f32"])
        while True:
            c = _norm("", rng.choice(["fwd", "bwd"]), _log(rng, 1, 16384), _width(rng, 64, 7168), t,
                      rng.choice([t, "f32"]), rng.random() < 0.5)
            if c["rows"] * c["d"] <= 4096 * 7168:
                break
    elif op == "quant":
        while True:
            c = _quant("", _log(rng, 1, 8192), rng.randint(1, 8), _width(rng, 64, 7168, 16), rng.choice(["bf16", "f16", "f32"]))
            if c["tokens"] * c["k"] * c["d"] <= 4096 * 8 * 2048:
                break
    elif op == "product":
        while True:
            e = _log(rng, 1, 256)
            c = _product("", _log(rng, 1, 4096), rng.randint(1, min(8, e)), e, _width(rng, 64, 7168), _width(rng, 64, 7168, 16),
                         rng.choice(["bf16", "f16"]), rng.choice(["normal", "biased", "zipf"]))
            rows = c["tokens"] * c["k"]
            # no dearer than the listed ones: their arithmetic, their weights, and the plain form's padded rows
            if (rows * c["n"] * c["kdim"] <= 32768 * 1536 * 2048 and e * c["n"] * c["kdim"] <= 128 * 1536 * 2048
                    and e * rows * (c["n"] + c["kdim"]) <= 2 ** 33):
                break
    else:
        while True:
            e = _log(rng, 1, 256)
            k = rng.randint(1, min(8, e))
            c = _layer("", _log(rng, 1, 32), k, e, _width(rng, 64, 7168, 64), _width(rng, 64, 2048, 64), rng.choice(["bf16", "f16"]))
            if e * c["d"] * c["f"] <= 2 ** 30 and c["tokens"] * k * c["d"] * c["f"] <= 64 * 7168 * 2048:
                break
    del c["name"]
    return c


# -------------------------------------------------------------------- inputs
def _logits(g, tokens, experts, k, how):
    logits = torch.randn(tokens, experts, generator=g, device=DEV)
    if how == "biased":
        logits += 0.5 * torch.randn(experts, generator=g, device=DEV)
    elif how == "zipf":
        rank = torch.randperm(experts, generator=g, device=DEV).float() + 1
        u = torch.rand(tokens, experts, generator=g, device=DEV).clamp_(1e-7, 1 - 1e-7)
        logits = -1.1 * torch.log(rank) - torch.log(-torch.log(u))
        if experts >= 16 * k:  # the rarest experts get no rows
            logits[:, rank > experts - experts // 16] = -math.inf
    return logits


def _segments(logits, k):
    """Offsets of the experts' segments, the assignment at each permuted row, and the longest segment."""
    experts = logits.shape[1]
    flat = logits.topk(k, dim=1).indices.reshape(-1)
    order = torch.sort(flat, stable=True).indices.to(torch.int32)
    counts = torch.bincount(flat, minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return offsets, order, int(counts.max())


def _randn(g, dtype, scale, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).mul_(scale).to(dtype)


def _weights(g, dtype, scale, experts, n, k):
    """Made in pieces: the 32-bit numbers of all experts would take twice their room."""
    w = torch.empty(experts, n, k, dtype=dtype, device=DEV)
    step = max(1, (1 << 28) // (n * k))
    for i in range(0, experts, step):
        m = min(step, experts - i)
        if dtype == torch.int8:
            v = torch.randn(m, n, k, generator=g, device=DEV).mul_(scale).round_().clamp_(-127, 127)
        else:
            v = torch.randn(m, n, k, generator=g, device=DEV).mul_(scale)
        w[i:i + m] = v.to(dtype)
    return w


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    t = TYPES[case["dtype"]]
    s = dict(case)
    if case["op"] == "norm":
        rows, d, p = case["rows"], case["d"], TYPES[case["ptype"]]
        s["gamma"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(p)
        s["beta"] = (0.1 * torch.randn(d, generator=g, device=DEV)).to(p)
        # a stream's rows: a few channels far larger than the others, means off zero
        channel = torch.exp(0.5 * torch.randn(d, generator=g, device=DEV))
        x = torch.randn(rows, d, generator=g, device=DEV).mul_(channel).add_(0.3 * torch.randn(rows, 1, generator=g, device=DEV))
        s["x"] = x.mul_(2.0).to(t)  # backward: the stream that was normalised
        if case["dir"] == "fwd":
            s["y"] = _randn(g, t, 0.8, rows, d) if case["residual"] else None
        else:
            s["dh"] = _randn(g, t, 0.1, rows, d)
            s["dx_out"] = _randn(g, t, 0.1, rows, d) if case["residual"] else None
    elif case["op"] == "quant":
        tokens, k, d = case["tokens"], case["k"], case["d"]
        channel = torch.exp(0.5 * torch.randn(d, generator=g, device=DEV))
        s["x"] = torch.randn(tokens, d, generator=g, device=DEV).mul_(channel).to(t)
        s["row_map"] = None
        if k > 1:  # rows in the experts' order: `sorted` of a permutation
            _, s["row_map"], _ = _segments(_logits(g, tokens, max(16, k), k, "normal"), k)
    elif case["op"] == "product":
        e, n, k = case["experts"], case["n"], case["kdim"]
        rows = case["tokens"] * case["k"]
        s["offsets"], _, s["longest"] = _segments(_logits(g, case["tokens"], e, case["k"], case["route"]), case["k"])
        s["x"] = torch.randn(rows, k, generator=g, device=DEV).mul_(32).round_().clamp_(-127, 127).to(torch.int8)
        s["x_scale"] = (0.5 + torch.rand(rows, generator=g, device=DEV)) / 32
        s["w"] = _weights(g, torch.int8, 32, e, n, k)
        s["w_scale"] = (0.5 + torch.rand(e, n, generator=g, device=DEV)) / (32 * math.sqrt(k))
    else:
        e, d, f = case["experts"], case["d"], case["f"]
        s["x"] = _randn(g, t, 1.0, case["tokens"], d)
        s["logits"] = _logits(g, case["tokens"], e, case["k"], "normal")
        s["w13"] = _weights(g, t, d ** -0.5, e, 2 * f, d)
        s["w2"] = _weights(g, t, f ** -0.5, e, d, f)
    if own:
        # what a program keeps between calls: the workspace
        import bit_quantized_expert_moe_gb300 as moe
        s["moe"] = moe
        if case["op"] == "norm" and case["dir"] == "bwd":
            s["ws"] = moe.workspace(moe.layer_norm_backward_workspace_size(rows, d))
        elif case["op"] == "product":
            s["ws"] = moe.workspace(moe.grouped_mm_i8_workspace_size(rows, e, n, k))
        elif case["op"] == "layer":
            s["ws"] = moe.workspace(moe.expert_layer_workspace_size(case["tokens"], case["k"], e, d, f))
    return s


# ------------------------------------------------------- one pass: framework
def _run_own(s):
    moe = s["moe"]
    if s["op"] == "norm":
        if s["dir"] == "fwd":
            x_out, h = moe.layer_norm(s["x"], s["y"], s["gamma"], s["beta"], eps=EPS)
            return {"x_out": x_out, "h": h} if s["residual"] else {"h": h}
        dx, dgamma, dbeta = moe.layer_norm_backward(s["x"], s["dh"], s["dx_out"], s["gamma"], s["beta"], eps=EPS, ws=s["ws"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if s["op"] == "quant":
        codes, scales = moe.quantize_rows(s["x"], s["row_map"], s["k"])
        return {"codes": codes, "scales": scales}
    if s["op"] == "product":
        return {"y": moe.grouped_mm_i8(s["x"], s["x_scale"], s["w"], s["w_scale"], s["offsets"],
                                       dtype=TYPES[s["dtype"]], ws=s["ws"])}
    ids = torch.empty(s["tokens"], s["k"], dtype=torch.int32, device=DEV)
    out = moe.expert_layer(s["x"], s["logits"], s["w13"], s["w2"], s["k"], ids=ids, ws=s["ws"])
    return {"out": out, "ids": ids}


# ------------------------------------------------------ one pass: plain form
def _plain_norm(s):
    t, p = TYPES[s["dtype"]], TYPES[s["ptype"]]
    x, gamma, beta = s["x"].float(), s["gamma"].float(), s["beta"].float()
    if s["dir"] == "fwd" and s["residual"]:
        x = x + s["y"].float()
    c = x - x.mean(1, keepdim=True)
    r = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
    n = c * r
    if s["dir"] == "fwd":
        h = (n * gamma + beta).to(t)
        return {"x_out": x.to(t), "h": h} if s["residual"] else {"h": h}
    dh = s["dh"].float()
    v = dh * gamma
    dx = r * (v - v.mean(1, keepdim=True) - n * (v * n).mean(1, keepdim=True))
    if s["residual"]:
        dx = dx + s["dx_out"].float()
    return {"dx": dx.to(t), "dgamma": (dh * n).sum(0).to(p), "dbeta": dh.sum(0).to(p)}


def _plain_quant(s):
    x = s["x"]
    if s["row_map"] is not None:
        x = x[s["row_map"].long() // s["k"]]
    top = x.abs().amax(1, keepdim=True)
    # 64 bits: a value next to the border between two codes
    codes = torch.round(x.double() * 127 / top.double().clamp_min(1e-300))
    return {"codes": codes.to(torch.int8), "scales": (top.float() / 127)[:, 0]}


def _plain_product(s):
    t = TYPES[s["dtype"]]
    start = s["offsets"][:-1].long()
    rows, experts = s["x"].shape[0], s["experts"]
    r = torch.arange(rows, device=DEV)
    e = torch.searchsorted(s["offsets"][1:].long(), r, right=True)
    scale = s["x_scale"][:, None] * s["w_scale"][e]
    if rows < experts:  # most experts have no rows: a matrix for each row
        y = torch.bmm(s["w"][e].float(), s["x"].float()[:, :, None])[:, :, 0]
        return {"y": (y * scale).to(t)}
    at = r - start[e]
    x = torch.zeros(experts, s["longest"], s["kdim"], device=DEV)
    x[e, at] = s["x"].float()
    y = torch.empty(experts, s["longest"], s["n"], device=DEV)
    for i in range(0, experts, 32):  # some experts' weights in 32 bits at a time
        torch.bmm(x[i:i + 32], s["w"][i:i + 32].float().transpose(1, 2), out=y[i:i + 32])
    return {"y": (y[e, at] * scale).to(t)}


def _plain_layer(s):
    f, x = s["f"], s["x"].float()
    order = torch.sort(s["logits"], dim=1, descending=True, stable=True)  # ties go to the lowest expert
    ids, top = order.indices[:, :s["k"]], order.values[:, :s["k"]]
    p = torch.exp(top - top[:, :1])
    p = p / p.sum(1, keepdim=True)
    out = torch.zeros_like(x)
    for j in range(s["k"]):
        gu = torch.bmm(s["w13"][ids[:, j]].float(), x[:, :, None])[:, :, 0]
        a, u = gu[:, :f], gu[:, f:]
        h = a / (1 + torch.exp(-a)) * u
        out += p[:, j:j + 1] * torch.bmm(s["w2"][ids[:, j]].float(), h[:, :, None])[:, :, 0]
    return {"out": out.to(TYPES[s["dtype"]]), "ids": ids.to(torch.int32)}


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "quant": _plain_quant, "product": _plain_product, "layer": _plain_layer}[state["op"]](state)


# ---------------------------------------------------------------------- work
def _touched(tokens, k, experts):
    """Experts that get a token, on average, where all are as likely."""
    return max(1, round(experts * (1 - (1 - k / experts) ** tokens)))


def work(case):
    b = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        rows, d = case["rows"], case["d"]
        pb = 4 if case["ptype"] == "f32" else 2
        if case["dir"] == "fwd":
            return {"bytes": b * rows * d * (4 if case["residual"] else 2) + 2 * pb * d, "flops": 9 * rows * d}
        return {"bytes": b * rows * d * (4 if case["residual"] else 3) + 3 * pb * d, "flops": 18 * rows * d}
    if case["op"] == "quant":
        rows = case["tokens"] * case["k"]
        read = case["tokens"] * case["d"] * b + (4 * rows if case["k"] > 1 else 0)
        return {"bytes": read + rows * (case["d"] + 4), "flops": 4 * rows * case["d"]}
    experts = _touched(case["tokens"], case["k"], case["experts"])
    if case["op"] == "product":
        rows, n, k = case["tokens"] * case["k"], case["n"], case["kdim"]
        if case["route"] == "zipf" and case["experts"] >= 16 * case["k"]:
            experts = min(experts, case["experts"] - case["experts"] // 16)
        return {"bytes": experts * n * (k + 4) + rows * (k + 4) + 2 * rows * n, "flops": 2 * rows * n * k}
    d, f, tokens = case["d"], case["f"], case["tokens"]
    return {"bytes": 6 * experts * d * f + 4 * tokens * d + 4 * tokens * (case["experts"] + case["k"]),
            "flops": 6 * tokens * case["k"] * d * f}


# ------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The operators' definitions in 64 bits, a row, an expert or a token's choice at a time."""
    s = prepare(case, seed)
    if case["op"] == "norm":
        d = case["d"]
        x = s["x"].double()
        if case["dir"] == "fwd" and case["residual"]:
            x += s["y"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        std = torch.sqrt(var + EPS)
        n = (x - mean) / std
        if case["dir"] == "fwd":
            h = torch.addcmul(s["beta"].double(), n, s["gamma"].double())
            return {"x_out": x, "h": h} if case["residual"] else {"h": h}
        dh = s["dh"].double()
        v = dh * s["gamma"].double()
        along = torch.einsum("td,td->t", v, n)[:, None] / d
        dx = (v - v.sum(1, keepdim=True) / d - along * n) / std
        if case["residual"]:
            dx += s["dx_out"].double()
        return {"dx": dx, "dgamma": torch.einsum("td,td->d", dh, n), "dbeta": dh.sum(0)}
    if case["op"] == "quant":
        scales = torch.linalg.vector_norm(s["x"].double(), ord=math.inf, dim=1) / 127
        codes = torch.empty(case["tokens"] * case["k"], case["d"], dtype=torch.int8, device=DEV)
        row = torch.arange(case["tokens"], device=DEV) if s["row_map"] is None else torch.div(
            s["row_map"].long(), case["k"], rounding_mode="floor")
        top = scales * 127
        for i in range(0, len(row), 4096):
            r = row[i:i + 4096]
            v = s["x"].index_select(0, r).double()
            # one division of exact numbers: what is next to a border falls on the right side
            codes[i:i + 4096] = torch.round(torch.where(top[r, None] > 0, 127 * v / top[r, None], v)).to(torch.int8)
        return {"codes": codes, "scales": scales[row]}
    if case["op"] == "product":
        cut = s["offsets"].tolist()
        y = torch.zeros(case["tokens"] * case["k"], case["n"], dtype=torch.float64, device=DEV)
        for e in range(case["experts"]):
            i, j = cut[e], cut[e + 1]
            if i < j:
                a = s["x"][i:j].double() * s["x_scale"][i:j].double().unsqueeze(1)
                y[i:j] = a @ (s["w"][e].double() * s["w_scale"][e].double().unsqueeze(1)).t()
        return {"y": y}
    x, lg, f, k = s["x"].double(), s["logits"].double().cpu(), case["f"], case["k"]
    ids = torch.empty(case["tokens"], k, dtype=torch.int32)
    out = torch.zeros(case["tokens"], case["d"], dtype=torch.float64, device=DEV)
    for i in range(case["tokens"]):
        row = lg[i].tolist()
        best = sorted(range(len(row)), key=lambda e: (-row[e], e))[:k]
        p = torch.softmax(lg[i][best], 0).tolist()
        ids[i] = torch.tensor(best, dtype=torch.int32)
        for e, w in zip(best, p):
            a = s["w13"][e, :f].double() @ x[i]
            u = s["w13"][e, f:].double() @ x[i]
            out[i] += w * (s["w2"][e].double() @ (a * torch.sigmoid(a) * u))
    return {"out": out, "ids": ids.to(DEV)}
