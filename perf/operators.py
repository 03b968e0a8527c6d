"""Cases that time the 16-bit expert operators: the products grouped by expert,
the gated activation with the routing weight, and the norms around a block.

`run` computes one pass of one operator: with elementary torch operations in
32 bits where `own` is false, through the framework's entry points where it is
true.  `exact` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


# --------------------------------------------------------------------- cases
def _grouped(name, direction, tokens, k, experts, n, kk, dtype, route):
    return {"name": name, "op": "grouped", "dir": direction, "tokens": tokens, "k": k, "experts": experts,
            "n": n, "kdim": kk, "dtype": dtype, "route": route}


def _swiglu(name, direction, tokens, k, f, dtype):
    return {"name": name, "op": "swiglu", "dir": direction, "tokens": tokens, "k": k, "f": f, "dtype": dtype}


def _norm(name, direction, rows, d, dtype, ptype, gates):
    return {"name": name, "op": "norm", "dir": direction, "rows": rows, "d": d, "dtype": dtype, "ptype": ptype,
            "gates": gates}


def listed():
    return [
        # gate_up of one token's 8 experts: single-stream decoding, bound by reading 8 experts' weights
        _grouped("experts 1 token", "fwd", 1, 8, 128, 1536, 2048, "bf16", "normal"),
        # down projection of a decode batch of 64 tokens: nearly every expert read for about four rows
        _grouped("experts 64 tokens", "fwd", 64, 8, 128, 2048, 768, "bf16", "normal"),
        # gate_up of a long prompt with Zipf-skewed experts: segments from empty to thousands of rows
        _grouped("experts 4096 skewed", "fwd", 4096, 8, 128, 1536, 2048, "bf16", "zipf"),
        # down projection of the large layer at 512 tokens: 7.5 GB of fp16 weights, about 16 rows an expert
        _grouped("experts large 512", "fwd", 512, 8, 256, 7168, 2048, "f16", "normal"),
        # training step of gate_up at 4096 tokens: gradients of the rows and of every expert's weights
        _grouped("experts grad 4096", "bwd", 4096, 8, 128, 1536, 2048, "bf16", "biased"),
        # a small fine-tuning batch with odd segments and widths that are multiples of 8 alone
        _grouped("experts grad ragged", "bwd", 619, 2, 8, 520, 264, "f16", "biased"),
        # gated activation of one token's 8 rows: a decode step, where latency counts
        _swiglu("gate 1 token", "fwd", 1, 8, 768, "bf16"),
        # gradient of the gated activation and of the routing weights over a long prompt
        _swiglu("gate grad 4096", "bwd", 4096, 8, 768, "bf16"),
        # the norms around a block for two concurrent requests
        _norm("norm 2 rows", "fwd", 2, 2048, "bf16", "bf16", 1),
        # the norms around a block of the large layer over a prompt, gate per channel
        _norm("norm 4096", "fwd", 4096, 7168, "bf16", "bf16", 1),
        # their gradients in training, parameters kept in 32 bits
        _norm("norm grad 4096", "bwd", 4096, 2048, "bf16", "f32", 1),
        # the same with one gate for each of 33 sequences of 35 rows and an odd width
        _norm("norm grad ragged", "bwd", 1155, 1288, "f16", "f16", 33),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A multiple of 8."""
    v = max(lo, _log(rng, lo, hi) // 8 * 8)
    return v + 8 if v == 3072 else v


def _tokens(rng, hi, k=1):
    v = _log(rng, 1, hi)
    return v + 1 if v * k == 3072 else v


def draw(rng):
    op = rng.choice(["grouped", "grouped", "swiglu", "norm"])
    direction = rng.choice(["fwd", "bwd"])
    if op == "grouped":
        top = work(listed()[4])["flops"]
        while True:
            e = _log(rng, 1, 256)
            k = rng.randint(1, min(8, e))
            c = _grouped("", direction, _tokens(rng, 4096, k), k, e, _width(rng, 64, 7168), _width(rng, 64, 7168),
                         rng.choice(["bf16", "f16"]), rng.choice(["normal", "biased", "zipf"]))
            w = work(c)
            rows = c["tokens"] * k
            # no dearer than the listed ones: their arithmetic and their weights
            if w["flops"] <= top and e * c["n"] * c["kdim"] <= 128 * 1536 * 2048 and e * rows * (c["n"] + c["kdim"]) <= 2 ** 33:
                break
    elif op == "swiglu":
        k = rng.randint(1, 8)
        while True:
            c = _swiglu("", direction, _tokens(rng, 4096, k), k, _width(rng, 64, 4096), rng.choice(["bf16", "f16", "f32"]))
            if c["f"] != 1536 and c["tokens"] * k * c["f"] <= 4096 * 8 * 768:
                break
    else:
        g = rng.choice([1, 1, _log(rng, 1, 64)])
        s = max(1, _log(rng, 1, 4096) // g)
        t = rng.choice(["bf16", "f16", "f32"])
        s = s + 1 if g * s == 3072 else s
        c = _norm("", direction, g * s, _width(rng, 64, 7168), t, rng.choice([t, "f32"]), g)
    del c["name"]
    return c


# -------------------------------------------------------------------- inputs
def _route(g, tokens, k, experts, how):
    """Offsets of the experts' segments and the assignment at each permuted row."""
    logits = torch.randn(tokens, experts, generator=g, device=DEV)
    if how == "biased":
        logits += 0.5 * torch.randn(experts, generator=g, device=DEV)
    elif how == "zipf":
        rank = torch.randperm(experts, generator=g, device=DEV).float() + 1
        u = torch.rand(tokens, experts, generator=g, device=DEV).clamp_(1e-7, 1 - 1e-7)
        logits = -1.1 * torch.log(rank) - torch.log(-torch.log(u))
        if experts >= 16 * k:  # the rarest experts get no rows
            logits[:, rank > experts - experts // 16] = -math.inf
    top, ids = logits.topk(k, dim=1)
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices.to(torch.int32)
    counts = torch.bincount(flat, minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return offsets, order, torch.softmax(top, dim=1).reshape(-1).contiguous(), int(counts.max())


def _randn(g, dtype, scale, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).mul_(scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    t = TYPES[case["dtype"]]
    s = dict(case)
    if case["op"] == "grouped":
        e, n, k = case["experts"], case["n"], case["kdim"]
        rows = case["tokens"] * case["k"]
        s["offsets"], _, _, s["longest"] = _route(g, case["tokens"], case["k"], e, case["route"])
        w = torch.empty(e, n, k, dtype=t, device=DEV)
        step = max(1, (1 << 28) // (n * k))
        for i in range(0, e, step):  # in pieces: the 32-bit numbers of 7.5 GB of weights would take 15 GB
            w[i:i + step] = _randn(g, t, k ** -0.5, min(step, e - i), n, k)
        s["x"] = _randn(g, t, 1.0, rows, k)
        s["w"] = w
        if case["dir"] == "bwd":
            s["dy"] = _randn(g, t, 0.1, rows, n)
    elif case["op"] == "swiglu":
        rows = case["tokens"] * case["k"]
        # the experts' number sets only the order of the rows
        _, s["row_map"], s["row_w"], _ = _route(g, case["tokens"], case["k"], max(16, case["k"]), "normal")
        s["gu"] = _randn(g, t, 1.5, rows, 2 * case["f"])
        if case["dir"] == "bwd":
            s["dh"] = _randn(g, t, 0.1, rows, case["f"])
    else:
        rows, d, p = case["rows"], case["d"], TYPES[case["ptype"]]
        s["alpha"] = 0.7
        s["gamma_post"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(p)
        s["gamma_pre"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(p)
        s["gate"] = torch.sigmoid(torch.randn(case["gates"], d, generator=g, device=DEV)).to(p)
        s["y"] = _randn(g, t, 0.8, rows, d)
        s["x"] = _randn(g, t, 2.0, rows, d)  # backward: the stream after the block
        if case["dir"] == "bwd":
            s["dx_out"] = _randn(g, t, 0.1, rows, d)
            s["dh"] = _randn(g, t, 0.1, rows, d)
    if own:
        # what a program keeps between calls: the workspace
        import bit_quantized_expert_moe_gb300 as moe
        s["moe"] = moe
        if case["op"] == "grouped":
            s["ws"] = moe.workspace(moe.grouped_mm_workspace_size(rows, e, n, k))
        elif case["op"] == "norm" and case["dir"] == "bwd":
            s["ws"] = moe.workspace(moe.block_norm_backward_workspace_size(rows, d, case["gates"]))
    return s


# ------------------------------------------------------- one pass: framework
def _run_own(s):
    moe = s["moe"]
    if s["op"] == "grouped":
        if s["dir"] == "fwd":
            return {"y": moe.grouped_mm(s["x"], s["w"], s["offsets"], ws=s["ws"])}
        return {"dx": moe.grouped_mm_dx(s["dy"], s["w"], s["offsets"], ws=s["ws"]),
                "dw": moe.grouped_mm_dw(s["dy"], s["x"], s["offsets"], ws=s["ws"])}
    if s["op"] == "swiglu":
        if s["dir"] == "fwd":
            return {"h": moe.swiglu(s["gu"], s["row_w"], s["row_map"])}
        dgu, dw = moe.swiglu_backward(s["dh"], s["gu"], s["row_w"], s["row_map"])
        return {"dgu": dgu, "drow_w": dw}
    p = {"gamma_post": s["gamma_post"], "gate": s["gate"], "gamma_pre": s["gamma_pre"], "alpha": s["alpha"], "eps": EPS}
    if s["dir"] == "fwd":
        x_out, h = moe.block_norm(s["x"], s["y"], **p)
        return {"x_out": x_out, "h": h}
    dx, dy, dpost, dgate, dpre = moe.block_norm_backward(s["x"], s["y"], s["dx_out"], s["dh"], **p, ws=s["ws"])
    return {"dx": dx, "dy": dy, "dgamma_post": dpost, "dgate": dgate, "dgamma_pre": dpre}


# ------------------------------------------------------ one pass: plain form
def _padded(s):
    """Of every permuted row: its expert and its place among the expert's rows."""
    start = s["offsets"][:-1].long()
    rows = s["x"].shape[0]
    r = torch.arange(rows, device=DEV)
    e = torch.searchsorted(s["offsets"][1:].long(), r, right=True)
    return e, r - start[e], s["longest"]


def _pad(v, e, at, longest, experts):
    out = torch.zeros(experts, longest, v.shape[1], device=DEV)
    out[e, at] = v.float()
    return out


def _run_plain(s):
    t = TYPES[s["dtype"]]
    if s["op"] == "grouped":
        e, at, longest = _padded(s)
        if s["dir"] == "fwd" and len(e) < s["experts"]:  # most experts have no rows: a matrix for each row
            return {"y": torch.bmm(s["w"][e].float(), s["x"].float()[:, :, None])[:, :, 0].to(t)}
        w = s["w"].float()
        if s["dir"] == "fwd":
            x = _pad(s["x"], e, at, longest, s["experts"])
            return {"y": torch.bmm(x, w.transpose(1, 2))[e, at].to(t)}
        dy = _pad(s["dy"], e, at, longest, s["experts"])
        dx = torch.bmm(dy, w)[e, at].to(t)
        x = _pad(s["x"], e, at, longest, s["experts"])
        return {"dx": dx, "dw": torch.bmm(dy.transpose(1, 2), x).to(t)}
    if s["op"] == "swiglu":
        f = s["f"]
        a, u = s["gu"][:, :f].float(), s["gu"][:, f:].float()
        at = s["row_map"].long()
        w = s["row_w"][at][:, None]
        sig = 1 / (1 + torch.exp(-a))
        if s["dir"] == "fwd":
            return {"h": (w * (a * sig) * u).to(t)}
        dh = s["dh"].float()
        da = w * dh * u * sig * (1 + a * (1 - sig))
        du = w * dh * (a * sig)
        drow = torch.zeros_like(s["row_w"])
        drow[at] = (dh * (a * sig) * u).sum(1)
        return {"dgu": torch.cat([da, du], 1).to(t), "drow_w": drow}
    p = TYPES[s["ptype"]]
    x, y = s["x"].float(), s["y"].float()
    post, pre, gates = s["gamma_post"].float(), s["gamma_pre"].float(), s["gates"]
    per = s["rows"] // gates
    gate = s["gate"].float().repeat_interleave(per, 0) if gates > 1 else s["gate"].float()
    r1 = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
    n = y * r1 * post
    if s["dir"] == "fwd":
        xo = x + s["alpha"] * gate * n
        return {"x_out": xo.to(t), "h": (xo * torch.rsqrt((xo * xo).mean(1, keepdim=True) + EPS) * pre).to(t)}
    dh = s["dh"].float()
    r2 = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    v = dh * pre
    d = s["dx_out"].float() + r2 * v - x * r2 ** 3 * (v * x).mean(1, keepdim=True)
    dn = s["alpha"] * gate * d
    q = dn * post
    dy = r1 * q - y * r1 ** 3 * (q * y).mean(1, keepdim=True)
    return {"dx": d.to(t), "dy": dy.to(t), "dgamma_post": (dn * y * r1).sum(0).to(p),
            "dgate": (s["alpha"] * d * n).reshape(gates, per, -1).sum(1).to(p),
            "dgamma_pre": (dh * x * r2).sum(0).to(p)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------- work
def work(case):
    b = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "grouped":
        rows, n, k = case["tokens"] * case["k"], case["n"], case["kdim"]
        weights = case["experts"] * n * k
        if case["dir"] == "bwd":
            return {"bytes": b * (2 * weights + 2 * rows * k + rows * n), "flops": 4 * rows * n * k}
        # an expert without rows is not read: at most one for each row
        return {"bytes": b * (min(case["experts"], rows) * n * k + rows * (n + k)), "flops": 2 * rows * n * k}
    if case["op"] == "swiglu":
        rows, f = case["tokens"] * case["k"], case["f"]
        if case["dir"] == "bwd":
            return {"bytes": b * 5 * rows * f + 12 * rows, "flops": 16 * rows * f}
        return {"bytes": b * 3 * rows * f + 8 * rows, "flops": 7 * rows * f}
    rows, d = case["rows"], case["d"]
    pb = (4 if case["ptype"] == "f32" else 2) * (2 + case["gates"]) * d
    if case["dir"] == "bwd":
        return {"bytes": b * 6 * rows * d + 2 * pb, "flops": 30 * rows * d}
    return {"bytes": b * 4 * rows * d + pb, "flops": 11 * rows * d}


# ------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The operators' definitions in 64 bits, an expert or a row at a time."""
    s = prepare(case, seed)
    if case["op"] == "grouped":
        cut = s["offsets"].tolist()
        rows = s["x"].shape[0]
        out = {}
        if case["dir"] == "fwd":
            out["y"] = torch.zeros(rows, case["n"], dtype=torch.float64, device=DEV)
        else:
            out["dx"] = torch.zeros(rows, case["kdim"], dtype=torch.float64, device=DEV)
            out["dw"] = torch.zeros(case["experts"], case["n"], case["kdim"], dtype=torch.float64, device=DEV)
        for e in range(case["experts"]):
            i, j = cut[e], cut[e + 1]
            if i == j:
                continue
            we = s["w"][e].double()
            if case["dir"] == "fwd":
                out["y"][i:j] = s["x"][i:j].double() @ we.t()
            else:
                dye = s["dy"][i:j].double()
                out["dx"][i:j] = dye @ we
                out["dw"][e] = dye.t() @ s["x"][i:j].double()
        return out
    if case["op"] == "swiglu":
        f = case["f"]
        gu = s["gu"].double()
        a, u = gu[:, :f], gu[:, f:]
        w = torch.take(s["row_w"].double(), s["row_map"].long()).unsqueeze(1)
        if case["dir"] == "fwd":
            return {"h": w * a * torch.sigmoid(a) * u}
        dh = s["dh"].double()
        silu = a * torch.sigmoid(a)
        slope = torch.sigmoid(a) + silu * torch.sigmoid(-a)
        drow = torch.empty_like(s["row_w"], dtype=torch.float64)
        drow.scatter_(0, s["row_map"].long(), torch.einsum("rf,rf->r", dh, silu * u))
        return {"dgu": torch.cat([dh * w * u * slope, dh * w * silu], dim=1), "drow_w": drow}
    d, gates, rows = case["d"], case["gates"], case["rows"]
    per = rows // gates
    shape = (gates, per, d)
    x, y = s["x"].double().view(shape), s["y"].double().view(shape)
    gate = s["gate"].double().view(gates, 1, d) * s["alpha"]
    post, pre = s["gamma_post"].double(), s["gamma_pre"].double()
    rms = lambda v: torch.sqrt(torch.linalg.vector_norm(v, dim=2, keepdim=True) ** 2 / d + EPS)  # noqa: E731
    yn = y / rms(y)
    if case["dir"] == "fwd":
        xo = x + gate * post * yn
        return {"x_out": xo.reshape(rows, d), "h": (xo / rms(xo) * pre).reshape(rows, d)}

    def back(v, dv):
        """Gradient of v / rms(v) along dv."""
        m = rms(v)
        vn = v / m
        return (dv - vn * (dv * vn).sum(2, keepdim=True) / d) / m

    dh = s["dh"].double().view(shape)
    dx = s["dx_out"].double().view(shape) + back(x, dh * pre)
    return {"dx": dx.reshape(rows, d), "dy": back(y, dx * gate * post).reshape(rows, d),
            "dgamma_post": (dx * gate * yn).sum((0, 1)), "dgate": (dx * s["alpha"] * post * yn).sum(1),
            "dgamma_pre": (dh * x / rms(x)).sum((0, 1))}
