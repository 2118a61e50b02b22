"""The operators of an MoE layer around the expert's activation cast, as they are measured: the residual
addition with the root-mean-square norm and its FP8 output, the routing of tokens to experts, both with their
gradients, and the experts' matrix-vector products with 4-bit weights.

``run`` computes a case either in plain torch operations (``own`` false) or with the package's entry points
(``own`` true); ``exact`` gives the same outputs from the definitions in 64 bits."""
import math

import torch

own = False  # which of the two forms run() takes

DEV = "cuda"
BF16, FP32, FP8, E8M0 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e8m0fnu
FLT_MAX = torch.finfo(torch.float32).max
DTYPES = {"bf16": BF16, "fp32": FP32}
# the package's tk_scale_fmt and tk_dtype values
SCALE_FMT = {"fp32": 0, "ue8m0": 1, "fp32_col": 2, "ue8m0_col": 3}
TK_DTYPE = {"bf16": 0, "fp32": 1, "fp8": 2}
SCORING = {"sigmoid": 0, "softmax": 1}
NORM_PARTS = 512  # rows of the norm's backward workspace
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---- the cases ------------------------------------------------------------------------------------------------


def _norm(name, n, hidden, dtype, residual, group, scale, keep):
    # keep: the normalised bf16 rows and 1/rms come back too (a router reads the first, a backward pass the second)
    return {"name": name, "op": "norm", "n": n, "hidden": hidden, "dtype": dtype, "residual": residual,
            "group": group, "scale": scale, "keep": keep}


def _norm_bwd(name, n, hidden, dtype, dresidual):
    return {"name": name, "op": "norm_bwd", "n": n, "hidden": hidden, "dtype": dtype, "dresidual": dresidual}


def _route(name, tokens, experts, k, groups, keep, scoring, bias, norm, dtype, masked):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "k": k, "groups": groups, "keep": keep,
            "scoring": scoring, "bias": bias, "norm": norm, "dtype": dtype, "masked": masked}


def _route_bwd(name, tokens, experts, k, scoring, norm, dtype):
    return {"name": name, "op": "route_bwd", "tokens": tokens, "experts": experts, "k": k, "scoring": scoring,
            "norm": norm, "dtype": dtype}


def _gemv(name, tokens, k, experts, out, inner, x, x_group, slots, scale, group, dtype):
    # k = 0: one matrix for every token; slots: each (token, choice) has an input row of its own
    return {"name": name, "op": "gemv", "tokens": tokens, "k": k, "experts": experts, "out": out, "in": inner, "x": x,
            "x_group": x_group, "slots": slots, "scale": scale, "group": group, "dtype": dtype}


def listed():
    return [
        # one decode step of a small batch: the layer's residual stream is added, normed and cast for the experts
        _norm("norm_decode", 8, 7168, "bf16", True, 128, "fp32", True),
        # prefill of 16384 tokens: per-block FP8 with power-of-two scales, what the backward needs kept
        _norm("norm_prefill", 16384, 7168, "bf16", True, 128, "ue8m0", True),
        # an fp32 stream, odd row count, groups of 96 columns that straddle lanes, no residual
        _norm("norm_fp32_odd", 1021, 2016, "fp32", False, 96, "fp32", False),
        # training: gradient of the norm, with the gradient that arrives through the residual stream
        _norm_bwd("norm_backward", 8192, 4096, "bf16", True),
        # a short ragged batch in fp32
        _norm_bwd("norm_backward_short", 333, 1024, "fp32", False),
        # one decode step: 256 experts in 8 groups keeping 4, sigmoid scores with the balancing bias
        _route("route_decode", 8, 256, 8, 8, 4, "sigmoid", True, True, "fp32", 0.0),
        # the same for a prefill
        _route("route_prefill", 16384, 256, 8, 8, 4, "sigmoid", True, True, "fp32", 0.0),
        # softmax scores without groups from bf16 logits, a tenth of the experts masked off (dropped devices)
        _route("route_softmax", 32768, 64, 6, 1, 1, "softmax", False, False, "bf16", 0.1),
        # training: gradients to the logits, sparse (sigmoid, renormalised) and dense (softmax over all)
        _route_bwd("route_backward", 16384, 256, 8, "sigmoid", True, "fp32"),
        _route_bwd("route_backward_soft", 4096, 160, 6, "softmax", False, "bf16"),
        # decode of one token: its 8 experts' gate and up rows, FP8 activations with a scale per 128 columns
        _gemv("gemv_gate_up", 1, 8, 256, 4096, 7168, "fp8", 128, False, "ue8m0", 32, "bf16"),
        # 16 tokens: the down projection of each (token, expert) row, FP8 with one scale a row
        _gemv("gemv_down", 16, 8, 64, 7168, 2048, "fp8", 0, True, "ue8m0", 32, "bf16"),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "route", "route", "route_bwd", "gemv", "gemv", "gemv"])
    if op in ("norm", "norm_bwd"):
        hidden = 8 * (2 * _between(rng, 8, 1023) + 1)
        if rng.random() < 0.5:
            hidden = rng.choice([1024, 2048, 4096, 7168, 8192, 16384])
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        n = _between(rng, 1, min(16384, 60_000_000 // hidden))
        if op == "norm_bwd":
            return {k: v for k, v in _norm_bwd("", n, hidden, dtype, rng.random() < 0.7).items() if k != "name"}
        fits = [g for g in (8, 16, 32, 64, 96, 128, 224, 256, 512, 896, 1024, 2048) if hidden % g == 0]
        c = _norm("", n, hidden, dtype, rng.random() < 0.7, rng.choice([0] + fits),
                  rng.choice(["fp32", "ue8m0", "fp32_col", "ue8m0_col"]), rng.random() < 0.6)
        return {k: v for k, v in c.items() if k != "name"}
    if op in ("route", "route_bwd"):
        tokens = _between(rng, 1, 32768)
        scoring, dtype, norm = rng.choice(["sigmoid", "softmax"]), rng.choice(["fp32", "bf16"]), rng.random() < 0.7
        if op == "route_bwd":
            experts = rng.choice([8, 33, 64, 100, 128, 160, 256, 384, 512])
            k = rng.choice([1, 2, 4, 6, 8])
            return {a: v for a, v in _route_bwd("", tokens, experts, k, scoring, norm, dtype).items() if a != "name"}
        experts, groups, keep = rng.choice([(8, 1, 1), (33, 1, 1), (64, 1, 1), (100, 1, 1), (128, 1, 1), (160, 8, 3),
                                            (256, 8, 4), (256, 1, 1), (256, 4, 2), (384, 1, 1), (512, 16, 8), (96, 3, 2)])
        k = rng.choice([1, 2, 4, 6, 8])
        c = _route("", tokens, experts, k, groups, keep, scoring, rng.random() < 0.6, norm, dtype,
                   rng.choice([0.0, 0.0, 0.1, 0.97]))
        return {a: v for a, v in c.items() if a != "name"}
    inner = 32 * (2 * _between(rng, 4, 127) + 1)
    if rng.random() < 0.6:
        inner = rng.choice([1024, 2048, 4096, 7168])
    out = _between(rng, 100, 8191) | 1
    if rng.random() < 0.6:
        out = rng.choice([1024, 2048, 4096, 7168])
    scale = rng.choice(["ue8m0", "ue8m0", "fp32"])
    groups = [g for g in ((0, 32, 64, 128, 256) if scale == "ue8m0" else (0, 128, 256)) if g == 0 or inner % g == 0]
    x = rng.choice(["bf16", "fp8", "fp8e"])
    xg = 0 if x == "bf16" else rng.choice([g for g in ((0, 32, 128) if x == "fp8e" else (0, 128)) if g == 0 or inner % g == 0])
    k = rng.choice([0, 0, 2, 4, 8])
    most = max(1, 800_000_000 // (out * inner * max(1, k)))
    tokens = _between(rng, 1, min(64, most))
    experts = rng.choice([8, 16, 32, 64]) if k else 1
    c = _gemv("", tokens, k, experts, out, inner, x, xg, bool(k) and rng.random() < 0.5, scale, rng.choice(groups),
              rng.choice(["bf16", "bf16", "fp32"]))
    return {a: v for a, v in c.items() if a != "name"}


def work(case):
    c, op = case, case["op"]
    if op == "norm":
        e, n, h = 2 if c["dtype"] == "bf16" else 4, c["n"], c["hidden"]
        per = e * (1 + 2 * c["residual"]) + 1 + 2 * c["keep"]
        scales = n * (h // (c["group"] or h)) * (4 if c["scale"].startswith("fp32") else 1)
        return {"bytes": n * h * per + scales + 4 * n * c["keep"] + 4 * h, "flops": 8 * n * h}
    if op == "norm_bwd":
        e, n, h = 2 if c["dtype"] == "bf16" else 4, c["n"], c["hidden"]
        return {"bytes": n * h * e * (3 + c["dresidual"]) + 4 * n + 8 * h, "flops": 10 * n * h}
    if op == "route":
        e, t, ex = 2 if c["dtype"] == "bf16" else 4, c["tokens"], c["experts"]
        return {"bytes": t * ex * e + 8 * t * c["k"] + 4 * ex * c["bias"], "flops": 10 * t * ex}
    if op == "route_bwd":
        e, t, ex = 2 if c["dtype"] == "bf16" else 4, c["tokens"], c["experts"]
        dense = c["scoring"] == "softmax" and not c["norm"]
        return {"bytes": t * ex * e + t * (ex if dense else c["k"]) * e + 8 * t * c["k"],
                "flops": (10 * t * ex if dense else 10 * t * c["k"])}
    t, k, ex, out, inner = c["tokens"], max(1, c["k"]), c["experts"], c["out"], c["in"]
    used = ex * (1 - (1 - k / ex) ** t) if c["k"] else 1  # experts that some token chose, on average
    rows = t * k if c["slots"] else t
    xb = rows * inner * (2 if c["x"] == "bf16" else 1)
    per_row = inner / 2 + (inner // (c["group"] or inner)) * (1 if c["scale"] == "ue8m0" else 4)
    return {"bytes": int(used * out * per_row + xb + t * k * out * (2 if c["dtype"] == "bf16" else 4)),
            "flops": 2 * t * k * out * inner}


# ---- the inputs -----------------------------------------------------------------------------------------------


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) % (1 << 62))
    return g


def _scale_buffer(fmt, n, groups):
    if fmt == "fp32":
        return torch.zeros((n, groups), dtype=FP32, device=DEV)
    if fmt == "ue8m0":
        return torch.zeros((n, groups), dtype=torch.uint8, device=DEV).view(E8M0)
    if fmt == "fp32_col":
        return torch.zeros((groups, -(-n // 4) * 4), dtype=FP32, device=DEV)
    return torch.zeros((groups, -(-n // 16) * 16), dtype=torch.uint8, device=DEV).view(E8M0)


def _fp8_rows(g, rows, inner, kind, group):
    """FP8 codes and scales of normal rows, as a cast leaves them: one scale for `group` columns (0: for the row)."""
    x = torch.randn((rows, inner), generator=g, device=DEV)
    x = x.view(rows, inner // (group or inner), group or inner)
    top = x.abs().amax(-1, keepdim=True)
    if kind == "fp8e":
        k = torch.ceil(torch.log2(top / 448.0))
        codes = (x * torch.exp2(-k)).clamp(-448, 448).to(FP8)
        scales = (k + 127).to(torch.uint8).view(E8M0)
    else:
        codes, scales = (x * (448.0 / top)).clamp(-448, 448).to(FP8), top / 448.0
    return codes.view(rows, inner), scales.view(rows, -1).contiguous()


def prepare(case, seed):
    c, g = case, _generator(seed)
    s = {"case": c}

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEV)

    op = c["op"]
    if op == "norm":
        n, h, dt = c["n"], c["hidden"], DTYPES[c["dtype"]]
        s["x"] = normal(n, h).to(dt)
        s["residual"] = (normal(n, h) * 4).to(dt) if c["residual"] else None
        s["weight"] = 1 + 0.25 * normal(h)
        s["residual_out"] = torch.empty((n, h), dtype=dt, device=DEV) if c["residual"] else None
        s["y"] = torch.empty((n, h), dtype=BF16, device=DEV) if c["keep"] else None
        s["rstd"] = torch.empty((n,), dtype=FP32, device=DEV) if c["keep"] else None
        s["codes"] = torch.empty((n, h), dtype=FP8, device=DEV)
        s["scales"] = _scale_buffer(c["scale"], n, h // (c["group"] or h))
    elif op == "norm_bwd":
        n, h, dt = c["n"], c["hidden"], DTYPES[c["dtype"]]
        s["h"] = (normal(n, h) * 4).to(dt)
        s["weight"] = 1 + 0.25 * normal(h)
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(-1) + 1e-6)
        s["dy"] = normal(n, h).to(dt)
        s["dresidual"] = normal(n, h).to(dt) if c["dresidual"] else None
        s["dx"] = torch.empty((n, h), dtype=dt, device=DEV)
        s["dweight"] = torch.empty((h,), dtype=FP32, device=DEV)
        s["workspace"] = torch.empty((NORM_PARTS, h), dtype=FP32, device=DEV)
    elif op in ("route", "route_bwd"):
        t, e, k, dt = c["tokens"], c["experts"], c["k"], DTYPES[c["dtype"]]
        logits = 2 * normal(t, e)
        if c.get("masked"):
            logits = torch.where(uniform(t, e) < c["masked"], -math.inf, logits)
        s["logits"] = logits.to(dt)
        if op == "route":
            s["bias"] = 0.1 * normal(e) if c["bias"] else None
            s["idx"] = torch.empty((t, k), dtype=torch.int32, device=DEV)
            s["weight"] = torch.empty((t, k), dtype=FP32, device=DEV)
        else:
            idx = torch.topk(logits, k, dim=-1).indices.to(torch.int32)
            s["idx"] = torch.where(uniform(t, k) < 0.01, -1, idx).contiguous()  # a few slots were dropped
            s["dweight"] = normal(t, k)
            s["dlogits"] = torch.empty((t, e), dtype=dt, device=DEV)
    else:
        t, k, e, out, inner = c["tokens"], c["k"], c["experts"], c["out"], c["in"]
        rows = t * max(1, k) if c["slots"] else t
        if c["x"] == "bf16":
            s["x"], s["x_scales"] = normal(rows, inner).to(BF16), None
        else:
            s["x"], s["x_scales"] = _fp8_rows(g, rows, inner, c["x"], c["x_group"])
        s["codes"] = torch.randint(0, 256, (e, out, inner // 2), generator=g, device=DEV, dtype=torch.uint8)
        groups = inner // (c["group"] or inner)
        if c["scale"] == "ue8m0":
            s["scales"] = torch.randint(118, 123, (e, out, groups), generator=g, device=DEV, dtype=torch.uint8).view(E8M0)
        else:
            s["scales"] = 0.002 + 0.03 * uniform(e, out, groups)
        s["idx"] = torch.topk(uniform(t, e), k, dim=-1).indices.to(torch.int32).contiguous() if k else None
        s["y"] = torch.empty((t * max(1, k), out), dtype=DTYPES[c["dtype"]], device=DEV)
    return s


# ---- one pass -------------------------------------------------------------------------------------------------


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


def _own(s):
    import moe_activation_bit_amd as tk
    c, op = s["case"], s["case"]["op"]
    if op == "norm":
        rc = tk.tk_rmsnorm_cast_fp8(s["x"], s["residual"], TK_DTYPE[c["dtype"]], s["weight"], c["n"], c["hidden"], 1e-6,
                                    c["group"], SCALE_FMT[c["scale"]], s["residual_out"], s["y"], s["rstd"], s["codes"],
                                    s["scales"])
        out = {m: s[m] for m in ("codes", "scales", "residual_out", "y", "rstd")}
    elif op == "norm_bwd":
        rc = tk.tk_rmsnorm_backward(s["dy"], s["h"], TK_DTYPE[c["dtype"]], s["weight"], s["rstd"], s["dresidual"], c["n"],
                                    c["hidden"], s["dx"], s["dweight"], s["workspace"])
        out = {"dx": s["dx"], "dweight": s["dweight"]}
    elif op == "route":
        rc = tk.tk_route(s["logits"], TK_DTYPE[c["dtype"]], s["bias"], c["tokens"], c["experts"], c["k"], c["groups"],
                         c["keep"], SCORING[c["scoring"]], c["norm"], 2.5, s["idx"], s["weight"])
        out = {"idx": s["idx"], "weight": s["weight"]}
    elif op == "route_bwd":
        rc = tk.tk_route_backward(s["dweight"], s["idx"], s["logits"], TK_DTYPE[c["dtype"]], c["tokens"], c["experts"],
                                  c["k"], SCORING[c["scoring"]], c["norm"], 2.5, s["dlogits"])
        out = {"dlogits": s["dlogits"]}
    else:
        rc = tk.tk_expert_gemv_fp4(s["x"], s["x_scales"], TK_DTYPE["bf16" if c["x"] == "bf16" else "fp8"],
                                   SCALE_FMT["ue8m0" if c["x"] == "fp8e" else "fp32"], c["x_group"], s["idx"], c["tokens"],
                                   max(1, c["k"]), c["slots"], s["codes"], s["scales"], SCALE_FMT[c["scale"]], c["group"],
                                   c["experts"], c["out"], c["in"], TK_DTYPE[c["dtype"]], s["y"])
        out = {"y": s["y"]}
    if rc != 0:
        raise RuntimeError(tk.tk_status_str(rc))
    return out


def _plain_norm(s):
    c = s["case"]
    n, h, G = c["n"], c["hidden"], c["group"] or c["hidden"]
    a = s["x"].float() if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["x"].dtype).float()
    rstd = 1.0 / torch.sqrt((a * a).sum(-1) / h + 1e-6)
    y = a * rstd[:, None] * s["weight"]
    top = y.view(n, h // G, G).abs().amax(-1)
    if c["scale"].startswith("fp32"):
        scales, inv = top / 448.0, (448.0 / top).clamp(max=FLT_MAX)
    else:
        m, e = torch.frexp(top)  # top = m * 2^e, 448 = 0.875 * 2^9
        k = (e - 9 + (m > 0.875).to(torch.int32)).clamp(min=-127)
        k = torch.where(top == 0, -127, k)
        scales, inv = (k + 127).to(torch.uint8), torch.ldexp(torch.ones_like(top), -k)
    codes = (y.view(n, h // G, G) * inv[..., None]).clamp(-448, 448).to(FP8).view(n, h)
    if c["scale"].endswith("_col"):
        cols = torch.zeros(s["scales"].shape, dtype=scales.dtype, device=DEV)
        cols[:, :n] = scales.t()
        scales = cols
    if not c["scale"].startswith("fp32"):
        scales = scales.view(E8M0)
    return {"codes": codes, "scales": scales, "residual_out": a.to(s["x"].dtype) if c["residual"] else None,
            "y": y.to(BF16) if c["keep"] else None, "rstd": rstd if c["keep"] else None}


def _plain_norm_bwd(s):
    h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
    g = dy * s["weight"]
    hat = h * rstd
    dx = rstd * (g - hat * ((g * hat).sum(-1, keepdim=True) / h.shape[1]))
    if s["dresidual"] is not None:
        dx = dx + s["dresidual"].float()
    return {"dx": dx.to(s["h"].dtype), "dweight": (dy * hat).sum(0)}


def _plain_scores(logits, scoring):
    """Scores in 64 bits; masked experts (-inf) score 0, and so does a row that the mask leaves empty."""
    x = logits.double()
    if scoring == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, 1.0, total)


def _plain_route(s):
    c = s["case"]
    t, e, ng = c["tokens"], c["experts"], c["groups"]
    logits = s["logits"]
    score = _plain_scores(logits, c["scoring"])
    live = logits > -math.inf
    if s["bias"] is None and ng == 1:
        key = logits.float()  # either score grows with the logit
    else:
        key = score.float()  # the order is that of the rounded scores: those next to each other are computed in 64 bits
        if s["bias"] is not None:
            key = key + s["bias"]
        key = torch.where(live, key, -math.inf)
    if ng > 1:
        best = torch.sort(key.view(t, ng, e // ng), dim=-1, descending=True).values[..., :2]
        total = best[..., 0] + torch.where(best[..., 1] > -math.inf, best[..., 1], 0.0)
        kept = torch.sort(total, dim=-1, descending=True, stable=True).indices[:, :c["keep"]]
        drop = torch.ones((t, ng), dtype=torch.bool, device=DEV).scatter_(1, kept, False)
        key = torch.where(drop[..., None].expand(t, ng, e // ng).reshape(t, e), -math.inf, key)
    top = torch.sort(key, dim=-1, descending=True, stable=True)
    idx = top.indices[:, :c["k"]]
    absent = top.values[:, :c["k"]] == -math.inf
    w = torch.where(absent, 0.0, torch.gather(score, 1, idx))
    if c["norm"]:
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total == 0, 1.0, total)
    return {"idx": torch.where(absent, -1, idx).to(torch.int32), "weight": (w * 2.5).float()}


def _plain_route_bwd(s):
    c = s["case"]
    x, absent = s["logits"].float(), s["idx"] < 0
    idx = s["idx"].clamp(min=0).long()
    dw = torch.where(absent, 0.0, s["dweight"] * 2.5)
    if c["scoring"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        score = torch.exp(x - x.amax(-1, keepdim=True))
        score = score / score.sum(-1, keepdim=True)
    w = torch.where(absent, 0.0, torch.gather(score, 1, idx))
    if c["norm"]:
        total = w.sum(-1, keepdim=True)
        total = torch.where(total == 0, 1.0, total)
        dw = torch.where(absent, 0.0, (dw - (dw * w).sum(-1, keepdim=True) / total) / total)
    if c["scoring"] == "sigmoid":
        d = torch.zeros_like(x).scatter_add_(1, idx, dw * w * (1.0 - w))
    else:
        d = torch.zeros_like(x).scatter_add_(1, idx, dw * w) - score * (dw * w).sum(-1, keepdim=True)
    return {"dlogits": d.to(s["logits"].dtype)}


def _plain_fp4(codes, scales):
    """The 4-bit weights' values: the low half of a byte is the even column."""
    table = torch.tensor(E2M1, dtype=FP32, device=DEV)
    c = torch.stack([codes & 15, codes >> 4], -1).view(*codes.shape[:-1], -1)
    w = table[c.to(torch.int32)]
    return (w.view(*scales.shape, -1) * scales.float()[..., None]).view(*w.shape)


def _plain_gemv(s):
    c = s["case"]
    t, k = c["tokens"], max(1, c["k"])
    x = s["x"].float()
    if s["x_scales"] is not None:
        x = (x.view(*s["x_scales"].shape, -1) * s["x_scales"].float()[..., None]).view(*x.shape)
    if s["idx"] is None:
        y = x @ _plain_fp4(s["codes"][0], s["scales"][0]).t()
    else:
        e = s["idx"].reshape(-1).long()
        w = _plain_fp4(s["codes"][e], s["scales"][e])
        if not c["slots"]:
            x = x.repeat_interleave(k, 0)
        y = torch.bmm(w, x[:, :, None])[:, :, 0]
    return {"y": y.to(s["y"].dtype)}


_PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "route": _plain_route, "route_bwd": _plain_route_bwd,
          "gemv": _plain_gemv}


# ---- the definitions in 64 bits -------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    c, op, D = case, case["op"], torch.float64
    if op == "norm":
        n, h, G = c["n"], c["hidden"], c["group"] or c["hidden"]
        a = s["x"].to(D)
        if s["residual"] is not None:
            a = (a + s["residual"].to(D)).to(s["x"].dtype).to(D)
        rstd = (a.square().mean(1) + 1e-6).pow(-0.5)
        y = torch.einsum("nh,n,h->nh", a, rstd, s["weight"].to(D))
        parts = y.reshape(n, -1, G)
        top = parts.abs().max(2).values
        if c["scale"].startswith("fp32"):
            scales, step = top / 448, top / 448
        else:
            exponent = torch.ceil(torch.log2(top / 448)).clamp(min=-127)
            scales, step = exponent.exp2(), exponent.exp2()
        codes = torch.where(step[..., None] > 0, parts / step[..., None], 0.0).clamp(-448, 448).to(FP32).to(FP8)
        if c["scale"].endswith("_col"):
            full = torch.zeros(s["scales"].shape, dtype=D, device=DEV)
            full += 0.0 if c["scale"] == "fp32_col" else 2.0 ** -127  # the value of an unwritten zero byte
            full[:, :n] = scales.T
            scales = full
        return {"codes": codes.view(n, h), "scales": scales, "residual_out": a if c["residual"] else None,
                "y": y if c["keep"] else None, "rstd": rstd if c["keep"] else None}
    if op == "norm_bwd":
        h, dy, r, w = (s[m].to(D) for m in ("h", "dy", "rstd", "weight"))
        dot = torch.einsum("nh,nh,h->n", h, dy, w)
        dx = r[:, None] * w * dy - (r ** 3 * dot / h.shape[1])[:, None] * h
        if s["dresidual"] is not None:
            dx += s["dresidual"].to(D)
        return {"dx": dx, "dweight": torch.einsum("nh,nh,n->h", dy, h, r)}
    if op == "route":
        return _exact_route(c, s)
    if op == "route_bwd":
        x, dw = s["logits"].to(D), s["dweight"].to(D) * 2.5
        t, e = x.shape
        chosen = torch.zeros((t, e + 1), dtype=D, device=DEV)
        up = torch.zeros((t, e + 1), dtype=D, device=DEV)
        at = torch.where(s["idx"] < 0, e, s["idx"]).long()
        chosen.scatter_(1, at, 1.0)
        up.scatter_(1, at, dw)
        chosen, up = chosen[:, :e], up[:, :e]
        up = up * chosen
        if c["scoring"] == "sigmoid":
            p = torch.sigmoid(x)
            if c["norm"]:
                total = (p * chosen).sum(1, keepdim=True).clamp(min=1e-300)
                up = chosen * (up * total - (up * p * chosen).sum(1, keepdim=True)) / total ** 2
            return {"dlogits": up * p * torch.sigmoid(-x)}
        p = torch.softmax(x, 1)
        if c["norm"]:
            p = p * chosen
            p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
        return {"dlogits": p * (up - (up * p).sum(1, keepdim=True))}
    t, k = c["tokens"], max(1, c["k"])
    x = s["x"].to(D)
    if s["x_scales"] is not None:
        x = x * s["x_scales"].to(FP32).to(D).repeat_interleave(x.shape[1] // s["x_scales"].shape[1], 1)
    lut = torch.tensor(E2M1, dtype=D, device=DEV)
    rows = []
    for r in range(t * k):
        e = 0 if s["idx"] is None else int(s["idx"][r // k, r % k])
        b = s["codes"][e].to(torch.int32)
        w = torch.empty((c["out"], c["in"]), dtype=D, device=DEV)
        w[:, 0::2], w[:, 1::2] = lut[b % 16], lut[b // 16]
        w *= s["scales"][e].to(FP32).to(D).repeat_interleave(c["in"] // s["scales"].shape[2], 1)
        rows.append(w @ x[r if c["slots"] else r // k])
    return {"y": torch.stack(rows)}


def _exact_route(c, s):
    import numpy as np
    x = s["logits"].float().cpu().numpy().astype(np.float64)
    t, e = x.shape
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if c["scoring"] == "sigmoid":
            p = np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))
        else:
            top = x.max(1, keepdims=True)
            p = np.exp(x - np.where(np.isinf(top), 0, top))
            p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
    bias = None if s["bias"] is None else s["bias"].cpu().numpy()
    key = x.astype(np.float32) if bias is None and c["groups"] == 1 else p.astype(np.float32)
    key = key if bias is None else key + bias
    key = np.where(np.isinf(x), np.float32(-np.inf), key).astype(np.float32)
    per = e // c["groups"]
    if c["groups"] > 1:
        two = np.partition(key.reshape(t, c["groups"], per), per - 2, axis=2)[:, :, -2:]
        total = (two[:, :, 1] + np.where(np.isinf(two[:, :, 0]), np.float32(0), two[:, :, 0])).astype(np.float32)
        rank = np.argsort(np.argsort(-total, axis=1, kind="stable"), axis=1, kind="stable")
        key = np.where(np.repeat(rank, per, axis=1) < c["keep"], key, np.float32(-np.inf))
    idx = np.argsort(-key, axis=1, kind="stable")[:, :c["k"]]
    gone = np.isinf(np.take_along_axis(key, idx, 1))
    w = np.where(gone, 0.0, np.take_along_axis(p, idx, 1))
    if c["norm"]:
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
    return {"idx": torch.from_numpy(np.where(gone, -1, idx).astype(np.int32)), "weight": torch.from_numpy(w * 2.5)}
