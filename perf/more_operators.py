"""Real calls of the framework's operators around its expert products, and their plain forms.

Four operators (include/nvfp4.h):
- nvfp4_route, nvfp4_route_backward: scores of the experts, the choice of each
  token's, their weights and the order of the rows by expert;
- nvfp4_dispatch, nvfp4_combine, nvfp4_combine_backward: rows into that order,
  and back as weighted sums;
- nvfp4_rmsnorm, nvfp4_rmsnorm_backward: root-mean-square norm with the
  residual's addition, out in bf16 or in int8 with a scale per row;
- nvfp4_bf16_linear, nvfp4_bf16_linear_backward: a product with bias,
  activation and residual in its epilogue, dense or grouped by expert.
`own` chooses between the framework's calls and the plain forms.
"""
import math

import torch

own = False

EPS = 1e-6
GELU = math.sqrt(2.0 / math.pi)


def listed():
    return [
        # a batch of decoding requests through a router with a balance bias and groups: latency
        {"name": "route decode", "op": "route", "pass": "fwd", "rows": 16, "experts": 64, "k": 8, "groups": 8, "kept": 4,
         "score": "sigmoid", "bias": True, "renorm": True, "dtype": "fp32", "pad": 0.0},
        # a training batch of 16384 tokens, softmax scores, no bias
        {"name": "route softmax", "op": "route", "pass": "fwd", "rows": 16384, "experts": 128, "k": 8, "groups": 1, "kept": 1,
         "score": "softmax", "bias": False, "renorm": True, "dtype": "fp32", "pad": 0.0},
        # the same length through sigmoid scores, a balance bias and groups, with padded tokens
        {"name": "route groups", "op": "route", "pass": "fwd", "rows": 16384, "experts": 256, "k": 8, "groups": 8, "kept": 4,
         "score": "sigmoid", "bias": True, "renorm": True, "dtype": "bf16", "pad": 0.03},
        # gradients of the logits from those of the weights
        {"name": "route backward", "op": "route", "pass": "bwd", "rows": 16384, "experts": 256, "k": 8, "groups": 1, "kept": 1,
         "score": "softmax", "bias": False, "renorm": False, "dtype": "fp32", "pad": 0.0},
        # the experts' answers to a few decoding requests, weighted and added to the residual
        {"name": "combine decode", "op": "move", "pass": "combine", "rows": 7, "k": 8, "cols": 2048, "weights": True,
         "residual": True, "from": "bf16", "out": "bf16", "pad": 0.0},
        # a training batch's tokens into the experts' order
        {"name": "dispatch", "op": "move", "pass": "dispatch", "rows": 8192, "k": 4, "cols": 5120, "weights": False,
         "residual": False, "from": "bf16", "out": "bf16", "pad": 0.0},
        # gradients of the combination: to the experts' rows and to the weights; odd sizes, padded tokens
        {"name": "combine backward", "op": "move", "pass": "bwd", "rows": 4001, "k": 6, "cols": 2568, "weights": True,
         "residual": False, "from": "bf16", "out": "bf16", "pad": 0.05},
        # one token before an int8 product
        {"name": "norm one token int8", "op": "norm", "pass": "int8", "rows": 1, "cols": 5120, "residual": True,
         "x": "bf16", "stream": "bf16", "weight": "bf16"},
        # a prompt or a training batch
        {"name": "norm", "op": "norm", "pass": "fwd", "rows": 8192, "cols": 5120, "residual": True,
         "x": "bf16", "stream": "bf16", "weight": "bf16"},
        # its gradients, with the one that comes along the residual
        {"name": "norm backward", "op": "norm", "pass": "bwd", "rows": 8192, "cols": 5120, "residual": True,
         "x": "bf16", "stream": "bf16", "weight": "fp32"},
        # an expert layer's first product with bias and activation, its sums before the activation kept for the backward pass
        {"name": "linear experts", "op": "linear", "pass": "fwd", "rows": 8192, "experts": 8, "skew": 0.5, "n": 5120, "k": 2560,
         "act": "relu2", "bias": True, "residual": False, "pre": True, "out": "bf16"},
        # gradients through that activation, and of the biases
        {"name": "linear backward", "op": "linear", "pass": "bwd", "rows": 8192, "experts": 8, "skew": 0.5, "n": 5120, "k": 2560,
         "act": "relu2", "bias": True, "residual": False, "pre": True, "out": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["route", "move", "norm", "linear"])
    some = rng.choice([0.0, 0.0, 0.04])
    if op == "route":
        which = rng.choice(["fwd", "fwd", "bwd"])
        groups = rng.choice([1, 1, 2, 4, 8]) if which == "fwd" else 1
        experts = groups * _log_int(rng, 4, max(4, 256 // groups))
        kept = rng.randint(1, groups)
        return {"op": op, "pass": which, "rows": _log_int(rng, 1, 16384), "experts": experts,
                "k": min(rng.randint(1, 8), kept * (experts // groups)), "groups": groups, "kept": kept,
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "renorm": rng.random() < 0.6,
                "dtype": rng.choice(["fp32", "bf16"]), "pad": some}
    if op == "move":
        which = rng.choice(["dispatch", "combine", "combine", "bwd"])
        k, cols = rng.randint(1, 8), 8 * _log_int(rng, 8, 640)
        return {"op": op, "pass": which, "rows": _log_int(rng, 1, max(1, min(16384, 400_000_000 // ((4 * k + 8) * cols)))), "k": k, "cols": cols,
                "weights": which == "bwd" or (which == "combine" and rng.random() < 0.6),
                "residual": which == "combine" and rng.random() < 0.5,
                "from": "bf16" if which == "dispatch" else rng.choice(["bf16", "fp32"]),
                "out": rng.choice(["bf16", "fp32"]) if which == "combine" else "bf16", "pad": some}
    if op == "norm":
        which = rng.choice(["fwd", "int8", "bwd"])
        return {"op": op, "pass": which, "rows": _log_int(rng, 1, 4096), "cols": 16 * _log_int(rng, 4, 320),
                "residual": rng.random() < 0.7, "x": rng.choice(["bf16", "bf16", "fp32"]),
                "stream": rng.choice(["bf16", "fp32"]), "weight": rng.choice(["bf16", "fp32"])}
    n, k = (8 * _log_int(rng, 16, 640) for _ in range(2))
    which, experts = rng.choice(["fwd", "fwd", "bwd"]), rng.choice([0, 0, _log_int(rng, 1, 32)])
    act = rng.choice(["none", "relu2", "silu", "gelu"]) if which == "fwd" else rng.choice(["relu2", "silu", "gelu"])
    return {"op": op, "pass": which, "rows": _log_int(rng, 1, 4096), "n": n, "k": k,
            "experts": min(experts, max(1, 8 * 5120 * 2560 // (n * k))) if experts else 0, "skew": round(rng.uniform(0.0, 1.0), 2),
            "act": act, "bias": which == "bwd" or rng.random() < 0.6, "residual": which == "fwd" and rng.random() < 0.5,
            "pre": act != "none" and (which == "bwd" or rng.random() < 0.5), "out": rng.choice(["bf16", "fp32"]) if which == "fwd" else "bf16"}


def _dtype(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def prepare(case, seed):
    g = _generator(seed)
    return {"route": _prepare_route, "move": _prepare_move, "norm": _prepare_norm, "linear": _prepare_linear}[case["op"]](case, seed, g)


def _padding(case, g):
    """Which tokens are padding: their logits are all minus infinity."""
    return torch.rand(case["rows"], generator=g, device="cuda") < case["pad"]


def _prepare_route(case, seed, g):
    T, E = case["rows"], case["experts"]
    # some experts are liked more than others
    logits = (1.5 * _randn(g, T, E) + 0.5 * _randn(g, 1, E))
    logits[_padding(case, g)] = -math.inf
    s = {"case": case, "logits": logits.to(_dtype(case["dtype"])), "bias": 0.1 * _randn(g, E) if case["bias"] else None}
    if case["pass"] == "bwd":
        s["experts"] = _choose(case, s["logits"], s["bias"])[0]
        s["dweights"] = 1e-2 * _randn(g, T, case["k"])
    return s


def _prepare_move(case, seed, g):
    T, k, cols = case["rows"], case["k"], case["cols"]
    # places in an expert order: each token to k experts of 4 k
    pick = torch.rand(T, 4 * k, generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32)
    pick[_padding(case, g)] = -1
    rows, _ = _places(pick, 4 * k)
    s = {"case": case, "rows": rows}
    if case["pass"] == "dispatch":
        s["x"] = _randn(g, T, cols).bfloat16()
    else:
        s["o"] = _randn(g, T * k, cols).to(_dtype(case["from"]))
        s["weights"] = torch.rand(T, k, generator=g, device="cuda").softmax(1) if case["weights"] else None
        s["residual"] = _randn(g, T, cols).to(_dtype(case["out"])) if case["residual"] else None
    if case["pass"] == "bwd":
        s["dy"] = (1e-2 * _randn(g, T, cols)).bfloat16()
    if case["pass"] != "combine":  # the rows behind the last place are nobody's: left as they were
        s["buffer"] = torch.zeros(T * k, cols, dtype=torch.bfloat16, device="cuda")
    return s


def _prepare_norm(case, seed, g):
    T, cols = case["rows"], case["cols"]
    # a few large channels, rows of unequal size
    x = _randn(g, T, cols) * torch.exp(0.5 * _randn(g, 1, cols)) * torch.exp(0.3 * _randn(g, T, 1))
    s = {"case": case, "weight": (1.0 + 0.2 * _randn(g, cols)).to(_dtype(case["weight"]))}
    if case["pass"] == "bwd":
        s["h"] = x.to(_dtype(case["stream"]))
        s["dy"] = (1e-2 * _randn(g, T, cols)).to(_dtype(case["x"]))
        s["dh"] = (1e-2 * _randn(g, T, cols)).to(_dtype(case["stream"])) if case["residual"] else None
    else:
        s["x"] = x.to(_dtype(case["x"]))
        s["residual"] = (2.0 * _randn(g, T, cols)).to(_dtype(case["stream"])) if case["residual"] else None
    return s


def _expert_rows(case):
    """Rows of each expert: proportional to 1 / rank^skew, rounded so that they add up."""
    share = [1.0 / (e + 1) ** case["skew"] for e in range(case["experts"])]
    total, done, rows = sum(share), 0, []
    for e in range(case["experts"]):
        upto = round(case["rows"] * sum(share[:e + 1]) / total)
        rows.append(upto - done)
        done = upto
    return rows


def _prepare_linear(case, seed, g):
    T, E, N, K = case["rows"], case["experts"], case["n"], case["k"]
    s = {"case": case, "ends": None, "most": T}
    if E:
        rows = _expert_rows(case)
        turn = seed % len(rows)  # which expert is busiest differs from batch to batch
        rows = rows[turn:] + rows[:turn]
        s["ends"], s["most"] = torch.cumsum(torch.tensor(rows, device="cuda"), 0).int(), max(rows)
    if case["pass"] == "bwd":
        s["pre"] = _randn(g, T, N).bfloat16()
        s["dy"] = (1e-2 * _randn(g, T, N)).bfloat16()
        return s
    s["x"] = _randn(g, T, K).bfloat16()
    s["w"] = _randn(g, *((E, N, K) if E else (N, K))).mul_(K ** -0.5).bfloat16()
    s["bias"] = 0.3 * _randn(g, *((E, N) if E else (N,))) if case["bias"] else None
    s["residual"] = _randn(g, T, N).to(_dtype(case["out"])) if case["residual"] else None
    return s


# ---- the plain forms ----

def _scores(case, logits):
    """Scores in 64 bits: a choice between two experts goes by their last bits."""
    l = logits.double()
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(torch.isfinite(top), top, 0.0))
    return e / e.sum(1, keepdim=True).clamp(min=1e-300)


def _choose(case, logits, bias):
    """The experts of each token (T x k, -1: none) and the scores of all."""
    T, E, k, G = case["rows"], case["experts"], case["k"], case["groups"]
    s = _scores(case, logits)
    c = s if bias is None else s + bias.double()
    c = torch.where(torch.isfinite(logits), c, -math.inf)
    allowed = torch.isfinite(c)
    if case["kept"] < G:
        best = c.view(T, G, E // G).sort(dim=2, descending=True)[0][:, :, :2]
        value = torch.where(torch.isfinite(best), best, 0.0).sum(2)
        value = torch.where(torch.isfinite(best[:, :, 0]), value, -math.inf)
        order = value.sort(dim=1, descending=True, stable=True)[1][:, :case["kept"]]
        group = torch.zeros(T, G, dtype=torch.bool, device=c.device).scatter_(1, order, True)
        allowed = allowed & group.repeat_interleave(E // G, 1)
    # without a bias the logits have the scores' order, and ties only where they are equal
    by = torch.where(allowed, logits.double() if bias is None else c, -math.inf)
    picked = by.sort(dim=1, descending=True, stable=True)[1][:, :k]
    return torch.where(allowed.gather(1, picked), picked, -1).to(torch.int32), s


def _weights(case, s, experts):
    w = s.gather(1, experts.clamp(min=0).long()) * (experts >= 0)
    return w / w.sum(1, keepdim=True).clamp(min=1e-300) if case["renorm"] else w


def _places(experts, E):
    """The place of each slot when they are sorted by expert, then token, and each expert's end."""
    flat = torch.where(experts < 0, E, experts).flatten().long()
    sorted_, order = flat.sort(dim=0, stable=True)
    rows = torch.empty_like(order)
    rows[order] = torch.arange(len(flat), device=flat.device)
    ends = torch.searchsorted(sorted_, torch.arange(E, device=flat.device), right=True)
    return torch.where(flat < E, rows, -1).view(experts.shape).int(), ends.int()


def _plain_route(s):
    case = s["case"]
    if case["pass"] == "fwd":
        experts, scores = _choose(case, s["logits"], s["bias"])
        rows, ends = _places(experts, case["experts"])
        return {"experts": experts, "weights": _weights(case, scores, experts).float(), "rows": rows, "ends": ends}
    scores, there = _scores(case, s["logits"]).float(), s["experts"] >= 0
    at = s["experts"].clamp(min=0).long()
    g, p = s["dweights"] * there, scores.gather(1, at) * there
    if case["renorm"]:
        rest = 1.0 - p if case["score"] == "sigmoid" else 1.0
        p = p / p.sum(1, keepdim=True).clamp(min=1e-30)
        d = p * (g - (g * p).sum(1, keepdim=True)) * rest
        out = torch.zeros_like(scores).scatter_add_(1, at, d * there)
    elif case["score"] == "sigmoid":
        out = torch.zeros_like(scores).scatter_add_(1, at, g * p * (1.0 - p))
    else:
        out = torch.zeros_like(scores).scatter_add_(1, at, g * p) - scores * (g * p).sum(1, keepdim=True)
    return out.to(s["logits"].dtype)


def _plain_move(s):
    case, rows = s["case"], s["rows"]
    at, there = rows.clamp(min=0).long(), rows >= 0
    if case["pass"] == "dispatch":
        token = torch.arange(case["rows"], device=rows.device)[:, None].expand_as(rows)
        s["buffer"][at[there]] = s["x"][token[there]]
        return s["buffer"]
    o = s["o"][at].float() * there[..., None]  # T x k x cols
    if case["pass"] == "combine":
        y = (o * s["weights"][..., None]).sum(1) if case["weights"] else o.sum(1)
        if case["residual"]:
            y = y + s["residual"].float()
        return y.to(_dtype(case["out"]))
    dy = s["dy"].float()[:, None]
    s["buffer"][at[there]] = (dy * s["weights"][..., None])[there].bfloat16()
    return {"rows": s["buffer"], "weights": (dy * o).sum(2)}


def _plain_norm(s):
    case, w = s["case"], s["weight"].float()
    if case["pass"] == "bwd":
        h, dy = s["h"].float(), s["dy"].float()
        rstd = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        xhat, u = h * rstd, dy * w
        dx = rstd * (u - xhat * (u * xhat).mean(1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(_dtype(case["stream"])), "dweight": (dy * xhat).sum(0)}
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * w
    out = {} if s["residual"] is None else {"h": h.to(_dtype(case["stream"]))}
    if case["pass"] == "fwd":
        return {**out, "y": y.bfloat16()}
    top = y.abs().amax(1, keepdim=True)
    codes = torch.round(y * (127.0 / torch.where(top > 0, top, 1.0)))
    return {**out, "codes": codes.bfloat16(), "scales": (top / 127.0).view(-1)}  # (the whole numbers as bf16 holds them)


def _act(name, z):
    if name == "relu2":
        return z.clamp(min=0.0).square()
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.tanh(GELU * (z + 0.044715 * z ** 3)))
    return z


def _act_slope(name, z):
    if name == "relu2":
        return 2.0 * z.clamp(min=0.0)
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    t = torch.tanh(GELU * (z + 0.044715 * z ** 3))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * GELU * (1.0 + 3 * 0.044715 * z * z)


def _by_expert(rows, ends, most):
    """rows (T x C) as E x most x C, zeros behind each expert's rows; also the places that hold rows."""
    begins = torch.cat([ends.new_zeros(1), ends[:-1]])
    at = begins[:, None] + torch.arange(most, device=rows.device, dtype=torch.int32)[None]
    there = at < ends[:, None]
    return rows[torch.where(there, at, 0).long()].float() * there[..., None], there


def _plain_linear(s):
    case, ends = s["case"], s["ends"]
    if case["pass"] == "bwd":
        dz = s["dy"].float() * _act_slope(case["act"], s["pre"].float())
        db = dz.sum(0) if ends is None else _by_expert(dz, ends, s["most"])[0].sum(1)
        return {"dpre": dz.bfloat16(), "dbias": db}
    if ends is None:
        z = s["x"].float() @ s["w"].float().t()
        if case["bias"]:
            z = z + s["bias"]
    else:
        x, there = _by_expert(s["x"], ends, s["most"])
        z = torch.bmm(x, s["w"].float().transpose(1, 2))
        if case["bias"]:
            z = z + s["bias"][:, None]
        z = z[there]
    y = _act(case["act"], z)
    if case["residual"]:
        y = y + s["residual"].float()
    y = y.to(_dtype(case["out"]))
    return {"y": y, "pre": z.bfloat16()} if case["pre"] else y


# ---- the framework's calls ----

def _own_route(s):
    import quantize_precision_gemm_amd as q
    case = s["case"]
    score = q.SIGMOID if case["score"] == "sigmoid" else q.SOFTMAX
    if case["pass"] == "bwd":
        return q.nvfp4_route_backward(s["logits"], s["experts"], s["dweights"], score, renormalise=case["renorm"],
                                      out_dtype=s["logits"].dtype)
    if "plan" not in s:  # a layer keeps its buffers from batch to batch
        s["plan"] = q.Routing.empty(case["rows"], case["experts"], case["k"], s["logits"].device)
    r = q.nvfp4_route(s["logits"], case["k"], score, bias=s["bias"], groups=case["groups"], groups_kept=case["kept"],
                      renormalise=case["renorm"], out=s["plan"])
    return {"experts": r.experts, "weights": r.weights, "rows": r.rows, "ends": r.ends}


def _own_move(s):
    import quantize_precision_gemm_amd as q
    case = s["case"]
    if case["pass"] == "dispatch":
        return q.nvfp4_dispatch(s["x"], s["rows"], out=s["buffer"])
    if case["pass"] == "combine":
        return q.nvfp4_combine(s["o"], s["rows"], s["weights"], residual=s["residual"], out_dtype=_dtype(case["out"]))
    rows, weights = q.nvfp4_combine_backward(s["dy"], s["o"], s["rows"], s["weights"], out=s["buffer"])
    return {"rows": rows, "weights": weights}


def _own_norm(s):
    import quantize_precision_gemm_amd as q
    case = s["case"]
    if case["pass"] == "bwd":
        dx, dweight = q.nvfp4_rmsnorm_backward(s["dy"], s["h"], s["weight"], EPS, dh=s["dh"], out_dtype=_dtype(case["stream"]))
        return {"dx": dx, "dweight": dweight}
    call = q.nvfp4_rmsnorm if case["pass"] == "fwd" else q.nvfp4_rmsnorm_i8
    y, h = call(s["x"], s["weight"], EPS, residual=s["residual"])
    out = {} if h is None else {"h": h}
    if case["pass"] == "fwd":
        return {**out, "y": y}
    return {**out, "codes": y.codes.bfloat16(), "scales": y.scales}


def _own_linear(s):
    import quantize_precision_gemm_amd as q
    case = s["case"]
    act = {"none": q.ACT_NONE, "relu2": q.ACT_RELU2, "silu": q.ACT_SILU, "gelu": q.ACT_GELU}[case["act"]]
    if case["pass"] == "bwd":
        dpre, dbias = q.nvfp4_bf16_linear_backward(s["dy"], s["pre"], act, ends=s["ends"])
        return {"dpre": dpre, "dbias": dbias}
    got = q.nvfp4_bf16_linear(s["x"], s["w"], ends=s["ends"], bias=s["bias"], activation=act, residual=s["residual"],
                              with_pre=case["pre"], out_dtype=_dtype(case["out"]))
    return {"y": got[0], "pre": got[1]} if case["pre"] else got


def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _own_route, "move": _own_move, "norm": _own_norm, "linear": _own_linear}[op](state)
    return {"route": _plain_route, "move": _plain_move, "norm": _plain_norm, "linear": _plain_linear}[op](state)


def work(case):
    def size(key):
        return 2 if case[key] == "bf16" else 4
    T = case["rows"]
    if case["op"] == "route":
        E, k = case["experts"], case["k"]
        if case["pass"] == "bwd":  # renormalised weights need the chosen logits alone
            read = k if case["renorm"] or case["score"] == "sigmoid" else E
            return {"bytes": T * (size("dtype") * (read + E) + 8 * k), "flops": 6 * T * E}
        return {"bytes": T * (size("dtype") * E + 12 * k) + 4 * E * (2 if case["bias"] else 1), "flops": 4 * T * E}
    if case["op"] == "move":
        k, cols, there = case["k"], case["cols"], 1.0 - case["pad"]
        if case["pass"] == "dispatch":
            return {"bytes": int(T * (there * cols * 2 * (1 + k) + 4 * k)), "flops": 0}
        if case["pass"] == "combine":
            out = size("out") * (2 if case["residual"] else 1)
            return {"bytes": int(T * (there * k * cols * size("from") + cols * out + (8 if case["weights"] else 4) * k)),
                    "flops": 2 * T * k * cols}
        return {"bytes": int(T * (there * cols * (2 + k * (size("from") + 2)) + 12 * k)), "flops": 3 * T * k * cols}
    if case["op"] == "norm":
        cols, n = case["cols"], T * case["cols"]
        if case["pass"] == "bwd":
            moved = size("x") + size("stream") * (3 if case["residual"] else 2)
            return {"bytes": n * moved + cols * (size("weight") + 4), "flops": 9 * n}
        moved = size("x") + (2 * size("stream") if case["residual"] else 0) + (2 if case["pass"] == "fwd" else 1)
        return {"bytes": n * moved + cols * size("weight"), "flops": 5 * n}
    E, N, K = max(case["experts"], 1), case["n"], case["k"]
    if case["pass"] == "bwd":
        return {"bytes": 6 * T * N + 4 * E * N, "flops": 6 * T * N}
    seen = sum(1 for r in _expert_rows(case) if r) if case["experts"] else 1
    out = size("out") * (2 if case["residual"] else 1) + (2 if case["pre"] else 0)
    return {"bytes": 2 * T * K + 2 * seen * N * K + T * N * out + (4 * seen * N if case["bias"] else 0), "flops": 2 * T * N * K}


# ---- the operators' definitions in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "move": _exact_move, "norm": _exact_norm, "linear": _exact_linear}[case["op"]](s)


def _exact_route(s):
    case, l = s["case"], s["logits"].double()
    T, E, k, G = case["rows"], case["experts"], case["k"], case["groups"]
    open_ = l > -math.inf
    score = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l.masked_fill(~open_, -1e300), 1) * open_
    if case["pass"] == "bwd":  # through the Jacobian of what was chosen
        z = l.masked_fill(~open_, -1e300).requires_grad_()
        at, there = s["experts"].clamp(min=0).long(), (s["experts"] >= 0).double()
        full = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, 1)
        w = full.gather(1, at) * there
        if case["renorm"]:
            w = w / (w.sum(1, keepdim=True) + (there.sum(1, keepdim=True) == 0))
        return torch.autograd.grad(w, z, s["dweights"].double() * there)[0] * open_
    choice = score + (s["bias"].double() if case["bias"] else 0.0)
    choice[~open_] = -math.inf
    if case["kept"] < G:
        value = choice.view(T, G, -1).topk(min(2, E // G), 2)[0].clamp(min=-1e200).sum(2)
        earlier = torch.ones(G, G, dtype=torch.bool, device=choice.device).tril(-1)
        above = (value[:, None, :] > value[:, :, None]) | ((value[:, None, :] == value[:, :, None]) & earlier)
        gone = above.sum(2) >= case["kept"]  # so many groups come before it
        choice[gone.repeat_interleave(E // G, 1)] = -math.inf
    # one after the other: the largest left, the first of equals
    left = choice.clone() if case["bias"] else torch.where(choice > -math.inf, l, -math.inf)
    picked = []
    for _ in range(k):
        top, at = left.max(1)
        at = (left == top[:, None]).int().argmax(1)
        picked.append(torch.where(top > -math.inf, at, -1))
        left[torch.arange(T, device=l.device), at] = -math.inf
    experts = torch.stack(picked, 1)
    w = score.gather(1, experts.clamp(min=0)) * (experts >= 0)
    if case["renorm"]:
        w = w / (w.sum(1, keepdim=True) + (w.sum(1, keepdim=True) == 0))
    return {"experts": None, "weights": w, "rows": None, "ends": None}


def _exact_move(s):
    case, rows = s["case"], s["rows"].long()
    T, k, cols = case["rows"], case["k"], case["cols"]
    slots = torch.zeros(T * k + 1, dtype=torch.long, device="cuda")
    slots[rows.flatten()] = torch.arange(T * k, device="cuda")  # (the last entry takes the empty slots)
    used = int((rows >= 0).sum())
    slots = slots[:used]
    if case["pass"] == "dispatch":
        out = torch.zeros(T * k, cols, dtype=torch.double, device="cuda")
        out[:used] = s["x"].double()[slots // k]
        return out
    w = s["weights"].double().flatten()[slots][:, None] if case["weights"] else 1.0
    if case["pass"] == "combine":
        y = s["residual"].double() if case["residual"] else torch.zeros(T, cols, dtype=torch.double, device="cuda")
        return y.index_add(0, slots // k, s["o"][:used].double() * w)
    out = torch.zeros(T * k, cols, dtype=torch.double, device="cuda")
    dy = s["dy"].double()[slots // k]
    out[:used] = dy * w
    dw = torch.zeros(T * k, dtype=torch.double, device="cuda")
    dw[slots] = torch.linalg.vecdot(dy, s["o"][:used].double())
    return {"rows": out, "weights": dw.view(T, k)}


def _exact_norm(s):
    case, w = s["case"], s["weight"].double()
    if case["pass"] == "bwd":
        h = s["h"].double().requires_grad_()
        w.requires_grad_()
        y = h / torch.sqrt((h ** 2).sum(1, keepdim=True) / case["cols"] + EPS) * w
        dx, dweight = torch.autograd.grad(y, (h, w), s["dy"].double())
        return {"dx": dx + (s["dh"].double() if case["residual"] else 0.0), "dweight": dweight}
    h = s["x"].double() + (s["residual"].double() if case["residual"] else 0.0)
    y = h / torch.sqrt((h ** 2).sum(1, keepdim=True) / case["cols"] + EPS) * w
    out = {"h": h} if case["residual"] else {}
    if case["pass"] == "fwd":
        return {**out, "y": y}
    scale = y.abs().max(1).values / 127.0
    return {**out, "codes": torch.round(y / torch.where(scale > 0, scale, 1.0)[:, None]), "scales": scale}


def _exact_linear(s):
    case, parts, begin = s["case"], [], 0
    ends = [case["rows"]] if s["ends"] is None else s["ends"].tolist()
    functions = {"none": lambda z: z, "relu2": lambda z: torch.relu(z) ** 2, "silu": torch.nn.functional.silu,
                 "gelu": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}
    if case["pass"] == "bwd":
        z = s["pre"].double().requires_grad_()
        dz = torch.autograd.grad(functions[case["act"]](z), z, s["dy"].double())[0]
        for end in ends:
            parts.append(dz[begin:end].sum(0))
            begin = end
        return {"dpre": dz, "dbias": parts[0] if s["ends"] is None else torch.stack(parts)}
    for e, end in enumerate(ends):
        at = () if s["ends"] is None else e
        z = s["x"][begin:end].double() @ s["w"][at].double().t()
        parts.append(z + s["bias"][at].double() if case["bias"] else z)
        begin = end
    z = torch.cat(parts)
    y = functions[case["act"]](z)
    if case["residual"]:
        y = y + s["residual"].double()
    return {"y": y, "pre": z} if case["pre"] else y
