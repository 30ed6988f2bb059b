"""The operators of an FP8 decoder layer's gated half, dense or with experts: cases, inputs, plain forms and exact values.

  route    the experts of each token with their weights, and the plan that sorts the choices by expert (its gradient too)
  experts  the experts' scaled products: FP8 rows, gathered by the plan, against each expert's FP8 weights
  gated    z = act(gate) * up to FP8 codes; in training the input's 8-bit checkpoint and the gradient taken from it
  combine  the weighted sum of a token's experts on top of the residual (its gradient too)

`own` chooses between the plain forms (torch products, sums, exponentials, sorts, comparisons and indexing in 32
bits; 64 where choices are ordered) and the library's entry points.  Codes are returned as the float8 values they
stand for.
"""
import math

import torch

own = False

DEV = "cuda"
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-12  # floor of a group's amax
KEPT = 128   # columns of a checkpoint's group
GROUP = {"row": 0, "group128": 128, "group32": 32}


def _route(name, tokens, experts, k, score="softmax", bias=False, groups=1, top=1, best=1, renorm=True, scale=1.0,
           dtype="fp32", padded=0, train=False):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "k": k, "score": score, "bias": bias,
            "groups": groups, "top": top, "best": best, "renorm": renorm, "scale": scale, "dtype": dtype,
            "padded": padded, "train": train}


def _experts(name, tokens, experts, k, cols, depth, gather=True, fmt="e4m3", skew=1.0):
    return {"name": name, "op": "experts", "tokens": tokens, "experts": experts, "k": k, "cols": cols, "depth": depth,
            "gather": gather, "fmt": fmt, "skew": skew}


def _gated(name, rows, cols, dtype="bf16", scales="row", fmt="e4m3", act="silu", pad=0, train=False):
    return {"name": name, "op": "gated", "rows": rows, "cols": cols, "dtype": dtype, "scales": scales, "fmt": fmt,
            "act": act, "pad": pad, "train": train}


def _combine(name, tokens, experts, k, cols, dtype="bf16", residual=True, train=False):
    return {"name": name, "op": "combine", "tokens": tokens, "experts": experts, "k": k, "cols": cols, "dtype": dtype,
            "residual": residual, "train": train}


def listed():
    return [
        # one generated token: the latency between the router's product and the experts'
        _route("route_token", 1, 64, 8),
        # a batch of prompts, padded at its end: sigmoid scores, a balancing bias, 4 of 8 groups
        _route("route_prompts", 8192, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5, padded=300),
        # a training micro-batch: softmax weights as they are, forward and gradient
        _route("route_train", 16384, 64, 6, renorm=False, dtype="bf16", train=True),
        # one generated token through its experts' gate and up projection
        _experts("experts_token", 1, 64, 8, 4096, 7168),
        # one step of a decode batch: a few rows for each expert, every weight is read
        _experts("experts_step", 64, 128, 8, 4096, 7168),
        # a short ragged chunk through the down projection, popular and idle experts side by side
        _experts("experts_ragged", 701, 32, 4, 7168, 2048, gather=False, skew=2.5),
        # prompts, about 1024 rows for each expert
        _experts("experts_prompts", 8192, 32, 4, 4096, 7168),
        # one generated token's experts
        _gated("gated_token", 8, 2048),
        # a prefill batch of a dense layer with intermediate size 29568
        _gated("gated_prefill", 4096, 29568),
        # a block-scaled training micro-batch, odd rows inside a wider buffer: codes, checkpoint, gradient
        _gated("gated_train", 8189, 7168, scales="group128", pad=64, train=True),
        # one step of a decode batch: the sum of each token's experts on the residual
        _combine("combine_step", 64, 128, 8, 7168),
        # a training micro-batch: the sum, and the gradients of the experts' rows and of the weights
        _combine("combine_train", 4096, 64, 8, 7168, train=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "gated", "combine"])
    experts, train = rng.choice([8, 16, 32, 60, 64, 128, 160, 256, 512]), rng.random() < 0.5
    k = rng.randint(1, min(16, experts // 4))
    if op == "route":
        groups = rng.choice([1, 1, 2, 4])
        top = rng.randint(max(1, -(-groups * k // experts)), groups)
        k = min(k, experts // groups * top)
        best = rng.choice([1, 2]) if groups > 1 else 1
        tokens = _log(rng, 1, min(16384, (1 << 21) // experts))
        c = _route("", tokens, experts, k, rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5, groups, top, best,
                   rng.random() < 0.6, rng.choice([1.0, 2.5]), rng.choice(["fp32", "bf16"]),
                   rng.choice([0, 0, tokens // 5]), train)
    elif op == "experts":
        experts = min(experts, 128)
        cols, depth = 16 * _log(rng, 4, 512), 128 * _log(rng, 1, 64)
        experts = max(8, min(experts, (3 << 30) // (cols * depth)))
        k = min(k, experts)
        tokens = _log(rng, 1, max(1, min(16384 // k, (1 << 39) // (cols * depth * k))))
        c = _experts("", tokens, experts, k, cols, depth, rng.random() < 0.6, rng.choice(["e4m3", "e4m3", "e5m2"]),
                     rng.choice([0.3, 1.0, 2.5]))
    elif op == "gated":
        cols = 16 * _log(rng, 4, 1848)
        rows = _log(rng, 1, min(16384, (1 << 25) // cols))
        c = _gated("", rows, cols, rng.choice(["bf16", "bf16", "fp32"]), rng.choice(sorted(GROUP)),
                   rng.choice(["e4m3", "e4m3", "e5m2"]), rng.choice(["silu", "gelu"]), rng.choice([0, 16, 48]), train)
    else:
        cols = 16 * _log(rng, 4, 512)
        tokens = _log(rng, 1, min(16384, (1 << 27) // (cols * k)))
        c = _combine("", tokens, experts, k, cols, rng.choice(["bf16", "bf16", "fp32"]), rng.random() < 0.7, train)
    del c["name"]
    return c


def _choices(case):
    """[tokens x k] experts of each token (CPU), some experts more popular than others."""
    gen = torch.Generator().manual_seed(case["tokens"] * 1000003 + case["experts"] * 1009 + case["k"])
    like = case.get("skew", 1.0) * torch.randn(case["experts"], generator=gen)
    u = torch.rand(case["tokens"], case["experts"], generator=gen).clamp_min(1e-9)
    return (like - (-u.log()).log()).topk(case["k"], 1).indices


def work(case):
    if case["op"] == "route":
        n, b = case["tokens"] * case["experts"], TYPES[case["dtype"]].itemsize
        moved = n * b + 16 * case["tokens"] * case["k"]
        if case["train"]:
            moved += n * b + 4 * case["tokens"] * case["k"]
        return {"bytes": moved, "flops": (20 if case["train"] else 10) * n}
    if case["op"] == "experts":
        ids, n, d = _choices(case), case["cols"], case["depth"]
        touched = len(ids.unique())
        rows = case["tokens"] if case["gather"] else ids.numel()
        return {"bytes": touched * n * (d + 4) + rows * (d + 4) + 2 * ids.numel() * n, "flops": 2 * ids.numel() * n * d}
    if case["op"] == "gated":
        n, b = case["rows"] * case["cols"], TYPES[case["dtype"]].itemsize
        moved = n * (2 * b + 1)
        if case["train"]:  # the checkpoint written and read, dz read, dx and z written
            moved += 4 * n + n * 4 * b
        return {"bytes": moved, "flops": (60 if case["train"] else 20) * n}
    n, b, k = case["tokens"] * case["cols"], TYPES[case["dtype"]].itemsize, case["k"]
    moved = n * b * (k + 1 + case["residual"])
    if case["train"]:
        moved += n * b * (1 + 2 * k)
    return {"bytes": moved, "flops": 2 * n * k * (4 if case["train"] else 1)}


# ---- inputs ---------------------------------------------------------------------------------------------------


def _wide(rows, cols, pad, dtype, gen, scale=1.0):
    """A [rows x cols] view of a buffer with rows of cols + pad."""
    t = torch.randn(rows, cols + pad, device=DEV, generator=gen) * scale
    return t.to(dtype)[:, :cols]


def _image(codes):
    """Fragment-ordered image of codes [N x K]: the lanes' first, then their last 16 bytes of 16 rows x 128 columns."""
    n, k = codes.shape
    return codes.view(n // 16, 16, k // 128, 4, 2, 16).permute(0, 2, 4, 3, 1, 5).contiguous().view(-1)


def _prepare_route(case, gen):
    T, E, k, dtype = case["tokens"], case["experts"], case["k"], TYPES[case["dtype"]]
    s = dict(case)
    logits = 1.5 * torch.randn(T, E, device=DEV, generator=gen) + torch.randn(E, device=DEV, generator=gen)
    if case["padded"]:
        logits[T - case["padded"]:] = -math.inf
    s["logits"] = logits.to(dtype)
    s["bias"] = 0.1 * torch.randn(E, device=DEV, generator=gen) if case["bias"] else None
    s["ids"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
    s["weights"] = torch.empty(T, k, device=DEV)
    s["slots"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
    s["order"] = torch.full((T * k,), -1, dtype=torch.int32, device=DEV)
    s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    if case["train"]:
        s["dweights"] = torch.randn(T, k, device=DEV, generator=gen)
        s["dlogits"] = torch.empty(T, E, dtype=dtype, device=DEV)
    return s


def _prepare_experts(case, gen):
    T, E, k, N, K, fmt = (case[c] for c in ("tokens", "experts", "k", "cols", "depth", "fmt"))
    s = dict(case)
    ids = _choices(case).to(DEV)
    flat, order = ids.view(-1).sort(stable=True)
    s["order"] = order.to(torch.int32)
    s["offsets"] = torch.searchsorted(flat, torch.arange(E + 1, device=DEV)).to(torch.int32)
    s["counts"] = torch.bincount(flat, minlength=E).tolist()
    rows = T if case["gather"] else T * k
    x = torch.randn(rows, K, device=DEV, generator=gen) * (1 + 5 * torch.rand(K, device=DEV, generator=gen) ** 8)
    s["scale_a"] = x.abs().amax(1, keepdim=True) / FMAX[fmt]
    s["a"] = (x / s["scale_a"]).to(F8[fmt]).view(torch.uint8)
    s["b"] = torch.empty(E, N, K, dtype=torch.uint8, device=DEV)
    s["scale_b"] = torch.empty(E, N, device=DEV)
    s["image"] = torch.empty(E * N * K, dtype=torch.uint8, device=DEV)  # the weights laid out once
    for e in range(E):
        w = torch.randn(N, K, device=DEV, generator=gen) / math.sqrt(K)
        s["scale_b"][e] = w.abs().amax(1) / FMAX["e4m3"]
        s["b"][e] = (w / s["scale_b"][e][:, None]).to(F8["e4m3"]).view(torch.uint8)
        s["image"][e * N * K:(e + 1) * N * K] = _image(s["b"][e])
    s["y"] = torch.empty(T * k, N, dtype=torch.bfloat16, device=DEV)
    return s


def _prepare_gated(case, gen):
    rows, cols, pad, dtype = case["rows"], case["cols"], case["pad"], TYPES[case["dtype"]]
    s = dict(case)
    s["x"] = _wide(rows, 2 * cols, pad, dtype, gen, 1.5)
    s["x"][:, :: max(1, cols // 5)] *= 8  # a few outlier channels, as activations have
    s["q"] = torch.empty(rows, cols, dtype=torch.uint8, device=DEV)
    s["scale"] = torch.empty(rows, -(-cols // (GROUP[case["scales"]] or cols)), device=DEV)
    if case["train"]:
        s["kept"] = torch.empty(rows, 2 * cols, dtype=torch.uint8, device=DEV)
        s["kept_scale"] = torch.empty(rows, 2, -(-cols // KEPT), device=DEV)
        s["dz"] = _wide(rows, cols, pad, dtype, gen, 0.01)
        s["dx"] = torch.empty(rows, 2 * cols, dtype=dtype, device=DEV)
        s["z"] = torch.empty(rows, cols, dtype=dtype, device=DEV)
    return s


def _prepare_combine(case, gen):
    T, E, k, C, dtype = case["tokens"], case["experts"], case["k"], case["cols"], TYPES[case["dtype"]]
    s = dict(case)
    ids = torch.rand(T, E, device=DEV, generator=gen).topk(k, 1).indices
    order = ids.view(-1).sort(stable=True).indices
    s["slots"] = torch.empty(T * k, dtype=torch.int32, device=DEV)
    s["slots"][order] = torch.arange(T * k, dtype=torch.int32, device=DEV)
    s["slots"] = s["slots"].view(T, k)
    w = torch.rand(T, k, device=DEV, generator=gen)
    s["weights"] = w / w.sum(1, keepdim=True)
    s["x"] = _wide(T * k, C, 0, dtype, gen)
    s["res"] = _wide(T, C, 0, dtype, gen, 2.0) if case["residual"] else None
    s["y"] = torch.empty(T, C, dtype=dtype, device=DEV)
    if case["train"]:
        s["dy"] = _wide(T, C, 0, dtype, gen, 0.01)
        s["dx"] = torch.empty(T * k, C, dtype=dtype, device=DEV)
        s["dweights"] = torch.empty(T, k, device=DEV)
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return {"route": _prepare_route, "experts": _prepare_experts, "gated": _prepare_gated,
            "combine": _prepare_combine}[case["op"]](case, gen)


# ---- the library's entry points -------------------------------------------------------------------------------


def _run_own(s):
    import dynamic_scaling_scaled_amd as rt

    if s["op"] == "route":
        score = rt.SOFTMAX if s["score"] == "softmax" else rt.SIGMOID
        rt.fp8_expert_route(s["logits"], s["ids"], s["weights"], s["slots"], s["order"], s["offsets"], score=score,
                            bias=s["bias"], groups=s["groups"], top_groups=s["top"], group_best=s["best"],
                            renormalise=s["renorm"], scale=s["scale"])
        out = _route_outputs(s)
        if s["train"]:
            rt.fp8_expert_route_backward(s["logits"], s["ids"], s["dweights"], s["dlogits"], score=score,
                                         renormalise=s["renorm"], scale=s["scale"])
            out["dlogits"] = s["dlogits"]
        return out
    if s["op"] == "experts":
        E, N, K = s["b"].shape
        rt.fp8_expert_gemm(s["a"], rt.E4M3 if s["fmt"] == "e4m3" else rt.E5M2, (1, 0), s["scale_a"],
                           rt.PackedWeights(s["image"], E * N, K), rt.E4M3, (1, 0), s["scale_b"], s["offsets"], s["y"],
                           order=s["order"] if s["gather"] else None, choices=s["k"] if s["gather"] else 1)
        return {"y": s["y"]}
    if s["op"] == "gated":
        act, fmt = rt.SILU if s["act"] == "silu" else rt.GELU, rt.E4M3 if s["fmt"] == "e4m3" else rt.E5M2
        rt.fp8_gated_quantize(s["x"], (1, GROUP[s["scales"]]), fmt, rt.DYNAMIC, EPS, False, s["scale"], s["q"], act=act,
                              kept=s.get("kept"), kept_scale=s.get("kept_scale"))
        out = {"codes": s["q"].view(F8[s["fmt"]]), "scale": s["scale"]}
        if s["train"]:
            rt.fp8_gated_backward(s["dz"], s["kept"], s["kept_scale"], s["dx"], act=act, z=s["z"])
            out |= {"kept": s["kept"].view(F8["e4m3"]), "kept_scale": s["kept_scale"], "dx": s["dx"], "z": s["z"]}
        return out
    rt.fp8_expert_combine(s["x"], s["slots"], s["weights"], s["y"], residual=s["res"])
    out = {"y": s["y"]}
    if s["train"]:
        rt.fp8_expert_combine_backward(s["dy"], s["x"], s["slots"], s["weights"], s["dx"], s["dweights"])
        out |= {"dx": s["dx"], "dweights": s["dweights"]}
    return out


def _route_outputs(s):
    return {c: s[c] for c in ("ids", "weights", "slots", "order", "offsets")}


# ---- the plain forms ------------------------------------------------------------------------------------------


def _scores(s):
    """(binary64 logits with absent experts at -inf, scores)"""
    l = s["logits"].double()
    l = torch.where(l.isnan(), -math.inf, l)
    if s["score"] == "sigmoid":
        return l, torch.sigmoid(l)
    p = (l - l.amax(1, keepdim=True).clamp_min(-1e300)).exp()
    return l, p / p.sum(1, keepdim=True).clamp_min(1e-300)


def _plain_route(s):
    T, E, k, G = s["tokens"], s["experts"], s["k"], s["groups"]
    l, p = _scores(s)
    absent = l == -math.inf
    key = l if s["bias"] is None else (p + s["bias"].double()).masked_fill(absent, -math.inf)
    if G > 1:
        top = (p if s["bias"] is None and s["best"] == 2 else key).masked_fill(absent, -math.inf)
        top = top.view(T, G, -1).topk(s["best"], 2).values
        group = top[:, :, 0] if s["best"] == 1 else top[:, :, 0] + top[:, :, 1].masked_fill(top[:, :, 1] == -math.inf, 0)
        rank = group.sort(dim=1, descending=True, stable=True).indices
        kept = torch.zeros(T, G, dtype=torch.bool, device=DEV).scatter_(1, rank[:, :s["top"]], True)
        key = key.masked_fill(~kept.repeat_interleave(E // G, 1), -math.inf)
    best, ids = (x[:, :k] for x in key.sort(dim=1, descending=True, stable=True))
    there = best > -math.inf
    w = p.gather(1, ids) * there
    if s["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    s["weights"].copy_(w * s["scale"])
    ids = torch.where(there, ids, -1)
    s["ids"].copy_(ids)
    by_expert, order = torch.where(there, ids, E).view(-1).sort(stable=True)
    place = torch.arange(T * k, device=DEV)
    s["slots"].view(-1)[order] = torch.where(by_expert < E, place, -1).int()
    s["order"].copy_(torch.where(by_expert < E, order, s["order"]))
    s["offsets"].copy_(torch.searchsorted(by_expert, torch.arange(E + 1, device=DEV)))
    out = _route_outputs(s)
    if s["train"]:
        there, at = s["ids"] >= 0, s["ids"].long().clamp_min(0)
        p = p.float()
        pc = p.gather(1, at) * there
        g = s["dweights"] * s["scale"] * there
        if s["renorm"]:
            total = pc.sum(1, keepdim=True)
            g = torch.where(total > 0, (g - (g * pc).sum(1, keepdim=True) / total) / total, 0.0) * there
        dp = torch.zeros_like(p).scatter_add_(1, at, g)
        if s["score"] == "softmax":
            d = p * (dp - (dp * p).sum(1, keepdim=True))
        else:
            d = dp * p * (1 - p)
        s["dlogits"].copy_(d)
        out["dlogits"] = s["dlogits"]
    return out


def _plain_experts(s):
    a = s["a"].view(F8[s["fmt"]]).float() * s["scale_a"]
    if s["gather"]:
        a = a[s["order"].long() // s["k"]]
    at = 0
    for e, n in enumerate(s["counts"]):
        if n:
            w = s["b"][e].view(F8["e4m3"]).float() * s["scale_b"][e][:, None]
            s["y"][at:at + n] = torch.matmul(a[at:at + n], w.T)
            at += n
    return {"y": s["y"]}


def _quantize(v, g, fmt):
    """(codes, scales) of the rows' 1 x g groups, the last one short (g = 0: the row)."""
    rows, cols = v.shape
    vg = torch.nn.functional.pad(v, (0, -cols % (g or cols))).view(rows, -1, g or cols)
    a = vg.abs().amax(2).clamp_min(EPS)
    top = torch.full_like(a, FMAX[fmt])
    codes = (vg * (top / a)[:, :, None]).clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt])
    return codes.view(torch.uint8).view(rows, -1)[:, :cols].contiguous().view(F8[fmt]), a / top


GELU_A, GELU_B = math.sqrt(2 / math.pi), 0.044715


def _act(g, kind):
    """(act(g), its derivative)"""
    if kind == "silu":
        c = torch.sigmoid(g)
        return g * c, c * (1 + g * (1 - c))
    t = torch.tanh(GELU_A * (g + GELU_B * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * GELU_A * (1 + 3 * GELU_B * g * g)


def _plain_gated(s):
    cols = s["cols"]
    gate, up = s["x"][:, :cols].float(), s["x"][:, cols:].float()
    codes, scale = _quantize(_act(gate, s["act"])[0] * up, GROUP[s["scales"]], s["fmt"])
    out = {"codes": codes, "scale": scale}
    if s["train"]:
        (cg, sg), (cu, su) = _quantize(gate, KEPT, "e4m3"), _quantize(up, KEPT, "e4m3")
        gate, up = (c.float() * sc.repeat_interleave(KEPT, 1)[:, :cols] for c, sc in ((cg, sg), (cu, su)))
        f, df = _act(gate, s["act"])
        dz = s["dz"].float()
        kept = torch.cat([cg.view(torch.uint8), cu.view(torch.uint8)], 1).view(F8["e4m3"])
        out |= {"kept": kept, "kept_scale": torch.stack([sg, su], 1),
                "dx": torch.cat([dz * up * df, dz * f], 1).to(s["x"].dtype), "z": (f * up).to(s["x"].dtype)}
    return out


def _plain_combine(s):
    x = s["x"][s["slots"].long()].float()  # [tokens x k x cols]
    y = (s["weights"][:, :, None] * x).sum(1)
    if s["res"] is not None:
        y = y + s["res"].float()
    out = {"y": y.to(s["x"].dtype)}
    if s["train"]:
        dy = s["dy"].float()
        s["dx"][s["slots"].long()] = (s["weights"][:, :, None] * dy[:, None]).to(s["x"].dtype)
        out |= {"dx": s["dx"], "dweights": (dy[:, None] * x).sum(2)}
    return out


def run(s):
    if own:
        return _run_own(s)
    return {"route": _plain_route, "experts": _plain_experts, "gated": _plain_gated, "combine": _plain_combine}[s["op"]](s)


# ---- exact values ---------------------------------------------------------------------------------------------


def _exact_route(case, s):
    """The weights, and their gradient by the chain rule over the chosen scores, in 64 bits; whole numbers are compared as they are."""
    l = s["logits"].double()
    if case["score"] == "softmax":
        p = torch.nan_to_num(torch.softmax(l, 1), nan=0.0)  # (rows without an expert)
    else:
        p = 1 / (1 + torch.exp(-l))
    pick, E, G = p if s["bias"] is None else p + s["bias"].double(), case["experts"], case["groups"]
    if s["bias"] is None and case["best"] == 1:
        pick = l
    order = pick if s["bias"] is not None else l
    order = torch.where(l > -math.inf, order, -math.inf)
    if G > 1:
        per = torch.where(l > -math.inf, pick, -math.inf).reshape(-1, G, E // G).sort(2, descending=True).values
        total = per[:, :, 0].clone()
        if case["best"] == 2:
            total += torch.where(per[:, :, 1] > -math.inf, per[:, :, 1], 0.0)
        place = torch.argsort(torch.argsort(-total, dim=1, stable=True), dim=1)
        order = torch.where((place < case["top"])[:, :, None].expand(-1, -1, E // G).reshape(-1, E), order, -math.inf)
    ids = torch.argsort(-order, dim=1, stable=True)[:, :case["k"]]
    mask = torch.zeros_like(p).scatter_(1, ids, 1.0) * (order > -math.inf)
    chosen = p * mask
    norm = chosen.sum(1, keepdim=True) if case["renorm"] else torch.ones_like(p[:, :1])
    safe = torch.where(norm > 0, norm, 1.0)
    out = {"ids": None, "weights": (case["scale"] * chosen / safe).gather(1, ids), "slots": None, "order": None, "offsets": None}
    if case["train"]:
        dw = torch.zeros_like(p).scatter_(1, ids, s["dweights"].double()) * mask * case["scale"]
        if case["renorm"]:  # w = chosen / norm
            dw = mask * (dw / safe - (dw * chosen).sum(1, keepdim=True) / safe ** 2)
            dw = torch.where(norm > 0, dw, 0.0)
        slope = p * dw
        out["dlogits"] = slope - p * slope.sum(1, keepdim=True) if case["score"] == "softmax" else slope - p * slope
    return out


def _exact_experts(case, s):
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
    bounds, order = s["offsets"].tolist(), s["order"].long()
    for e in range(case["experts"]):
        lo, hi = bounds[e], bounds[e + 1]
        if lo == hi:
            continue
        rows = order[lo:hi] // case["k"] if case["gather"] else torch.arange(lo, hi, device=DEV)
        dots = s["a"][rows].view(F8[case["fmt"]]).double() @ s["b"][e].view(F8["e4m3"]).double().T
        y[lo:hi] = dots * s["scale_a"][rows].double() * s["scale_b"][e].double()[None]
    return {"y": y}


def _exact_gated(case, s):
    """In 64 bits, a group at a time; codes as the value over its scale before the cast rounds it."""
    cols, rows, top = case["cols"], case["rows"], FMAX[case["fmt"]]

    def act(g):
        if case["act"] == "silu":
            return g / (1 + torch.exp(-g))
        return g / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))

    def slope(g):  # of the same, with c = sigmoid(u): act = g c, act' = c + g c (1 - c) u'
        u, du = g, 1.0
        if case["act"] == "gelu":
            u, du = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3), 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * g * g)
        c = 1 / (1 + torch.exp(-u))
        return c + g * c * (1 - c) * du

    gate, up = s["x"][:, :cols].double(), s["x"][:, cols:].double()
    z = act(gate) * up
    step, codes, scale = GROUP[case["scales"]] or cols, torch.empty_like(z), []
    for c in range(0, cols, step):
        part = z[:, c:c + step]
        scale.append(part.abs().max(1).values.clamp_min(EPS) / top)
        codes[:, c:c + step] = part / scale[-1][:, None]
    out = {"codes": codes, "scale": torch.stack(scale, 1)}
    if case["train"]:
        # the gradient is that of the checkpoint: its codes are rounded values, as the operator's definition has them
        kept, ks = torch.empty(rows, 2 * cols, dtype=torch.float64, device=DEV), torch.empty(s["kept_scale"].shape, dtype=torch.float64, device=DEV)
        back = torch.empty_like(kept)
        for h in range(2):
            for i, c in enumerate(range(0, cols, KEPT)):
                v = s["x"][:, h * cols + c:h * cols + min(c + KEPT, cols)]
                a = v.float().abs().max(1).values.clamp_min(EPS)
                full = torch.full_like(a, 448.0)
                at = slice(h * cols + c, h * cols + c + v.shape[1])
                kept[:, at] = (v.float() * (full / a)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).double()
                back[:, at] = kept[:, at] * (a / full).double()[:, None]
                ks[:, h, i] = a.double() / 448
        g, u, dz = back[:, :cols], back[:, cols:], s["dz"].double()
        out |= {"kept": kept, "kept_scale": ks, "dx": torch.cat([dz * u * slope(g), dz * act(g)], 1), "z": act(g) * u}
    return out


def _exact_combine(case, s):
    y = s["res"].double() if case["residual"] else torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
    out = {"y": y}
    if case["train"]:
        out["dx"] = torch.zeros(s["x"].shape, dtype=torch.float64, device=DEV)
        out["dweights"] = torch.empty(s["weights"].shape, dtype=torch.float64, device=DEV)
    for j in range(case["k"]):
        at, w = s["slots"][:, j].long(), s["weights"][:, j].double()[:, None]
        rows = s["x"][at].double()
        y += w * rows
        if case["train"]:
            dy = s["dy"].double()
            out["dx"].index_copy_(0, at, w * dy)
            out["dweights"][:, j] = (dy * rows).sum(1)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "experts": _exact_experts, "gated": _exact_gated, "combine": _exact_combine}[case["op"]](case, s)
