"""The operators of an FP8 decoder layer around the scaled GEMMs: cases, inputs, plain forms and exact values.

  norm    h = x + residual, y = RMSnorm(h) * weight, FP8 codes of y with their scales (the GEMM's operand)
  grad    the gradient of that norm for h (with the residual path's gradient added) and for the weight
  append  new keys and values written into a paged cache of FP8 codes, one scale for each page and head
  attend  attention over that cache: single tokens, chunks of a prompt, whole prompts

`own` chooses between the plain forms (torch products, sums, exponentials, comparisons and indexing in 32 bits)
and the library's entry points.  Codes are returned as the float8 values they stand for.
"""
import math
import random

import torch

own = False

DEV = "cuda"
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-12  # floor of a group's amax
NORM_EPS = 1e-6
GROUP = {"row": 0, "group128": 128, "group32": 32, "tensor": 0}


def _norm(name, rows, cols, dtype="bf16", residual=True, scales="row", fmt="e4m3", pad=0):
    return {"name": name, "op": "norm", "rows": rows, "cols": cols, "dtype": dtype, "residual": residual,
            "scales": scales, "fmt": fmt, "pad": pad}


def _grad(name, rows, cols, dtype="bf16", residual=True, pad=0):
    return {"name": name, "op": "grad", "rows": rows, "cols": cols, "dtype": dtype, "residual": residual, "pad": pad}


def _append(name, seqs, new, before, heads, dim, page, dtype="bf16", fmt="e4m3", pow2=False):
    return {"name": name, "op": "append", "seqs": seqs, "new": new, "before": before, "heads": heads, "dim": dim,
            "page": page, "dtype": dtype, "fmt": fmt, "pow2": pow2}


def _attend(name, seqs, new, before, heads, group, dim, page, fmt="e4m3", causal=True, window=0, even=False):
    return {"name": name, "op": "attend", "seqs": seqs, "new": new, "before": before, "heads": heads, "group": group,
            "dim": dim, "page": page, "fmt": fmt, "causal": causal, "window": window, "even": even}


def listed():
    return [
        # one generated token of a model with hidden size 8192: the latency of a step's norm
        _norm("norm_one_token", 1, 8192),
        # a prefill batch at the same hidden size, per-token scales
        _norm("norm_prefill", 4096, 8192),
        # a block-scaled layer (1x128 groups) on an odd token count, rows inside a wider buffer
        _norm("norm_groups", 8189, 7168, scales="group128", pad=64),
        # a small fine-tuning batch in 32 bits
        _grad("grad_small", 257, 1024, dtype="fp32"),
        # a training micro-batch at hidden size 8192
        _grad("grad_batch", 4096, 8192),
        # one step of a decode batch: one token into each sequence's last page
        _append("append_step", 64, 1, 4096, 8, 128, 64),
        # ragged prompts entering the cache, each going on in a page that is partly filled
        _append("append_prompts", 5, 4001, 777, 8, 128, 16),
        # a single request's decode step: latency
        _attend("attend_one", 1, 1, 1000, 8, 8, 128, 16),
        # a decode batch of ragged lengths
        _attend("attend_batch", 64, 1, 8191, 8, 8, 128, 64),
        # two requests with long contexts
        _attend("attend_long", 2, 1, 131071, 8, 8, 128, 128, even=True),
        # a whole prompt, causal
        _attend("attend_prompt", 1, 8192, 0, 8, 8, 128, 64, even=True),
        # chunks of prompts of uneven lengths behind uneven contexts, a sliding window, E5M2 codes
        _attend("attend_chunks", 6, 701, 6001, 4, 5, 64, 32, fmt="e5m2", window=1024),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["norm", "grad", "append", "attend", "attend", "attend"])
    if op in ("norm", "grad"):
        cols = 16 * _log(rng, 4, 1024)
        rows = _log(rng, 1, min(16384, (1 << 25) // cols))
        dtype, residual, pad = rng.choice(["bf16", "bf16", "fp32"]), rng.random() < 0.7, rng.choice([0, 16, 48])
        if op == "grad":
            c = _grad("", rows, cols, dtype, residual, pad)
        else:
            c = _norm("", rows, cols, dtype, residual, rng.choice(sorted(GROUP)), rng.choice(["e4m3", "e4m3", "e5m2"]), pad)
    elif op == "append":
        seqs = _log(rng, 1, 128)
        new = 1 if rng.random() < 0.5 else _log(rng, 2, max(3, 16384 // seqs))
        c = _append("", seqs, new, rng.choice([0, _log(rng, 1, 4096)]), rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128]),
                    rng.choice([16, 32, 64, 128]), rng.choice(["bf16", "bf16", "fp32"]), rng.choice(["e4m3", "e4m3", "e5m2"]),
                    rng.random() < 0.3)
    else:
        heads, group, dim = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8, 16]), rng.choice([64, 128])
        seqs = _log(rng, 1, 64)
        if rng.random() < 0.5:
            new, before = rng.choice([1, 1, 1, 2, 5]), _log(rng, 1, min(131072, 262144 // seqs))
        else:
            seqs = min(seqs, 8)
            new = _log(rng, 17, max(18, 4096 // seqs))
            before = rng.choice([0, _log(rng, 1, 8192 // seqs)])
        c = _attend("", seqs, new, before, heads, group, dim, rng.choice([16, 32, 64, 128]),
                    rng.choice(["e4m3", "e4m3", "e5m2"]), rng.random() < 0.85, rng.choice([0, 0, _log(rng, 16, 4096)]),
                    rng.random() < 0.3)
    del c["name"]
    return c


def _lengths(case):
    """New tokens and tokens already cached of each sequence: the first has the most, the others are ragged."""
    if case.get("even") or case["seqs"] == 1:
        return [case["new"]] * case["seqs"], [case["before"]] * case["seqs"]
    rng = random.Random(case["seqs"] * 1000003 + case["new"] * 1009 + case["before"])
    new = [case["new"]] + [rng.randint(1, case["new"]) for _ in range(case["seqs"] - 1)]
    before = [case["before"]] + [rng.randint(0, case["before"]) for _ in range(case["seqs"] - 1)]
    return new, before


def _visible(case):
    """Visible (query, key) pairs, and keys that some query sees, over all sequences."""
    pairs = keys = 0
    for n, b in zip(*_lengths(case)):
        w, L = case["window"] or (b + n), b + n
        first = torch.arange(b, b + n, dtype=torch.int64)  # the queries' positions
        last = first + 1 if case["causal"] else torch.full_like(first, L)
        lo = (first - w + 1).clamp_min(0) if case["window"] else torch.zeros_like(first)
        pairs += int((last - lo).sum())
        keys += L - int(lo[0])
    return pairs, keys


def work(case):
    if case["op"] in ("norm", "grad"):
        n, b = case["rows"] * case["cols"], TYPES[case["dtype"]].itemsize
        if case["op"] == "norm":
            moved = n * (b * (1 + 2 * case["residual"]) + 1)
            return {"bytes": moved + b * case["cols"], "flops": 6 * n}
        return {"bytes": n * b * (3 + case["residual"]) + 6 * case["cols"], "flops": 10 * n}
    new, before = _lengths(case)
    if case["op"] == "append":
        n = 2 * sum(new) * case["heads"] * case["dim"]
        return {"bytes": n * (TYPES[case["dtype"]].itemsize + 1), "flops": 4 * n}
    pairs, keys = _visible(case)
    q = sum(new) * case["heads"] * case["group"] * case["dim"]
    kv = 2 * keys * case["heads"] * (case["dim"] + 4 / case["page"])
    return {"bytes": kv + 4 * q, "flops": 4 * pairs * case["heads"] * case["group"] * case["dim"]}


def _wide(rows, cols, pad, dtype, gen, scale=1.0):
    """A [rows x cols] view of a buffer with rows of cols + pad."""
    t = torch.randn(rows, cols + pad, device=DEV, generator=gen) * scale
    return t.to(dtype)[:, :cols]


def _paged(case, gen):
    """The plan that a serving program keeps: where each sequence's new tokens are, its length, its pages."""
    new, before = _lengths(case)
    page = case["page"]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    lens = [n + b for n, b in zip(new, before)]
    per = [-(-x // page) for x in lens]
    width = max(per)
    pages = sum(per) + 3  # a few that belong to nobody
    order = torch.randperm(pages, device=DEV, generator=gen).to(torch.int32)
    table = torch.full((case["seqs"], width), -1, dtype=torch.int32, device=DEV)
    used = torch.arange(width, device=DEV)[None, :] < torch.tensor(per, device=DEV)[:, None]
    table[used] = order[:sum(per)]
    s = {"op": case["op"], "table": table, "pages": pages, "page": page, "max_new": max(new), "max_kv": max(lens),
         "start": torch.tensor(starts, dtype=torch.int32, device=DEV),
         "len": torch.tensor(lens, dtype=torch.int32, device=DEV), "tokens": starts[-1], "fmt": case["fmt"]}
    return s


def _cache(case, s, gen, spread):
    """A cache in use: every slot holds codes under its page's scale (also slots that no sequence owns yet)."""
    shape = (s["pages"], case["heads"], case["page"], case["dim"])
    channel = 1 + spread * torch.rand(case["dim"], device=DEV, generator=gen) ** 8  # a few loud channels
    x = torch.randn(shape, device=DEV, generator=gen) * channel
    scale = (x.abs().amax((2, 3)) / FMAX[case["fmt"]]).contiguous()
    return (x / scale[:, :, None, None]).to(F8[case["fmt"]]).view(torch.uint8), scale


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if case["op"] in ("norm", "grad"):
        rows, cols, pad, dtype = case["rows"], case["cols"], case["pad"], TYPES[case["dtype"]]
        s = {"op": case["op"]}
        s["weight"] = (1 + 0.2 * torch.randn(cols, device=DEV, generator=gen)).to(dtype)
        s["res"] = _wide(rows, cols, pad, dtype, gen, 2.0) if case["residual"] else None
        if case["op"] == "grad":
            s["dy"] = _wide(rows, cols, pad, dtype, gen, 0.01)
            s["h"] = _wide(rows, cols, pad, dtype, gen, 2.0)
            s["rstd"] = (s["h"].float().square().mean(1) + NORM_EPS).rsqrt()
            if case["residual"]:
                s["res"] = s["res"] * 0.01
            s["dx"] = torch.empty(rows, cols, dtype=dtype, device=DEV)
            s["dweight"] = torch.empty(cols, device=DEV)
            return s
        x = _wide(rows, cols, pad, dtype, gen)
        x[:, :: max(1, cols // 5)] *= 20  # a few outlier channels, as activations have
        s |= {"x": x, "fmt": case["fmt"], "scales": case["scales"]}
        groups = 1 if not GROUP[case["scales"]] else -(-cols // GROUP[case["scales"]])
        s["q"] = torch.empty(rows, cols, dtype=torch.uint8, device=DEV)
        s["h"] = torch.empty(rows, cols, dtype=dtype, device=DEV) if case["residual"] else None
        s["rstd"] = torch.empty(rows, device=DEV)
        if case["scales"] == "tensor":  # a delayed scale: given, and the amax that its history takes next
            s["scale"] = torch.full((1, 1), 8.0 / FMAX[case["fmt"]], device=DEV)
            s["amax"] = torch.empty(1, 1, device=DEV)
        else:
            s["scale"], s["amax"] = torch.empty(rows, groups, device=DEV), None
        return s
    s = _paged(case, gen)
    s["k"], s["ks"] = _cache(case, s, gen, 6.0)
    s["v"], s["vs"] = _cache(case, s, gen, 1.0)
    if case["op"] == "append":
        both = torch.randn(s["tokens"], 2 * case["heads"], case["dim"], device=DEV, generator=gen)
        both[:: 7] *= 1.5  # some tokens are louder than what their page has seen
        s["new"] = both.to(TYPES[case["dtype"]])
        s["pow2"] = case["pow2"]
        if case["pow2"]:
            for name in ("ks", "vs"):
                s[name] = torch.exp2(torch.ceil(torch.log2(s[name])))
        return s
    heads = case["heads"] * case["group"]
    s["q"] = torch.randn(s["tokens"], heads, case["dim"], device=DEV, generator=gen).to(torch.bfloat16)
    s["y"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(s["tokens"], heads, device=DEV)
    s |= {"causal": case["causal"], "window": case["window"], "sm_scale": 1.0 / math.sqrt(case["dim"])}
    return s


# ---- the library's entry points -------------------------------------------------------------------------------


def _run_own(s):
    import dynamic_scaling_scaled_amd as rt

    if s["op"] == "norm":
        g, fmt = GROUP[s["scales"]], rt.E4M3 if s["fmt"] == "e4m3" else rt.E5M2
        given = s["scales"] == "tensor"
        rt.fp8_rmsnorm_quantize(s["x"], s["weight"], NORM_EPS, (0, 0) if given else (1, g), fmt,
                                rt.GIVEN if given else rt.DYNAMIC, EPS, False, s["scale"], s["q"], residual=s["res"],
                                h=s["h"], rstd=s["rstd"], amax_out=s["amax"])
        return _norm_outputs(s, s["q"].view(F8[s["fmt"]]), s["scale"], s["h"], s["rstd"], s["amax"])
    if s["op"] == "grad":
        rt.fp8_rmsnorm_backward(s["dy"], s["h"], s["weight"], s["rstd"], s["dx"], s["dweight"], dresidual=s["res"])
        return {"dx": s["dx"], "dweight": s["dweight"]}
    fmt = rt.E4M3 if s["fmt"] == "e4m3" else rt.E5M2
    if s["op"] == "append":
        heads = s["k"].shape[1]
        rt.fp8_kv_append(s["new"][:, :heads], s["new"][:, heads:], s["k"], s["v"], s["ks"], s["vs"], fmt, s["table"],
                         s["start"], s["len"], s["max_new"], EPS, s["pow2"])
        return {"k": s["k"].view(F8[s["fmt"]]), "v": s["v"].view(F8[s["fmt"]]), "ks": s["ks"], "vs": s["vs"]}
    rt.fp8_paged_attention(s["q"], s["k"], s["v"], s["ks"], s["vs"], fmt, s["table"], s["start"], s["len"], s["max_new"],
                           s["max_kv"], s["sm_scale"], s["y"], causal=s["causal"], window=s["window"], lse=s["lse"])
    return {"y": s["y"], "lse": s["lse"]}


def _norm_outputs(s, codes, scale, h, rstd, amax):
    out = {"codes": codes, "rstd": rstd}
    if s["scales"] != "tensor":
        out["scale"] = scale
    else:
        out["amax"] = amax
    if h is not None:
        out["h"] = h
    return out


# ---- the plain forms ------------------------------------------------------------------------------------------


def _cast(v, fmt):
    return v.clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt])


def _scale_of(amax, fmt, pow2=False):
    """(s, r): the scale kept with the codes and the multiplier of the cast."""
    a = amax.clamp_min(EPS)
    s, r = a / FMAX[fmt], FMAX[fmt] / a
    if pow2:
        m, e = torch.frexp(s)  # s = m 2^e, m in [0.5, 1)
        s = torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))
        r = 1 / s
    return s, r


def _plain_norm(s):
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    rstd = (h.square().mean(1) + NORM_EPS).rsqrt()
    y = h * rstd[:, None] * s["weight"].float()
    rows, cols = y.shape
    g, amax = GROUP[s["scales"]] or cols, None
    if s["scales"] == "tensor":
        scale, r, amax = s["scale"], 1 / s["scale"], y.abs().amax().view(1, 1)
        codes = _cast(y * r, s["fmt"])
    else:
        fill = (-cols) % g
        yg = torch.nn.functional.pad(y, (0, fill)).view(rows, -1, g)
        scale, r = _scale_of(yg.abs().amax(2), s["fmt"])
        codes = _cast(yg * r[:, :, None], s["fmt"]).view(rows, -1)[:, :cols].contiguous()
    return _norm_outputs(s, codes, scale, h.to(s["x"].dtype) if s["h"] is not None else None, rstd, amax)


def _plain_grad(s):
    dy, n = s["dy"].float(), s["h"].float() * s["rstd"][:, None]
    g = dy * s["weight"].float()
    dx = s["rstd"][:, None] * (g - n * (g * n).mean(1, keepdim=True))
    if s["res"] is not None:
        dx = dx + s["res"].float()
    return {"dx": dx.to(s["dy"].dtype), "dweight": (dy * n).sum(0)}


def _token_places(s):
    """Each new token's sequence and position, and the position at which its sequence's new tokens begin."""
    t = torch.arange(s["tokens"], device=DEV)
    seq = torch.searchsorted(s["start"].long(), t, right=True) - 1
    first = s["len"].long() - (s["start"][1:] - s["start"][:-1]).long()
    return seq, first[seq] + t - s["start"].long()[seq], first


def _plain_append_one(s, x, cache, scale):
    page, fmt = s["page"], s["fmt"]
    seq, pos, first = _token_places(s)
    key = seq * s["table"].shape[1] + pos // page
    touched, place = torch.unique(key, return_inverse=True)
    tseq, tpage = touched // s["table"].shape[1], touched % s["table"].shape[1]
    at = s["table"][tseq, tpage].long()
    x = x.float()
    amax = torch.zeros(len(touched), x.shape[1], device=DEV)
    amax = amax.scatter_reduce_(0, place[:, None].expand(-1, x.shape[1]), x.abs().amax(2), "amax")
    cand, r = _scale_of(amax, fmt, s["pow2"])
    fill = (first[tseq] - tpage * page).clamp(0, page)  # tokens that the page held before
    old = torch.where((fill > 0)[:, None], scale[at], torch.zeros_like(cand))
    keep = old > cand
    new, r = torch.where(keep, old, cand), torch.where(keep, 1 / old, r)
    grown = (fill > 0)[:, None] & ~keep & (old != cand)
    held = cache[at].view(F8[fmt])
    again = _cast(held.float() * (old / new)[:, :, None, None], fmt).view(torch.uint8)
    slot = torch.arange(page, device=DEV)
    change = grown[:, :, None, None] & (slot[None, :] < fill[:, None])[:, None, :, None]
    cache[at] = torch.where(change, again, held.view(torch.uint8))
    scale[at] = new
    cache[at[place], :, pos % page] = _cast(x * r[place][:, :, None], fmt).view(torch.uint8)


def _plain_append(s):
    heads = s["k"].shape[1]
    _plain_append_one(s, s["new"][:, :heads], s["k"], s["ks"])
    _plain_append_one(s, s["new"][:, heads:], s["v"], s["vs"])
    return {"k": s["k"].view(F8[s["fmt"]]), "v": s["v"].view(F8[s["fmt"]]), "ks": s["ks"], "vs": s["vs"]}


def _gather(s, cache, scale):
    """[sequence, head, position, dim] values of the cache."""
    at = s["table"].long().clamp_min(0)
    x = cache[at].view(F8[s["fmt"]]).float() * scale[at][:, :, :, None, None]
    return x.transpose(1, 2).reshape(at.shape[0], cache.shape[1], -1, cache.shape[3])


def _plain_attend(s):
    seq, pos, first = _token_places(s)
    k, v = _gather(s, s["k"], s["ks"]), _gather(s, s["v"], s["vs"])
    seqs, heads, length, dim = k.shape
    group, row = s["q"].shape[1] // heads, torch.arange(s["tokens"], device=DEV) - s["start"].long()[seq]
    q = torch.zeros(seqs, s["max_new"], heads, group, dim, device=DEV)
    q[seq, row] = s["q"].float().view(-1, heads, group, dim)
    q = q.permute(0, 2, 3, 1, 4).reshape(seqs, heads, group * s["max_new"], dim)
    p = torch.matmul(q, k.transpose(2, 3).contiguous()) * s["sm_scale"]
    p = p.view(seqs, heads, group, s["max_new"], length)
    j = torch.arange(length, device=DEV)
    at = first[:, None] + torch.arange(s["max_new"], device=DEV)
    seen = (j < s["len"].long()[:, None])[:, None, :].expand(seqs, s["max_new"], length)
    if s["causal"]:
        seen = seen & (j <= at[:, :, None])
    if s["window"]:
        seen = seen & (j > at[:, :, None] - s["window"])
    p = p.masked_fill_(~seen[:, None, None], -math.inf)
    top = p.amax(4, keepdim=True).clamp_min(-1e30)
    p = p.sub_(top).exp_()
    total = p.sum(4, keepdim=True)
    y = torch.matmul(p.view(seqs, heads, -1, length), v).view(seqs, heads, group, s["max_new"], dim)
    y = torch.where(total > 0, y / total, torch.zeros_like(y))
    lse = (top + total.log()).squeeze(4)
    y = y.permute(0, 3, 1, 2, 4)[seq, row].reshape(s["tokens"], -1, dim)
    lse = lse.permute(0, 3, 1, 2)[seq, row].reshape(s["tokens"], -1)
    return {"y": y.to(s["q"].dtype), "lse": lse}


def run(s):
    if own:
        return _run_own(s)
    return {"norm": _plain_norm, "grad": _plain_grad, "append": _plain_append, "attend": _plain_attend}[s["op"]](s)


# ---- exact values ---------------------------------------------------------------------------------------------


def _exact_norm(case, s):
    """In 64 bits; the codes as y / s before the cast rounds them."""
    h = s["x"].double()
    if case["residual"]:
        h += s["res"].double()
    cols, top = h.shape[1], FMAX[case["fmt"]]
    rstd = ((h * h).sum(1) / cols + NORM_EPS) ** -0.5
    y = h * rstd[:, None] * s["weight"].double()[None, :]
    out = {"rstd": rstd}
    if case["scales"] == "tensor":
        out |= {"amax": y.abs().max().view(1, 1), "codes": (y / s["scale"].double()).clamp(-top, top)}
    else:
        scale, codes = [], torch.empty_like(y)
        step = GROUP[case["scales"]] or cols
        for c in range(0, cols, step):
            part = y[:, c:c + step]
            sc = part.abs().max(1).values.clamp_min(EPS) / top
            scale.append(sc)
            codes[:, c:c + step] = part / sc[:, None]
        out |= {"scale": torch.stack(scale, 1), "codes": codes}
    if case["residual"]:
        out["h"] = h
    return out


def _exact_grad(case, s):
    dy, h, w, c = s["dy"].double(), s["h"].double(), s["weight"].double(), s["rstd"].double()[:, None]
    cols = h.shape[1]
    # y_j = w_j h_j c, c = (mean h^2 + eps)^(-1/2):  dy_j/dh_i = w_j c (1[i = j] - c^2 h_i h_j / cols)
    dot = (dy * w * h).sum(1, keepdim=True)
    dx = c * w * dy - c ** 3 * h * dot / cols
    if case["residual"]:
        dx += s["res"].double()
    return {"dx": dx, "dweight": (dy * h * c).sum(0)}


def _exact_append(case, s):
    """In 64 bits, page after page; codes that this call writes as the value over its scale."""
    new, before = _lengths(case)
    out, top, page, heads = {}, FMAX[case["fmt"]], case["page"], case["heads"]
    table = s["table"].tolist()
    for name, sname, x in (("k", "ks", s["new"][:, :heads]), ("v", "vs", s["new"][:, heads:])):
        codes, scale, t = s[name].view(F8[case["fmt"]]).double(), s[sname].double(), 0
        for b in range(case["seqs"]):
            pos, end = before[b], before[b] + new[b]
            while pos < end:
                stop = min(end, (pos // page + 1) * page)
                at, off = table[b][pos // page], pos % page
                part = x[t:t + stop - pos].double().transpose(0, 1)
                sc = part.abs().amax((1, 2)).clamp_min(EPS) / top
                if case["pow2"]:
                    sc = 2.0 ** torch.ceil(torch.log2(sc))
                if off:
                    old = scale[at].clone()
                    sc = torch.maximum(old, sc)
                    codes[at, :, :off] *= (old / sc)[:, None, None]
                codes[at, :, off:off + stop - pos] = part / sc[:, None, None]
                scale[at] = sc
                t, pos = t + stop - pos, stop
        out[name], out[sname] = codes, scale
    return out


def _exact_attend(case, s):
    new, before = _lengths(case)
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    start = 0
    for b in range(case["seqs"]):
        n, length = new[b], new[b] + before[b]
        at = s["table"][b, : -(-length // case["page"])].long()
        i = torch.arange(before[b], length, device=DEV)[:, None]
        j = torch.arange(length, device=DEV)[None, :]
        hidden = torch.zeros(n, length, dtype=torch.bool, device=DEV)
        if case["causal"]:
            hidden |= j > i
        if case["window"]:
            hidden |= i - j >= case["window"]
        for head in range(case["heads"]):
            k, v = (s[c][at, head].view(F8[case["fmt"]]).double().mul(s[sc][at, head].double()[:, None, None])
                    .reshape(-1, case["dim"])[:length] for c, sc in (("k", "ks"), ("v", "vs")))
            for h in range(head * case["group"], (head + 1) * case["group"]):
                z = s["q"][start:start + n, h].double() @ k.T * s["sm_scale"]
                z[hidden] = -math.inf
                lse[start:start + n, h] = torch.logsumexp(z, 1)
                y[start:start + n, h] = torch.softmax(z, 1) @ v
        start += n
    return {"y": y, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "grad": _exact_grad, "append": _exact_append, "attend": _exact_attend}[case["op"]](case, s)
