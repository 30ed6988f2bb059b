"""64-bit references of the gated half of a decoder layer (routing, the experts' products, the gated
activation with its checkpoint, the weighted sum), written from the formulas in plain Python and torch on
the CPU, and the error bounds the tests hold the kernels to.  u = 2^-24 is binary32's unit roundoff."""
import math

import torch

import layer_ref as lr

U = lr.U
FLT_MAX = torch.finfo(torch.float32).max
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative


def route(logits, k, score="softmax", bias=None, groups=1, top=1, best=1, renorm=True, scale=1.0):
    """(ids [tokens][k], weights [tokens][k], bound of the weights' relative error) token after token.  A bias of -Inf or
    NaN switches its expert off for the choice."""
    ids, weights, bounds = [], [], []
    for row in logits.double().tolist():
        E = len(row)
        l = [-math.inf if math.isnan(x) else min(x, FLT_MAX) for x in row]
        there = [x > -math.inf for x in l]
        m = max(l)
        if score == "softmax":
            e = [math.exp(x - m) if t else 0.0 for x, t in zip(l, there)]
            total = sum(e)
            p = [x / total if total else 0.0 for x in e]
        else:
            p = [(1 / (1 + math.exp(-x)) if x > -700 else math.exp(x)) if t else 0.0 for x, t in zip(l, there)]
        with_bias = p if bias is None else [x + b for x, b in zip(p, bias.double().tolist())]
        key = l if bias is None else with_bias
        there = [t and x > -math.inf for t, x in zip(there, key)]  # (False for NaN)
        open_ = set(range(E))
        if groups > 1:
            n, found = E // groups, []
            for g in range(groups):
                by = with_bias if bias is not None or best == 2 else l
                have = sorted((by[e] for e in range(g * n, g * n + n) if there[e]), reverse=True)
                if have:
                    found.append((-(have[0] + (have[1] if best == 2 and len(have) > 1 else 0.0)), g))
            open_ = {e for _, g in sorted(found)[:top] for e in range(g * n, g * n + n)}
        order = sorted((e for e in open_ if there[e]), key=lambda e: (-key[e], e))[:k]
        if renorm and order:  # relative to the largest: p itself may be too small for a number
            a = {e: (l[e] if score == "softmax" else min(l[e], 0.0)) for e in order}
            M = max(a.values())
            q = {e: math.exp(a[e] - M) / (1.0 if score == "softmax" else 1 + math.exp(-abs(l[e]))) for e in order}
            total = sum(q.values())
            w = [scale * q[e] / total for e in order]
            spread = M - min(a.values())
        else:
            w = [scale * p[e] for e in order]
            spread = m - min(l[e] for e in order) if score == "softmax" and order else 0.0
        ids.append(order + [-1] * (k - len(order)))
        weights.append(w + [0.0] * (k - len(order)))
        # exponentials (2 u each, and u of their argument), sums of up to 16 + 6 or k terms, quotients, products
        bounds.append((48 + 2 * min(spread, 100.0)) * U)
    return torch.tensor(ids, dtype=torch.int32), torch.tensor(weights, dtype=torch.float64), torch.tensor(bounds)[:, None]


def plan(ids, experts):
    """(slots, order without its tail, offsets) of the choices sorted by expert, then token."""
    flat = [(e, i) for i, e in enumerate(ids.view(-1).tolist()) if e >= 0]
    order = [i for _, i in sorted(flat)]
    slots = torch.full((ids.numel(),), -1, dtype=torch.int32)
    for s, i in enumerate(order):
        slots[i] = s
    counts = [0] * experts
    for e, _ in flat:
        counts[e] += 1
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
    return slots.view(ids.shape), torch.tensor(order, dtype=torch.int32), offsets


def route_grad(logits, ids, dw, score, renorm, scale):
    """(dlogits, sum of its terms' magnitudes) in double."""
    l = logits.double()
    l = torch.where(l.isnan(), -math.inf, l).clamp_max(FLT_MAX)
    out, terms = torch.zeros_like(l), torch.zeros_like(l)
    for t in range(l.shape[0]):
        e = torch.tensor([i for i in ids[t].tolist() if 0 <= i < l.shape[1]], dtype=torch.long)
        g = scale * dw[t, :].double()[[j for j, i in enumerate(ids[t].tolist()) if 0 <= i < l.shape[1]]]
        if not len(e):
            continue
        lc = l[t, e]
        if renorm:
            a = lc if score == "softmax" else lc.clamp_max(0)
            q = torch.exp(a - a.max()) / (1 if score == "softmax" else 1 + torch.exp(-lc.abs()))
            w = q / q.sum()
            f = 1.0 if score == "softmax" else 1 / (1 + torch.exp(lc))
            out[t, e] += w * (g - (w * g).sum()) * f
            terms[t, e] += w * (g.abs() + (w * g.abs()).sum()) * f
        elif score == "softmax":
            p = torch.softmax(l[t], 0)
            full = torch.zeros_like(p)
            full[e] = g
            out[t] = p * (full - (p * full).sum())
            terms[t] = p * (full.abs() + (p * full.abs()).sum())
        else:
            p = 1 / (1 + torch.exp(-lc))
            out[t, e] += g * p * (1 - p)
            terms[t, e] += (g * p * (1 - p)).abs()
    return out, terms


def experts(a, fa, sa, order, choices, b, sb, offsets, slots):
    """(y, bound without the output's rounding) of the experts' products; a [rows x K] and b [E x N x K] codes,
    sb [E x N].  The matrix cores lose less than 7 2^-13 of the largest |product| of each run of 8, and binary32
    accumulation less than 2^-23 of the sum of magnitudes at each of K / 8 + 16 steps."""
    E, N, K = b.shape
    y, tol = torch.zeros(slots, N, dtype=torch.float64), torch.zeros(slots, N, dtype=torch.float64)
    written = torch.zeros(slots, dtype=torch.bool)
    da, db = lr.decode(a, fa), lr.decode(b, 0)
    for e in range(E):
        for s in range(max(0, int(offsets[e])), min(slots, int(offsets[e + 1]))):
            written[s] = True
            r = s if order is None else int(order[s]) // choices if int(order[s]) >= 0 else -1
            if not 0 <= r < a.shape[0]:
                continue
            prod = da[r][None] * db[e]
            scale = sa[r].double() * sb[e].double()
            y[s] = prod.sum(1) * scale
            mag = prod.abs()
            tol[s] = (7 * 2.0 ** -13 * mag.view(N, -1, 8).amax(2).sum(1)
                      + ((K // 8 + 16) * 2.0 ** -23 + 4 * U) * mag.sum(1)) * scale.abs()
    return y, tol, written


GELU_A, GELU_B = math.sqrt(2 / math.pi), 0.044715


def act(g, kind):
    """(act(g), act'(g), |v|, |dv/dg|) in double, act = g sigmoid(v)."""
    v, dv = (g, torch.ones_like(g)) if kind == 0 else (2 * GELU_A * (g + GELU_B * g ** 3), 2 * GELU_A * (1 + 3 * GELU_B * g * g))
    c = torch.sigmoid(v)
    return g * c, c + g * c * (1 - c) * dv, v.abs(), dv


def gated_bound(v):
    """Relative error of g c u: v in 4 roundings, its product with log2 e and the exponential's argument 2 more, the
    hardware's exponential, reciprocal 2 u each, a sum and two products."""
    return (6 * v + 16) * U


def kept(x, fmt, eps):
    """(codes, scales) of one half of the checkpoint, every step one binary32 operation."""
    rows, cols = x.shape
    n = -(-cols // 128)
    xg = torch.nn.functional.pad(x.float(), (0, 128 * n - cols)).view(rows, n, 128)
    a = xg.abs().amax(2)
    a[xg.isnan().any(2)] = math.nan
    s, r = lr.scale_of(a, fmt, eps, False)
    return lr.cast(xg * r[:, :, None], fmt).view(rows, -1)[:, :cols], s
