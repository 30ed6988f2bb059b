"""64-bit references of the decoder-layer operators (norm to FP8 and its
gradient, the paged cache's append, attention over the cache), written from the
formulas in plain torch on the CPU, and the error bounds the tests hold the
kernels to.  u = 2^-24 is binary32's unit roundoff."""
import math

import torch

U = 2.0 ** -24
FMAX = (448.0, 57344.0)
MANT = (3, 2)     # mantissa bits of E4M3, E5M2
EMIN = (-6, -14)  # exponent of the smallest normal
F8 = (torch.float8_e4m3fn, torch.float8_e5m2)


def decode(codes, fmt):
    return codes.view(F8[fmt]).double()


def spacing(v, fmt):
    """Distance between neighbouring FP8 values around |v| (double)."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -40))).clamp_min(EMIN[fmt])
    return 2.0 ** (e - MANT[fmt])


def pow2_up(s):
    m, e = torch.frexp(s)
    return torch.where(m == 0.5, s, torch.ldexp(torch.ones_like(s), e))


def codes_off(codes, v, fmt, delta):
    """How many codes are not a correct rounding of some value within
    |v| delta of v (v = y / s in double, saturating)."""
    top = FMAX[fmt]
    lo, hi = v - v.abs() * delta, v + v.abs() * delta
    got = decode(codes, fmt)
    half = 0.5 * spacing(torch.maximum(lo.abs(), hi.abs()), fmt)
    return int(((got < lo.clamp(-top, top) - half) | (got > hi.clamp(-top, top) + half) | ~got.isfinite()).sum())


def norm(x, res, w, eps):
    """(h, rstd, y) in double."""
    h = x.double() if res is None else x.double() + res.double()
    rstd = 1.0 / torch.sqrt((h * h).mean(1) + eps)
    return h, rstd, h * rstd[:, None] * w.double()


def group_amax(y, g):
    """[rows x groups] amax of 1 x g groups, the last one short (g = 0: the row)."""
    rows, cols = y.shape
    g = g or cols
    return torch.nn.functional.pad(y.abs(), (0, -cols % g)).view(rows, -1, g).amax(2)


def spread(t, g, cols):
    """Per-group values repeated over their columns."""
    return t.repeat_interleave(g or cols, 1)[:, :cols]


def norm_grad(dy, h, w, rstd, dres):
    """(dx, dweight, bound of |dx|'s rounding terms, bound of dweight's) in double."""
    dy, n, c = dy.double(), h.double() * rstd.double()[:, None], rstd.double()[:, None]
    g = dy * w.double()
    dx = c * (g - n * (g * n).mean(1, keepdim=True))
    terms = c * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if dres is not None:
        dx = dx + dres.double()
        terms = terms + dres.double().abs()
    return dx, (dy * n).sum(0), terms, (dy * n).abs().sum(0)


class Batch:
    """A batch over a paged cache: sequence b brings new[b] tokens behind before[b]; `before` may be
    negative (kv_len below the number of new tokens)."""

    def __init__(self, new, before, page, seed=0, spare=2, extra_width=1):
        self.new, self.before, self.page = list(new), list(before), page
        self.lens = [n + b for n, b in zip(new, before)]
        per = [-(-max(0, x) // page) for x in self.lens]
        self.width = max(max(per), 1) + extra_width
        self.pages = sum(per) + spare
        g = torch.Generator().manual_seed(seed)
        order = torch.randperm(self.pages, generator=g)
        # entries behind a sequence's pages: values that must never be used as an index
        self.table = torch.full((len(self.new), self.width), 2 ** 30, dtype=torch.int32)
        self.table[:, ::2] = -7
        at = 0
        for b, p in enumerate(per):
            self.table[b, :p] = order[at:at + p].to(torch.int32)
            at += p
        self.start = torch.tensor([0] + self.new).cumsum(0).to(torch.int32)
        self.kv_len = torch.tensor(self.lens, dtype=torch.int32)
        self.tokens = int(self.start[-1])
        self.max_new, self.max_kv = max(1, max(self.new)), max(1, max(self.lens))


def scale_of(amax, fmt, eps, pow2):
    """The scale rule in binary32: (s, r)."""
    a = torch.maximum(amax, torch.tensor(eps, dtype=torch.float32))
    top = torch.full_like(a, FMAX[fmt])  # number / tensor would multiply by a rounded reciprocal
    s, r = a / top, top / a
    if pow2:
        s = pow2_up(s)
        r = 1.0 / s
    bad = ~amax.isfinite()
    nan = torch.tensor(math.nan)
    return torch.where(bad, nan, s), torch.where(bad, nan, r)


def cast(v, fmt):
    """Saturating cast of binary32 values; NaN -> 0x7F."""
    c = v.clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt]).view(torch.uint8)
    return torch.where(v.isnan(), torch.tensor(0x7F, dtype=torch.uint8), c)


def append(bt, x, cache, scale, fmt, eps, pow2):
    """New tokens x [tokens x heads x dim] into cache / scale (CPU tensors, updated in place), page after
    page: every step is one binary32 operation, so the result is compared bit for bit."""
    x = x.float()
    for b in range(len(bt.new)):
        first, t0 = bt.before[b], int(bt.start[b])
        pos = max(0, first)
        held = pos
        while pos < bt.lens[b]:
            lp = pos // bt.page
            end = min(bt.lens[b], (lp + 1) * bt.page)
            pg, part = int(bt.table[b, lp]), x[t0 + pos - first:t0 + end - first].transpose(0, 1)
            if 0 <= pg < cache.shape[0]:
                s, r = scale_of(part.abs().amax((1, 2)), fmt, eps, pow2)
                s[part.isnan().any(2).any(1)] = math.nan
                r[s.isnan()] = math.nan
                fill = max(0, held - lp * bt.page)
                if fill:
                    for hd in range(x.shape[1]):
                        old = scale[pg, hd].clone()
                        if not (s[hd] >= old) and not s[hd].isnan():
                            s[hd], r[hd] = old, 1.0 / old
                        elif s[hd] != old:
                            was = cache[pg, hd, :fill].view(F8[fmt]).float()
                            cache[pg, hd, :fill] = cast(was * (old / s[hd]), fmt)
                off = pos % bt.page
                cache[pg, :, off:off + end - pos] = cast(part * r[:, None, None], fmt)
                scale[pg] = s
            pos = end


def attend(bt, q, kc, vc, ks, vs, fmt, sm, causal, window):
    """(y, lse, bound of y, bound of lse) in double; hidden positions are left out of every sum."""
    T, QH, D = q.shape
    heads = kc.shape[1]
    y = torch.zeros(T, QH, D, dtype=torch.float64)
    lse = torch.full((T, QH), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(y), torch.zeros_like(lse)
    q = q.double()
    for b in range(len(bt.new)):
        length = min(max(0, bt.lens[b]), bt.width * bt.page)
        pos = torch.arange(length)
        pg = bt.table[b][pos // bt.page].long()
        there = (pg >= 0) & (pg < kc.shape[0])
        pg = pg.clamp(0, kc.shape[0] - 1)
        for i in range(bt.new[b]):
            t, at = int(bt.start[b]) + i, bt.before[b] + i
            seen = there.clone()
            if causal:
                seen &= pos <= at
            if window:
                seen &= pos > at - window
            j = pos[seen]
            if not len(j):
                continue
            p = pg[j]
            k = decode(kc[p, :, j % bt.page], fmt) * ks[p].double()[:, :, None]  # [n, heads, D]
            v = decode(vc[p, :, j % bt.page], fmt) * vs[p].double()[:, :, None]
            k, v = (u.repeat_interleave(QH // heads, 1) for u in (k, v))
            z = sm * (q[t][None] * k).sum(2)
            # binary32 dot product of exact products, then two scale multiplications
            dz = (D + 6) * U * abs(sm) * (q[t][None] * k).abs().sum(2).max(0).values + 4 * U * z.abs().max(0).values
            m = z.max(0).values
            w = torch.exp(z - m)
            l = w.sum(0)
            y[t] = (w[:, :, None] * v).sum(0) / l[:, None]
            lse[t] = m + torch.log(l)
            # exp2 of the shifted score (a few u of its argument's size), weights rounded to fp16
            # (2^-11, or 2^-25 of the largest where subnormal), binary32 sums, bf16 output
            arg = (z - m).abs().max(0).values
            rel = 2 * dz + 4 * U * (arg + 2) + 2.0 ** -11 + (len(j) + 8) * U
            mass = (w[:, :, None] * v.abs()).sum(0)
            low = torch.clamp(2.0 ** -25 * v.abs().amax((0, 2))[None] * len(j), min=0).T
            tol[t] = 2.0 ** -8 * y[t].abs() + (rel[:, None] * mass + low) / l[:, None] + 1e-30
            ltol[t] = dz + 4 * U * (arg + 2) + (len(j) + 8) * U + 4 * U * lse[t].abs()
    return y, lse, tol, ltol
