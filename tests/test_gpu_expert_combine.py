"""fp8_expert_combine and its gradient against 64-bit references.  Bounds: k products and k + 1 sums in binary32
and the output's rounding; a dot product adds at most cols / 128 + 8 terms a thread, 6 shuffles and 16 waves."""
import math

import pytest
import torch

import expert_ref as ref

pytestmark = pytest.mark.gpu

U = ref.U


@pytest.fixture(scope="module")
def rt():
    import dynamic_scaling_scaled_amd as rt

    rt.lib()
    return rt


def inputs(tokens, k, cols, dtype, rows=None, pad=0, seed=0):
    g = torch.Generator().manual_seed(seed + tokens * 7 + cols)
    rows = rows or tokens * k
    x = torch.randn(rows, cols + pad, generator=g).to(dtype).cuda()[:, :cols]
    res = (2 * torch.randn(tokens, cols + pad, generator=g)).to(dtype).cuda()[:, :cols]
    dy = torch.randn(tokens, cols + 2 * pad, generator=g).to(dtype).cuda()[:, :cols]
    slots = torch.randperm(max(rows, tokens * k), generator=g)[:tokens * k].to(torch.int32).view(tokens, k).cuda()
    return x, res, dy, slots, torch.rand(tokens, k, generator=g).cuda()


def expected(x, slots, w, res, dy):
    x, w, dy, at = x.cpu().double(), w.cpu().double(), dy.cpu().double(), slots.cpu().long()
    there = (at >= 0) & (at < x.shape[0])
    rows = torch.where(there[:, :, None], x[at.clamp(0, x.shape[0] - 1)], 0.0)
    terms = torch.where(there[:, :, None], w[:, :, None] * rows, 0.0)
    y, mass = terms.sum(1), terms.abs().sum(1)
    if res is not None:
        y, mass = y + res.cpu().double(), mass + res.cpu().double().abs()
    return y, mass, (dy[:, None] * rows).sum(2), (dy[:, None] * rows).abs().sum(2), there


def check(rt, tokens, k, cols, dtype=torch.bfloat16, residual=True, change=None, alias=False, **kw):
    x, res, dy, slots, w = inputs(tokens, k, cols, dtype, **kw)
    if change:
        change(x, slots, w)
    want, mass, dots, dmass, there = expected(x, slots, w, res if residual else None, dy)
    y = res if alias else torch.full((tokens, cols), 7.0, dtype=dtype, device="cuda")
    rt.fp8_expert_combine(x, slots, w, y, residual=res if residual else None)
    tol = (k + 2) * U * mass + ref.HALF[dtype] * want.abs() + 2.0 ** -133
    assert bool(((y.cpu().double() - want).abs() <= tol).all())
    dx, dw = torch.full_like(x, 7.0), torch.full((tokens, k), 7.0, device="cuda")
    rt.fp8_expert_combine_backward(dy, x, slots, w, dx, dw)
    assert bool(((dw.cpu().double() - dots).abs() <= (cols / 128 + 40) * U * dmass).all())
    rows = torch.full(x.shape, 7.0, dtype=dtype)
    part = (w.cpu()[:, :, None] * dy.cpu().float()[:, None]).to(dtype)  # one product, one rounding
    rows[slots.cpu().long()[there]] = part[there]
    assert torch.equal(dx.cpu(), rows)


@pytest.mark.parametrize("cols", [8, 64, 512, 520, 2048, 7168, 8200])
@pytest.mark.parametrize("k", [1, 2, 8, 9, 16, 32])
def test_sizes(rt, cols, k):
    check(rt, 3, k, cols, pad=8)
    check(rt, 5, k, cols, dtype=torch.float32, residual=False)


def test_many_tokens(rt):
    check(rt, 3000, 2, 72)
    check(rt, 700, 8, 264, alias=True)
    check(rt, 1, 8, 16384)


def test_slots_outside(rt):
    """Choices without a slot count for nothing, whatever their weight; rows of no slot stay as they were."""
    def change(x, slots, w):
        slots[0, 1] = -1
        slots[1] = -1
        slots[2, 0], slots[3, 2] = x.shape[0], 2 ** 31 - 1
        slots[4, 1] = -2 ** 31
        w[0, 1] = math.nan
        w[2, 0] = math.inf
    check(rt, 9, 3, 136, rows=40, change=change)
    check(rt, 9, 3, 136, dtype=torch.float32, residual=False, change=change)


def test_not_finite(rt):
    """A row that is not finite reaches its own token alone."""
    x, res, dy, slots, w = inputs(6, 2, 64, torch.bfloat16)
    x[slots[2, 1].long()] = math.nan
    x[slots[3, 0].long(), 5] = math.inf
    y = torch.empty_like(res)
    rt.fp8_expert_combine(x, slots, w, y, residual=res)
    dx, dw = torch.zeros_like(x), torch.empty(6, 2, device="cuda")
    rt.fp8_expert_combine_backward(dy, x, slots, w, dx, dw)
    bad = ~y.isfinite().all(1)
    assert bad.cpu().tolist() == [False, False, True, True, False, False] and int((~y[3].isfinite()).sum()) == 1
    assert bool(dw[2, 1].isnan()) and bool(dx.isfinite().all()) and int((~dw.isfinite()).sum()) == 2


def test_gradient_in_place(rt):
    x, _, dy, slots, w = inputs(20, 4, 264, torch.bfloat16)
    dx, dw, dw2 = torch.empty_like(x), torch.empty(20, 4, device="cuda"), torch.empty(20, 4, device="cuda")
    rt.fp8_expert_combine_backward(dy, x, slots, w, dx, dw)
    rt.fp8_expert_combine_backward(dy, x, slots, w, x, dw2)
    assert torch.equal(x, dx) and torch.equal(dw, dw2)


def test_gradient_against_differences(rt):
    """The sum is linear in rows and weights: a unit step changes <y, dy> by the gradient."""
    x, res, dy, slots, w = inputs(4, 3, 32, torch.float32)
    dx, dw = torch.zeros_like(x), torch.empty_like(w)
    rt.fp8_expert_combine_backward(dy, x, slots, w, dx, dw)

    def loss(x, w):
        y = torch.empty_like(res)
        rt.fp8_expert_combine(x, slots, w, y, residual=res)
        return float((y.double() * dy.double()).sum())
    base = loss(x, w)
    for t, j, c in ((0, 0, 0), (3, 2, 31), (1, 1, 17)):
        x2, w2 = x.clone(), w.clone()
        x2[slots[t, j].long(), c] += 1.0
        w2[t, j] += 1.0
        assert abs(loss(x2, w) - base - float(dx[slots[t, j].long(), c])) < 1e-4
        assert abs(loss(x, w2) - base - float(dw[t, j])) < 1e-4


def test_graph(rt):
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x, res, dy, slots, w = inputs(50, 4, 520, torch.bfloat16)
        y, dx, dw = torch.empty_like(res), torch.empty_like(x), torch.empty_like(w)

        def call(y, dx, dw):
            rt.fp8_expert_combine(x, slots, w, y, residual=res)
            rt.fp8_expert_combine_backward(dy, x, slots, w, dx, dw)
        call(y, dx, dw)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(y, dx, dw)
        for seed in range(3):
            for a, b in zip((x, res, dy, slots, w), inputs(50, 4, 520, torch.bfloat16, seed=seed + 1)):
                a.copy_(b)
            g.replay()
            s.synchronize()
            want = torch.empty_like(y), torch.empty_like(dx), torch.empty_like(dw)
            call(*want)
            assert all(torch.equal(a, b) for a, b in zip(want, (y, dx, dw)))
