"""fp8_expert_route and its gradient against 64-bit references: choices and plan exactly, weights and
gradients within the bounds of expert_ref (each exponential 2 u and u of its argument, sums, quotients)."""
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


def run(rt, logits, k, score="softmax", bias=None, groups=1, top=1, best=1, renorm=True, scale=1.0, planned=True, out=None):
    tokens, experts = logits.shape
    o = out or {"ids": torch.full((tokens, k), -7, dtype=torch.int32, device="cuda"),
                "weights": torch.full((tokens, k), -7.0, device="cuda")}
    if planned and out is None:
        o |= {"slots": torch.full((tokens, k), -7, dtype=torch.int32, device="cuda"),
              "order": torch.full((tokens * k,), -7, dtype=torch.int32, device="cuda"),
              "offsets": torch.full((experts + 1,), -7, dtype=torch.int32, device="cuda")}
    rt.fp8_expert_route(logits, **o, score=rt.SOFTMAX if score == "softmax" else rt.SIGMOID, bias=bias, groups=groups,
                        top_groups=top, group_best=best, renormalise=renorm, scale=scale)
    return o


def check(rt, logits, k, bias=None, **kw):
    """logits: on the GPU, of any stride."""
    o = {n: t.cpu() for n, t in run(rt, logits, k, bias=bias, **kw).items()}
    ids, weights, rel = ref.route(logits.cpu().float(), k, bias=None if bias is None else bias.cpu(), **kw)
    assert torch.equal(o["ids"], ids)
    assert bool(((o["weights"].double() - weights).abs() <= rel * weights.abs() + 2.0 ** -149).all())
    slots, order, offsets = ref.plan(ids, logits.shape[1])
    assert torch.equal(o["slots"], slots) and torch.equal(o["offsets"], offsets)
    assert torch.equal(o["order"][:len(order)], order) and bool((o["order"][len(order):] == -7).all())


def logits_of(tokens, experts, dtype=torch.float32, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed + tokens * 31 + experts)
    x = 1.5 * torch.randn(tokens, experts + pad, generator=g) + torch.randn(experts + pad, generator=g)
    return x.to(dtype).cuda()[:, :experts]


CHOICES = [dict(), dict(renorm=False), dict(score="sigmoid", scale=2.5), dict(score="sigmoid", renorm=False),
           dict(groups=4, top=2), dict(groups=4, top=2, best=2), dict(groups=4, top=3, best=2, score="sigmoid")]


@pytest.mark.parametrize("experts,k", [(8, 1), (8, 8), (60, 4), (64, 6), (100, 7), (128, 8), (160, 8), (256, 8), (512, 16),
                                       (1000, 32), (1024, 10)])
@pytest.mark.parametrize("tokens", [1, 17])
def test_experts(rt, experts, k, tokens):
    for i, kw in enumerate(CHOICES):
        if experts // kw.get("groups", 1) * kw.get("top", 1) < k:
            kw = dict(kw, top=kw["groups"])
        g = torch.Generator().manual_seed(i)
        bias = (0.1 * torch.randn(experts, generator=g)).cuda()
        dtype = torch.bfloat16 if i % 2 else torch.float32
        check(rt, logits_of(tokens, experts, dtype, i, pad=i), k, **kw)
        check(rt, logits_of(tokens, experts, dtype, i, pad=i), k, bias=bias, **kw)


@pytest.mark.parametrize("tokens", [2, 63, 64, 65, 96, 97, 500, 2049])
def test_tokens(rt, tokens):
    """One workgroup, several, a short last one; the plan in one kernel and in two."""
    check(rt, logits_of(tokens, 24, torch.bfloat16), 3)
    check(rt, logits_of(tokens, 256, seed=3), 8, score="sigmoid", groups=8, top=4, best=2, bias=logits_of(1, 256)[0] * 0.05)


@pytest.mark.parametrize("tokens,experts,k,kw", [
    (700, 600, 5, dict(score="sigmoid")), (2500, 200, 6, dict(groups=2, top=1, best=2)), (5000, 256, 3, dict()),
    (4200, 40, 4, dict(groups=5, top=2, best=2)), (1500, 120, 9, dict(score="sigmoid", groups=3, top=2))])
def test_blocks_of_tokens(rt, tokens, experts, k, kw):
    """Blocks of 8, 16 and 32 tokens, one and two rounds of a workgroup's runs; groups that are no runs of lanes."""
    bias = logits_of(1, experts, seed=5)[0] * 0.02
    check(rt, logits_of(tokens, experts, seed=9), k, bias=bias, **kw)


def test_many_tokens(rt):
    """More than 256 workgroups, blocks of 32 and of 64 tokens: the plan against a stable sort of the ids."""
    for tokens, experts, k in ((16385, 8, 2), (9000, 64, 6), (40000, 16, 4), (70001, 128, 1)):
        o = run(rt, logits_of(tokens, experts), k)
        flat = o["ids"].view(-1).long()
        by, order = flat.sort(stable=True)
        assert torch.equal(o["order"].long(), order)
        assert torch.equal(o["offsets"].long(), torch.searchsorted(by, torch.arange(experts + 1, device="cuda")))
        assert torch.equal(o["slots"].view(-1)[order].long(), torch.arange(tokens * k, device="cuda"))


@pytest.mark.parametrize("groups,top,best", [(1, 1, 1), (2, 1, 2), (4, 2, 1), (4, 2, 2), (16, 5, 2), (64, 33, 1)])
@pytest.mark.parametrize("biased", [False, True])
def test_ties(rt, groups, top, best, biased):
    """Few distinct values: equal keys go to the lower expert, equal groups to the lower group."""
    g = torch.Generator().manual_seed(groups)
    x = torch.randint(-2, 2, (70, 64), generator=g).float().cuda()
    x[3] = 0.0
    x[4, ::2], x[4, 1::2] = 0.0, -0.0
    bias = torch.randint(0, 2, (64,), generator=g).float().cuda() if biased else None
    for score in ("softmax", "sigmoid"):
        check(rt, x, min(6, 64 // groups * top), bias=bias, score=score, groups=groups, top=top, best=best)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_absent_experts(rt, score, renorm, biased):
    """-Inf and NaN are absent: rows with all, some, fewer than k and none; +Inf is the largest finite value."""
    x = logits_of(40, 32, seed=9)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, 3:] = -math.inf
    x[3, :31] = math.nan
    x[4, ::2] = -math.inf
    x[5, 7] = math.inf
    x[6, 9:11] = math.inf
    x[7] = torch.finfo(torch.float32).min
    x[8, :16] = -math.inf  # two whole groups
    x[9, 1:8] = -math.inf  # one expert of its group
    bias = (0.3 * torch.randn(32, generator=torch.Generator().manual_seed(1))).cuda() if biased else None
    for kw in (dict(), dict(groups=4, top=2, best=1), dict(groups=4, top=2, best=2)):
        check(rt, x, 6, bias=bias, score=score, renorm=renorm, **kw)
    check(rt, x[:2], 6, bias=bias, score=score, renorm=renorm)  # no expert at all


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_too_small_for_a_number(rt, score):
    """Far logits: chosen by their bias, p itself underflows; renormalised weights are still the scores' ratio."""
    x = torch.full((4, 16), -300.0).cuda()
    x[:, 0] = 90.0
    x[1, 1:] -= torch.arange(15).cuda() * 0.25
    x[2] = -200.0
    x[3] = 200.0
    bias = torch.zeros(16).cuda()
    bias[8:] = 4.0
    check(rt, x, 4, bias=bias, score=score)
    check(rt, x, 4, score=score)


def test_choice_alone(rt):
    """Without a plan, and a bias of the type's ends."""
    x = logits_of(100, 48)
    o = run(rt, x, 5, planned=False)
    ids, _, _ = ref.route(x.cpu(), 5)
    assert torch.equal(o["ids"].cpu(), ids)
    bias = torch.zeros(48).cuda()
    bias[5], bias[6] = 3e38, -3e38
    check(rt, x, 32, bias=bias, score="sigmoid", renorm=False)


def grad(rt, x, ids, dw, dl, score="softmax", renorm=True, scale=1.0):
    rt.fp8_expert_route_backward(x, ids, dw, dl, score=rt.SOFTMAX if score == "softmax" else rt.SIGMOID, renormalise=renorm,
                                 scale=scale)


def check_grad(rt, x, ids, dw, score, renorm, scale, inplace=False):
    dl = x.clone() if inplace else torch.full_like(x, 7.0)
    grad(rt, dl if inplace else x, ids, dw, dl, score, renorm, scale)
    want, terms = ref.route_grad(x.cpu().float(), ids.cpu(), dw.cpu(), score, renorm, scale)
    l = x.cpu().double().clamp(-200, 200)
    l = torch.where(l.isnan(), 0.0, l)
    spread = (l.max(1).values - l.min(1).values)[:, None]
    tol = (96 + 4 * spread) * U * terms + ref.HALF[x.dtype] * want.abs() + 2.0 ** -133
    assert bool(((dl.cpu().double() - want).abs() <= tol).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("experts,k", [(8, 8), (60, 4), (64, 6), (130, 8), (256, 8), (512, 16), (1024, 32)])
def test_gradient(rt, score, renorm, experts, k):
    for tokens, dtype in ((1, torch.float32), (33, torch.bfloat16), (70, torch.float32)):
        x = logits_of(tokens, experts, dtype, 5, pad=3)
        ids = run(rt, x, k, score=score)["ids"]
        dw = torch.randn(tokens, k, generator=torch.Generator().manual_seed(k)).cuda()
        check_grad(rt, x, ids, dw, score, renorm, 2.5)
    check_grad(rt, x, ids, dw, score, renorm, 1.0, inplace=True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_of_odd_choices(rt, score, renorm):
    """Places without an expert, ids outside the experts, absent experts, rows without any."""
    x = logits_of(8, 20, seed=2)
    x[2, 4:] = -math.inf
    x[3] = -math.inf
    x[5, ::3] = math.nan
    ids = run(rt, x, 6, score=score)["ids"]
    ids[0, 2], ids[1, 1], ids[4] = 20, 2 ** 31 - 1, -1
    ids[6, 0] = -2 ** 31
    check_grad(rt, x, ids, torch.randn(8, 6, generator=torch.Generator().manual_seed(1)).cuda(), score, renorm, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(rt, score, renorm):
    """Central differences of the 64-bit weights (step 1e-4: error of 1e-8 of the third derivative's size)."""
    x, k = logits_of(6, 12, seed=4), 4
    ids = run(rt, x, k, score=score)["ids"]
    dw = torch.randn(6, k, generator=torch.Generator().manual_seed(2))
    dl = torch.empty_like(x)
    grad(rt, x, ids, dw.cuda(), dl, score, renorm, 1.5)
    base, at = x.cpu().double(), ids.cpu().long()

    def loss(l):
        p = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
        w = p.gather(1, at)
        if renorm:
            w = w / w.sum(1, keepdim=True)
        return (1.5 * w * dw.double()).sum(1)

    h = 1e-4
    for e in range(12):
        step = torch.zeros(12, dtype=torch.float64)
        step[e] = h
        diff = (loss(base + step) - loss(base - step)) / (2 * h)
        assert bool(((dl[:, e].cpu().double() - diff).abs() < 1e-5).all())


def test_streams_and_repeats(rt):
    """Another stream than the current one, and the same bits again and again."""
    x = logits_of(3000, 64)
    first = run(rt, x, 6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        again = {n: torch.full_like(t, -9) for n, t in first.items()}
        torch.cuda.current_stream().synchronize()
        rt.fp8_expert_route(x, **again, stream=s)
        s.synchronize()
        assert all(torch.equal(again[n], first[n]) for n in first)


def test_graph(rt):
    """Captured and replayed on new logits, with other calls between the replays."""
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x = logits_of(400, 64)
        out = run(rt, x, 6, score="sigmoid")
        dw, dl = torch.randn(400, 6, device="cuda"), torch.empty_like(x)
        grad(rt, x, out["ids"], dw, dl, "sigmoid")
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            run(rt, x, 6, score="sigmoid", out=out)
            grad(rt, x, out["ids"], dw, dl, "sigmoid")
        for seed in range(4):
            x.copy_(logits_of(400, 64, seed=seed))
            g.replay()
            s.synchronize()
            want = run(rt, x, 6, score="sigmoid")
            assert all(torch.equal(want[n], out[n]) for n in want)
            d2 = torch.empty_like(x)
            grad(rt, x, want["ids"], dw, d2, "sigmoid")
            assert torch.equal(d2, dl)
