"""fp8_expert_gemm against 64-bit products of the codes' values (bound: expert_ref.experts)."""
import pytest
import torch

import expert_ref as ref
import layer_ref as lr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rt():
    import dynamic_scaling_scaled_amd as rt

    rt.lib()
    return rt


def codes(shape, fmt, g):
    return (torch.randn(shape, generator=g) * 20).clamp(-lr.FMAX[fmt], lr.FMAX[fmt]).to(lr.F8[fmt]).view(torch.uint8)


def weights(rt, E, N, K, g):
    b = codes((E, N, K), 0, g)
    return b, rt.fp8_pack_weights16(b.view(E * N, K).cuda())


def check(rt, counts, N, K, fa=0, out=torch.bfloat16, choices=1, gather=False, ga=(1, 0), gb="channel", pad=0, spare=0,
          seed=0, change=None):
    """counts: slots of each expert; gather: rows of a by order // choices; spare: rows of y behind the last expert."""
    g = torch.Generator().manual_seed(seed + 13 * N + K)
    E, S = len(counts), sum(counts) + spare
    rows = -(-S // choices) if gather else S
    a = torch.zeros(rows, K + pad, dtype=torch.uint8)
    a[:, :K] = codes((rows, K), fa, g)
    b, image = weights(rt, E, N, K, g)
    sa = torch.rand(rows if ga == (1, 0) else 1, 1, generator=g) + 0.5
    sb = torch.rand(E, N if gb == "channel" else 1, generator=g) + 0.5
    if gb == "tensor":
        sb = sb[:1]
    gran = {"channel": (1, 0), "expert": (N, 0), "tensor": (0, 0)}[gb]
    order = torch.randperm(S, generator=g).to(torch.int32) if gather else None
    offsets = torch.tensor([0] + list(counts)).cumsum(0).to(torch.int32)
    if change:
        change(order, offsets)
    y = torch.full((S, N + pad), 7.0, dtype=out).cuda()
    rt.fp8_expert_gemm(a.cuda()[:, :K], fa, ga, sa.cuda(), image, rt.E4M3, gran, sb.cuda(), offsets.cuda(), y[:, :N],
                       order=None if order is None else order.cuda(), choices=choices)
    want, tol, written = ref.experts(a[:, :K].contiguous(), fa, sa.expand(rows, 1), order, choices, b,
                                     sb.expand(E, N), offsets, S)
    got = y.cpu()
    assert bool((got[:, N:] == 7).all()) and bool((got[~written] == 7).all())
    err = (got[:, :N].double() - want).abs()
    assert bool((err <= tol + ref.HALF[out] * (want.abs() + tol))[written].all())


@pytest.mark.parametrize("counts", [(1,), (16,), (17,), (0, 1, 0), (3, 0, 0, 5, 1), (15, 16, 17, 33), (0, 0, 70), (40, 40)])
@pytest.mark.parametrize("N,K", [(16, 128), (48, 256), (80, 640)])
def test_counts(rt, counts, N, K):
    check(rt, counts, N, K)
    check(rt, counts, N, K, gather=True, choices=3, out=torch.float32, pad=16)


@pytest.mark.parametrize("rows", [5, 20, 50, 100, 130, 200, 257, 300])
def test_rows_of_an_expert(rt, rows):
    """Every tile height, whole and partial, beside an idle and a small expert."""
    check(rt, (rows, 0, rows // 2, rows), 64, 256, spare=3)
    check(rt, (rows, 0, rows // 2, rows), 272, 384, gather=True, choices=2)


@pytest.mark.parametrize("kw", [dict(), dict(fa=1, out=torch.float32, gather=True, choices=3, pad=32),
                                dict(out=torch.float32, ga=(0, 0), gb="expert"), dict(fa=1, gather=True, spare=9, gb="tensor")])
@pytest.mark.parametrize("counts", [(150, 140), (300, 70, 200, 130, 240), (257, 1, 300)])
@pytest.mark.parametrize("N", [16, 272])
def test_many_rows_and_deep(rt, counts, N, kw):
    """The tiles of 256 slots, with each number of blocks of 64."""
    check(rt, counts, N, 2176, **kw)


@pytest.mark.parametrize("fa", [0, 1])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ga", [(1, 0), (0, 0)])
@pytest.mark.parametrize("gb", ["channel", "expert", "tensor"])
@pytest.mark.parametrize("counts", [(3, 6), (30, 20), (150, 140)])
def test_types_and_scales(rt, fa, out, ga, gb, counts):
    check(rt, counts, 64, 256, fa=fa, out=out, ga=ga, gb=gb, pad=32)


@pytest.mark.parametrize("K", [128, 256, 384, 1152, 4096])
@pytest.mark.parametrize("counts", [(2, 1), (20, 30), (120, 90), (280, 300)])
def test_depths(rt, K, counts):
    check(rt, counts, 32, K)


@pytest.mark.parametrize("N", [16, 256, 528, 2048])
@pytest.mark.parametrize("counts", [(4, 4), (70, 2), (260, 5)])
def test_widths(rt, N, counts):
    check(rt, counts, N, 128, gather=True, choices=2)


def test_many_experts(rt):
    g = torch.Generator().manual_seed(1)
    check(rt, torch.randint(0, 5, (200,), generator=g).tolist(), 32, 128, gather=True, choices=2)
    check(rt, torch.randint(0, 2, (1024,), generator=g).tolist(), 16, 128)
    check(rt, [0] * 63 + [300] + [0] * 64 + [1], 64, 256)


@pytest.mark.parametrize("rows", [6, 90, 260])
def test_untrusted_plan(rt, rows):
    """Offsets past the slots, falling, negative; rows of a that are not there: bounded, and such slots are 0."""
    def change(order, offsets):
        offsets[0] = -5
        offsets[-1] = 2 ** 31 - 1
        if order is not None:
            order[0], order[3], order[5] = -1, 2 ** 31 - 1, -2 ** 31
    check(rt, (rows, rows, 2), 64, 256, change=change)
    check(rt, (rows, rows, 2), 64, 256, gather=True, choices=2, change=change)

    def falling(order, offsets):  # expert 1 ends before it starts; expert 2 takes the rest
        offsets[1], offsets[2] = rows, 0
    g = torch.Generator().manual_seed(3)
    a, (b, image) = codes((2 * rows, 256), 0, g), weights(rt, 3, 64, 256, g)
    one = torch.ones(1, 1).cuda()
    offsets = torch.tensor([0, rows, 0, 0], dtype=torch.int32)
    y = torch.full((2 * rows, 64), 7.0).cuda()
    rt.fp8_expert_gemm(a.cuda(), 0, (0, 0), one, image, 0, (0, 0), one, offsets.cuda(), y)
    want, tol, written = ref.experts(a, 0, torch.ones(2 * rows, 1), None, 1, b, torch.ones(3, 64), offsets, 2 * rows)
    assert bool((y.cpu()[~written] == 7).all()) and bool(((y.cpu().double() - want).abs() <= tol + 2.0 ** -23 * want.abs())[written].all())


def test_no_slot_at_all(rt):
    check(rt, (0, 0, 0), 64, 256, spare=20)
    check(rt, (0, 0, 0), 64, 256, spare=300, gather=True, choices=2)


def test_not_finite(rt):
    """A row of NaN codes stays in its own slots; what the other rows of its tile hold is untouched."""
    for n in (8, 100, 260):
        g = torch.Generator().manual_seed(n)
        a, (b, image) = codes((n, 256), 0, g), weights(rt, 2, 64, 256, g)
        one = torch.ones(1, 1).cuda()
        offsets = torch.tensor([0, n // 2, n], dtype=torch.int32).cuda()
        y, y2 = torch.empty(n, 64).cuda(), torch.empty(n, 64).cuda()
        rt.fp8_expert_gemm(a.cuda(), 0, (0, 0), one, image, 0, (0, 0), one, offsets, y)
        a[3] = 0x7F
        rt.fp8_expert_gemm(a.cuda(), 0, (0, 0), one, image, 0, (0, 0), one, offsets, y2)
        assert bool(y2[3].isnan().all())
        y2[3] = y[3]
        assert torch.equal(y, y2)


def test_large_against_double(rt):
    """Sizes of real layers, on the GPU in 64 bits; the bound of a dot product's loss as a whole: 7 2^-13 of
    the products' sum of magnitudes, and bf16's half step."""
    for E, S, N, K in ((16, 100, 2048, 2048), (4, 1500, 1024, 2048)):
        g = torch.Generator(device="cuda").manual_seed(S)
        a = torch.randn(S, K, device="cuda", generator=g).mul(20).clamp(-448, 448).to(torch.float8_e4m3fn)
        b = torch.randn(E, N, K, device="cuda", generator=g).mul(20).clamp(-448, 448).to(torch.float8_e4m3fn)
        image = rt.fp8_pack_weights16(b.view(torch.uint8).view(E * N, K))
        cuts = torch.randint(0, S + 1, (E - 1,), generator=torch.Generator().manual_seed(S)).sort().values.tolist()
        offsets = [0] + cuts + [S]
        sa, sb = torch.rand(S, 1, device="cuda", generator=g), torch.rand(E, N, device="cuda", generator=g)
        y = torch.empty(S, N, dtype=torch.bfloat16, device="cuda")
        plan = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        rt.fp8_expert_gemm(a.view(torch.uint8), 0, (1, 0), sa, image, 0, (1, 0), sb, plan, y)
        again = torch.empty_like(y)
        rt.fp8_expert_gemm(a.view(torch.uint8), 0, (1, 0), sa, image, 0, (1, 0), sb, plan, again)
        assert torch.equal(y, again)
        for e in range(E):
            lo, hi = offsets[e], offsets[e + 1]
            x, w = a[lo:hi].double(), b[e].double().T.contiguous()
            scale = sa[lo:hi].double() * sb[e].double()[None]
            want, mag = (x @ w) * scale, (x.abs() @ w.abs()) * scale
            assert bool(((y[lo:hi].double() - want).abs() <= 7 * 2.0 ** -13 * mag + 2.0 ** -8 * want.abs() * 1.01).all())


def test_graph(rt):
    """One captured call, replayed on other plans."""
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.Generator().manual_seed(2)
        E, S, N, K = 6, 40, 64, 256
        a, (_, image) = codes((S, K), 0, g).cuda(), weights(rt, E, N, K, g)
        sa, sb = torch.rand(S, 1, generator=g).cuda(), torch.rand(E, N, generator=g).cuda()
        offsets, order = torch.zeros(E + 1, dtype=torch.int32).cuda(), torch.zeros(S, dtype=torch.int32).cuda()
        y = torch.empty(S, N, device="cuda")

        def call(y):
            rt.fp8_expert_gemm(a, 0, (1, 0), sa, image, 0, (1, 0), sb, offsets, y, order=order, choices=1)
        call(y)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call(y)
        for i in range(4):
            cuts = torch.randint(0, S + 1, (E - 1,), generator=g).sort().values
            offsets.copy_(torch.cat([torch.zeros(1), cuts, torch.full((1,), S)]).to(torch.int32))
            order.copy_(torch.randperm(S, generator=g).to(torch.int32))
            y.fill_(7.0)
            graph.replay()
            s.synchronize()
            want = torch.full_like(y, 7.0)
            call(want)
            assert torch.equal(y, want)
