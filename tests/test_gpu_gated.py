"""fp8_gated_quantize and fp8_gated_backward against 64-bit references, the checkpoint bit for bit (bounds: expert_ref)."""
import math

import pytest
import torch

import expert_ref as ref
import layer_ref as lr

pytestmark = pytest.mark.gpu

U = ref.U
EPS = 1e-12


@pytest.fixture(scope="module")
def rt():
    import dynamic_scaling_scaled_amd as rt

    rt.lib()
    return rt


def wide(rows, cols, pad, dtype, g, scale=1.0):
    return (torch.randn(rows, cols + pad, generator=g) * scale).to(dtype).cuda()[:, :cols]


def check(rt, rows, cols, dtype=torch.bfloat16, act=0, gran=(1, 0), fmt=0, mode=0, pow2=False, pad=0, keep=True, kf=0,
          live=None, spread=2.0, seed=0, extra=None):
    g = torch.Generator().manual_seed(seed + rows * 131 + cols)
    x = wide(rows, 2 * cols, pad, dtype, g, spread)
    x[:, ::7] *= 3
    if extra:
        extra(x)
    n = rt.scale_shape((rows, cols), gran)
    scale = torch.full(n, -1.0).cuda() if mode == rt.DYNAMIC else torch.full(n, 40.0 / lr.FMAX[fmt]).cuda()
    inv = torch.full(n, -1.0).cuda() if mode == rt.DYNAMIC else None
    amax = torch.full(n, -1.0).cuda()
    q = torch.full((rows, cols + pad), 0xAA, dtype=torch.uint8).cuda()
    kept = torch.full((rows, 2 * cols + pad), 0xAA, dtype=torch.uint8).cuda() if keep else None
    ks = torch.full((rows, 2, -(-cols // 128)), -1.0).cuda() if keep else None
    count = None if live is None else torch.tensor([live], dtype=torch.int32).cuda()
    rt.fp8_gated_quantize(x, gran, fmt, mode, EPS, pow2, scale, q[:, :cols], act=act, inv_scale=inv, amax_out=amax,
                          kept=kept[:, :2 * cols] if keep else None, kept_scale=ks, kept_fmt=kf, live=count)
    torch.cuda.synchronize()
    L = rows if live is None else max(0, min(rows, live))
    assert bool((q[:, cols:] == 0xAA).all()) and bool((q[L:] == 0xAA).all())
    xc = x.cpu()[:L]
    if keep:
        assert bool((kept[:, 2 * cols:] == 0xAA).all()) and bool((kept[L:] == 0xAA).all()) and bool((ks[L:] == -1.0).all())
        for h in range(2 if L else 0):
            codes, s = ref.kept(xc[:, h * cols:(h + 1) * cols], kf, EPS)
            assert torch.equal(kept[:L, h * cols:(h + 1) * cols].cpu(), codes)
            assert torch.equal(ks[:L, h].cpu(), s)
    if not L:
        return
    f, _, v, _ = ref.act(xc[:, :cols].double(), act)
    z = f * xc[:, cols:].double()
    rel = ref.gated_bound(v)
    am = z.abs().max().view(1, 1) if gran == (0, 0) else lr.group_amax(z, gran[1])
    err = (rel * z.abs()).max().view(1, 1) if gran == (0, 0) else lr.group_amax(rel * z, gran[1])
    if gran != (0, 0):
        got = amax.cpu()[:L]
        if mode == rt.DYNAMIC:  # the scale rule on the observed amax, bit for bit
            s, r = lr.scale_of(got, fmt, EPS, pow2)
            assert torch.equal(scale.cpu()[:L], s) and torch.equal(inv.cpu()[:L], r)
            assert bool((scale[L:] == -1.0).all()) and bool((amax[L:] == -1.0).all())
    else:
        got = amax.cpu()
    assert bool(((got.double() - am).abs() <= err + U * am).all())
    sc = scale.cpu().double()
    sc = sc if gran == (0, 0) else lr.spread(sc[:L], gran[1], cols)
    assert lr.codes_off(q[:L, :cols].cpu().contiguous(), z / sc, fmt, rel + 8 * U) == 0


@pytest.mark.parametrize("cols", [16, 64, 144, 512, 528, 2048, 8192, 8208, 16400, 29568, 65536])
def test_widths(rt, cols):
    check(rt, 3, cols, pad=16)
    check(rt, 3, cols, gran=(1, 128), act=1)


@pytest.mark.parametrize("gran", [(1, 0), (1, 16), (1, 32), (1, 64), (1, 128), (1, 256), (1, 512), (0, 0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("act", [0, 1])
def test_granularities(rt, gran, dtype, fmt, act):
    mode = rt.GIVEN if gran == (0, 0) else rt.DYNAMIC
    check(rt, 37, 1040, dtype=dtype, gran=gran, fmt=fmt, act=act, mode=mode, pad=48, kf=fmt)
    check(rt, 2, 2048, dtype=dtype, gran=gran, fmt=fmt, act=act, mode=mode, keep=False)


@pytest.mark.parametrize("gran", [(1, 16), (1, 128), (1, 512), (0, 0)])
@pytest.mark.parametrize("cols", [4096, 4112, 8208, 20000])
def test_few_wide_rows(rt, gran, cols):
    """Rows that are cut into chunks, whole and not, with groups short at the row's end."""
    mode = rt.GIVEN if gran == (0, 0) else rt.DYNAMIC
    check(rt, 5, cols, gran=gran, mode=mode, pad=16)
    check(rt, 7, cols, gran=gran, mode=mode, act=1, keep=False, live=None if gran == (0, 0) else 4)
    check_grad(rt, 6, cols, act=1, pad=16, live=4)


@pytest.mark.parametrize("gran", [(1, 0), (1, 32), (1, 128)])
def test_given_and_pow2(rt, gran):
    check(rt, 33, 784, gran=gran, mode=rt.GIVEN)
    check(rt, 33, 784, gran=gran, pow2=True)


@pytest.mark.parametrize("gran", [(1, 0), (1, 128), (0, 0)])
def test_many_rows(rt, gran):
    mode = rt.GIVEN if gran == (0, 0) else rt.DYNAMIC
    for rows, cols in ((20000, 32), (9001, 144), (3000, 1040)):
        check(rt, rows, cols, gran=gran, mode=mode)


@pytest.mark.parametrize("live", [-5, 0, 1, 20, 36, 37, 2 ** 31 - 1])
def test_live_rows(rt, live):
    for cols in (64, 1040):
        check(rt, 37, cols, live=live)
        check(rt, 37, cols, gran=(1, 128), live=live)
    if live > 0:
        check(rt, 37, 1040, gran=(0, 0), mode=rt.GIVEN, live=live)


@pytest.mark.parametrize("gran", [(1, 0), (1, 64)])
def test_values(rt, gran):
    """Zeros, gates far out on both sides (their activation's error stays that of the formula), tiny values."""
    def extra(x):
        x[0] = 0.0
        x[1] *= 2.0 ** -60
        x[2, :512] = -60.0
        x[3, :512] = 80.0
        x[4, :512:2] = -1000.0
        x[5, :512] = 1e30
    # (the reference's products of far gates are below every code: any small value rounds alike)
    for act in (0, 1):
        check(rt, 7, 512, dtype=torch.float32, act=act, gran=gran, extra=extra)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_not_finite(rt, dtype):
    """A NaN or an infinity makes its own group's scales NaN and its codes 0x7F, in the output and the checkpoint."""
    for gran, cols in (((1, 0), 256), ((1, 0), 1040), ((1, 128), 256)):
        x = torch.ones(4, 2 * cols, dtype=dtype).cuda()
        x[1, 130] = math.nan
        x[2, cols + 3] = math.inf
        q, ks = torch.zeros(4, cols, dtype=torch.uint8).cuda(), torch.zeros(4, 2, -(-cols // 128)).cuda()
        kept, s = torch.zeros(4, 2 * cols, dtype=torch.uint8).cuda(), torch.zeros(rt.scale_shape((4, cols), gran)).cuda()
        rt.fp8_gated_quantize(x, gran, rt.E4M3, rt.DYNAMIC, EPS, False, s, q, kept=kept, kept_scale=ks)
        bad = torch.zeros(s.shape, dtype=torch.bool)
        bad[1, 130 // 128 if gran[1] else 0] = bad[2, 0] = True
        assert torch.equal(s.isnan().cpu(), bad)
        assert torch.equal((q == 0x7F).cpu(), lr.spread(bad, gran[1], cols))
        kbad = torch.zeros(ks.shape, dtype=torch.bool)
        kbad[1, 0, 1] = kbad[2, 1, 0] = True
        assert torch.equal(ks.isnan().cpu(), kbad)
        both = torch.cat([lr.spread(kbad[:, 0], 128, cols), lr.spread(kbad[:, 1], 128, cols)], 1)
        assert torch.equal((kept == 0x7F).cpu(), both)


def check_grad(rt, rows, cols, dtype=torch.bfloat16, act=0, kf=0, pad=0, with_z=True, live=None, seed=0):
    g = torch.Generator().manual_seed(seed + rows * 17 + cols)
    n = -(-cols // 128)
    kept = torch.randint(0, 256, (rows, 2 * cols + pad), generator=g).to(torch.uint8)
    bad = lr.decode(kept, kf).isnan() | lr.decode(kept, kf).isinf()
    kept = torch.where(bad, torch.tensor(0x11, dtype=torch.uint8), kept)
    ks = torch.rand(rows, 2, n, generator=g) * (12.0 / lr.FMAX[kf])
    dz = wide(rows, cols, pad, dtype, g)
    dx = torch.full((rows, 2 * cols + pad), 7.0, dtype=dtype).cuda()
    z = torch.full((rows, cols + pad), 7.0, dtype=dtype).cuda() if with_z else None
    count = None if live is None else torch.tensor([live], dtype=torch.int32).cuda()
    rt.fp8_gated_backward(dz, kept.cuda()[:, :2 * cols], ks.cuda(), dx[:, :2 * cols], act=act,
                          z=None if z is None else z[:, :cols], kept_fmt=kf, live=count)
    L = rows if live is None else max(0, min(rows, live))
    assert bool((dx[:, 2 * cols:] == 7).all()) and bool((dx[L:] == 7).all())
    assert z is None or (bool((z[:, cols:] == 7).all()) and bool((z[L:] == 7).all()))
    half = [(lr.decode(kept[:, h * cols:(h + 1) * cols].contiguous(), kf).float() * lr.spread(ks[:, h], 128, cols)).double()
            for h in range(2)]
    f, df, v, dv = ref.act(half[0], act)
    d, rel = dz.cpu().double(), ref.gated_bound(v) + 8 * U
    out = ref.HALF[dtype]
    # The hardware's reciprocal returns 0 for a result below the smallest normal number: where e^-v passes
    # 2^126, c = 1 / (1 + e^-v) is off by its whole value, at most 2^-126, act(g) = g c by at most |g| 2^-126 and the slope by
    # (1 + |g| dv) 2^-126; `tiny` is the same for the outputs' own subnormal numbers.
    tiny, low = 2.0 ** -130, 2.0 ** -126 * half[0].abs()
    for got, want, terms, lost in (
            (dx[:, :cols], d * half[1] * df, (d * half[1]).abs() * (1 + f.abs() * dv), (d * half[1]).abs() * (2.0 ** -126 + low * dv)),
            (dx[:, cols:2 * cols], d * f, (d * f).abs(), d.abs() * low),
            (None if z is None else z[:, :cols], f * half[1], (f * half[1]).abs(), half[1].abs() * low)):
        if got is not None:
            err = (got.cpu().double() - want).abs()
            assert bool((err <= rel * terms + out * want.abs() + tiny + lost)[:L].all())


@pytest.mark.parametrize("cols", [16, 64, 144, 528, 2048, 29568])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient(rt, cols, act, dtype):
    check_grad(rt, 5, cols, dtype, act, kf=0, pad=16)
    check_grad(rt, 3, cols, dtype, act, kf=1, with_z=False)


def test_gradient_many_rows(rt):
    check_grad(rt, 20000, 32)
    check_grad(rt, 1000, 1040)
    for live in (-1, 0, 1, 17, 40, 2 ** 31 - 1):
        check_grad(rt, 40, 272, live=live)


@pytest.mark.parametrize("act", [0, 1])
def test_gradient_against_differences(rt, act):
    """Central differences of the 64-bit activation at the checkpoint's values (step 1e-4)."""
    x = torch.randn(4, 128, generator=torch.Generator().manual_seed(1)).cuda()
    q, s = torch.empty(4, 64, dtype=torch.uint8, device="cuda"), torch.empty(4, 1, device="cuda")
    kept, ks = torch.empty(4, 128, dtype=torch.uint8, device="cuda"), torch.empty(4, 2, 1, device="cuda")
    rt.fp8_gated_quantize(x, (1, 0), rt.E4M3, rt.DYNAMIC, EPS, False, s, q, act=act, kept=kept, kept_scale=ks)
    dx = torch.empty_like(x)
    rt.fp8_gated_backward(torch.ones(4, 64, device="cuda"), kept, ks, dx, act=act)
    back = (lr.decode(kept.cpu(), 0).view(4, 2, 64) * ks.cpu().double()).view(4, 2, 64)
    assert float((back.view(4, 128) - x.cpu().double()).norm() / x.cpu().double().norm()) < 2.0 ** -4
    gate, up, h = back[:, 0], back[:, 1], 1e-4
    dg = (ref.act(gate + h, act)[0] - ref.act(gate - h, act)[0]) / (2 * h) * up
    assert bool(((dx[:, :64].cpu().double() - dg).abs() < 1e-5).all())
    assert bool(((dx[:, 64:].cpu().double() - ref.act(gate, act)[0]).abs() < 1e-5).all())


@pytest.mark.parametrize("act", [0, 1])
def test_gradient_of_far_gates(rt, act):
    """Gates where the sigmoid has reached 0 or 1: the slope is 0 or 1, nothing overflows."""
    kept = torch.zeros(2, 64, dtype=torch.uint8)
    kept[0, :32] = 0x7E  # 448
    kept[1, :32] = 0xFE  # -448
    kept[:, 32:] = 0x38  # 1
    ks = torch.tensor([[[1e30], [1.0]], [[1e30], [1.0]]]).cuda()
    dx = torch.empty(2, 64, device="cuda")
    rt.fp8_gated_backward(torch.ones(2, 32, device="cuda"), kept.cuda(), ks, dx, act=act)
    assert bool((dx[0, :32] == 1).all()) and bool((dx[1] == 0).all()) and bool(dx.isfinite().all())


def test_graph(rt):
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        rows, cols = 50, 1040
        x, dz = torch.empty(rows, 2 * cols, device="cuda").bfloat16(), torch.empty(rows, cols, device="cuda").bfloat16()
        count = torch.tensor([rows], dtype=torch.int32, device="cuda")

        def buffers():
            return dict(q=torch.zeros(rows, cols, dtype=torch.uint8, device="cuda"), scale=torch.zeros(1, 1, device="cuda") + 0.01,
                        kept=torch.zeros(rows, 2 * cols, dtype=torch.uint8, device="cuda"), amax_out=torch.zeros(1, 1, device="cuda"),
                        kept_scale=torch.zeros(rows, 2, 9, device="cuda")), torch.zeros_like(x)

        def call(b, dx):
            rt.fp8_gated_quantize(x, (0, 0), rt.E4M3, rt.GIVEN, EPS, False, live=count, **b)
            rt.fp8_gated_backward(dz, b["kept"], b["kept_scale"], dx, live=count)
        b, dx = buffers()
        call(b, dx)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(b, dx)
        for live in (50, 0, 31, 50):
            x.normal_()
            dz.normal_()
            count.fill_(live)
            b2, dx2 = buffers()
            for n, t in b2.items():
                b[n].copy_(t)
            dx.zero_()
            g.replay()
            s.synchronize()
            call(b2, dx2)
            assert all(torch.equal(b[n], b2[n]) for n in b) and torch.equal(dx, dx2)
