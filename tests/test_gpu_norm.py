"""fp8_rmsnorm_quantize and fp8_rmsnorm_backward against 64-bit references.

Bounds (u = 2^-24): a thread adds at most 32 squares in sequence, then 6 shuffles and 16 waves, so the
sum of squares is within 56 u and rstd, at half of that plus mean, root and quotient, within 32 u.  h adds 1 u,
the two multiplications of y 2 u, the scale 2 u: every y / s is within 48 u + 16 u of its exact value."""
import numpy as np
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu

U = ref.U
RSTD, REL = 32 * U, 64 * U


@pytest.fixture(scope="module")
def rt():
    import dynamic_scaling_scaled_amd as rt

    rt.lib()
    return rt


def wide(rows, cols, pad, dtype, g, scale=1.0):
    return (torch.randn(rows, cols + pad, generator=g) * scale).to(dtype).cuda()[:, :cols]


def check_norm(rt, rows, cols, dtype=torch.bfloat16, residual=True, gran=(1, 0), fmt=0, pow2=False, pad=0, wt=None,
               mode=0, alias=None, seed=0, extra=None):
    g = torch.Generator().manual_seed(seed + rows * 131 + cols)
    x = wide(rows, cols, pad, dtype, g)
    x[:, ::7] *= 9
    res = wide(rows, cols, 2 * pad, dtype, g, 2.0) if residual else None
    w = (1 + 0.3 * torch.randn(cols, generator=g)).to(wt or dtype).cuda()
    if extra:
        extra(x, res, w)
    xc, rc = x.cpu().clone(), None if res is None else res.cpu().clone()
    ns = rt.scale_shape((rows, cols), gran)
    scale = torch.full(ns, -1.0).cuda() if mode == rt.DYNAMIC else torch.full(ns, 7.0 / ref.FMAX[fmt]).cuda()
    inv = torch.full(ns, -1.0).cuda() if mode == rt.DYNAMIC else None
    amax = torch.full(ns, -1.0).cuda()
    q = torch.full((rows, cols + pad), 0xAA, dtype=torch.uint8).cuda()
    h = x if alias == "x" else res if alias == "res" else torch.empty(rows, cols, dtype=dtype).cuda()
    rstd = torch.empty(rows).cuda()
    rt.fp8_rmsnorm_quantize(x, w, 1e-6, gran, fmt, mode, 1e-12, pow2, scale, q[:, :cols], residual=res, h=h,
                            rstd=rstd, inv_scale=inv, amax_out=amax)
    torch.cuda.synchronize()
    assert bool((q[:, cols:] == 0xAA).all())
    want_h = (xc.float() + (rc.float() if residual else 0)).to(dtype)
    assert torch.equal(h.cpu(), want_h)
    h64, r64, y = ref.norm(xc, rc, w.cpu(), 1e-6)
    assert bool(((rstd.cpu().double() - r64).abs() <= RSTD * r64).all())
    if gran == (0, 0):
        am = y.abs().max().view(1, 1)
    else:
        am = ref.group_amax(y, gran[1])
    assert bool(((amax.cpu().double() - am).abs() <= REL * am).all())
    if mode == rt.DYNAMIC:
        a = amax.cpu()  # the scale rule on the observed amax, bit for bit
        s, r = ref.scale_of(a, fmt, 1e-12, pow2)
        assert torch.equal(scale.cpu(), s) and torch.equal(inv.cpu(), r)
    sc = scale.cpu().double()
    sc = sc if gran == (0, 0) else ref.spread(sc, gran[1], cols)
    assert ref.codes_off(q[:, :cols].cpu().contiguous(), y / sc, fmt, REL) == 0


@pytest.mark.parametrize("cols", [16, 64, 528, 1024, 4096, 4112, 8192, 16384, 16400, 32768])
def test_widths(rt, cols):
    check_norm(rt, 5, cols, pad=16)
    check_norm(rt, 3, cols, gran=(1, 128))


@pytest.mark.parametrize("gran", [(1, 0), (1, 16), (1, 32), (1, 64), (1, 128), (1, 256), (1, 512), (0, 0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", [0, 1])
def test_granularities(rt, gran, dtype, fmt):
    mode = rt.GIVEN if gran == (0, 0) else rt.DYNAMIC
    check_norm(rt, 37, 1040, dtype=dtype, gran=gran, fmt=fmt, mode=mode, pad=48)
    check_norm(rt, 1, 2048, dtype=dtype, gran=gran, fmt=fmt, mode=mode, residual=False)


@pytest.mark.parametrize("gran", [(1, 0), (1, 32), (1, 128)])
def test_given_and_pow2(rt, gran):
    check_norm(rt, 33, 784, gran=gran, mode=rt.GIVEN)
    check_norm(rt, 33, 784, gran=gran, pow2=True)


def test_many_rows_and_types(rt):
    check_norm(rt, 9001, 64, gran=(0, 0), mode=rt.GIVEN)     # more rows than the grid's cap
    check_norm(rt, 9001, 144, gran=(1, 0))
    check_norm(rt, 700, 2064, gran=(1, 128))                  # several rows per workgroup
    check_norm(rt, 40, 512, dtype=torch.bfloat16, wt=torch.float32)
    check_norm(rt, 40, 512, dtype=torch.float32, wt=torch.bfloat16)


@pytest.mark.parametrize("alias", ["x", "res"])
@pytest.mark.parametrize("cols", [64, 8192, 16400])
def test_in_place(rt, alias, cols):
    check_norm(rt, 19, cols, alias=alias)


def test_zero_and_huge_rows(rt):
    def extra(x, res, w):
        x[1] = 0
        res[1] = 0
        x[2] = 1e-20
        res[2] = 0
    check_norm(rt, 6, 256, dtype=torch.float32, extra=extra)
    check_norm(rt, 6, 256, dtype=torch.float32, extra=extra, gran=(1, 32))


def test_non_finite_rows_stay_in_their_row(rt):
    rows, cols = 8, 640
    g = torch.Generator().manual_seed(3)
    x = torch.randn(rows, cols, generator=g).bfloat16().cuda()
    w = torch.ones(cols).bfloat16().cuda()

    def run(x):
        q = torch.zeros(rows, cols, dtype=torch.uint8).cuda()
        s = torch.zeros(rows, 1).cuda()
        rt.fp8_rmsnorm_quantize(x, w, 1e-6, (1, 0), rt.E4M3, rt.DYNAMIC, 1e-12, False, s, q)
        return q.cpu(), s.cpu()

    q0, s0 = run(x)
    bad = x.clone()
    bad[2, 77] = float("nan")
    bad[5, 600] = float("inf")
    q1, s1 = run(bad)
    ok = [i for i in range(rows) if i not in (2, 5)]
    assert torch.equal(q1[ok], q0[ok]) and torch.equal(s1[ok], s0[ok])
    assert bool(s1[[2, 5]].isnan().all()) and bool((q1[[2, 5]] == 0x7F).all())


def grad_inputs(rows, cols, dt, ht, pad, residual, seed=0):
    g = torch.Generator().manual_seed(seed + rows * 7 + cols)
    dy, h = wide(rows, cols, pad, dt, g, 0.1), wide(rows, cols, 2 * pad, ht, g, 3.0)
    w = (1 + 0.3 * torch.randn(cols, generator=g)).to(dt).cuda()
    res = wide(rows, cols, pad, dt, g, 0.1) if residual else None
    rstd = (1.0 / (h.float().square().mean(1) + 1e-6).sqrt())
    return dy, h, w, rstd, res


@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 8192), (3, 528), (65, 1024), (257, 4096), (600, 144), (1025, 2064),
                                       (9, 16400), (7, 32768)])
@pytest.mark.parametrize("dt,ht", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                   (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
def test_gradient(rt, rows, cols, dt, ht):
    """The row's dot product is within 60 u of its terms' size, each dx adds a few roundings: 80 u.  dweight adds
    at most rows / 256 + 64 terms in sequence."""
    residual = (rows + cols) % 2 == 1 or rows == 65
    dy, h, w, rstd, res = grad_inputs(rows, cols, dt, ht, 16, residual)
    dx = torch.full((rows, cols), 7.0, dtype=dt).cuda()
    dw = torch.full((cols,), 7.0).cuda()
    rt.fp8_rmsnorm_backward(dy, h, w, rstd, dx, dw, dresidual=res)
    want, wdw, terms, wterms = ref.norm_grad(dy.cpu(), h.cpu(), w.cpu(), rstd.cpu(), None if res is None else res.cpu())
    tol = 80 * U * terms + (2.0 ** -8 * want.abs() if dt == torch.bfloat16 else 0)
    assert bool(((dx.cpu().double() - want).abs() <= tol).all())
    assert bool(((dw.cpu().double() - wdw).abs() <= (rows / 256 + 72) * U * wterms).all())
    # without dweight, and in place of dy
    d2 = dy.clone()
    rt.fp8_rmsnorm_backward(d2, h, w, rstd, d2, None, dresidual=res)
    assert torch.equal(d2, dx)


def test_gradient_repeats(rt):
    dy, h, w, rstd, res = grad_inputs(1500, 4096, torch.bfloat16, torch.bfloat16, 0, True)
    outs = []
    for _ in range(3):
        dx, dw = torch.empty_like(dy), torch.empty(4096).cuda()
        rt.fp8_rmsnorm_backward(dy, h, w, rstd, dx, dw, dresidual=res)
        outs.append((dx.cpu(), dw.cpu()))
    assert all(torch.equal(a, outs[0][0]) and torch.equal(b, outs[0][1]) for a, b in outs)


def test_gradient_against_differences(rt):
    """The kernel's gradient against central differences of the forward formula in 64 bits (step 1e-4: the
    difference's own error is of order 1e-8 of the third derivative, 1e-6 here, beside binary32 rounding)."""
    rows, cols = 4, 32
    dy, h, w, _, _ = grad_inputs(rows, cols, torch.float32, torch.float32, 0, False)
    h64, w64, dy64 = h.cpu().double(), w.cpu().double(), dy.cpu().double()

    def loss(h, w):
        return (ref.norm(h, None, w, 1e-6)[2] * dy64).sum()

    num, numw, d = torch.zeros(rows, cols, dtype=torch.float64), torch.zeros(cols, dtype=torch.float64), 1e-4
    for i in range(rows):
        for j in range(cols):
            e = torch.zeros_like(h64)
            e[i, j] = d
            num[i, j] = (loss(h64 + e, w64) - loss(h64 - e, w64)) / (2 * d)
    for j in range(cols):
        e = torch.zeros_like(w64)
        e[j] = d
        numw[j] = (loss(h64, w64 + e) - loss(h64, w64 - e)) / (2 * d)
    # the forward's own rstd
    q, s, rstd = torch.empty(rows, cols, dtype=torch.uint8).cuda(), torch.empty(rows, 1).cuda(), torch.empty(rows).cuda()
    rt.fp8_rmsnorm_quantize(h, w, 1e-6, (1, 0), rt.E4M3, rt.DYNAMIC, 1e-12, False, s, q, rstd=rstd)
    dx, dw = torch.empty_like(dy), torch.empty(cols).cuda()
    rt.fp8_rmsnorm_backward(dy, h, w, rstd, dx, dw)
    assert float((dx.cpu().double() - num).abs().max()) <= 2e-6 * float(num.abs().max()) + 1e-7
    assert float((dw.cpu().double() - numw).abs().max()) <= 2e-6 * float(numw.abs().max()) + 1e-7


def test_other_stream_and_graph(rt):
    """On a stream of its own, captured after a warm-up, replayed on new inputs: every replay equals the
    eager call."""
    rows, cols = 300, 1024
    g = torch.Generator().manual_seed(1)
    st = torch.cuda.Stream()
    x, res = torch.empty(rows, cols).bfloat16().cuda(), torch.randn(rows, cols, generator=g).bfloat16().cuda()
    w = torch.ones(cols).bfloat16().cuda()
    dy, dx, dw = torch.randn(rows, cols, generator=g).bfloat16().cuda(), torch.empty(rows, cols).bfloat16().cuda(), torch.empty(cols).cuda()
    q, h = torch.empty(rows, cols, dtype=torch.uint8).cuda(), torch.empty(rows, cols).bfloat16().cuda()
    s, rstd, am = torch.full((1, 1), 0.02).cuda(), torch.empty(rows).cuda(), torch.empty(1, 1).cuda()

    def step():
        rt.fp8_rmsnorm_quantize(x, w, 1e-6, (0, 0), rt.E4M3, rt.GIVEN, 1e-12, False, s, q, residual=res, h=h,
                                rstd=rstd, amax_out=am)
        rt.fp8_rmsnorm_backward(dy, h, w, rstd, dx, dw)

    x.copy_(torch.randn(rows, cols, generator=g))
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step()
    for _ in range(4):
        x.copy_(torch.randn(rows, cols, generator=g))
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            graph.replay()
        st.synchronize()
        got = [t.clone() for t in (q, h, rstd, am, dx, dw)]
        with torch.cuda.stream(st):
            step()
        st.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (q, h, rstd, am, dx, dw)))
