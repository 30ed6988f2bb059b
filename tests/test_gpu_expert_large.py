"""The operators of the gated half of a decoder layer on matrices whose offsets pass 32 bits: the first and last rows."""
import pytest
import torch

import expert_ref as ref
import layer_ref as lr

pytestmark = pytest.mark.gpu

U = ref.U


@pytest.fixture(scope="module")
def rt():
    import dynamic_scaling_scaled_amd as rt

    rt.lib()
    yield rt
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows", [3, 40, 200])
def test_weights(rt, rows):
    """72 x 4096 x 16384 codes (4.8 GB): the last expert's products on each kernel."""
    E, N, K = 72, 4096, 16384
    g = torch.Generator(device="cuda").manual_seed(rows)
    b = torch.randint(0, 120, (E * N, K), dtype=torch.uint8, device="cuda", generator=g)
    image = rt.fp8_pack_weights16(b)
    counts = [rows] + [0] * (E - 2) + [rows] if rows > 3 else [rows] * E
    S = sum(counts)
    a = torch.randint(0, 120, (S, K), dtype=torch.uint8, device="cuda", generator=g)
    sa, sb = torch.full((S, 1), 2.0 ** -10).cuda(), torch.ones(E, N).cuda()
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    y = torch.empty(S, N, device="cuda")
    rt.fp8_expert_gemm(a, 0, (1, 0), sa, image, 0, (1, 0), sb, off, y)
    for e in (0, E - 1):
        lo, hi, n0 = int(off[e]), int(off[e + 1]), N - 32
        w = b[e * N + n0:(e + 1) * N].cpu()
        want, tol, _ = ref.experts(a[lo:lo + 3].cpu(), 0, sa[lo:lo + 3].cpu(), None, 1, w.view(1, 32, K), sb[e:e + 1, n0:].cpu(),
                                   [0, 3], 3)
        assert hi - lo == rows and bool(((y[lo:lo + 3, n0:].cpu().double() - want).abs() <= tol + ref.HALF[torch.float32] * want).all())


def test_activation_and_gradient(rt):
    rows, cols = 140000, 16384  # x 9.2 GB, checkpoint 4.6 GB
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, 2 * cols, dtype=torch.bfloat16, device="cuda", generator=g)
    q = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    for gran in ((1, 0), (1, 128)):
        n = rt.scale_shape((rows, cols), gran)
        s, kept = torch.empty(n, device="cuda"), torch.empty(rows, 2 * cols, dtype=torch.uint8, device="cuda")
        ks = torch.empty(rows, 2, cols // 128, device="cuda")
        rt.fp8_gated_quantize(x, gran, 0, rt.DYNAMIC, 1e-12, False, s, q, kept=kept, kept_scale=ks)
        for at in (slice(0, 2), slice(rows - 2, rows)):
            xc = x[at].cpu()
            f, _, v, _ = ref.act(xc[:, :cols].double(), 0)
            z = f * xc[:, cols:].double()
            sc = lr.spread(s[at].cpu().double(), gran[1], cols)
            assert lr.codes_off(q[at].cpu(), z / sc, 0, ref.gated_bound(v) + 8 * U) == 0
            for h in (0, 1):
                codes, scales = ref.kept(xc[:, h * cols:(h + 1) * cols], 0, 1e-12)
                assert torch.equal(kept[at, h * cols:(h + 1) * cols].cpu(), codes) and torch.equal(ks[at, h].cpu(), scales)
    dz, dx = x[:, :cols], torch.empty_like(x)
    rt.fp8_gated_backward(dz, kept, ks, dx)
    for at in (slice(0, 2), slice(rows - 2, rows)):
        gate, up = [(lr.decode(kept[at, h * cols:(h + 1) * cols].cpu().contiguous(), 0).float()
                     * lr.spread(ks[at, h].cpu(), 128, cols)).double() for h in (0, 1)]
        f, df, v, dv = ref.act(gate, 0)
        d, rel = dz[at].cpu().double(), ref.gated_bound(v) + 8 * U
        for got, want, terms in ((dx[at, :cols], d * up * df, (d * up).abs() * (1 + f.abs() * dv)), (dx[at, cols:], d * f, (d * f).abs())):
            err = (got.cpu().double() - want).abs()
            assert bool((err <= rel * terms + ref.HALF[torch.bfloat16] * want.abs() + 2.0 ** -126).all())


def test_sum_and_gradient(rt):
    rows, cols, k = 300000, 8192, 3  # 4.9 GB
    tokens = rows // k
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(rows, cols, dtype=torch.bfloat16, device="cuda", generator=g)
    slots = torch.arange(rows, dtype=torch.int32, device="cuda").flip(0).view(tokens, k)
    w = torch.rand(tokens, k, device="cuda", generator=g)
    y = torch.empty(tokens, cols, dtype=torch.bfloat16, device="cuda")
    rt.fp8_expert_combine(x, slots, w, y)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    rt.fp8_expert_combine_backward(y, x, slots, w, dx, dw)
    for t in (0, 1, tokens - 1):
        at = slots[t].long()
        r, c, d = x[at].cpu().double(), w[t].cpu().double()[:, None], y[t].cpu()
        terms = c * r
        assert bool(((d.double() - terms.sum(0)).abs() <= (k + 2) * U * terms.abs().sum(0) + 2.0 ** -8 * terms.sum(0).abs()).all())
        dots = d.double() * r
        assert bool(((dw[t].cpu().double() - dots.sum(1)).abs() <= (cols / 128 + 40) * U * dots.abs().sum(1)).all())
        assert torch.equal(dx[at].cpu(), (w[t].cpu()[:, None] * d.float()).bfloat16())
