"""fp8_paged_attention where one key outweighs all others: the others together still make the output, so each
of their small weights has to keep its bits.

Bound: a weight (times its page's v scale) is rounded to 11 bits, or, below 2^-22 of the row's largest, to a
multiple of 2^-32 of it: half of that is an absolute error for each key.  Scores and sums are binary32 (as in
layer_ref.attend), the output bf16."""
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu

U = ref.U
STEP = 2.0 ** -32  # spacing of the smallest weights, relative to the row's largest


@pytest.fixture(scope="module")
def rt():
    import dynamic_scaling_scaled_amd as rt

    rt.lib()
    return rt


def reference(q, k, v, s, sm):
    """(y, lse, bound of y, bound of lse) of rows q [r x d] over keys k [n x d], codes v [n x d] and their scales s [n], in double."""
    n, d = k.shape
    z = sm * (q @ k.T)
    dz = ((d + 6) * U * abs(sm) * (q.abs() @ k.abs().T).amax(1) + 4 * U * z.abs().amax(1))[:, None]
    m = z.amax(1, keepdim=True)
    w = torch.exp(z - m)
    l = w.sum(1, keepdim=True)
    y = (w * s) @ v / l
    rel = 2 * dz + 4 * U * ((z - m).abs().amax(1, keepdim=True) + 2) + 2.0 ** -11 + (n + 8) * U
    mass = (w * s) @ v.abs()
    low = 0.5 * STEP * (w * s).amax(1, keepdim=True) * v.abs().sum(0)
    tol = 2.0 ** -8 * y.abs() + (rel * mass + low) / l
    lse = (m + torch.log(l))[:, 0]
    return y, lse, tol, (dz + 4 * U * ((z - m).abs().amax(1, keepdim=True) + 2) + (n + 8) * U)[:, 0] + 4 * U * lse.abs()


def run(rt, n, dim, page, fmt, seqs, new, at, gap, loud, seed=3):
    """`seqs` sequences over the same n keys: key `at` scores `gap` above the rest, has a value of 0, and its page's v scale is `loud`
    times the others'."""
    g = torch.Generator().manual_seed(seed)
    pages, group = -(-n // page), 4
    k = 0.25 * torch.randn(pages * page, dim, generator=g)
    v = 0.5 + 1.5 * torch.rand(pages * page, dim, generator=g)
    k[:, 0], v[at] = 0, 0
    k[at, 0] = gap
    kc, vc = (ref.cast(t, fmt) for t in (k, v))
    s = torch.ones(pages)
    s[at // page] = loud
    q = 0.2 * torch.randn(seqs * new, group, dim, generator=g)
    q[:, :, 0] = 8
    q = q.bfloat16().cuda()
    order = torch.randperm(pages, generator=g)
    place = torch.argsort(order)  # page order[i] holds the keys of logical page i
    pool = [t.view(pages, 1, page, dim)[place].contiguous().cuda() for t in (kc, vc)]
    scales = [torch.ones(pages, 1).cuda(), s[place].view(pages, 1).contiguous().cuda()]
    table = order.to(torch.int32).cuda().expand(seqs, pages).contiguous()
    start = (torch.arange(seqs + 1) * new).to(torch.int32).cuda()
    kv_len = torch.full((seqs,), n, dtype=torch.int32).cuda()
    y, lse = torch.empty_like(q), torch.empty(q.shape[:2]).cuda()
    rt.fp8_paged_attention(q, *pool, *scales, fmt, table, start, kv_len, new, n, 0.125, y, causal=False, lse=lse)
    kd, vd = (ref.decode(t, fmt)[:n].cuda() for t in (kc, vc))
    sd = s.double().repeat_interleave(page)[:n].cuda()
    rows, got, lse = q.double().view(-1, dim), y.double().view(-1, dim), lse.double().view(-1)
    for i in range(0, len(rows), 1000):
        wy, wl, tol, ltol = reference(rows[i:i + 1000], kd, vd, sd, 0.125)
        off = (got[i:i + 1000] - wy).abs()
        assert bool((off <= tol).all()), "rows %d.., worst relative error %.3g" % (i, float((off / wy.abs()).max()))
        assert bool(((lse[i:i + 1000] - wl).abs() <= ltol).all())


# (sequences, new tokens): single tokens uncut and cut along the keys, prompts' kernel uncut and cut
SHAPES = [(520, 1), (2, 1), (400, 5), (3, 30)]


@pytest.mark.parametrize("seqs,new", SHAPES)
@pytest.mark.parametrize("gap,loud", [(13, 1), (16, 1), (18, 1), (13, 64)])
def test_one_dominant_key(rt, seqs, new, gap, loud):
    run(rt, 8192, 64, 16, 0, seqs, new, 0, gap, loud)


@pytest.mark.parametrize("seqs,new", SHAPES)
@pytest.mark.parametrize("dim,page,fmt", [(128, 64, 0), (128, 128, 1), (64, 32, 1)])
def test_types_and_places(rt, seqs, new, dim, page, fmt):
    run(rt, 5003, dim, page, fmt, seqs, new, 0, 16, 4.0)
    run(rt, 5003, dim, page, fmt, seqs, new, 1700, 16, 1.0)


@pytest.mark.parametrize("seqs,new", [(520, 1), (400, 5)])
def test_long_tail(rt, seqs, new):
    run(rt, 70000, 64, 128, 0, seqs, new, 0, 14, 1.0)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("fmt", [0, 1])
def test_smallest_codes_beside_the_largest(rt, new, dim, fmt):
    """Dimensions whose codes are the smallest subnormal beside others at the largest value: the former keep
    their own relative error."""
    n, page = 200, 16
    g = torch.Generator().manual_seed(8)
    pages = -(-n // page)
    c = torch.full((pages, 1, page, dim), 0x01, dtype=torch.uint8)
    c[..., 1::3] = 0x7E if fmt == 0 else 0x7B
    k = ref.cast(0.25 * torch.randn(pages, 1, page, dim, generator=g), fmt)
    q = torch.randn(new, 2, dim, generator=g).bfloat16().cuda()
    s, table = torch.ones(pages, 1).cuda(), torch.arange(pages, dtype=torch.int32).view(1, -1).cuda()
    start, kv_len = torch.tensor([0, new], dtype=torch.int32).cuda(), torch.tensor([n], dtype=torch.int32).cuda()
    y = torch.empty_like(q)
    rt.fp8_paged_attention(q, k.cuda(), c.cuda(), s, s, fmt, table, start, kv_len, new, n, 0.125, y)
    want = ref.decode(c[0, 0, 0], fmt)  # every key has the same value
    rel = 2.0 ** -8 + 2.0 ** -10 + (n + 64) * U
    assert bool(((y.cpu().double() - want).abs() <= rel * want).all())
