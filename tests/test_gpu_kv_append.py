"""fp8_kv_append against a page-by-page reference whose every step is one
binary32 operation: codes and scales are compared bit for bit, over the whole
cache, so that nothing else in it may change."""
import math

import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rt():
    import dynamic_scaling_scaled_amd as rt

    rt.lib()
    return rt


def cache(bt, heads, dim, fmt, pow2, seed):
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, 256, (bt.pages, heads, bt.page, dim), generator=g, dtype=torch.uint8)
    s = torch.exp(torch.randn(bt.pages, heads, generator=g)) * (2.0 / ref.FMAX[fmt])
    return c, ref.pow2_up(s) if pow2 else s


def run(rt, bt, heads, dim, fmt=0, dtype=torch.bfloat16, pow2=False, layout="fused", edit=None, seed=5):
    g = torch.Generator().manual_seed(seed)
    kc, ks = cache(bt, heads, dim, fmt, pow2, seed + 1)
    vc, vs = cache(bt, heads, dim, fmt, pow2, seed + 2)
    if layout == "fused":      # rows of [q | k | v]
        qkv = torch.randn(max(1, bt.tokens), 3 * heads, dim, generator=g).to(dtype)
        k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    else:                      # heads outermost
        kv = torch.randn(2, heads, max(1, bt.tokens), dim, generator=g).to(dtype)
        k, v = kv[0].transpose(0, 1), kv[1].transpose(0, 1)
    k[::3] *= 4
    if edit:
        edit(k, v, ks, vs)
    d = [t.cuda() for t in (kc, vc, ks, vs)]
    # .cuda() keeps the strides of a dense tensor only; give the views their base
    if layout == "fused":
        base = qkv.cuda()
        kd, vd = base[:, heads:2 * heads], base[:, 2 * heads:]
    else:
        base = kv.cuda()
        kd, vd = base[0].transpose(0, 1), base[1].transpose(0, 1)
    plan = [t.cuda() for t in (bt.table, bt.start, bt.kv_len)]
    for _ in range(2):  # the second call changes nothing
        rt.fp8_kv_append(kd, vd, *d, fmt, *plan, bt.max_new, 1e-12, pow2)
    ref.append(bt, k, kc, ks, fmt, 1e-12, pow2)
    ref.append(bt, v, vc, vs, fmt, 1e-12, pow2)
    for got, want in zip(d, (kc, vc, ks, vs)):
        got = got.cpu()
        if got.dtype == torch.float32:
            assert torch.equal(got.isnan(), want.isnan())
            assert torch.equal(got.nan_to_num(0), want.nan_to_num(0))
        else:
            assert torch.equal(got, want)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("fmt", [0, 1])
def test_ragged(rt, page, dim, fmt):
    new = [1, 0, 5, page, 2 * page + 3, 1, 1, 17]
    before = [0, 9, page - 2, 0, page // 2, page, page - 1, 3 * page + 7]
    run(rt, ref.Batch(new, before, page), 3, dim, fmt)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("layout", ["fused", "heads"])
def test_types_and_layouts(rt, dtype, pow2, layout):
    run(rt, ref.Batch([3, 40, 1], [30, 5, 63], 32), 5, 128, 0, dtype, pow2, layout)


def test_one_token_each(rt):
    n = 70
    run(rt, ref.Batch([1] * n, [13 * i % 97 for i in range(n)], 16), 8, 128)


def test_long_prompt(rt):
    run(rt, ref.Batch([1500], [7], 64), 2, 128)


def test_lengths_below_the_new_tokens(rt):
    """kv_len below the number of new tokens: the first ones have no position."""
    run(rt, ref.Batch([6, 4, 3], [-2, -4, -9], 16), 2, 64)


def test_missing_pages_and_bad_entries(rt):
    bt = ref.Batch([40, 40], [0, 10], 16)
    bt.table[0, 1] = -1
    bt.table[1, 2] = bt.pages  # one past the last
    run(rt, bt, 2, 64)
    bt = ref.Batch([40], [0], 16, extra_width=0)
    bt.kv_len[0] = 10 ** 6     # beyond the table: nothing there to write
    bt.before, bt.lens = [10 ** 6 - 40], [0]
    run(rt, bt, 2, 64)


def test_starts_out_of_order(rt):
    """seq_start is not trusted: starts that fall or pass the tokens give empty sequences."""
    bt = ref.Batch([5, 5], [0, 0], 16)
    k = torch.randn(10, 2, 64).bfloat16().cuda()
    c = [torch.zeros(bt.pages, 2, 16, 64, dtype=torch.uint8).cuda() for _ in range(2)]
    s = [torch.zeros(bt.pages, 2).cuda() for _ in range(2)]
    start = torch.tensor([8, 3, 10 ** 9], dtype=torch.int32).cuda()
    rt.fp8_kv_append(k, k, *c, *s, 0, bt.table.cuda(), start, bt.kv_len.cuda(), 5)
    torch.cuda.synchronize()
    assert int((s[0] != 0).sum()) == 2 and int((s[1] != 0).sum()) == 2  # sequence 1's page, both heads


def test_non_finite(rt):
    def edit(k, v, ks, vs):
        k[2, 0, 5] = math.nan
        v[30, 1, 9] = math.inf
        ks[3, 1] = math.nan
    run(rt, ref.Batch([20, 25, 1], [9, 0, 20], 16), 2, 64, edit=edit)


def test_zeros_and_extremes(rt):
    def edit(k, v, ks, vs):
        k[:5] = 0
        v[3] = 1e30
        v[4] = 1e-30
    run(rt, ref.Batch([5, 9], [12, 0], 16), 2, 64, dtype=torch.float32, edit=edit)


def test_tokens_past_the_bound_are_dropped(rt):
    """max_new is a bound: what passes it is not written."""
    bt = ref.Batch([12], [0], 16)
    k = torch.randn(12, 1, 64).bfloat16()
    c = [torch.zeros(bt.pages, 1, 16, 64, dtype=torch.uint8).cuda() for _ in range(2)]
    s = [torch.zeros(bt.pages, 1).cuda() for _ in range(2)]
    rt.fp8_kv_append(k.cuda(), k.cuda(), *c, *s, 0, bt.table.cuda(), bt.start.cuda(), bt.kv_len.cuda(), 7)
    pg = int(bt.table[0, 0])
    got = c[0][pg, 0].cpu()
    sc, r = ref.scale_of(k[:7].float().abs().max().view(1), 0, 1e-12, False)
    assert torch.equal(got[:7], ref.cast(k[:7, 0].float() * r, 0)) and int(got[7:].sum()) == 0
    assert float(s[0][pg, 0]) == float(sc)


def test_offsets_past_32_bits(rt):
    """A cache of more than 2^32 bytes: the last pages are written, and read by attention."""
    heads, page, dim = 8, 128, 128
    pages = (1 << 32) // (heads * page * dim) + 9
    kc = torch.zeros(pages, heads, page, dim, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    ks, vs = torch.zeros(pages, heads, device="cuda"), torch.zeros(pages, heads, device="cuda")
    g = torch.Generator().manual_seed(2)
    k = torch.randn(200, heads, dim, generator=g).bfloat16()
    table = torch.tensor([[pages - 1, pages - 5]], dtype=torch.int32).cuda()
    start, kv = torch.tensor([0, 200], dtype=torch.int32).cuda(), torch.tensor([200], dtype=torch.int32).cuda()
    rt.fp8_kv_append(k.cuda(), k.cuda(), kc, vc, ks, vs, 0, table, start, kv, 200)
    sc, r = ref.scale_of(k[:128].float().abs().amax((0, 2)), 0, 1e-12, False)
    want = ref.cast(k[:128].float().transpose(0, 1) * r[:, None, None], 0)
    assert torch.equal(kc[pages - 1].cpu(), want) and torch.equal(vc[pages - 1].cpu(), want)
    assert int(kc[: pages - 5].any()) == 0
    q = torch.randn(1, heads, dim, generator=g).bfloat16()
    y, lse = torch.empty(1, heads, dim, dtype=torch.bfloat16).cuda(), torch.empty(1, heads).cuda()
    bt = ref.Batch([1], [199], page)
    bt.table, bt.width = table.cpu(), 2
    small = torch.arange(pages - 5, pages)
    rt.fp8_paged_attention(q.cuda(), kc, vc, ks, vs, 0, table, torch.tensor([0, 1], dtype=torch.int32).cuda(), kv, 1,
                           200, dim ** -0.5, y, lse=lse)
    bt.table = bt.table - (pages - 5)
    wy, wl, tol, ltol = ref.attend(bt, q, kc[small.cuda()].cpu(), vc[small.cuda()].cpu(), ks[small.cuda()].cpu(),
                                   vs[small.cuda()].cpu(), 0, dim ** -0.5, True, 0)
    assert bool(((y.cpu().double() - wy).abs() <= tol).all())
