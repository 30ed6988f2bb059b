"""fp8_paged_attention against a 64-bit reference, query by query, with the
bounds that its roundings allow (layer_ref.attend).  What must count for nothing is filled with NaN
codes and scales: slots past a sequence's length, pages nobody owns, hidden positions."""
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


def make(bt, heads, dim, fmt, seed, poison=True):
    g = torch.Generator().manual_seed(seed)
    shape = (bt.pages, heads, bt.page, dim)
    out = []
    for loud in (4.0, 1.0):
        x = torch.randn(shape, generator=g) * (1 + loud * (torch.rand(dim, generator=g) > 0.9))
        s = x.abs().amax((2, 3)) / ref.FMAX[fmt] * (0.25 + torch.rand(bt.pages, heads, generator=g))
        out.append((ref.cast(x / s[:, :, None, None], fmt), s))
    (kc, ks), (vc, vs) = out
    if poison:
        owned = torch.zeros(bt.pages, bt.page, dtype=torch.bool)
        for b, n in enumerate(bt.lens):
            for j in range(max(0, min(n, bt.width * bt.page))):
                pg = int(bt.table[b, j // bt.page])
                if 0 <= pg < bt.pages:
                    owned[pg, j % bt.page] = True
        for c, s in ((kc, ks), (vc, vs)):
            c[~owned.unsqueeze(1).expand(-1, heads, -1)] = 0x7F
            s[~owned.any(1)] = math.nan
    return kc, vc, ks, vs


def run(rt, bt, heads, group, dim, fmt=0, causal=True, window=0, seed=11, layout="tokens", kv=None, qscale=1.0,
        sm=None, want_lse=True, max_kv=None, edit_q=None):
    g = torch.Generator().manual_seed(seed)
    kc, vc, ks, vs = kv if kv is not None else make(bt, heads, dim, fmt, seed + 1)
    T, QH = max(1, bt.tokens), heads * group
    q = (torch.randn(T, QH, dim, generator=g) * qscale).bfloat16()
    if edit_q:
        edit_q(q)
    sm = dim ** -0.5 if sm is None else sm
    if layout == "tokens":
        qd, y = q.cuda(), torch.full((T, QH, dim), 7.0, dtype=torch.bfloat16).cuda()
    elif layout == "heads":    # heads outermost
        qd = q.transpose(0, 1).contiguous().cuda().transpose(0, 1)
        y = torch.full((QH, T, dim), 7.0, dtype=torch.bfloat16).cuda().transpose(0, 1)
    else:                      # rows of [q | k | v], output rows wider than the heads
        base = torch.zeros(T, QH + 2 * heads, dim, dtype=torch.bfloat16)
        base[:, :QH] = q
        qd = base.cuda()[:, :QH]
        y = torch.full((T, QH + 1, dim), 7.0, dtype=torch.bfloat16).cuda()[:, :QH]
    lse = torch.full((T, QH), 7.0).cuda() if want_lse else None
    rt.fp8_paged_attention(qd, kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), fmt, bt.table.cuda(), bt.start.cuda(),
                           bt.kv_len.cuda(), bt.max_new, max_kv or bt.max_kv, sm, y, causal=causal, window=window,
                           lse=lse)
    wy, wl, tol, ltol = ref.attend(bt, q, kc, vc, ks, vs, fmt, sm, causal, window)
    y = y.cpu().double()
    assert torch.equal(y.isnan(), wy.isnan())
    off = (y - wy).abs() > tol
    assert not bool(off[~wy.isnan()].any()), "%d of %d, worst %.3g against %.3g" % (
        int(off.sum()), off.numel(), float((y - wy).abs().nan_to_num(0).max()), float(tol.max()))
    if want_lse:
        l = lse.cpu().double()
        none = wl == -math.inf
        assert bool((l[none] == -math.inf).all()) and torch.equal(l.isnan(), wl.isnan())
        fine = wl.isfinite()
        assert bool(((l - wl).abs()[fine] <= ltol[fine]).all())
    return y


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("fmt", [0, 1])
def test_single_tokens(rt, page, dim, fmt):
    before = [0, 1, 14, 15, 16, 17, 31, 62, 63, 64, 127, 128, 129, 500, 1023]
    run(rt, ref.Batch([1] * len(before), before, page), 2, 4, dim, fmt)


@pytest.mark.parametrize("group", [1, 2, 5, 7, 8, 16, 20])
@pytest.mark.parametrize("new", [1, 2, 3])
def test_head_groups(rt, group, new):
    run(rt, ref.Batch([new] * 3, [0, 33, 300], 32), 2, group, 128)


@pytest.mark.parametrize("heads", [1, 3, 8])
def test_heads(rt, heads):
    run(rt, ref.Batch([1, 1], [700, 41], 64), heads, 4, 64)


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts(rt, page, dim, causal):
    run(rt, ref.Batch([130, 1, 0, 65, 40], [0, 77, 5, 200, 31], page), 2, 3, dim, causal=causal)


@pytest.mark.parametrize("window", [1, 2, 16, 33, 100])
@pytest.mark.parametrize("new", [1, 50])
@pytest.mark.parametrize("causal", [True, False])
def test_windows(rt, window, new, causal):
    run(rt, ref.Batch([new, new], [150, 7], 16), 2, 4, 64, causal=causal, window=window)


def test_longer_prompt(rt):
    run(rt, ref.Batch([300], [130], 64), 1, 4, 128, fmt=1)


@pytest.mark.parametrize("causal,window,fmt", [(True, 0, 0), (True, 37, 1), (False, 0, 0)])
def test_many_rows(rt, causal, window, fmt):
    """Enough (token, head) rows for the widest workgroups, ragged, with a missing page and values that are
    not finite where some rows see them."""
    bt = ref.Batch([64] * 15 + [50], [(37 * i) % 90 for i in range(16)], 16)
    bt.table[3, 2] = -1
    kc, vc, ks, vs = make(bt, 8, 128, fmt, 21)
    vc[int(bt.table[5, bt.lens[5] // 16 - 1]), 1, 3, 7] = 0x7F
    vs[int(bt.table[6, 1]), 2] = math.nan
    run(rt, bt, 8, 16, 128, fmt, causal=causal, window=window, kv=(kc, vc, ks, vs))


@pytest.mark.parametrize("seqs", [40, 64, 70])
def test_many_sequences(rt, seqs):
    """More (sequence, head) pairs than CUs: the longest go first, equal and empty ones among them."""
    before = [(61 * i) % 157 if i % 3 else 64 for i in range(seqs)]
    before[5], before[7], before[11] = -1, -1, 700
    run(rt, ref.Batch([1] * seqs, before, 16), 8, 2, 64)
    run(rt, ref.Batch([2] * seqs, before, 32), 8, 1, 128, window=50)


@pytest.mark.parametrize("dim,heads,group", [(128, 2, 4), (64, 1, 5), (128, 2, 17)])
def test_prompts_among_single_tokens(rt, dim, heads, group):
    """Sequences with one, few, many and no new tokens in one call, short and long contexts: both kernels run,
    with and without their keys cut."""
    run(rt, ref.Batch([1, 70, 0, 3, 1, 4, 200, 1, 5], [900, 0, 7, 40, 2600, 5, 30, 0, 1300], 16), heads, group, dim)
    run(rt, ref.Batch([1, 40, 2], [5000, 10, 1], 32), heads, group, dim, window=2000)
    run(rt, ref.Batch([1, 40] + [1] * 30, [50, 300] + [17 * i for i in range(30)], 64), heads, group, dim, causal=False)


def test_long_context(rt):
    run(rt, ref.Batch([1, 1, 2], [9000, 20, 4000], 64), 2, 8, 128)
    run(rt, ref.Batch([1], [9000], 16), 1, 4, 64, window=5000)


def test_bound_on_the_length_is_a_hint(rt):
    """max_kv chooses the split of the work only: longer sequences are still computed."""
    run(rt, ref.Batch([1, 1], [5000, 100], 32), 1, 4, 64, max_kv=64)
    run(rt, ref.Batch([40], [900], 32), 1, 4, 64, max_kv=1)


@pytest.mark.parametrize("new", [1, 6, 40])
def test_queries_that_see_nothing(rt, new):
    """kv_len 0, and below the number of new tokens: those rows are 0 with lse -Inf."""
    y = run(rt, ref.Batch([new, new, new], [-new, -new + 1, 20], 16), 2, 4, 64)
    assert bool((y[:new] == 0).all())


def test_missing_pages(rt):
    bt = ref.Batch([1, 70], [400, 30], 16)
    bt.table[0, 3] = -1
    bt.table[0, 10] = bt.pages
    bt.table[1, 0:2] = -1      # its first queries see nothing
    run(rt, bt, 2, 4, 64)
    bt = ref.Batch([1], [300], 64)
    bt.table[0, :] = -1
    run(rt, bt, 1, 2, 128)


@pytest.mark.parametrize("layout", ["heads", "fused"])
@pytest.mark.parametrize("new", [1, 40])
def test_layouts(rt, layout, new):
    run(rt, ref.Batch([new, 3], [100, 0], 32), 2, 4, 128, layout=layout)
    run(rt, ref.Batch([new, 3], [100, 0], 32), 2, 4, 64, layout=layout, want_lse=False)


@pytest.mark.parametrize("new", [2, 9, 80])
@pytest.mark.parametrize("fmt,code", [(0, 0x7F), (0, 0xFF), (1, 0x7F), (1, 0xFF), (1, 0x7C), (1, 0xFC)])
def test_non_finite_values_reach_only_who_sees_them(rt, fmt, new, code):
    """A NaN (or E5M2 infinity) in a later token's key or value leaves earlier queries as they are."""
    bt = ref.Batch([new, new], [50, 0], 16)
    kc, vc, ks, vs = make(bt, 2, 64, fmt, 3)
    for b in range(2):
        j = bt.lens[b] - 1 - new // 3
        vc[int(bt.table[b, j // 16]), 0, j % 16, 5] = code
        j = bt.lens[b] - 1
        kc[int(bt.table[b, j // 16]), 1, j % 16, 9] = 0x7F
    run(rt, bt, 2, 4, 64, fmt, kv=(kc, vc, ks, vs))
    run(rt, bt, 2, 4, 64, fmt, kv=(kc, vc, ks, vs), window=3)


@pytest.mark.parametrize("new", [1, 33])
def test_non_finite_scales(rt, new):
    bt = ref.Batch([new, new], [64, 40], 16)
    kc, vc, ks, vs = make(bt, 2, 128, 0, 4)
    vs[int(bt.table[0, (bt.lens[0] - 1) // 16]), 0] = math.nan
    ks[int(bt.table[1, (bt.lens[1] - 1) // 16]), 1] = math.nan
    run(rt, bt, 2, 4, 128, kv=(kc, vc, ks, vs))


@pytest.mark.parametrize("new", [1, 40])
def test_scales_of_very_different_size(rt, new):
    """Pages whose scales differ by many powers of two, zero pages among them."""
    bt = ref.Batch([new, new], [300, 90], 16)
    kc, vc, ks, vs = make(bt, 2, 64, 0, 5)
    g = torch.Generator().manual_seed(9)
    vs *= torch.exp2(torch.randint(-20, 20, vs.shape, generator=g).float())
    vs[::5] = 1e-12 / 448
    run(rt, bt, 2, 4, 64, kv=(kc, vc, ks, vs))
    vs *= 2.0 ** -90
    run(rt, bt, 2, 4, 64, kv=(kc, vc, ks, vs))
    vs *= 2.0 ** 170
    run(rt, bt, 2, 4, 64, kv=(kc, vc, ks, vs))


@pytest.mark.parametrize("new", [1, 40])
def test_sharp_and_flat_scores(rt, new):
    bt = ref.Batch([new, new], [200, 1], 32)
    run(rt, bt, 2, 4, 128, qscale=30.0)
    run(rt, bt, 2, 4, 128, qscale=0.0)
    run(rt, bt, 2, 4, 128, sm=-0.3)
    run(rt, bt, 2, 4, 128, sm=0.0)


def test_infinite_query(rt):
    def edit(q):
        q[0, 0, 3] = math.inf
        q[1, 1, 3] = math.nan
    bt = ref.Batch([1, 1, 1], [40, 60, 20], 16)
    y = run(rt, bt, 1, 2, 64, kv=make(bt, 1, 64, 0, 6), edit_q=lambda q: None)
    g = torch.Generator().manual_seed(11)
    q = torch.randn(3, 2, 64, generator=g).bfloat16()
    edit(q)
    kc, vc, ks, vs = make(bt, 1, 64, 0, 6)
    out = torch.empty(3, 2, 64, dtype=torch.bfloat16).cuda()
    rt.fp8_paged_attention(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), 0, bt.table.cuda(), bt.start.cuda(),
                           bt.kv_len.cuda(), 1, bt.max_kv, 0.125, out)
    out = out.cpu().double()
    assert bool(out[0, 0].isnan().all()) and bool(out[1, 1].isnan().all())
    for t, h in ((0, 1), (1, 0), (2, 0), (2, 1)):
        assert torch.equal(out[t, h], y[t, h])


@pytest.mark.parametrize("new,before", [(1, 3000), (60, 100)])
def test_repeats_and_streams(rt, new, before):
    """The same call again, on the default stream and on another, gives the same bits; so does a captured
    graph on every replay."""
    bt = ref.Batch([new, new], [before, before // 2], 16)
    kc, vc, ks, vs = (t.cuda() for t in make(bt, 2, 128, 0, 7))
    plan = [t.cuda() for t in (bt.table, bt.start, bt.kv_len)]
    q = torch.randn(bt.tokens, 8, 128).bfloat16().cuda()
    st = torch.cuda.Stream()
    y, lse = torch.empty_like(q), torch.empty(bt.tokens, 8).cuda()

    def call():
        rt.fp8_paged_attention(q, kc, vc, ks, vs, 0, *plan, bt.max_new, bt.max_kv, 0.09, y, lse=lse)

    call()
    torch.cuda.synchronize()
    first = y.clone(), lse.clone()
    for _ in range(3):
        with torch.cuda.stream(st):
            y.zero_()
            call()
        st.synchronize()
        assert torch.equal(y, first[0]) and torch.equal(lse, first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        call()
    for k in range(4):
        q.copy_(torch.randn(bt.tokens, 8, 128))
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            graph.replay()
        st.synchronize()
        got = y.clone()
        with torch.cuda.stream(st):
            call()
        st.synchronize()
        assert torch.equal(got, y)
