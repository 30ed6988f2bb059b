"""fp8_paged_attention over caches of zeros and of tiny values, whose v scales are the smallest that fp8_kv_append
writes: 2^-96 (the least eps) over the format's largest value.  The sums of weights over scales pass 2^112 for each key.
And over the largest values."""
import math

import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu

U = ref.U
EPS = 2.0 ** -96


@pytest.fixture(scope="module")
def rt():
    import dynamic_scaling_scaled_amd as rt

    rt.lib()
    return rt


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("n,rise", [(300, 0.0), (80000, 0.0), (80000, 5.0)])
@pytest.mark.parametrize("seqs,new", [(1, 1), (520, 1), (400, 5), (1, 40)])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -97, 2.0 ** 127])
def test_long_context_of_extreme_values(rt, fmt, n, rise, seqs, new, size):
    """All sequences read one page of equal keys and values over and over; with `rise` the keys of the first page score
    that much less.  Bounds: a score is within 16 u of terms of at most 6, a sum of n equal terms within (n + 8) u, the
    weights are rounded to 11 bits, the output to bf16."""
    dim, page, group = 64, 16, 4
    k = torch.full((2 * page, 1, dim), 0.0).bfloat16()
    k[page:, 0, 0] = rise
    v = torch.full((2 * page, 1, dim), size).bfloat16()
    caches = [torch.zeros(2, 1, page, dim, dtype=torch.uint8).cuda() for _ in range(2)]
    scales = [torch.zeros(2, 1).cuda() for _ in range(2)]
    one = [torch.tensor(t, dtype=torch.int32).cuda() for t in ([[0, 1]], [0, 2 * page], [2 * page])]
    rt.fp8_kv_append(k.cuda(), v.cuda(), *caches, *scales, fmt, *one, 2 * page, EPS)
    vs = float(scales[1][0, 0])
    assert vs == float(torch.tensor(max(EPS, size), dtype=torch.float32) / ref.FMAX[fmt])
    pages = -(-n // page)
    table = torch.ones(seqs, pages, dtype=torch.int32)
    table[:, 0] = 0
    q = torch.zeros(seqs * new, group, dim).bfloat16()
    q[:, :, 0] = 1
    start = (torch.arange(seqs + 1) * new).to(torch.int32).cuda()
    kv_len = torch.full((seqs,), n, dtype=torch.int32).cuda()
    y, lse = torch.empty(q.shape, dtype=torch.bfloat16).cuda(), torch.empty(q.shape[:2]).cuda()
    rt.fp8_paged_attention(q.cuda(), *caches, *scales, fmt, table.cuda(), start, kv_len, new, n, 1.0, y, causal=False, lse=lse)
    up = float(ref.decode(caches[0][1, 0, 0, :1].cpu(), fmt)) * float(scales[0][1, 0])
    want = up + math.log(page * math.exp(-up) + (n - page))
    off = (lse.double() - want).abs().max()
    assert float(off) <= 16 * U * 6 + (n + 8) * U + 4 * U * abs(want), float(off)
    value = float(ref.decode(caches[1][1, 0, 0, :1].cpu(), fmt)) * vs
    assert float((y.double() - value).abs().max()) <= (2.0 ** -8 + 2.0 ** -11 + (n + 64) * U) * value
