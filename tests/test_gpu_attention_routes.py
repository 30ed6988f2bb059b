"""fp8_paged_attention on the routes that few calls take: the widest workgroups with their keys cut, alone and
beside single tokens; bounds looser than the batch; windows of any size."""
import pytest
import torch

import layer_ref as ref
from test_gpu_paged_attention import make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rt():
    import dynamic_scaling_scaled_amd as rt

    rt.lib()
    return rt


# 256-row tiles need 64 of them and sequences over 8 heads by the bounds; few tokens leave the CUs free, so keys are cut
NEW = [10, 20, 1, 0, 9, 1, 1, 2, 1, 3, 1, 2, 5, 1, 6, 1]
BEFORE = [700, 3, 620, 40, 0, 17, 5, 30, 1, 9, 61, 0, 12, 3, 2, 15]


@pytest.mark.parametrize("group", [16, 17])   # with single tokens on their own kernel, and all on one
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 90), (False, 0)])
def test_widest_workgroups_with_cut_keys(rt, group, causal, window):
    bt = ref.Batch(NEW, BEFORE, 32)
    bt.max_new = 64
    bt.table[0, 5] = -1
    run(rt, bt, 8, group, 128, causal=causal, window=window)


def test_bounds_looser_than_the_batch(rt):
    bt = ref.Batch([1, 30, 2], [300, 5, 40], 16)
    for max_new, max_kv in ((33, 10 ** 6), (1 << 20, 1 << 40)):
        bt.max_new, bt.max_kv = max_new, max_kv
        run(rt, bt, 2, 4, 64)
        run(rt, bt, 2, 4, 128, causal=False, window=37)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 62, 2 ** 63 - 1])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new", [1, 40])
def test_a_window_wider_than_any_sequence_hides_nothing(rt, window, causal, new):
    """kv_len below the number of new tokens among them: those queries stand before position 0."""
    bt = ref.Batch([new, 3, 4], [2000, -2, 0], 16)
    kc, vc, ks, vs = (t.cuda() for t in make(bt, 2, 64, 0, 12))
    q = torch.randn(bt.tokens, 8, 64, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    plan = [t.cuda() for t in (bt.table, bt.start, bt.kv_len)]

    def call(window):
        y, lse = torch.full_like(q, 7.0), torch.full((bt.tokens, 8), 7.0).cuda()
        rt.fp8_paged_attention(q, kc, vc, ks, vs, 0, *plan, bt.max_new, bt.max_kv, 0.125, y, causal=causal,
                               window=window, lse=lse)
        return y, lse

    assert all(torch.equal(a, b) for a, b in zip(call(window), call(0)))
