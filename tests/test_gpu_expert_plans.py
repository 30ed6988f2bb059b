"""fp8_expert_gemm on plans that no router writes, where experts claim the same slots, and on shallow products with so
many slots an expert that they take the tiles of 256 slots (bound: expert_ref.experts)."""
import pytest
import torch

import expert_ref as ref
import layer_ref as lr
from test_gpu_expert_gemm import check, codes, weights
from test_gpu_expert_offsets import kernel

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rt():
    import dynamic_scaling_scaled_amd as rt

    rt.lib()
    return rt


@pytest.mark.parametrize("counts,K", [((2100,), 128), ((2140, 2201), 128), ((2300, 2060), 128), ((1100,), 256),
                                      ((1150, 1177), 256), ((1270, 1060), 256)])
def test_shallow_and_tall(rt, counts, K):
    """One and two stages of the tiles of 256 slots: full ones and last ones of 1 to 4 blocks, both formats and outputs."""
    for N, kw in ((48, dict(out=torch.float32)), (272, dict(fa=1, gather=True, choices=2, pad=16)),
                  (16, dict(fa=1, out=torch.float32, spare=5)), (32, dict(ga=(0, 0), gb="expert"))):
        assert kernel(sum(counts) + kw.get("spare", 0), len(counts), N, K) == "tile256"
        check(rt, counts, N, K, **kw)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,K", [(6, 256), (40, 256), (90, 256), (260, 2176), (700, 2176)])
def test_claims_of_the_same_slots(rt, out, rows, K):
    """Each number of a claimed slot is that of one of its claims, or still open where more is claimed than there are slots;
    rows behind the slots and columns beside y are left as they were."""
    N, pad, S = 272, 16, 2 * rows
    for offsets in ([0, rows, 0, S], [0, S, 0, S, 0, S, 0, S], [S // 2, S, 0, 3, S - 1, S, 2 ** 31 - 1, 0, S],
                    [0, S] * 20, [-2 ** 31, 2 ** 31 - 1] * 8):
        E = len(offsets) - 1
        g = torch.Generator().manual_seed(rows)
        a, (b, image) = codes((S, K), 0, g), weights(rt, E, N, K, g)
        one = torch.ones(1, 1).cuda()
        y = torch.full((S + 4, N + pad), 7.0, dtype=out).cuda()
        rt.fp8_expert_gemm(a.cuda(), 0, (0, 0), one, image, 0, (0, 0), one, torch.tensor(offsets, dtype=torch.int32).cuda(),
                           y[:S, :N])
        got = y.cpu()
        assert bool((got[S:] == 7).all()) and bool((got[:, N:] == 7).all())
        look = sorted({0, 1, rows - 1, rows, S - 2, S - 1})  # rows of the slots
        some = got[look, :N].double()
        fits = some == 7
        da = lr.decode(a[look], 0)
        for e in range(E):
            claimed = torch.tensor([max(offsets[e], 0) <= s < offsets[e + 1] for s in look])
            prod = lr.decode(b[e], 0)[None] * da[:, None]
            want, mag = prod.sum(2), prod.abs()
            tol = 7 * 2.0 ** -13 * mag.view(len(look), N, -1, 8).amax(3).sum(2) + ((K // 8 + 16) * 2.0 ** -23 + 4 * ref.U) * mag.sum(2)
            fits |= claimed[:, None] & ((some - want).abs() <= tol + ref.HALF[out] * (want.abs() + tol))
        assert bool(fits.all())
