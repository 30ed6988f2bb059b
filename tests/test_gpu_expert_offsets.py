"""fp8_expert_gemm where offsets pass 32 bits, on each of its kernels: a weight image of more than 4 GiB, and rows of a up to
just under the 2^32 bytes that the call allows.  `kernel` states the library's choice, so that every case is known to run the
kernel that it names; the slots behind the last expert's make up the average that the choice goes by."""
import pytest
import torch

import expert_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rt():
    import dynamic_scaling_scaled_amd as rt

    rt.lib()
    yield rt
    torch.cuda.empty_cache()


def kernel(slots, E, N, K):
    """The kernel of a call: streams of 16 or 32 slots, tiles of 64 or 256."""
    a, cols, cus = -(-slots // E), -(-N // 256), torch.cuda.get_device_properties(0).multi_processor_count
    units = min(E, slots) * cols
    if a <= 8 or (a <= 16 and units < cus):
        return "stream16"
    if a <= 32 and units < cus:
        return "stream32"
    return "tile64" if a <= 64 or a * K <= 1 << 18 or (a <= 128 and units <= cus) else "tile256"


def at(y, rows, cols):
    return y[rows][:, cols].cpu().double()


@pytest.mark.parametrize("name,E,N,K,average,first,last", [
    ("stream16", 72, 4096, 16384, 7, 13, 9), ("stream32", 140, 256, 131072, 20, 33, 47),
    ("tile64", 72, 4096, 16384, 40, 70, 131), ("tile256", 72, 4096, 16384, 130, 200, 300)])
def test_weights(rt, name, E, N, K, average, first, last):
    """4.7 to 4.8 GB of codes: the products of the first and the last expert, their first and last rows and columns."""
    S = average * E
    assert kernel(S, E, N, K) == name and E * N * K > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(average)
    b = torch.randint(0, 120, (E * N, K), dtype=torch.uint8, device="cuda", generator=g)
    image = rt.fp8_pack_weights16(b)
    a = torch.randint(0, 120, (first + last, K), dtype=torch.uint8, device="cuda", generator=g)
    sa, sb = torch.full((first + last, 1), 2.0 ** -10).cuda(), torch.ones(E, N).cuda()
    off = torch.tensor([0] + [first] * (E - 1) + [first + last], dtype=torch.int32).cuda()
    y = torch.full((S, N), 7.0, device="cuda")
    rt.fp8_expert_gemm(a, 0, (1, 0), sa, image, 0, (1, 0), sb, off, y)
    assert bool((y[first + last:] == 7).all())
    for e, lo, hi in ((0, 0, first), (E - 1, first, first + last)):
        rows = [lo, (lo + hi) // 2, hi - 1]
        for c in (slice(0, 16), slice(N - 16, N)):
            w = b[e * N:(e + 1) * N][c].cpu().view(1, 16, K)
            want, tol, _ = ref.experts(a[rows].cpu(), 0, sa[rows].cpu(), None, 1, w, torch.ones(1, 16), [0, 3], 3)
            assert bool(((at(y, rows, c) - want).abs() <= tol + ref.HALF[torch.float32] * want).all())


@pytest.mark.parametrize("name,average", [("stream16", 4), ("stream32", 24), ("tile64", 60), ("tile256", 200)])
def test_rows_of_a(rt, name, average):
    """131071 rows 32768 bytes apart, 2^32 - 32768 bytes: slots of the first and last rows and around the middle."""
    E, N, K, rows, ld = 4, 512, 4096, 131071, 32768
    S = average * E
    assert kernel(S, E, N, K) == name and (rows + 1) * ld == 1 << 32
    g = torch.Generator(device="cuda").manual_seed(average)
    a = torch.randint(0, 120, (rows, ld), dtype=torch.uint8, device="cuda", generator=g)
    b = torch.randint(0, 120, (E * N, K), dtype=torch.uint8, device="cuda", generator=g)
    sa = torch.rand(rows, 1, device="cuda", generator=g) * 2.0 ** -10
    order = torch.randint(0, rows, (S,), generator=torch.Generator().manual_seed(average)).to(torch.int32)
    order[:6] = torch.tensor([rows - 1, 0, rows // 2, rows // 2 + 1, 2 ** 31 - 1, rows])
    order[-2:] = torch.tensor([rows - 1, rows - 2])
    off = torch.arange(E + 1, dtype=torch.int32) * average
    y = torch.empty(S, N, device="cuda")
    rt.fp8_expert_gemm(a[:, :K], 0, (1, 0), sa, rt.fp8_pack_weights16(b), 0, (1, 0), torch.ones(E, N).cuda(), off.cuda(), y,
                       order=order.cuda())
    pick = order.long().clamp_max(rows - 1)
    few = a[pick.cuda()][:, :K].cpu().contiguous()
    places = torch.where(order.long() < rows, torch.arange(S), -1).to(torch.int32)
    c = slice(N - 16, N)
    want, tol, _ = ref.experts(few, 0, sa[pick.cuda()].cpu(), places, 1, b.view(E, N, K)[:, c].cpu(), torch.ones(E, 16), off, S)
    assert bool(((at(y, slice(0, S), c) - want).abs() <= tol + ref.HALF[torch.float32] * want).all())
