"""The gated half's calls on two streams at once, from one thread and from two: each stream has its own counts and partials, so
the results are those of calls one after the other, bit for bit; and a graph of a smaller batch than the stream was warmed
up with."""
import threading

import pytest
import torch

from test_gpu_expert_route import logits_of

pytestmark = pytest.mark.gpu

TOKENS, E, K, N, D = 3000, 64, 4, 256, 512


@pytest.fixture(scope="module")
def rt():
    import dynamic_scaling_scaled_amd as rt

    rt.lib()
    return rt


class Job:
    """Routing in several blocks, products, an activation with one given scale and its observed amax, sum, gradients."""

    def __init__(self, rt, seed, tokens=TOKENS):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.rt, S = rt, tokens * K
        self.logits = logits_of(tokens, E, seed=seed)
        self.a = torch.randint(0, 120, (tokens, D), dtype=torch.uint8, device="cuda", generator=g)
        self.image = rt.fp8_pack_weights16(torch.randint(0, 120, (E * 2 * N, D), dtype=torch.uint8, device="cuda", generator=g))
        self.one = torch.full((1, 1), 2.0 ** -10, device="cuda")  # (products of about 0.5, codes of about 150)
        ints = dict(dtype=torch.int32, device="cuda")
        self.out = dict(ids=torch.zeros(tokens, K, **ints), weights=torch.zeros(tokens, K, device="cuda"),
                        slots=torch.zeros(tokens, K, **ints), order=torch.zeros(S, **ints), offsets=torch.zeros(E + 1, **ints),
                        both=torch.zeros(S, 2 * N, dtype=torch.bfloat16, device="cuda"),
                        z=torch.zeros(S, N, dtype=torch.uint8, device="cuda"), amax=torch.zeros(1, 1, device="cuda"),
                        y=torch.zeros(tokens, 2 * N, dtype=torch.bfloat16, device="cuda"), dx=torch.zeros(S, 2 * N, dtype=torch.bfloat16, device="cuda"),
                        dw=torch.zeros(tokens, K, device="cuda"), dl=torch.zeros(tokens, E, device="cuda"))

    def __call__(self, stream=None):
        rt, o = self.rt, self.out
        rt.fp8_expert_route(self.logits, o["ids"], o["weights"], o["slots"], o["order"], o["offsets"], stream=stream)
        rt.fp8_expert_gemm(self.a, 0, (0, 0), self.one, self.image, 0, (0, 0), self.one, o["offsets"], o["both"], order=o["order"],
                           choices=K, stream=stream)
        rt.fp8_gated_quantize(o["both"], (0, 0), 0, rt.GIVEN, 1e-12, False, self.one, o["z"], amax_out=o["amax"],
                              live=o["offsets"][E:], stream=stream)
        rt.fp8_expert_combine(o["both"], o["slots"], o["weights"], o["y"], stream=stream)
        rt.fp8_expert_combine_backward(o["y"], o["both"], o["slots"], o["weights"], o["dx"], o["dw"], stream=stream)
        rt.fp8_expert_route_backward(self.logits, o["ids"], o["dw"], o["dl"], stream=stream)

    def clear(self):
        for t in self.out.values():
            t.zero_()


def prepared(rt, **kw):
    jobs = [Job(rt, s, **kw) for s in (1, 2)]
    want = []
    for job in jobs:
        job()
        torch.cuda.synchronize()
        want.append({n: t.clone() for n, t in job.out.items()})
        assert all(bool((t != 0).any()) for t in want[-1].values())
    return jobs, want


def test_two_streams(rt):
    jobs, want = prepared(rt)
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        for job in jobs:
            job.clear()
        torch.cuda.synchronize()
        for _ in range(4):
            for job, s in zip(jobs, streams):
                job(s)
        torch.cuda.synchronize()
        for job, w in zip(jobs, want):
            assert all(torch.equal(job.out[n], w[n]) for n in w)


def test_two_threads(rt):
    jobs, want = prepared(rt)
    streams = [torch.cuda.Stream() for _ in jobs]
    for job in jobs:
        job.clear()
    torch.cuda.synchronize()
    threads = [threading.Thread(target=lambda j=j, s=s: [j(s) for _ in range(10)]) for j, s in zip(jobs, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for job, w in zip(jobs, want):
        assert all(torch.equal(job.out[n], w[n]) for n in w)


@pytest.mark.parametrize("tokens", [1, 65, 2048])
def test_smaller_batch_captured(rt, tokens):
    """The stream is warmed up with 3000 tokens; the counts of 2048 take as many blocks again as those of 2049."""
    jobs, want = prepared(rt, tokens=tokens)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        Job(rt, 3)(s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        jobs[0](s)
    for _ in range(3):
        jobs[0].clear()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        jobs[1]()  # on the current stream
        torch.cuda.synchronize()
        for job, w in zip(jobs, want):
            assert all(torch.equal(job.out[n], w[n]) for n in w)
