"""The gated half of a dense decoder layer from the library's entry points: codes -> gates and ups -> gated activation (and
the 8-bit checkpoint) -> second product; its input's and weights' gradients; the whole of it captured and replayed.

Bounds (2-norm, relative to the half in 32 bits): E4M3 rounds a value by 2.6% of it (root mean square), E5M2 by 5.2%.  Codes
of the input and of weights put 3.7% on gates and ups; their product, with an activation whose slope is near 1, has 5 to
6%, and codes of it and of the second weights add 3.7%: about 6.5% in all, 12% is the limit.  The input's gradient has
codes in E5M2 and weights twice (5.8% each) and, between them, gates and ups with 3.7% and the checkpoint's 2.6% (4.5%
each, 6.5% of the products): about 10.5%, 18% is the limit.  The second weights' gradient multiplies codes in E5M2 (5.2%)
with codes (2.6%) of the product computed again (6.5%): 8.7%, the limit is 15%; the first ones' the gradient of gates and
ups (8.7%, codes 5.2%) with codes of the input (2.6%): 10.5%, the limit is 18%."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

EPS = 1e-12


@pytest.fixture(scope="module")
def rt():
    import dynamic_scaling_scaled_amd as rt

    rt.lib()
    return rt


class Half:
    """w_in [2 inter x hidden], w_out [hidden x inter]; grouped: 1 x 128 scales with 128 x 128 for the weights, else rows'."""

    def __init__(self, rt, hidden, inter, act, grouped):
        g = torch.Generator().manual_seed(hidden + inter)
        self.rt, self.hidden, self.inter, self.act = rt, hidden, inter, act
        self.ga, self.gw = ((1, 128), (128, 128)) if grouped else ((1, 0), (1, 0))
        self.w_in = (torch.randn(2 * inter, hidden, generator=g) / math.sqrt(hidden)).bfloat16().cuda()
        self.w_out = (torch.randn(hidden, inter, generator=g) / math.sqrt(inter)).bfloat16().cuda()
        self.up, self.down = self.codes(self.w_in, self.gw), self.codes(self.w_out, self.gw)
        self.up_t, self.down_t = (self.codes(w.T.contiguous(), self.gw) for w in (self.w_in, self.w_out))

    def codes(self, x, gran, fmt=0):
        q = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
        s = torch.empty(self.rt.scale_shape(x.shape, gran), device="cuda")
        self.rt.fp8_quantize(x, gran, fmt, self.rt.DYNAMIC, EPS, False, s, None, q)
        return q, s

    def columns(self, x, fmt):
        """Codes of x transposed, with a scale for each column of x."""
        rows, cols = x.shape
        q, qt = (torch.empty(s, dtype=torch.uint8, device="cuda") for s in ((rows, cols), (cols, rows)))
        s = torch.empty(1, cols, device="cuda")
        self.rt.fp8_quantize_transpose(x, (0, 1), fmt, self.rt.DYNAMIC, EPS, False, s, None, q, qt)
        return qt, s

    def product(self, a, fmt, w, out):
        y = torch.empty(a[0].shape[0], w[0].shape[0], dtype=out, device="cuda")
        self.rt.fp8_scaled_gemm(a[0], fmt, self.ga, a[1], w[0], 0, self.gw, w[1], y)
        return y

    def weight_gradient(self, d, x):
        y = torch.empty(d.shape[1], x.shape[1], device="cuda")
        (a, sa), (b, sb) = self.columns(d, 1), self.columns(x, 0)
        self.rt.fp8_scaled_gemm(a, 1, (1, 0), sa, b, 0, (1, 0), sb, y)
        return y

    def __call__(self, x, dy):
        """(y, dx, gradient of w_in, of w_out); the weights' need a multiple of 16 tokens."""
        rt, rows = self.rt, x.shape[0]
        both = self.product(self.codes(x, self.ga), 0, self.up, torch.bfloat16)
        z8 = torch.empty(rows, self.inter, dtype=torch.uint8, device="cuda")
        sz = torch.empty(rt.scale_shape(z8.shape, self.ga), device="cuda")
        kept = torch.empty(rows, 2 * self.inter, dtype=torch.uint8, device="cuda")
        ks = torch.empty(rows, 2, -(-self.inter // rt.KEPT_GROUP), device="cuda")
        rt.fp8_gated_quantize(both, self.ga, rt.E4M3, rt.DYNAMIC, EPS, False, sz, z8, act=self.act, kept=kept, kept_scale=ks)
        y = self.product((z8, sz), 0, self.down, torch.bfloat16)
        dz = self.product(self.codes(dy, self.ga, 1), 1, self.down_t, torch.bfloat16)
        dboth, z = torch.empty_like(both), torch.empty_like(dz)
        rt.fp8_gated_backward(dz, kept, ks, dboth, act=self.act, z=z)
        dx = self.product(self.codes(dboth, self.ga, 1), 1, self.up_t, torch.bfloat16)
        if rows % 16:
            return y, dx
        return y, dx, self.weight_gradient(dboth, x), self.weight_gradient(dy, z)

    def reference(self, x, dy):
        x, w_in, w_out = (t.float().requires_grad_() for t in (x, self.w_in, self.w_out))
        gate, up = (x @ w_in.T).chunk(2, 1)
        f = torch.nn.functional.silu(gate) if self.act == self.rt.SILU else torch.nn.functional.gelu(gate, approximate="tanh")
        y = (f * up) @ w_out.T
        y.backward(dy.float())
        return y.detach(), x.grad, w_in.grad, w_out.grad


def inputs(rows, hidden, seed=0):
    g = torch.Generator().manual_seed(rows + seed)
    return [torch.randn(rows, hidden, generator=g).bfloat16().cuda() for _ in range(2)]


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("hidden,inter", [(512, 640), (1024, 384)])
@pytest.mark.parametrize("rows", [1, 16, 77, 400])
def test_half_and_gradients(rt, grouped, act, hidden, inter, rows):
    half = Half(rt, hidden, inter, act, grouped)
    x, dy = inputs(rows, hidden)
    for got, want, limit in zip(half(x, dy), half.reference(x, dy), (0.12, 0.18, 0.18, 0.15)):
        assert float((got.float() - want).norm() / want.norm()) < limit


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("rows", [1, 160])
def test_captured_and_replayed(rt, grouped, rows):
    """In one graph, replayed on new inputs with eager work on another stream in between: as without it, bit for bit."""
    half = Half(rt, 512, 256, 0, grouped)
    data = [inputs(rows, 512, i) for i in range(4)]
    want = [[t.clone() for t in half(*d)] for d in data]
    x, dy = (t.clone() for t in data[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        half(x, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = half(x, dy)
    for i in (1, 2, 3, 0):
        x.copy_(data[i][0])
        dy.copy_(data[i][1])
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            graph.replay()
        other = half(*data[(i + 1) % 4])  # this stream's own memory
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
        assert all(torch.equal(a, b) for a, b in zip(other, want[(i + 1) % 4]))
