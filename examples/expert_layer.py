"""The gated half of a decoder layer in FP8, with experts, from the library's entry points:

  norm (+ residual) -> codes -> routing -> gates and ups of the chosen experts -> gated activation -> codes (and an
  8-bit checkpoint) -> the experts' second product -> weighted sum (+ residual)

A batch of tokens and a single one go through the layer; then one training step takes the gradients of the layer's
input and of the router through it, the experts' weights being FP8 codes that stay as they are.  Run it from the
repository's root on an MI355X:  python examples/expert_layer.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dynamic_scaling_scaled_amd as rt  # noqa: E402

NORM_EPS, EPS = 1e-6, 1e-12


def codes(x, fmt=rt.E4M3):
    """FP8 codes of x's rows and their scales."""
    q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    s = torch.empty(x.shape[0], 1, device=x.device)
    rt.fp8_quantize(x, (1, 0), fmt, rt.DYNAMIC, EPS, False, s, None, q)
    return q, s


class Weights:
    """[experts x N x K] as per-channel E4M3 codes in the products' layout, laid out once."""

    def __init__(self, w):
        self.experts, self.N, self.K = w.shape
        q, s = codes(w.reshape(-1, self.K).contiguous())
        self.image, self.scale = rt.fp8_pack_weights16(q), s

    def __call__(self, a, fmt, scale, plan, gather=False):
        """a's rows through their experts; gather: a holds tokens, not slots."""
        slots, order, offsets = plan
        y = torch.empty(order.numel(), self.N, dtype=torch.bfloat16, device=a.device)
        rt.fp8_expert_gemm(a, fmt, (1, 0), scale, self.image, rt.E4M3, (1, 0), self.scale, offsets, y,
                           order=order if gather else None, choices=slots.shape[1])
        return y


class Experts:
    def __init__(self, hidden, inter, experts, k, act=rt.SILU, score=rt.SOFTMAX, groups=1, top_groups=1, biased=False, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.hidden, self.inter, self.experts, self.k, self.act = hidden, inter, experts, k, act
        self.choice = dict(score=score, groups=groups, top_groups=top_groups, group_best=2 if groups > 1 else 1,
                           bias=(0.1 * torch.randn(experts, generator=g)).cuda() if biased else None)
        self.norm = (1 + 0.1 * torch.randn(hidden, generator=g)).bfloat16().cuda()
        self.router = (torch.randn(experts, hidden, generator=g) / math.sqrt(hidden)).cuda()
        self.w_in = (torch.randn(experts, 2 * inter, hidden, generator=g) / math.sqrt(hidden)).bfloat16().cuda()
        self.w_out = (torch.randn(experts, hidden, inter, generator=g) / math.sqrt(inter)).bfloat16().cuda()
        self.up, self.down = Weights(self.w_in), Weights(self.w_out)
        # the same weights along their other axis, for the gradient of what they multiply
        self.up_t, self.down_t = Weights(self.w_in.transpose(1, 2)), Weights(self.w_out.transpose(1, 2))

    def __call__(self, x, residual, train=False):
        """(output, what the gradients need): the output is the layer's sum with h = x + residual."""
        tokens, S = x.shape[0], x.shape[0] * self.k
        ints = dict(dtype=torch.int32, device=x.device)
        q8, s8 = torch.empty(tokens, self.hidden, dtype=torch.uint8, device=x.device), torch.empty(tokens, 1, device=x.device)
        h, rstd = torch.empty_like(x), torch.empty(tokens, device=x.device)
        rt.fp8_rmsnorm_quantize(x, self.norm, NORM_EPS, (1, 0), rt.E4M3, rt.DYNAMIC, EPS, False, s8, q8,
                                residual=residual, h=h, rstd=rstd)
        n = (h.float() * rstd[:, None]) * self.norm.float()
        logits = n @ self.router.T
        ids, weights = torch.empty(tokens, self.k, **ints), torch.empty(tokens, self.k, device=x.device)
        plan = (torch.empty(tokens, self.k, **ints), torch.empty(S, **ints), torch.empty(self.experts + 1, **ints))
        rt.fp8_expert_route(logits, ids, weights, *plan, **self.choice)
        slots, _, offsets = plan
        both = self.up(q8, rt.E4M3, s8, plan, gather=True)
        z8, sz = torch.empty(S, self.inter, dtype=torch.uint8, device=x.device), torch.empty(S, 1, device=x.device)
        kept = kept_scale = None
        if train:
            kept = torch.empty(S, 2 * self.inter, dtype=torch.uint8, device=x.device)
            kept_scale = torch.empty(S, 2, -(-self.inter // rt.KEPT_GROUP), device=x.device)
        rt.fp8_gated_quantize(both, (1, 0), rt.E4M3, rt.DYNAMIC, EPS, False, sz, z8, act=self.act, kept=kept,
                              kept_scale=kept_scale, live=offsets[self.experts:])
        out = self.down(z8, rt.E4M3, sz, plan)
        y = torch.empty_like(x)
        rt.fp8_expert_combine(out, slots, weights, y, residual=h)
        return y, (h, rstd, logits, ids, weights, plan, kept, kept_scale, out)

    def gradients(self, dy, saved):
        """(dx, dlogits): of the norm's input (the residual's own path included) and of the router's logits."""
        h, rstd, logits, ids, weights, plan, kept, kept_scale, out = saved
        slots, _, offsets = plan
        S = out.shape[0]
        dout, dweights = torch.empty_like(out), torch.empty_like(weights)
        rt.fp8_expert_combine_backward(dy, out, slots, weights, dout, dweights)
        dlogits = torch.empty_like(logits)
        rt.fp8_expert_route_backward(logits, ids, dweights, dlogits, score=self.choice["score"])
        dz = self.down_t(*self._given(dout), plan)
        dboth = torch.empty(S, 2 * self.inter, dtype=torch.bfloat16, device=dy.device)
        rt.fp8_gated_backward(dz, kept, kept_scale, dboth, act=self.act, live=offsets[self.experts:])
        dslots = self.up_t(*self._given(dboth), plan)
        dn = torch.empty_like(dy)  # a token's gradient: its slots' sum, and the router's
        rt.fp8_expert_combine(dslots, slots, torch.ones_like(weights), dn, residual=(dlogits @ self.router).bfloat16())
        dx = torch.empty_like(dy)
        rt.fp8_rmsnorm_backward(dn, h, self.norm, rstd, dx, dresidual=dy)
        return dx, dlogits

    @staticmethod
    def _given(d):
        q, s = codes(d, rt.E5M2)  # gradients: the wider range
        return q, rt.E5M2, s


def reference(layer, x, residual, ids):
    """The same layer without FP8, in 32 bits, with the experts `ids` and weights by its own logits (which it also
    returns); differentiable in x."""
    h = x + residual
    n = h * (h.square().mean(1, keepdim=True) + NORM_EPS).rsqrt() * layer.norm.float()
    logits = n @ layer.router.T
    logits.retain_grad() if logits.requires_grad else None
    chosen = logits.gather(1, ids.long())
    w = chosen.softmax(1) if layer.choice["score"] == rt.SOFTMAX else chosen.sigmoid() / chosen.sigmoid().sum(1, keepdim=True)
    y = h
    for e in range(layer.experts):
        t, j = (ids == e).nonzero(as_tuple=True)
        gate, up = (n[t] @ layer.w_in[e].float().T).chunk(2, 1)
        z = (torch.nn.functional.silu(gate) if layer.act == rt.SILU else torch.nn.functional.gelu(gate, approximate="tanh")) * up
        y = y.index_add(0, t, (z @ layer.w_out[e].float().T) * w[t, j][:, None])
    return y, h, logits


def main(hidden=1024, inter=512, experts=16, k=4, tokens=(200, 1), seed=1, **kw):
    """Relative errors (2-norm) against the layer in 32 bits: for each count of tokens of the layer's own term and of the
    gradient that it adds to the input's; then of all logits' gradient."""
    g = torch.Generator().manual_seed(seed)
    layer = Experts(hidden, inter, experts, k, **kw)
    errors, routers = [], []
    for t in tokens:
        x, res, dy = (torch.randn(t, hidden, generator=g).bfloat16().cuda() for _ in range(3))
        y, saved = layer(x, res, train=True)
        h, ids = saved[0], saved[3]
        xf = x.float().requires_grad_()
        want, hf, logits = reference(layer, xf, res.float(), ids)
        want.backward(dy.float())
        term = (want - hf).detach()
        errors.append(float((y.float() - h.float() - term).norm() / term.norm()))
        dx, dlogits = layer.gradients(dy, saved)
        own = xf.grad - dy.float()
        errors.append(float((dx.float() - dy.float() - own).norm() / own.norm()))
        routers.append((dlogits, logits.grad))
    got, want = (torch.cat(r) for r in zip(*routers))
    return errors + [float((got - want).norm() / want.norm())]


if __name__ == "__main__":
    batch, batch_grad, one, one_grad, router = main()
    print("relative errors against the layer in 32 bits: 200 tokens %.3f, gradient %.3f; one token %.3f, gradient %.3f; "
          "router's gradient %.3f" % (batch, batch_grad, one, one_grad, router))
