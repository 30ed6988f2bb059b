"""The attention half of a decoder layer in FP8, from the library's entry points:

  norm (+ residual) -> codes -> QKV GEMM -> keys and values into the paged cache ->
  attention over it -> codes -> output GEMM -> the next norm takes the sum

A batch of prompts goes through the layer, then some steps of one token for
each sequence; then one training step's gradient of the norm.  Run it from the repository's root on
an MI355X:  python examples/decoder_layer.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dynamic_scaling_scaled_amd as rt  # noqa: E402

NORM_EPS, EPS = 1e-6, 1e-12


class Attention:
    """Weights of one layer: per-channel E4M3 codes, laid out once."""

    def __init__(self, hidden, q_heads, kv_heads, dim, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.hidden, self.q_heads, self.kv_heads, self.dim = hidden, q_heads, kv_heads, dim
        self.norm = (1 + 0.1 * torch.randn(hidden, generator=g)).bfloat16().cuda()
        self.w_qkv = (torch.randn((q_heads + 2 * kv_heads) * dim, hidden, generator=g) / math.sqrt(hidden)).bfloat16().cuda()
        self.w_out = (torch.randn(hidden, q_heads * dim, generator=g) / math.sqrt(q_heads * dim)).bfloat16().cuda()
        self.qkv, self.qkv_scale = self._codes(self.w_qkv)
        self.out, self.out_scale = self._codes(self.w_out)

    @staticmethod
    def _codes(x):
        q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
        s = torch.empty(x.shape[0], 1, device=x.device)
        rt.fp8_quantize(x, (1, 0), rt.E4M3, rt.DYNAMIC, EPS, False, s, None, q)
        return q, s

    def __call__(self, x, residual, cache, plan):
        """(output, h): h = x + residual, which the next norm's residual is."""
        tokens = x.shape[0]
        q8, s8 = torch.empty(tokens, self.hidden, dtype=torch.uint8, device=x.device), torch.empty(tokens, 1, device=x.device)
        h = torch.empty_like(x)
        rt.fp8_rmsnorm_quantize(x, self.norm, NORM_EPS, (1, 0), rt.E4M3, rt.DYNAMIC, EPS, False, s8, q8,
                                residual=residual, h=h)
        qkv = torch.empty(tokens, self.qkv.shape[0], dtype=torch.bfloat16, device=x.device)
        rt.fp8_scaled_gemm(q8, rt.E4M3, (1, 0), s8, self.qkv, rt.E4M3, (1, 0), self.qkv_scale, qkv)
        heads = qkv.view(tokens, -1, self.dim)
        q, k, v = heads.split([self.q_heads, self.kv_heads, self.kv_heads], 1)
        rt.fp8_kv_append(k, v, *cache.tensors, rt.E4M3, plan.table, plan.start, plan.kv_len, plan.max_new)
        y = torch.empty(tokens, self.q_heads, self.dim, dtype=torch.bfloat16, device=x.device)
        rt.fp8_paged_attention(q, *cache.tensors, rt.E4M3, plan.table, plan.start, plan.kv_len, plan.max_new,
                               plan.max_kv, self.dim ** -0.5, y)
        y8, sy = self._codes(y.view(tokens, -1))
        out = torch.empty_like(x)
        rt.fp8_scaled_gemm(y8, rt.E4M3, (1, 0), sy, self.out, rt.E4M3, (1, 0), self.out_scale, out)
        return out, h


class Cache:
    """Pages of FP8 codes with one scale for each page and head."""

    def __init__(self, pages, heads, page, dim):
        self.page = page
        self.tensors = [torch.zeros(pages, heads, page, dim, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.tensors += [torch.zeros(pages, heads, device="cuda") for _ in range(2)]


class Plan:
    """Which tokens a call brings (`new` of each sequence), and where they live."""

    def __init__(self, table, new, lens):
        start = [0]
        for n in new:
            start.append(start[-1] + n)
        self.table, self.max_new, self.max_kv = table, max(new), max(lens)
        self.start = torch.tensor(start, dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")


def reference(layer, x, residual, lens):
    """The same layer without FP8, in 32 bits, over whole sequences."""
    h = x.float() + residual.float()
    n = h * (h.square().mean(1, keepdim=True) + NORM_EPS).rsqrt() * layer.norm.float()
    heads = (n @ layer.w_qkv.float().T).view(x.shape[0], -1, layer.dim)
    q, k, v = heads.split([layer.q_heads, layer.kv_heads, layer.kv_heads], 1)
    out, at = [], 0
    for length in lens:
        kk, vv = (t[at:at + length].repeat_interleave(layer.q_heads // layer.kv_heads, 1).transpose(0, 1).contiguous() for t in (k, v))
        z = q[at:at + length].transpose(0, 1) @ kk.transpose(1, 2).contiguous() * layer.dim ** -0.5
        z = z.masked_fill(torch.ones(length, length, device=z.device).triu(1).bool(), -math.inf)
        out.append((z.softmax(-1) @ vv).transpose(0, 1).reshape(length, -1))
        at += length
    return torch.cat(out) @ layer.w_out.float().T


def main(hidden=1024, q_heads=8, kv_heads=2, dim=128, page=16, lens=(70, 5, 33), steps=3, seed=1):
    """Relative error (2-norm) of the prompts' and the steps' outputs against the 32-bit layer."""
    g = torch.Generator().manual_seed(seed)
    layer = Attention(hidden, q_heads, kv_heads, dim)
    total = [n + steps for n in lens]
    width = -(-max(total) // page)
    cache = Cache(len(lens) * width, kv_heads, page, dim)
    table = torch.randperm(len(lens) * width, generator=g).to(torch.int32).view(len(lens), width).cuda()
    x = torch.randn(sum(total), hidden, generator=g).bfloat16().cuda()
    res = torch.randn(sum(total), hidden, generator=g).bfloat16().cuda()
    first = torch.tensor([0] + total).cumsum(0).tolist()
    rows = [torch.arange(first[b], first[b] + lens[b]) for b in range(len(lens))]
    got = torch.empty_like(x)
    prompt = torch.cat(rows).cuda()
    got[prompt], h = layer(x[prompt], res[prompt], cache, Plan(table, list(lens), list(lens)))
    for t in range(steps):
        at = torch.tensor([first[b] + lens[b] + t for b in range(len(lens))]).cuda()
        got[at], _ = layer(x[at], res[at], cache, Plan(table, [1] * len(lens), [n + t + 1 for n in lens]))
    want = reference(layer, x, res, total)
    step = torch.ones(len(x), dtype=torch.bool, device="cuda")
    step[prompt] = False
    errors = [float((got[i].float() - want[i]).norm() / want[i].norm()) for i in (prompt, step)]
    # the norm's gradient, as a training step takes it
    dy, dx, dw = torch.randn_like(h), torch.empty_like(h), torch.empty(hidden, device="cuda")
    rstd = (h.float().square().mean(1) + NORM_EPS).rsqrt()
    rt.fp8_rmsnorm_backward(dy, h, layer.norm, rstd, dx, dw, dresidual=dy)
    torch.cuda.synchronize()
    return errors


if __name__ == "__main__":
    prompt_error, step_error = main()
    print("relative error against the layer in 32 bits: prompts %.3f, single tokens %.3f" % (prompt_error, step_error))
