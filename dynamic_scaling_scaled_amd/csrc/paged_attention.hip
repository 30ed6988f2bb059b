// paged_attention.hip -- attention over a paged cache of FP8 codes with one
// scale for each page and head.
//
// One wave per query and head: each lane scores one of 64 positions, the
// softmax's running maximum and sum are joined over the wave, and each lane
// then adds its share of the head's dimensions for all 64.
#include "paged_common.h"

namespace fp8rt {

namespace {

template <int F, int D>
__global__ void __launch_bounds__(64) k_attend(AttendArgs a, int64_t grid_n) {
  constexpr int E = D / 64;  // dimensions of one lane
  __shared__ float qs[D];
  const int lane = threadIdx.x;
  const int64_t b = blockIdx.x / grid_n;
  const int64_t i = blockIdx.x % grid_n;
  const int64_t h = blockIdx.y;
  const SeqSpan s = seq_span(a.p, b);
  if (i >= s.n) return;
  const int64_t tok = s.tok0 + i, at = s.first + i;
  const int head = static_cast<int>(h / (a.q_heads / a.p.heads));
  const int page = a.p.page;
  for (int e = 0; e < E; ++e) {
    const int d = lane * E + e;
    qs[d] = __uint_as_float(static_cast<uint32_t>(a.q[tok * a.ldq + h * a.hdq + d]) << 16);
  }
  __syncthreads();
  int64_t lo = 0, hi = s.len;
  if (a.causal && at + 1 < hi) hi = at + 1;
  if (a.window > 0 && at - a.window + 1 > 0) lo = at - a.window + 1;
  float m = -INFINITY, l = 0.0f, y[E] = {};
  for (int64_t j0 = lo / 16 * 16; j0 < hi; j0 += 64) {
    const int64_t j = j0 + lane;
    const bool inside = j >= lo && j < hi;
    const int32_t pg = inside ? page_of(a.p, b, j / page) : -1;
    const bool seen = pg >= 0;
    float z = -INFINITY, vs = 0.0f;
    if (seen) {
      const uint32_t* k = reinterpret_cast<const uint32_t*>(
          a.kc + ((int64_t(pg) * a.p.heads + head) * page + j % page) * D);
      float dot = 0.0f;
      for (int d = 0; d < D; d += 4) {
        float v[4];
        decode4<F>(k[d / 4], v);
        for (int t = 0; t < 4; ++t) dot += v[t] * qs[d + t];
      }
      z = dot * a.ks[int64_t(pg) * a.p.heads + head] * a.sm_scale;
      vs = a.vs[int64_t(pg) * a.p.heads + head];
    }
    float mt = z;
    for (int o = 32; o >= 1; o >>= 1) mt = fmaxf(mt, __shfl_xor(mt, o));
    const float mn = fmaxf(m, mt);
    const float base = mn == -INFINITY ? 0.0f : mn;
    const float fade = expf(m - base);
    const float p = expf(z - base);
    float sum = p;
    for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
    l = l * fade + sum;
    m = mn;
    for (int e = 0; e < E; ++e) y[e] *= fade;
    for (int t = 0; t < 64; ++t) {
      const int32_t pt = __shfl(pg, t);
      if (pt < 0) continue;
      const float w = __shfl(p, t) * __shfl(vs, t);
      const uint8_t* v = a.vc + ((int64_t(pt) * a.p.heads + head) * page + (j0 + t) % page) * D + lane * E;
      for (int e = 0; e < E; ++e) {
        float x[4];
        decode4<F>(v[e], x);
        y[e] += w * x[0];
      }
    }
  }
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
  for (int e = 0; e < E; ++e) {
    const __bf16 r = static_cast<__bf16>(y[e] * inv);
    a.y[tok * a.ldy + h * a.hdy + lane * E + e] = __builtin_bit_cast(uint16_t, r);
  }
  if (a.lse && lane == 0) a.lse[tok * a.q_heads + h] = l != 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace

hipError_t launch_paged_attention(const AttendArgs& a, hipStream_t st) {
  const int64_t gx = a.p.seqs * a.p.max_new;
  if (gx >= (int64_t(1) << 26)) return hipErrorInvalidValue;
  const dim3 grid(static_cast<uint32_t>(gx), static_cast<uint32_t>(a.q_heads));
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, dim3(64), 0, st, a, a.p.max_new); };
  if (a.p.fmt == FP8RT_E4M3)
    a.p.dim == 128 ? go(k_attend<kE4M3, 128>) : go(k_attend<kE4M3, 64>);
  else
    a.p.dim == 128 ? go(k_attend<kE5M2, 128>) : go(k_attend<kE5M2, 64>);
  return hipGetLastError();
}

}  // namespace fp8rt
