// kv_append.hip -- new keys and values into a paged FP8 cache with one scale
// for each page and head.
//
// A page and head that receives tokens is one wave's work: the maximum over
// what it receives, the scale (that of the page's earlier tokens if it is
// larger), the earlier tokens' codes again if the scale grew, the new codes.
// Bound by HBM for prompts (2 or 4 bytes read, 1 written per element; five ragged prompts of
// together 11.8 thousand tokens, 8 heads of 128, pages of 16: 16 to 18 us, 4.0 to 4.6 TB/s), by launch and two
// dependent loads for single tokens (64 sequences: 4.1 us).  A wave needs no barrier, and a page of up to 32 tokens
// (64 at 64 dimensions) is read once.
#include "paged_common.h"

namespace fp8rt {

namespace {

constexpr int kWaves = 4;

template <typename T, int F, int D>
__global__ void __launch_bounds__(64 * kWaves) k_kv_append(AppendArgs a, FastDiv pages_per_seq) {
  constexpr int L = D / 8;         // lanes of one token (an octet each)
  constexpr int kTok = 64 / L;     // tokens of one wave instruction
  const int lane = threadIdx.x & 63;
  const uint32_t b = pages_per_seq.div(blockIdx.x);
  const int pi = blockIdx.x - b * pages_per_seq.d;
  const int item = blockIdx.y * kWaves + (threadIdx.x >> 6);  // head, then keys / values
  if (item >= 2 * a.p.heads) return;
  const bool val = item >= a.p.heads;
  const int head = val ? item - a.p.heads : item;
  const SeqSpan s = seq_span(a.p, b);
  const int page = a.p.page, shift = 31 - __builtin_clz(page);
  // positions [lo, hi) of the new tokens that exist, then of those in this page
  int64_t lo = s.first > 0 ? s.first : 0, hi = s.first + s.n < s.len ? s.first + s.n : s.len;
  if (lo >= hi) return;
  const int64_t lp = (lo >> shift) + pi;
  const int64_t p0 = lp << shift;
  const int64_t before = lo;  // positions below it were there before this call
  lo = lo > p0 ? lo : p0;
  hi = hi < p0 + page ? hi : p0 + page;
  if (lo >= hi) return;
  const int32_t pg = page_of(a.p, b, lp);
  if (pg < 0) return;
  const int fill = before > p0 ? static_cast<int>(before - p0) : 0;  // earlier tokens of this page
  const int n = static_cast<int>(hi - lo);
  const T* src = static_cast<const T*>(val ? a.v : a.k);
  const int64_t ld = val ? a.ldv : a.ldk, hd = val ? a.hdv : a.hdk;
  src += (s.tok0 + (lo - s.first)) * ld + head * hd + (lane % L) * 8;
  uint8_t* dst = (val ? a.vc : a.kc) + ((int64_t(pg) * a.p.heads + head) * page) * D;
  float* scp = (val ? a.vs : a.ks) + int64_t(pg) * a.p.heads + head;
  const int t0 = lane / L;

  // the first kHeld octets of a lane (32 tokens at D = 128, 64 at D = 64) stay in registers,
  // what a larger page brings beyond them is read again, from the cache
  constexpr int kHeld = 8;
  Octet<T> held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int t = t0 + i * kTok;
    held[i].load(src + (t < n ? t : 0) * ld);  // (the maximum does not mind the first token again)
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) m = max(m, held[i].absmax_bits());
  for (int t = t0 + kHeld * kTok; t < n; t += kTok) {
    Octet<T> o;
    o.load(src + t * ld);
    m = max(m, o.absmax_bits());
  }
  m = wave_max_u32(m);
  float sc, r;
  scale_from_amax(__uint_as_float(m), Fmt<F>::kMax, a.eps, a.pow2 != 0, sc, r);
  if (fill > 0) {
    const float old = *scp;
    if (!(sc >= old) && !__builtin_isnan(sc)) {  // the page's scale stays (NaN stays NaN)
      sc = old;
      r = 1.0f / old;
    } else if (sc != old) {  // it grew: the earlier tokens' codes again
      const float again = old / sc;
      for (int t = t0; t < fill; t += kTok) {
        u32x2* p = reinterpret_cast<u32x2*>(dst + t * D + (lane % L) * 8);
        u32x2 c = *p;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float v[4];
          decode4<F>(c[i], v);
          c[i] = cvt4_nan<F>(v[0] * again, v[1] * again, v[2] * again, v[3] * again);
        }
        *p = c;
      }
    }
  }
  if (lane == 0) *scp = sc;
  const int slot = static_cast<int>(lo - p0);
  auto put = [&](const Octet<T>& o, int t) {
    const u32x2 c = u32x2{cvt4_nan<F>(o.get(0) * r, o.get(1) * r, o.get(2) * r, o.get(3) * r),
                          cvt4_nan<F>(o.get(4) * r, o.get(5) * r, o.get(6) * r, o.get(7) * r)};
    *reinterpret_cast<u32x2*>(dst + (slot + t) * D + (lane % L) * 8) = c;
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (t0 + i * kTok < n) put(held[i], t0 + i * kTok);
  for (int t = t0 + kHeld * kTok; t < n; t += kTok) {
    Octet<T> o;
    o.load(src + t * ld);
    put(o, t);
  }
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs& a, hipStream_t st) {
  const int per = static_cast<int>((a.p.max_new + a.p.page - 2) / a.p.page + 1);  // pages that max_new tokens can touch
  const int64_t gx = a.p.seqs * per;
  const dim3 grid(static_cast<uint32_t>(gx), static_cast<uint32_t>(ceil_div(2 * a.p.heads, kWaves)));
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, dim3(64 * kWaves), 0, st, a, FastDiv(per)); };
  auto by_fmt = [&](auto tag) {
    using T = decltype(tag);
    if (a.p.fmt == FP8RT_E4M3)
      a.p.dim == 128 ? go(k_kv_append<T, kE4M3, 128>) : go(k_kv_append<T, kE4M3, 64>);
    else
      a.p.dim == 128 ? go(k_kv_append<T, kE5M2, 128>) : go(k_kv_append<T, kE5M2, 64>);
  };
  if (a.xt == FP8RT_BF16)
    by_fmt(uint16_t{});
  else
    by_fmt(float{});
  return hipGetLastError();
}

}  // namespace fp8rt
