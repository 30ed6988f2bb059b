// norm.hip -- root-mean-square norm with the residual's addition and an FP8
// output (the next scaled GEMM's operand), and its gradient.
//
// With h = x + residual, c = (mean h^2 + e)^(-1/2):  y_j = h_j w_j c.  Since
// binary32 multiplication by c >= 0 is monotonic, max_j |y_j| is exactly
// fl(c max_j |h_j w_j|): the sum of squares and the row's maximum are one
// reduction round, and no element is visited twice before the cast.
// The gradient, from dy_i/dh_j = w_i c (1[i = j] - c^2 h_i h_j / cols):
//   dh_j = c (g_j - n_j mean_k(g_k n_k)),  g = dy w, n = h c;   dw_j = sum_rows dy_j n_j.
//
// Both are bound by HBM: the forward moves x, residual, h and one byte of code per element,
// the gradient dy, h, the residual's gradient and dx.  Up to 16384 columns a row stays in registers between its
// reduction and its use (fp32 rows of the forward spill 2 of them); workgroups loop over rows, the forward up to 16384
// and the gradient up to 8192 columns with the next
// row's loads in flight, since one row a workgroup leaves the memory idle during its reduction.  Above 16384
// columns a thread holds 4 octets, of which 32 to 46 registers (forward) and 78 to 93 (gradient) spill.
// Measured at 4096 x 8192 bf16 with residual: forward 45 us (5.2 TB/s), gradient 48 + 4 us for
// dweight's shares (5.3 TB/s); a device copy of as many bytes reaches 4.7 to 5.2.  4096 x 16384: 89 us (5.3 TB/s) and
// 109 (4.9); 4096 x 32768: 241 (3.9) and 499 (2.2).  8189 x 7168 in 1x128
// groups: 93 us (4.4 TB/s), the groups' scales (two exact quotients per group) taking the rest.  One
// row of 8192: 4.1 us, launch and one chain of loads and reductions.
#include <algorithm>

#include "device_common.h"
#include "internal.h"

namespace fp8rt {

namespace {

constexpr int kMaxWaves = 16;

// 8 weights from column c, fp32 or bf16.
__device__ __forceinline__ void load_weight(const void* w, int wt, int64_t c, float* out) {
  if (wt == FP8RT_BF16) {
    Octet<uint16_t> o;
    o.load(static_cast<const uint16_t*>(w) + c);
    widen(o, out);
  } else {
    Octet<float> o;
    o.load(static_cast<const float*>(w) + c);
    widen(o, out);
  }
}

// Sum of s and maximum of the bit patterns m over a row's threads, the same in
// all of them: L lanes of a wave (a power of two), or the workgroup (L = 0).  `sh`
// holds one pair per wave; the caller alternates two of them, so one barrier per round is enough.
__device__ __forceinline__ void row_sum_max(float& s, uint32_t& m, float2* sh, int L) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    if (L && o >= L) continue;
    s += __shfl_xor(s, o);
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), o)));
  }
  const int nw = blockDim.x >> 6;
  if (L || nw == 1) return;
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = make_float2(s, __uint_as_float(m));
  __syncthreads();
  s = 0.0f;
  m = 0;
  for (int i = 0; i < nw; ++i) {
    s += sh[i].x;
    m = max(m, __float_as_uint(sh[i].y));
  }
}

// How rows are laid over threads (chosen on the host, see shape_for): a row is L
// lanes of a wave, or the whole workgroup (L = 0).
struct RowShape {
  int L;
  int64_t rows_at_once;  // rows of the grid in one round
};

// ---------------------------------------------------------------------------
// Forward.  Thread t of a row holds octets t, t + threads, ... (NV of them) and their
// weights, over all rows of its workgroup; the next row's loads are in flight during this
// row's reduction and cast.
template <typename T, int F, int NV>
__global__ void __launch_bounds__(1024) k_rmsnorm_quantize(NormArgs a, RowShape shape, BlockPartial* part) {
  __shared__ float2 sh[2][kMaxWaves];
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.res);
  T* hp = static_cast<T*>(a.h);
  const int L = shape.L, per = L ? L : blockDim.x;  // threads of a row
  const int tr = L ? threadIdx.x & (L - 1) : threadIdx.x;
  const int octets = static_cast<int>(a.cols >> 3);
  const int64_t ng = (a.cols + a.ec - 1) / a.ec;
  const bool tensor = a.er != 1, rowwise = !tensor && a.ec == a.cols;
  const int seg = rowwise || tensor ? 0 : static_cast<int>(a.ec >> 3);  // lanes per group
  const float inv_cols = 1.0f / static_cast<float>(a.cols);
  const int64_t row0 = L ? (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) / L : blockIdx.x;
  const int64_t last = a.rows - 1;
  constexpr bool kHold = NV <= 2;  // weights held, the next row fetched early: 4 octets would spill
  float w[NV][8];
  auto weights = [&] {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int o = v * per + tr;
      load_weight(a.w, a.wt, (o < octets ? o : 0) * 8, w[v]);
    }
  };
  if (kHold) weights();
  Octet<T> xo[NV], ro[NV];
  auto load = [&](int64_t row) {  // (rows past the end load the last one again)
    const int64_t r = row < last ? row : last;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int o = v * per + tr;
      const int oc = o < octets ? o : 0;
      xo[v].load_nt(x + r * a.ldx + oc * 8);
      if (res) ro[v].load_nt(res + r * a.ldr + oc * 8);
    }
  };
  uint32_t seen = 0;  // tensor groups: max |y| of this thread's rows
  int round = 0;
  if (kHold) load(row0);
  // (the same number of rounds for every thread of a workgroup: rows are reduced together)
  for (int64_t base = 0; base < a.rows; base += shape.rows_at_once, round ^= 1) {
    const int64_t row = base + row0;
    const bool on = row < a.rows;
    if (!kHold) load(row);
    float h[NV][8];
    uint32_t om[NV];  // max |h w| of each octet
    float ss = 0.0f;
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const bool in = v * per + tr < octets;
      xo[v].keep_if(in);
      widen(xo[v], h[v]);
      if (res) {
        ro[v].keep_if(in);
        float r[8];
        widen(ro[v], r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[v][i] += r[i];
      }
    }
    if (kHold && base + shape.rows_at_once < a.rows) load(row + shape.rows_at_once);
    if (!kHold) weights();
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int o = v * per + tr;
      const bool in = o < octets;
      if (hp && in && on) store8(hp + row * a.ldh + o * 8, h[v]);
      om[v] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss += h[v][i] * h[v][i];
        h[v][i] *= w[v][i];  // from here on h * w
        om[v] = max(om[v], __float_as_uint(h[v][i]) & kAbsMask);
      }
      if (!in) om[v] = 0;  // (0 * a weight that is not finite)
      m = max(m, om[v]);
    }
    row_sum_max(ss, m, sh[round], L);
    const float rstd = 1.0f / sqrtf(ss * inv_cols + a.norm_eps);
    const bool first = tr == 0 && on;
    if (a.rstd && first) a.rstd[row] = rstd;
    const float row_amax = __uint_as_float(__float_as_uint(__uint_as_float(m) * rstd) & kAbsMask);
    if (on) seen = max(seen, __float_as_uint(row_amax));
    float s = 0.0f, r = 0.0f;
    if (!seg) {
      const int64_t g = tensor || !on ? 0 : row;
      if (a.mode == FP8RT_DYNAMIC) {
        scale_from_amax(row_amax, Fmt<F>::kMax, a.eps, a.pow2 != 0, s, r);
        if (first) {
          a.scale[g] = s;
          if (a.inv_scale) a.inv_scale[g] = r;
        }
      } else {
        r = a.inv_scale ? a.inv_scale[g] : 1.0f / a.scale[g];
      }
      if (!tensor && a.amax_out && first) a.amax_out[g] = row_amax;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int o = v * per + tr;
      const bool in = o < octets && on;
      if (seg) {
        uint32_t gm = om[v];
        for (int d = seg >> 1; d >= 1; d >>= 1)
          gm = max(gm, static_cast<uint32_t>(__shfl_xor(static_cast<int>(gm), d)));
        gm = __float_as_uint(__uint_as_float(gm) * rstd) & kAbsMask;  // = max |y|, as for a row
        const int64_t g = in ? row * ng + o / seg : 0;
        const bool lead = in && (o & (seg - 1)) == 0;
        if (a.mode == FP8RT_DYNAMIC) {
          scale_from_amax(__uint_as_float(gm), Fmt<F>::kMax, a.eps, a.pow2 != 0, s, r);
          if (lead) {
            a.scale[g] = s;
            if (a.inv_scale) a.inv_scale[g] = r;
          }
        } else {
          r = a.inv_scale ? a.inv_scale[g] : 1.0f / a.scale[g];
        }
        if (a.amax_out && lead) a.amax_out[g] = __uint_as_float(gm);
      }
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = h[v][i] * rstd * r;
      u32x2 c;
      if (a.mode == FP8RT_DYNAMIC) {  // a value that is not finite has made r NaN, and all codes with it
        c = u32x2{cvt4<F>(y[0], y[1], y[2], y[3]), cvt4<F>(y[4], y[5], y[6], y[7])};
        if (__builtin_isnan(r)) c = u32x2{0x7F7F7F7Fu, 0x7F7F7F7Fu};
      } else {
        c = u32x2{cvt4_nan<F>(y[0], y[1], y[2], y[3]), cvt4_nan<F>(y[4], y[5], y[6], y[7])};
      }
      if (in) *reinterpret_cast<u32x2*>(a.q + row * a.ldq + o * 8) = c;
    }
  }
  if (part) {
    float none = 0.0f;
    __syncthreads();
    row_sum_max(none, seen, sh[0], 0);
    if (threadIdx.x == 0) part[blockIdx.x] = BlockPartial{seen, 0u, 0u, 0u};
  }
}

// ---------------------------------------------------------------------------
// Gradient.  The same layout; a thread keeps its columns' share of dweight in
// registers over all its rows; rows side by side (L > 0) are added at the end, so that a
// workgroup writes one share of dweight.
template <typename T, typename H, int NV>
__global__ void __launch_bounds__(1024) k_rmsnorm_backward(NormGradArgs a, RowShape shape, float* dw_part) {
  __shared__ float2 sh[2][kMaxWaves];
  const T* dy = static_cast<const T*>(a.dy);
  const T* dres = static_cast<const T*>(a.dres);
  const H* hp = static_cast<const H*>(a.h);
  T* dx = static_cast<T*>(a.dx);
  const int L = shape.L, per = L ? L : blockDim.x;
  const int tr = L ? threadIdx.x & (L - 1) : threadIdx.x;
  const int octets = static_cast<int>(a.cols >> 3);
  const float inv_cols = 1.0f / static_cast<float>(a.cols);
  const int64_t row0 = L ? (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) / L : blockIdx.x;
  const int64_t last = a.rows - 1;
  constexpr bool kHold = NV == 1;  // as in the forward; dweight's sums take the registers of one octet
  float w[NV][8];
  auto weights = [&] {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int o = v * per + tr;
      load_weight(a.w, a.wt, (o < octets ? o : 0) * 8, w[v]);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[v][i] = o < octets ? w[v][i] : 0.0f;  // (0 * a weight that is not finite)
    }
  };
  if (kHold) weights();
  Octet<T> go[NV], ro[NV];
  Octet<H> ho[NV];
  float cn;
  auto load = [&](int64_t row) {
    const int64_t r = row < last ? row : last;
    cn = a.rstd[r];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int o = v * per + tr;
      const int oc = o < octets ? o : 0;
      go[v].load_nt(dy + r * a.lddy + oc * 8);
      ho[v].load_nt(hp + r * a.ldh + oc * 8);
      if (kHold && dres) ro[v].load_nt(dres + r * a.lddr + oc * 8);
    }
  };
  float dw[NV][8] = {};
  int round = 0;
  if (kHold) load(row0);
  for (int64_t base = 0; base < a.rows; base += shape.rows_at_once, round ^= 1) {
    const int64_t row = base + row0;
    const bool on = row < a.rows;
    if (!kHold) load(row);
    const float c = cn;
    float g[NV][8], n[NV][8];
    Octet<T> rs[NV];
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const bool in = v * per + tr < octets && on;
      go[v].keep_if(in);
      ho[v].keep_if(in);
      widen(go[v], g[v]);
      widen(ho[v], n[v]);
      if (kHold && dres) rs[v] = ro[v];
    }
    if (kHold && base + shape.rows_at_once < a.rows) load(row + shape.rows_at_once);
    if (!kHold) weights();
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const bool in = v * per + tr < octets && on;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n[v][i] = in ? n[v][i] * c : 0.0f;  // (0 * NaN outside the row)
        dw[v][i] += g[v][i] * n[v][i];
        g[v][i] *= w[v][i];
        dot += g[v][i] * n[v][i];
      }
    }
    uint32_t none = 0;
    row_sum_max(dot, none, sh[round], L);
    const float mean = dot * inv_cols;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int o = v * per + tr;
      if (o < octets && on) {
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = c * (g[v][i] - n[v][i] * mean);
        if (dres) {
          if (!kHold) rs[v].load_nt(dres + row * a.lddr + o * 8);
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] += rs[v].get(i);
        }
        store8(dx + row * a.lddx + o * 8, d);
      }
    }
  }
  if (!dw_part) return;
  float* share = dw_part + int64_t(blockIdx.x) * a.cols;
  if (L) {  // (NV = 1, 4 waves, cols <= 512)
    __shared__ __align__(16) float side[4][512];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      for (int d = L; d < 64; d <<= 1) dw[0][i] += __shfl_xor(dw[0][i], d);
    if (static_cast<int>(threadIdx.x & 63) < L && tr < octets) store8(&side[threadIdx.x >> 6][tr * 8], dw[0]);
    __syncthreads();
    for (int64_t c = threadIdx.x; c < a.cols; c += 256) share[c] = (side[0][c] + side[1][c]) + (side[2][c] + side[3][c]);
    return;
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int o = v * per + tr;
    if (o < octets) store8(share + o * 8, dw[v]);
  }
}

// dweight[j] = sum of the n shares in a fixed order: 16 slices of the shares for 64
// columns in one workgroup, several loads of 4 columns in flight, joined through LDS.
__global__ void __launch_bounds__(256) k_dweight_sum(const float* part, int n, int64_t cols, float* dw) {
  __shared__ __align__(16) float4 sh[16][16];
  const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
  const int64_t c = int64_t(blockIdx.x) * 64 + 4 * x;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c < cols) {
#pragma unroll 8
    for (int i = y; i < n; i += 16) {
      const float4 v = *reinterpret_cast<const float4*>(part + i * cols + c);
      s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
    }
  }
  sh[y][x] = s;
  __syncthreads();
  if (y == 0 && c < cols) {
    s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 16; ++i) s = make_float4(s.x + sh[i][x].x, s.y + sh[i][x].y, s.z + sh[i][x].z, s.w + sh[i][x].w);
    *reinterpret_cast<float4*>(dw + c) = s;
  }
}

// The layout of rows over threads.
//  - Up to 512 columns: a power of two of lanes a row, several rows a workgroup.
//  - Few rows (under 2 a CU): one octet a thread, the shortest chain.
//  - Many rows: nv_many octets a thread, looped over by threads_per_cu threads a CU.  Measured at
//    4096 x 8192 bf16 with residual, us for 1 / 2 / 4 octets: forward 59 / 49 / 74 with 1024 threads a
//    CU, 61 / 49 / 80 with 2048; gradient 53 / 101 / 302 (2 octets leave no registers for the next row, 4 spill) with
//    512, 56 / 107 / 280 with 2048.  One workgroup a row, no loop: 69 and 65.
struct Launch {
  RowShape shape;
  int nv, threads;
  int64_t grid;
};
Launch shape_for(int64_t rows, int64_t cols, int nv_many, int threads_per_cu) {
  const int64_t octets = cols >> 3;
  Launch g;
  if (octets <= 64) {
    int L = 2;
    while (L < octets) L <<= 1;
    g.nv = 1;
    g.threads = 256;
    g.grid = std::min<int64_t>(ceil_div(rows * L, 256), int64_t(device_cus()) * (threads_per_cu / 256));
    g.shape = RowShape{L, g.grid * (256 / L)};
    return g;
  }
  g.nv = rows >= 2 * device_cus() ? nv_many : 1;
  while (octets > int64_t(1024) * g.nv) g.nv <<= 1;
  g.threads = static_cast<int>(ceil_div(ceil_div(octets, g.nv), 64) * 64);
  g.grid = std::min<int64_t>(rows, int64_t(device_cus()) * std::max(1, threads_per_cu / g.threads));
  g.shape = RowShape{0, g.grid};
  return g;
}

}  // namespace

hipError_t launch_rmsnorm_quantize(const NormArgs& a, hipStream_t st) {
  const Launch g = shape_for(a.rows, a.cols, 2, 1024);
  const bool partials = a.er != 1 && a.amax_out;
  BlockPartial* part = nullptr;
  if (partials) {
    DevWorkspace* ws = nullptr;
    const hipError_t e = get_workspace(st, &ws);
    if (e != hipSuccess) return e;
    part = ws->pass2;  // (at most kMaxBlocks: shape_for's grids are a few per CU)
  }
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(g.grid), dim3(g.threads), 0, st, a, g.shape, part); };
  auto by_nv = [&](auto tag) {
    using T = decltype(tag);
    if (a.fmt == FP8RT_E4M3)
      g.nv == 1 ? go(k_rmsnorm_quantize<T, kE4M3, 1>) : g.nv == 2 ? go(k_rmsnorm_quantize<T, kE4M3, 2>)
                                                                 : go(k_rmsnorm_quantize<T, kE4M3, 4>);
    else
      g.nv == 1 ? go(k_rmsnorm_quantize<T, kE5M2, 1>) : g.nv == 2 ? go(k_rmsnorm_quantize<T, kE5M2, 2>)
                                                                 : go(k_rmsnorm_quantize<T, kE5M2, 4>);
  };
  if (a.xt == FP8RT_BF16)
    by_nv(uint16_t{});
  else
    by_nv(float{});
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && partials) e = launch_finish(part, static_cast<int>(g.grid), a.amax_out, nullptr, st);
  return e;
}

hipError_t launch_rmsnorm_backward(const NormGradArgs& a, hipStream_t st) {
  const Launch g = shape_for(a.rows, a.cols, 1, 512);  // (each workgroup costs a share of dweight)
  const int shares = static_cast<int>(g.grid);
  void* part = nullptr;
  if (a.dw) {
    const hipError_t e = get_scratch(st, size_t(shares) * a.cols * sizeof(float), &part);
    if (e != hipSuccess) return e;
  }
  float* dwp = static_cast<float*>(part);
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(g.grid), dim3(g.threads), 0, st, a, g.shape, dwp); };
  auto by_nv = [&](auto t, auto h) {
    using T = decltype(t);
    using H = decltype(h);
    g.nv == 1 ? go(k_rmsnorm_backward<T, H, 1>)
              : g.nv == 2 ? go(k_rmsnorm_backward<T, H, 2>) : go(k_rmsnorm_backward<T, H, 4>);
  };
  if (a.dyt == FP8RT_BF16)
    a.ht == FP8RT_BF16 ? by_nv(uint16_t{}, uint16_t{}) : by_nv(uint16_t{}, float{});
  else
    a.ht == FP8RT_BF16 ? by_nv(float{}, uint16_t{}) : by_nv(float{}, float{});
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && a.dw) {
    hipLaunchKernelGGL(k_dweight_sum, dim3(ceil_div(a.cols, 64)), dim3(256), 0, st, dwp, shares, a.cols, a.dw);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace fp8rt
