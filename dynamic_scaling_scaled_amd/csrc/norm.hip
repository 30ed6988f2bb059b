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
// the gradient dy, h, the residual's gradient and dx.  A row stays in
// registers between its reduction and its use, so every element is read once.
#include "device_common.h"
#include "internal.h"

namespace fp8rt {

namespace {

constexpr int kMaxWaves = 16;

template <typename T>
__device__ __forceinline__ void widen(const Octet<T>& o, float* out) {
#pragma unroll
  for (int i = 0; i < 8; ++i) out[i] = o.get(i);
}

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

// Two binary32 values rounded to nearest even onto bf16 (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x2 v;
  v[0] = static_cast<__bf16>(a);
  v[1] = static_cast<__bf16>(b);
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
  *reinterpret_cast<u32x4*>(p) =
      u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  u32x4 a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = __float_as_uint(v[i]);
    b[i] = __float_as_uint(v[i + 4]);
  }
  reinterpret_cast<u32x4*>(p)[0] = a;
  reinterpret_cast<u32x4*>(p)[1] = b;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Block-wide sum of s and maximum of the bit patterns m, the same in every
// thread.  `sh` holds one pair per wave; the caller alternates two of them, so
// one barrier per round is enough.
__device__ __forceinline__ void block_sum_max(float& s, uint32_t& m, float2* sh) {
  s = wave_sum(s);
  m = wave_max_u32(m);
  const int nw = blockDim.x >> 6;
  if (nw == 1) return;
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = make_float2(s, __uint_as_float(m));
  __syncthreads();
  s = 0.0f;
  m = 0;
  for (int i = 0; i < nw; ++i) {
    s += sh[i].x;
    m = max(m, __float_as_uint(sh[i].y));
  }
}

// ---------------------------------------------------------------------------
// Forward.  One workgroup per row at a time; thread t holds octets t, t +
// blockDim, ... (NV of them).
template <typename T, int F, int NV>
__global__ void __launch_bounds__(1024) k_rmsnorm_quantize(NormArgs a, BlockPartial* part) {
  __shared__ float2 sh[2][kMaxWaves];
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.res);
  T* hp = static_cast<T*>(a.h);
  const int octets = static_cast<int>(a.cols >> 3);
  const int64_t ng = (a.cols + a.ec - 1) / a.ec;
  const bool tensor = a.er != 1, rowwise = !tensor && a.ec == a.cols;
  const int seg = rowwise || tensor ? 0 : static_cast<int>(a.ec >> 3);  // lanes per group
  const float inv_cols = 1.0f / static_cast<float>(a.cols);
  uint32_t seen = 0;  // tensor groups: max |y| of this workgroup's rows
  int round = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, round ^= 1) {
    float h[NV][8];
    Octet<T> xo[NV], ro[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int o = v * blockDim.x + threadIdx.x;
      const int oc = o < octets ? o : 0;
      xo[v].load_nt(x + row * a.ldx + oc * 8);
      if (res) ro[v].load_nt(res + row * a.ldr + oc * 8);
    }
    float ss = 0.0f;
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int o = v * blockDim.x + threadIdx.x;
      const bool in = o < octets;
      xo[v].keep_if(in);
      widen(xo[v], h[v]);
      if (res) {
        ro[v].keep_if(in);
        float r[8];
        widen(ro[v], r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[v][i] += r[i];
      }
      if (hp && in) store8(hp + row * a.ldh + o * 8, h[v]);
      float w[8];
      load_weight(a.w, a.wt, (in ? o : 0) * 8, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss += h[v][i] * h[v][i];
        h[v][i] *= w[i];  // from here on h * w
        m = max(m, in ? __float_as_uint(h[v][i]) & kAbsMask : 0u);
      }
    }
    block_sum_max(ss, m, sh[round]);
    const float rstd = 1.0f / sqrtf(ss * inv_cols + a.norm_eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    const float row_amax = __uint_as_float(m) * rstd;
    seen = max(seen, __float_as_uint(row_amax) & kAbsMask);
    float s = 0.0f, r = 0.0f;
    if (!seg) {
      const int64_t g = tensor ? 0 : row;
      if (a.mode == FP8RT_DYNAMIC) {
        scale_from_amax(row_amax, Fmt<F>::kMax, a.eps, a.pow2 != 0, s, r);
        if (threadIdx.x == 0) {
          a.scale[g] = s;
          if (a.inv_scale) a.inv_scale[g] = r;
        }
      } else {
        r = a.inv_scale ? a.inv_scale[g] : 1.0f / a.scale[g];
      }
      if (!tensor && a.amax_out && threadIdx.x == 0) a.amax_out[g] = __uint_as_float(__float_as_uint(row_amax) & kAbsMask);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int o = v * blockDim.x + threadIdx.x;
      const bool in = o < octets;
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = h[v][i] * rstd;
      if (seg) {
        uint32_t gm = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) gm = max(gm, in ? __float_as_uint(y[i]) & kAbsMask : 0u);
        for (int d = seg >> 1; d >= 1; d >>= 1)
          gm = max(gm, static_cast<uint32_t>(__shfl_xor(static_cast<int>(gm), d)));
        const int64_t g = row * ng + (in ? o : 0) / seg;
        const bool first = in && (o & (seg - 1)) == 0;
        if (a.mode == FP8RT_DYNAMIC) {
          scale_from_amax(__uint_as_float(gm), Fmt<F>::kMax, a.eps, a.pow2 != 0, s, r);
          if (first) {
            a.scale[g] = s;
            if (a.inv_scale) a.inv_scale[g] = r;
          }
        } else {
          r = a.inv_scale ? a.inv_scale[g] : 1.0f / a.scale[g];
        }
        if (a.amax_out && first) a.amax_out[g] = __uint_as_float(gm);
      }
      if (in) {
        const u32x2 c = u32x2{cvt4_nan<F>(y[0] * r, y[1] * r, y[2] * r, y[3] * r),
                              cvt4_nan<F>(y[4] * r, y[5] * r, y[6] * r, y[7] * r)};
        *reinterpret_cast<u32x2*>(a.q + row * a.ldq + o * 8) = c;
      }
    }
  }
  if (part && threadIdx.x == 0) part[blockIdx.x] = BlockPartial{seen, 0u, 0u, 0u};
}

// ---------------------------------------------------------------------------
// Gradient.  Workgroup b takes rows b, b + gridDim, ...; a thread keeps its
// columns' share of dweight in registers over all its rows and writes it once.
template <typename T, typename H, int NV>
__global__ void __launch_bounds__(1024) k_rmsnorm_backward(NormGradArgs a, float* dw_part) {
  __shared__ float2 sh[2][kMaxWaves];
  const T* dy = static_cast<const T*>(a.dy);
  const T* dres = static_cast<const T*>(a.dres);
  const H* hp = static_cast<const H*>(a.h);
  T* dx = static_cast<T*>(a.dx);
  const int octets = static_cast<int>(a.cols >> 3);
  const float inv_cols = 1.0f / static_cast<float>(a.cols);
  float dw[NV][8] = {};
  int round = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, round ^= 1) {
    const float c = a.rstd[row];
    float g[NV][8], n[NV][8];
    Octet<T> go[NV];
    Octet<H> ho[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int o = v * blockDim.x + threadIdx.x;
      const int oc = o < octets ? o : 0;
      go[v].load_nt(dy + row * a.lddy + oc * 8);
      ho[v].load_nt(hp + row * a.ldh + oc * 8);
    }
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int o = v * blockDim.x + threadIdx.x;
      go[v].keep_if(o < octets);
      ho[v].keep_if(o < octets);
      widen(go[v], g[v]);
      widen(ho[v], n[v]);
      float w[8];
      load_weight(a.w, a.wt, (o < octets ? o : 0) * 8, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n[v][i] = o < octets ? n[v][i] * c : 0.0f;  // (0 * NaN outside the row)
        dw[v][i] += g[v][i] * n[v][i];
        g[v][i] *= w[i];
        dot += g[v][i] * n[v][i];
      }
    }
    uint32_t none = 0;
    block_sum_max(dot, none, sh[round]);
    const float mean = dot * inv_cols;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int o = v * blockDim.x + threadIdx.x;
      if (o < octets) {
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = c * (g[v][i] - n[v][i] * mean);
        if (dres) {
          Octet<T> ro;
          ro.load_nt(dres + row * a.lddr + o * 8);
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] += ro.get(i);
        }
        store8(dx + row * a.lddx + o * 8, d);
      }
    }
  }
  if (dw_part) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int o = v * blockDim.x + threadIdx.x;
      if (o < octets) store8(dw_part + int64_t(blockIdx.x) * a.cols + o * 8, dw[v]);
    }
  }
}

// dweight[j] = sum of the workgroups' shares in their order: 16 slices of the
// parts per column in one workgroup, joined through LDS.
__global__ void __launch_bounds__(1024) k_dweight_sum(const float* part, int n, int64_t cols, float* dw) {
  __shared__ float sh[16][64];
  const int64_t c = int64_t(blockIdx.x) * 64 + threadIdx.x;
  float s = 0.0f;
  if (c < cols)
    for (int i = threadIdx.y; i < n; i += 16) s += part[i * cols + c];
  sh[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < cols) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += sh[i][threadIdx.x];
    dw[c] = s;
  }
}

// Threads for `octets` octets at nv a thread: whole waves, at most 1024.
int threads_for(int64_t octets, int nv) { return static_cast<int>(ceil_div(ceil_div(octets, nv), 64) * 64); }

}  // namespace

hipError_t launch_rmsnorm_quantize(const NormArgs& a, hipStream_t st) {
  const int64_t octets = a.cols >> 3;
  const int nv = octets <= 1024 ? 1 : octets <= 2048 ? 2 : 4;
  const int threads = threads_for(octets, nv);
  const bool partials = a.er != 1 && a.amax_out;
  BlockPartial* part = nullptr;
  int64_t grid = a.rows;
  if (partials) {
    DevWorkspace* ws = nullptr;
    const hipError_t e = get_workspace(st, &ws);
    if (e != hipSuccess) return e;
    part = ws->pass2;
  }
  if (grid > kMaxBlocks) grid = kMaxBlocks;
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(grid), dim3(threads), 0, st, a, part); };
  auto by_nv = [&](auto tag) {
    using T = decltype(tag);
    if (a.fmt == FP8RT_E4M3)
      nv == 1 ? go(k_rmsnorm_quantize<T, kE4M3, 1>) : nv == 2 ? go(k_rmsnorm_quantize<T, kE4M3, 2>)
                                                               : go(k_rmsnorm_quantize<T, kE4M3, 4>);
    else
      nv == 1 ? go(k_rmsnorm_quantize<T, kE5M2, 1>) : nv == 2 ? go(k_rmsnorm_quantize<T, kE5M2, 2>)
                                                               : go(k_rmsnorm_quantize<T, kE5M2, 4>);
  };
  if (a.xt == FP8RT_BF16)
    by_nv(uint16_t{});
  else
    by_nv(float{});
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && partials) e = launch_finish(part, static_cast<int>(grid), a.amax_out, nullptr, st);
  return e;
}

hipError_t launch_rmsnorm_backward(const NormGradArgs& a, hipStream_t st) {
  const int64_t octets = a.cols >> 3;
  const int nv = octets <= 1024 ? 1 : octets <= 2048 ? 2 : 4;
  const int threads = threads_for(octets, nv);
  int64_t grid = a.rows < 512 ? a.rows : 512;
  void* part = nullptr;
  if (a.dw) {
    const hipError_t e = get_scratch(st, size_t(grid) * a.cols * sizeof(float), &part);
    if (e != hipSuccess) return e;
  }
  float* dwp = static_cast<float*>(part);
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(grid), dim3(threads), 0, st, a, dwp); };
  auto by_nv = [&](auto t, auto h) {
    using T = decltype(t);
    using H = decltype(h);
    nv == 1 ? go(k_rmsnorm_backward<T, H, 1>) : nv == 2 ? go(k_rmsnorm_backward<T, H, 2>) : go(k_rmsnorm_backward<T, H, 4>);
  };
  if (a.dyt == FP8RT_BF16)
    a.ht == FP8RT_BF16 ? by_nv(uint16_t{}, uint16_t{}) : by_nv(uint16_t{}, float{});
  else
    a.ht == FP8RT_BF16 ? by_nv(float{}, uint16_t{}) : by_nv(float{}, float{});
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && a.dw) {
    hipLaunchKernelGGL(k_dweight_sum, dim3(ceil_div(a.cols, 64)), dim3(64, 16), 0, st, dwp, static_cast<int>(grid),
                       a.cols, a.dw);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace fp8rt
