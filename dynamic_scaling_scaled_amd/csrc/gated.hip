// gated.hip -- gated activation with an FP8 output and an 8-bit checkpoint of its
// input, and its gradient from that checkpoint.
//
//   z = act(g) u,  act(g) = g c,  c = 1 / (1 + e^-v);  v = g (SiLU) or 2 sqrt(2/pi) (g + 0.044715 g^3) (GELU's tanh form)
//   dz/du = g c,   dz/dg = u (c + g c (1 - c) dv/dg)
#include <algorithm>

#include "device_common.h"
#include "internal.h"

namespace fp8rt {

namespace {

constexpr int kMaxWaves = 16;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kGeluA = 1.5957691216057307f;  // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// c of a gate: 1 / (1 + 2^(-v log2 e)).  The hardware's exponential and reciprocal (1 ulp each); an
// overflowing exponential gives c = 0.
template <int ACT>
__device__ __forceinline__ float gate_c(float g) {
  float v = g;
  if constexpr (ACT == FP8RT_GELU) v = kGeluA * (g + kGeluB * (g * g * g));
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * v));
}

// Rows that count.
__device__ __forceinline__ int64_t live_rows(const GatedArgs& a) {
  if (!a.live) return a.rows;
  const int64_t n = a.live[0];
  return n < 0 ? 0 : n < a.rows ? n : a.rows;
}

// Maximum over aligned runs of n lanes (a power of two up to 64).
__device__ __forceinline__ uint32_t run_max(uint32_t m, int n) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1)
    if (d < n) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), d)));
  return m;
}

template <int F>
__device__ __forceinline__ u32x2 codes8(const float* v, float r) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = v[i] * r;
  const u32x2 c = u32x2{cvt4<F>(y[0], y[1], y[2], y[3]), cvt4<F>(y[4], y[5], y[6], y[7])};
  return __builtin_isnan(r) ? u32x2{0x7F7F7F7Fu, 0x7F7F7F7Fu} : c;  // a value that is not finite has made r NaN
}

// The checkpoint of 8 columns of one half: groups of 128 columns are runs of 16 lanes (`lanes`, fewer
// when a row has fewer).
template <typename T>
__device__ __forceinline__ void keep8(const GatedArgs& a, const Octet<T>& x, const float* v, int64_t row, int half, int o,
                                      bool in, int lanes) {
  float s, r;
  scale_from_amax(__uint_as_float(run_max(in ? x.absmax_bits() : 0u, lanes)), fmax_of(a.kf), a.eps, false, s, r);
  if (!in) return;
  const u32x2 c = a.kf == FP8RT_E4M3 ? codes8<kE4M3>(v, r) : codes8<kE5M2>(v, r);
  *reinterpret_cast<u32x2*>(a.kept + row * a.ldk + half * a.cols + o * 8) = c;
  constexpr int kRun = kKeptGroup / 8;
  if ((o & (kRun - 1)) == 0) a.kept_scale[(row * 2 + half) * ((a.cols + kKeptGroup - 1) / kKeptGroup) + o / kRun] = s;
}

// z of 8 columns, with their checkpoint.
template <typename T, int ACT>
__device__ __forceinline__ void gated8(const GatedArgs& a, const Octet<T>& go, const Octet<T>& uo, int64_t row, int o,
                                       bool in, int lanes, float* z) {
  float g[8], u[8];
  widen(go, g);
  widen(uo, u);
  if (a.kept) {
    keep8(a, go, g, row, 0, o, in, lanes);
    keep8(a, uo, u, row, 1, o, in, lanes);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = in ? g[i] * gate_c<ACT>(g[i]) * u[i] : 0.0f;
}

__device__ __forceinline__ uint32_t absmax8(const float* z) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(z[i]) & kAbsMask);
  return m;
}

template <int F>
__device__ __forceinline__ void store_codes(const GatedArgs& a, const float* z, float r, int64_t row, int o) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = z[i] * r;
  *reinterpret_cast<u32x2*>(a.q + row * a.ldq + o * 8) =
      a.mode == FP8RT_DYNAMIC ? codes8<F>(z, r)
                              : u32x2{cvt4_nan<F>(y[0], y[1], y[2], y[3]), cvt4_nan<F>(y[4], y[5], y[6], y[7])};
}

// Scale of group g with maximum m: its multiplier, written out by the lane that leads.
template <int F>
__device__ __forceinline__ float group_scale(const GatedArgs& a, uint32_t m, int64_t g, bool lead) {
  float s, r;
  if (a.mode == FP8RT_DYNAMIC) {
    scale_from_amax(__uint_as_float(m), Fmt<F>::kMax, a.eps, a.pow2 != 0, s, r);
    if (lead) {
      a.scale[g] = s;
      if (a.inv_scale) a.inv_scale[g] = r;
    }
  } else {
    r = a.inv_scale ? a.inv_scale[g] : 1.0f / a.scale[g];
  }
  if (a.amax_out && lead && a.er == 1) a.amax_out[g] = __uint_as_float(m);
  return r;
}

// Groups inside a row, or one given scale for all: no row has to be held.  A workgroup takes `rows_per` rows, a thread
// an octet of one of them at a time; `opad`, the octets of a row rounded up to whole runs, keeps a group's lanes in line.
template <typename T, int F, int ACT>
__global__ void __launch_bounds__(256) k_gated_groups(GatedArgs a, int rows_per, FastDiv opad, BlockPartial* part) {
  const T* x = static_cast<const T*>(a.x);
  const int64_t row0 = int64_t(blockIdx.x) * rows_per, live = live_rows(a);
  const int octets = static_cast<int>(a.cols >> 3);
  const bool tensor = a.er != 1;
  const int seg = tensor ? 1 : static_cast<int>(a.ec >> 3);
  const int64_t ng = (a.cols + a.ec - 1) / a.ec;
  const int64_t left = live - row0;
  const uint32_t n = left <= 0 ? 0u : static_cast<uint32_t>(left < rows_per ? left : rows_per) * opad.d;
  uint32_t seen = 0;
  for (uint32_t base = 0; base < n; base += 256) {
    const uint32_t i = min(base + threadIdx.x, n - 1);
    const uint32_t rr = opad.div(i);
    const int o = static_cast<int>(i - rr * opad.d);
    const bool in = o < octets && base + threadIdx.x < n;
    const int64_t row = row0 + rr;
    const int oc = o < octets ? o : 0;
    Octet<T> go, uo;
    go.load_nt(x + row * a.ldx + oc * 8);
    uo.load_nt(x + row * a.ldx + a.cols + oc * 8);
    float z[8];
    gated8<T, ACT>(a, go, uo, row, o, in, kKeptGroup / 8, z);
    const uint32_t m = run_max(absmax8(z), seg);
    seen = max(seen, m);
    const int64_t g = tensor ? 0 : row * ng + oc / seg;
    const float r = group_scale<F>(a, m, g, !tensor && in && (o & (seg - 1)) == 0);
    if (in) store_codes<F>(a, z, r, row, o);
  }
  if (part) block_stats_store<4>(reinterpret_cast<u32x4*>(&part[blockIdx.x]), seen, 0u, 0u);
}

// One scale a row: z stays in registers between the row's maximum and its cast.  A row is L lanes of a wave (a power of
// two), or the whole workgroup (L = 0); a thread holds octets t, t + threads, ... (NV of them).
template <typename T, int F, int ACT, int NV>
__global__ void __launch_bounds__(1024) k_gated_rows(GatedArgs a, int L, int64_t rows_at_once) {
  __shared__ uint32_t sh[2][kMaxWaves];
  const T* x = static_cast<const T*>(a.x);
  const int per = L ? L : blockDim.x;
  const int tr = L ? threadIdx.x & (L - 1) : threadIdx.x;
  const int octets = static_cast<int>(a.cols >> 3);
  const int64_t live = live_rows(a);
  const int64_t row0 = L ? (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) / L : blockIdx.x;
  const int lanes = L && L < kKeptGroup / 8 ? L : kKeptGroup / 8;
  int round = 0;
  // (the same number of rounds for every thread of a workgroup: rows are reduced together)
  for (int64_t base = 0; base < live; base += rows_at_once, round ^= 1) {
    const int64_t row = base + row0;
    const bool on = row < live;
    const int64_t rc = on ? row : live - 1;
    Octet<T> go[NV], uo[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int o = v * per + tr;
      const int oc = o < octets ? o : 0;
      go[v].load_nt(x + rc * a.ldx + oc * 8);
      uo[v].load_nt(x + rc * a.ldx + a.cols + oc * 8);
    }
    float z[NV][8];
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int o = v * per + tr;
      gated8<T, ACT>(a, go[v], uo[v], rc, o, on && o < octets, lanes, z[v]);
      m = max(m, absmax8(z[v]));
    }
    if (L) {
      m = run_max(m, L);
    } else {
      m = wave_max_u32(m);
      if (blockDim.x > 64) {
        if ((threadIdx.x & 63) == 0) sh[round][threadIdx.x >> 6] = m;
        __syncthreads();
        for (int i = 0; i < static_cast<int>(blockDim.x >> 6); ++i) m = max(m, sh[round][i]);
      }
    }
    const float r = group_scale<F>(a, m, rc, tr == 0 && on);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int o = v * per + tr;
      if (on && o < octets) store_codes<F>(a, z[v], r, row, o);
    }
  }
}

// Gradient: 16 columns a thread, nothing shared between threads.
template <typename T, int KF, int ACT>
__global__ void __launch_bounds__(256) k_gated_backward(GatedArgs a, int rows_per, FastDiv per_row) {
  const T* dz = static_cast<const T*>(a.x);
  T* dx = static_cast<T*>(a.dx);
  T* zp = static_cast<T*>(a.z);
  const int64_t row0 = int64_t(blockIdx.x) * rows_per, live = live_rows(a);
  const int64_t left = live - row0;
  const uint32_t n = left <= 0 ? 0u : static_cast<uint32_t>(left < rows_per ? left : rows_per) * per_row.d;
  const int64_t ng = (a.cols + kKeptGroup - 1) / kKeptGroup;
  for (uint32_t i = threadIdx.x; i < n; i += 256) {
    const uint32_t rr = per_row.div(i);
    const int64_t row = row0 + rr, c = int64_t(i - rr * per_row.d) * 16;
    const uint8_t* kp = a.kept + row * a.ldk + c;
    const u32x4 kg = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(kp));
    const u32x4 ku = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(kp + a.cols));
    Octet<T> d[2];
    d[0].load_nt(dz + row * a.ldx + c);
    d[1].load_nt(dz + row * a.ldx + c + 8);
    const float sg = a.kept_scale[row * 2 * ng + c / kKeptGroup], su = a.kept_scale[(row * 2 + 1) * ng + c / kKeptGroup];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float g[8], u[8], dg[8], du[8], z[8];
      decode4<KF>(kg[2 * h], g);
      decode4<KF>(kg[2 * h + 1], g + 4);
      decode4<KF>(ku[2 * h], u);
      decode4<KF>(ku[2 * h + 1], u + 4);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float gv = g[k] * sg, uv = u[k] * su, dv = d[h].get(k);
        const float cc = gate_c<ACT>(gv);
        const float f = gv * cc;
        float t = f * (1.0f - cc);  // g c (1 - c) dv/dg: 0 where c has reached 0 or 1, whatever dv/dg
        if constexpr (ACT == FP8RT_GELU) t = t == 0.0f ? 0.0f : t * (kGeluA * (1.0f + 3.0f * kGeluB * (gv * gv)));
        z[k] = f * uv;
        du[k] = dv * f;
        dg[k] = dv * uv * (cc + t);
      }
      store8(dx + row * a.lddx + c + 8 * h, dg);
      store8(dx + row * a.lddx + a.cols + c + 8 * h, du);
      if (zp) store8(zp + row * a.ldz + c + 8 * h, z);
    }
  }
}

}  // namespace

hipError_t launch_gated_quantize(const GatedArgs& a, hipStream_t st) {
  const int64_t octets = a.cols >> 3;
  const bool rowwise = a.er == 1 && a.ec == a.cols;
  const bool partials = a.er != 1 && a.amax_out;
  if (rowwise) {
    int L = 0, nv = 1, threads = 256;
    int64_t grid, at_once;
    if (octets <= 64) {
      L = 2;
      while (L < octets) L <<= 1;
      grid = std::min<int64_t>(ceil_div(a.rows * L, 256), int64_t(device_cus()) * 8);
      at_once = grid * (256 / L);
    } else {
      while (octets > int64_t(1024) * nv) nv <<= 1;
      threads = static_cast<int>(ceil_div(ceil_div(octets, nv), 64) * 64);
      grid = at_once = std::min<int64_t>(a.rows, int64_t(device_cus()) * std::max(1, 2048 / threads));
    }
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(grid), dim3(threads), 0, st, a, L, at_once); };
    auto by_nv = [&](auto t, auto f, auto act) {
      using T = decltype(t);
      constexpr int F = decltype(f)::value, A = decltype(act)::value;
      switch (nv) {
        case 1: go(k_gated_rows<T, F, A, 1>); break;
        case 2: go(k_gated_rows<T, F, A, 2>); break;
        case 4: go(k_gated_rows<T, F, A, 4>); break;
        default: go(k_gated_rows<T, F, A, 8>); break;
      }
    };
    auto by_act = [&](auto t, auto f) {
      a.act == FP8RT_SILU ? by_nv(t, f, std::integral_constant<int, FP8RT_SILU>{})
                          : by_nv(t, f, std::integral_constant<int, FP8RT_GELU>{});
    };
    auto by_fmt = [&](auto t) {
      a.fmt == FP8RT_E4M3 ? by_act(t, std::integral_constant<int, kE4M3>{}) : by_act(t, std::integral_constant<int, kE5M2>{});
    };
    a.xt == FP8RT_BF16 ? by_fmt(uint16_t{}) : by_fmt(float{});
    return hipGetLastError();
  }
  BlockPartial* part = nullptr;
  if (partials) {
    DevWorkspace* ws = nullptr;
    const hipError_t e = get_workspace(st, &ws);
    if (e != hipSuccess) return e;
    part = ws->pass2;
  }
  const int64_t run = std::max<int64_t>(a.er == 1 ? a.ec >> 3 : 1, kKeptGroup / 8);
  const int64_t opad = ceil_div(octets, run) * run;
  // about four octets a thread; at most kMaxBlocks workgroups, one partial each (opad <= 8192 and
  // rows_per <= 2^18 rows keep a workgroup's count of octets in 32 bits)
  const int64_t rows_per = std::max(ceil_div(1024, opad), ceil_div(a.rows, kMaxBlocks));
  if (rows_per * opad >= (int64_t(1) << 32)) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(ceil_div(a.rows, rows_per)));
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, dim3(256), 0, st, a, static_cast<int>(rows_per), FastDiv(static_cast<uint32_t>(opad)), part);
  };
  auto by_act = [&](auto t, auto f) {
    using T = decltype(t);
    constexpr int F = decltype(f)::value;
    a.act == FP8RT_SILU ? go(k_gated_groups<T, F, FP8RT_SILU>) : go(k_gated_groups<T, F, FP8RT_GELU>);
  };
  auto by_fmt = [&](auto t) {
    a.fmt == FP8RT_E4M3 ? by_act(t, std::integral_constant<int, kE4M3>{}) : by_act(t, std::integral_constant<int, kE5M2>{});
  };
  a.xt == FP8RT_BF16 ? by_fmt(uint16_t{}) : by_fmt(float{});
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && partials) e = launch_finish(part, static_cast<int>(grid.x), a.amax_out, nullptr, st);
  return e;
}

hipError_t launch_gated_backward(const GatedArgs& a, hipStream_t st) {
  const int64_t per_row = a.cols >> 4;
  // about four pieces a thread; at most 2^20 workgroups
  const int64_t rows_per = std::max(ceil_div(1024, per_row), ceil_div(a.rows, int64_t(1) << 20));
  if (rows_per * per_row >= (int64_t(1) << 32)) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(ceil_div(a.rows, rows_per)));
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, dim3(256), 0, st, a, static_cast<int>(rows_per), FastDiv(static_cast<uint32_t>(per_row)));
  };
  auto by_act = [&](auto t, auto kf) {
    using T = decltype(t);
    constexpr int KF = decltype(kf)::value;
    a.act == FP8RT_SILU ? go(k_gated_backward<T, KF, FP8RT_SILU>) : go(k_gated_backward<T, KF, FP8RT_GELU>);
  };
  auto by_fmt = [&](auto t) {
    a.kf == FP8RT_E4M3 ? by_act(t, std::integral_constant<int, kE4M3>{}) : by_act(t, std::integral_constant<int, kE5M2>{});
  };
  a.xt == FP8RT_BF16 ? by_fmt(uint16_t{}) : by_fmt(float{});
  return hipGetLastError();
}

}  // namespace fp8rt
