// gated.hip -- gated activation with an FP8 output and an 8-bit checkpoint of its
// input, and its gradient from that checkpoint.
//
//   z = act(g) u,  act(g) = g c,  c = 1 / (1 + e^-v);  v = g (SiLU) or 2 sqrt(2/pi) (g + 0.044715 g^3) (GELU's tanh form)
//   dz/du = g c,   dz/dg = u (c + g c (1 - c) dv/dg)
//
// Bound by memory: bf16 reads 4 bytes and writes 1 for each of z's values, 2 more with the checkpoint; the gradient
// reads 4 and writes 4, 2 more with z.  Measured: 4096 rows of 29568 columns, one scale a row, 106 us (5.7 TB/s); 8189 of
// 7168 in groups of 128 with the checkpoint 92 us (4.5 TB/s: three exact scales and three casts for each 128 columns
// keep the vector units as busy as the memory) and the gradient with z 98 (6.0 TB/s).  One scale a row beside the checkpoint:
// 4096 of 16384 columns 82 to 95 us (4.9 to 5.7 TB/s), of 29568 209 (4.1), 2048 of 65536 377 (2.5: see k_gated_rows); fp32 rows
// without it 230 (4.7) and 291 (4.2), with it 286 for 29568 (4.7), and its gradient 460 (4.7).
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "internal.h"

namespace fp8rt {

namespace {

constexpr int kMaxWaves = 16;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kGeluA = 1.5957691216057307f;  // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// c of a gate: 1 / (1 + 2^(-v log2 e)).  The product is rounded before the exponential, which costs |v| u, v itself is
// rounded in up to 4 operations, and the hardware's exponential and reciprocal are off by 1 ulp each: (6 |v| + 16) u in all, for
// values that are next rounded to 8 bits or by a gradient's casts.  The reciprocal gives 0 for a c below 2^-126 (v below -87.3).
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

// Maximum over aligned runs of n lanes (a power of two up to 64): within 16 lanes by DPP operands (quad_perm, then
// mirrors, which pair the runs' halves), beyond them through LDS.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t m) {
  return max(m, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), CTRL, 0xF, 0xF, true)));
}
__device__ __forceinline__ uint32_t run_max(uint32_t m, int n) {
  if (n >= 2) m = dpp_max<0xB1>(m);   // quad_perm 1 0 3 2
  if (n >= 4) m = dpp_max<0x4E>(m);   // quad_perm 2 3 0 1
  if (n >= 8) m = dpp_max<0x141>(m);  // row_half_mirror
  if (n >= 16) m = dpp_max<0x140>(m);  // row_mirror
  if (n >= 32) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16)));
  if (n >= 64) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
  return m;
}

// The value of lane K of the lane's quad, or pair.
template <int K>
__device__ __forceinline__ float quad(float v) {
  return __uint_as_float(__builtin_amdgcn_mov_dpp(static_cast<int>(__float_as_uint(v)), K * 0x55, 0xF, 0xF, true));
}
template <int K>
__device__ __forceinline__ float pair(float v) {  // quad_perm K K K+2 K+2
  return __uint_as_float(__builtin_amdgcn_mov_dpp(static_cast<int>(__float_as_uint(v)), K * 0x55 + 0xA0, 0xF, 0xF, true));
}

// Codes of 8 values under the multiplier that their own group's maximum gave: no product passes F_max by more
// than its rounding, which the cast's own takes back, so nothing is clamped; a value that is not finite has made r NaN.
template <int F>
__device__ __forceinline__ u32x2 codes8(const float* v, float r) {
  u32x2 c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float* x = v + 4 * h;
    int w;
    if constexpr (F == kE4M3) {
      w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * r, x[1] * r, 0, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * r, x[3] * r, w, true);
    } else {
      w = __builtin_amdgcn_cvt_pk_bf8_f32(x[0] * r, x[1] * r, 0, false);
      w = __builtin_amdgcn_cvt_pk_bf8_f32(x[2] * r, x[3] * r, w, true);
    }
    c[h] = __builtin_isnan(r) ? 0x7F7F7F7Fu : static_cast<uint32_t>(w);
  }
  return c;
}

constexpr int kKeptRun = kKeptGroup / 8;  // lanes of a checkpoint's group

__device__ __forceinline__ void store_kept(const GatedArgs& a, const float* v, float r, int64_t row, int half, int o) {
  *reinterpret_cast<u32x2*>(a.kept + row * a.ldk + half * a.cols + o * 8) =
      a.kf == FP8RT_E4M3 ? codes8<kE4M3>(v, r) : codes8<kE5M2>(v, r);
}
__device__ __forceinline__ float* kept_scale_at(const GatedArgs& a, int64_t row, int half, int o) {
  return a.kept_scale + (row * 2 + half) * ((a.cols + kKeptGroup - 1) / kKeptGroup) + o / kKeptRun;
}

// z of 8 columns, 0 outside the row (selects on the loaded words: a condition on z became a branch for each
// element).
template <typename T, int ACT>
__device__ __forceinline__ void gated8(Octet<T>& go, Octet<T>& uo, bool in, float* g, float* u, float* z) {
  go.keep_if(in);
  uo.keep_if(in);
  widen(go, g);
  widen(uo, u);
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = g[i] * gate_c<ACT>(g[i]) * u[i];
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

// Octets of a chunk of a row, where few rows are cut into chunks.
constexpr uint32_t kChunk = 512;

// Groups inside a row, or one given scale for all: no row has to be held.  A workgroup takes `rows_per` rows or a chunk of
// one, a thread an octet at a time; `opad`, the octets of a row rounded up to whole runs, keeps a group's lanes in line.
template <typename T, int F, int ACT, bool KEPT>
__global__ void __launch_bounds__(256) k_gated_groups(GatedArgs a, int rows_per, FastDiv opad, FastDiv chunks, BlockPartial* part) {
  const T* x = static_cast<const T*>(a.x);
  const uint32_t block = chunks.div(blockIdx.x), chunk = blockIdx.x - block * chunks.d;
  const int64_t row0 = int64_t(block) * rows_per, live = live_rows(a);
  const int octets = static_cast<int>(a.cols >> 3);
  const bool tensor = a.er != 1;
  const int seg = tensor ? 1 : static_cast<int>(a.ec >> 3);
  const int64_t ng = (a.cols + a.ec - 1) / a.ec;
  const int64_t left = live - row0;
  const uint32_t all = left <= 0 ? 0u : static_cast<uint32_t>(left < rows_per ? left : rows_per) * opad.d;
  const uint32_t n = min(all, chunks.d > 1 ? (chunk + 1) * kChunk : all);  // this workgroup's octets end here
  uint32_t seen = 0;
  struct Place {  // octet o of row row0 + rr
    uint32_t rr;
    int o;
  };
  auto place = [&](uint32_t base) {
    const uint32_t i = min(base + threadIdx.x, n - 1), rr = opad.div(i);
    return Place{rr, static_cast<int>(i - rr * opad.d)};
  };
  Octet<T> go, uo;
  auto load = [&](const Place& p) {
    const T* at = x + (row0 + p.rr) * a.ldx + (p.o < octets ? p.o : 0) * 8;
    go.load_nt(at);
    uo.load_nt(at + a.cols);
  };
  Place p{0, 0};
  const uint32_t first = chunk * kChunk;
  if (first < n) load(p = place(first));
  for (uint32_t base = first; base < n; base += 256) {
    const int o = p.o;
    const bool in = o < octets && base + threadIdx.x < n;
    const int64_t row = row0 + p.rr;
    Octet<T> gc = go, uc = uo;
    if (base + 256 < n) load(p = place(base + 256));  // in flight during this octet's work
    float gv[8], uv[8], z[8];
    gated8<T, ACT>(gc, uc, in, gv, uv, z);
    const uint32_t m = run_max(absmax8(z), seg);
    seen = max(seen, m);
    const int64_t g = tensor ? 0 : row * ng + (o < octets ? o / seg : 0);
    const bool lead = !tensor && in && (o & (seg - 1)) == 0;
    float r;
    if constexpr (KEPT) {
      // Three scales, of which a lane works out one and hands it to its quad (exact quotients are what this kernel's
      // vector units spend most on): lanes 0 and 1 the checkpoint's, the others the output's.
      const uint32_t mg = run_max(gc.absmax_bits(), kKeptRun), mu = run_max(uc.absmax_bits(), kKeptRun);
      const int k = threadIdx.x & 3;
      const bool shared = seg >= 4 && a.mode == FP8RT_DYNAMIC;
      float s, rr;
      scale_from_amax(__uint_as_float(k == 0 ? mg : k == 1 ? mu : m), k < 2 ? fmax_of(a.kf) : Fmt<F>::kMax, a.eps,
                      k >= 2 && a.pow2 != 0, s, rr);
      if (in && (o & (kKeptRun - 1)) < 2) *kept_scale_at(a, row, k, o) = s;
      const float rg = quad<0>(rr), ru = quad<1>(rr);
      if (in) {
        store_kept(a, gv, rg, row, 0, o);
        store_kept(a, uv, ru, row, 1, o);
      }
      if (shared) {
        s = quad<2>(s);
        r = quad<2>(rr);
        if (lead) {
          a.scale[g] = s;
          if (a.inv_scale) a.inv_scale[g] = r;
          if (a.amax_out) a.amax_out[g] = __uint_as_float(m);
        }
      } else {
        r = group_scale<F>(a, m, g, lead);
      }
    } else {
      r = group_scale<F>(a, m, g, lead);
    }
    if (in) store_codes<F>(a, z, r, row, o);
  }
  if (part) block_stats_store<4>(reinterpret_cast<u32x4*>(&part[blockIdx.x]), seen, 0u, 0u);
}

// One scale a row: z stays in registers between the row's maximum and its cast, with the next row's loads in flight.  A row
// is L lanes of a wave (a power of two), or the whole workgroup (L = 0); a thread holds octets t, t + threads, ... (NV of
// them).  1024 threads leave 128 registers each.  What is left over goes to scratch memory: 18 of them for bf16 rows of 4 octets
// with a checkpoint (past 16384 columns), 79 to 93 for 8 octets with one (past 32768), 34 for fp32 rows of 8 octets without.
template <typename T, int F, int ACT, int NV, bool KEPT>
__global__ void __launch_bounds__(1024) k_gated_rows(GatedArgs a, int lanes_per_row, int64_t rows_at_once) {
  __shared__ uint32_t sh[2][kMaxWaves];
  const int L = NV == 1 ? lanes_per_row : 0;  // (several octets a thread: always the whole workgroup, rows uniform)
  const T* x = static_cast<const T*>(a.x);
  const int per = L ? L : blockDim.x;
  const int tr = L ? threadIdx.x & (L - 1) : threadIdx.x;
  const int octets = static_cast<int>(a.cols >> 3);
  const int64_t live = live_rows(a);
  if (live == 0) return;
  const int64_t row0 = L ? (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) / L : blockIdx.x;
  const int lanes = L && L < kKeptRun ? L : kKeptRun;
  constexpr bool kHold = NV * sizeof(T) <= 8;  // (more loads in flight than that would only be spilled)
  Octet<T> go[NV], uo[NV];
  auto load = [&](int64_t row) {  // (rows past the end load the last one again)
    const T* gp = x + (row < live ? row : live - 1) * a.ldx;
    const T* up = gp + a.cols;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const uint32_t o = v * per + tr;
      const uint32_t oc = o < static_cast<uint32_t>(octets) ? o * 8 : 0;
      go[v].load_nt(gp + oc);
      uo[v].load_nt(up + oc);
    }
  };
  if (kHold) load(row0);
  int round = 0;
  // (the same number of rounds for every thread of a workgroup: rows are reduced together)
  for (int64_t base = 0; base < live; base += rows_at_once, round ^= 1) {
    const int64_t row = base + row0;
    const bool on = row < live;
    if (!kHold) load(row);
    float z[NV][8];
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int o = v * per + tr;
      if constexpr (NV >= 4 && sizeof(T) == 2) asm volatile("" : "+v"(go[v].raw), "+v"(uo[v].raw));
      const bool in = on && o < octets;
      float gv[8], uv[8];
      gated8<T, ACT>(go[v], uo[v], in, gv, uv, z[v]);
      m = max(m, absmax8(z[v]));
      if constexpr (KEPT) {  // even lanes work out the gates' scale, odd ones the ups'
        const uint32_t mg = run_max(go[v].absmax_bits(), lanes), mu = run_max(uo[v].absmax_bits(), lanes);
        float s, r;
        scale_from_amax(__uint_as_float(threadIdx.x & 1 ? mu : mg), fmax_of(a.kf), a.eps, false, s, r);
        const float rg = pair<0>(r), ru = pair<1>(r);  // (the smallest rows are two lanes)
        if (in) {
          if ((o & (kKeptRun - 1)) < 2) *kept_scale_at(a, row, threadIdx.x & 1, o) = s;
          store_kept(a, gv, rg, row, 0, o);
          store_kept(a, uv, ru, row, 1, o);
        }
      }
      if (NV >= 4) __builtin_amdgcn_sched_barrier(0);  // one octet's temporaries at a time: else they spill
    }
    if (kHold && base + rows_at_once < live) load(row + rows_at_once);
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
    const float r = group_scale<F>(a, m, on ? row : 0, tr == 0 && on);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int o = v * per + tr;
      if (on && o < octets) store_codes<F>(a, z[v], r, row, o);
    }
  }
}

// Gradient: 8 columns a thread, nothing shared between threads.
template <typename T, int KF, int ACT>
__global__ void __launch_bounds__(256) k_gated_backward(GatedArgs a, int rows_per, FastDiv octets, FastDiv chunks) {
  const T* dz = static_cast<const T*>(a.x);
  T* dx = static_cast<T*>(a.dx);
  T* zp = static_cast<T*>(a.z);
  const uint32_t block = chunks.div(blockIdx.x), chunk = blockIdx.x - block * chunks.d;
  const int64_t row0 = int64_t(block) * rows_per, live = live_rows(a);
  const int64_t left = live - row0;
  const uint32_t all = left <= 0 ? 0u : static_cast<uint32_t>(left < rows_per ? left : rows_per) * octets.d;
  const uint32_t n = min(all, chunks.d > 1 ? (chunk + 1) * kChunk : all);
  const int64_t ng = (a.cols + kKeptGroup - 1) / kKeptGroup;
  struct Piece {
    int64_t row;
    uint32_t c;
    u32x2 g, u;
    Octet<T> d;
    float sg, su;
  };
  auto load = [&](uint32_t i) {
    Piece p;
    const uint32_t rr = octets.div(i);
    p.row = row0 + rr;
    p.c = (i - rr * octets.d) * 8;
    const uint8_t* kp = a.kept + p.row * a.ldk + p.c;
    p.g = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(kp));
    p.u = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(kp + a.cols));
    p.d.load_nt(dz + p.row * a.ldx + p.c);
    const float* s = a.kept_scale + p.row * 2 * ng + p.c / kKeptGroup;
    p.sg = s[0];
    p.su = s[ng];
    return p;
  };
  Piece next;
  const uint32_t first = chunk * kChunk + threadIdx.x;
  if (first < n) next = load(first);
  for (uint32_t i = first; i < n; i += 256) {
    const Piece p = next;
    if (i + 256 < n) next = load(i + 256);  // in flight during this piece's work
    float g[8], u[8], dg[8], du[8], z[8];
    decode4<KF>(p.g[0], g);
    decode4<KF>(p.g[1], g + 4);
    decode4<KF>(p.u[0], u);
    decode4<KF>(p.u[1], u + 4);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float gv = g[k] * p.sg, uv = u[k] * p.su, dv = p.d.get(k);
      const float cc = gate_c<ACT>(gv);
      const float f = gv * cc;
      float t = f * (1.0f - cc);  // g c (1 - c) dv/dg: 0 where c has reached 0 or 1, whatever dv/dg
      if constexpr (ACT == FP8RT_GELU) t = t == 0.0f ? 0.0f : t * (kGeluA * (1.0f + 3.0f * kGeluB * (gv * gv)));
      z[k] = f * uv;
      du[k] = dv * f;
      dg[k] = dv * uv * (cc + t);
    }
    T* out = dx + p.row * a.lddx + p.c;
    store8(out, dg);
    store8(out + a.cols, du);
    if (zp) store8(zp + p.row * a.ldz + p.c, z);
  }
}

// Chunks that each row is cut into: few rows otherwise leave CUs idle (54 rows of 23776 columns in groups
// of 128: 6.2 us, whole rows 15.4).
int row_chunks(int64_t rows, int64_t rows_per, int64_t octets) {
  const int64_t chunks = ceil_div(octets, kChunk);
  return rows_per == 1 && rows < 4 * device_cus() && rows * chunks <= kMaxBlocks ? static_cast<int>(chunks) : 1;
}

// Calls f with the types of a call: input, format, activation, checkpoint.
template <typename Fn>
void by_kind(const GatedArgs& a, Fn&& f) {
  using std::integral_constant;
  auto by_kept = [&](auto t, auto fmt, auto act) { a.kept ? f(t, fmt, act, std::true_type{}) : f(t, fmt, act, std::false_type{}); };
  auto by_act = [&](auto t, auto fmt) {
    a.act == FP8RT_SILU ? by_kept(t, fmt, integral_constant<int, FP8RT_SILU>{})
                        : by_kept(t, fmt, integral_constant<int, FP8RT_GELU>{});
  };
  auto by_fmt = [&](auto t) {
    a.fmt == FP8RT_E4M3 ? by_act(t, integral_constant<int, kE4M3>{}) : by_act(t, integral_constant<int, kE5M2>{});
  };
  a.xt == FP8RT_BF16 ? by_fmt(uint16_t{}) : by_fmt(float{});
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
      nv = a.rows < 2 * device_cus() ? 1 : a.kept || a.xt == FP8RT_F32 ? 2 : 4;
      while (octets > int64_t(1024) * nv) nv <<= 1;
      threads = static_cast<int>(ceil_div(ceil_div(octets, nv), 64) * 64);
      grid = at_once = std::min<int64_t>(a.rows, int64_t(device_cus()) * std::max(1, 1024 / threads));
    }
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(grid), dim3(threads), 0, st, a, L, at_once); };
    auto by_nv = [&](auto t, auto f, auto act, auto kept) {
      using T = decltype(t);
      constexpr int F = decltype(f)::value, A = decltype(act)::value;
      constexpr bool K = decltype(kept)::value;
      switch (nv) {
        case 1: go(k_gated_rows<T, F, A, 1, K>); break;
        case 2: go(k_gated_rows<T, F, A, 2, K>); break;
        case 4: go(k_gated_rows<T, F, A, 4, K>); break;
        default: go(k_gated_rows<T, F, A, 8, K>); break;
      }
    };
    by_kind(a, by_nv);
    return hipGetLastError();
  }
  BlockPartial* part = nullptr;
  if (partials) {
    DevWorkspace* ws = nullptr;
    const hipError_t e = get_workspace(st, &ws);
    if (e != hipSuccess) return e;
    part = ws->pass2;
  }
  const int64_t run = std::max<int64_t>(a.er == 1 ? a.ec >> 3 : 1, kKeptRun);
  const int64_t opad = ceil_div(octets, run) * run;
  // about four octets a thread; at most kMaxBlocks workgroups, one partial each (opad <= 8192 and
  // rows_per <= 2^18 keep a workgroup's count of octets in 32 bits)
  const int64_t rows_per = std::max(ceil_div(1024, opad), ceil_div(a.rows, kMaxBlocks));
  const int chunks = row_chunks(a.rows, rows_per, opad);
  const dim3 grid(static_cast<unsigned>(ceil_div(a.rows, rows_per) * chunks));
  by_kind(a, [&](auto t, auto f, auto act, auto kept) {
    hipLaunchKernelGGL((k_gated_groups<decltype(t), decltype(f)::value, decltype(act)::value, decltype(kept)::value>), grid,
                       dim3(256), 0, st, a, static_cast<int>(rows_per), FastDiv(static_cast<uint32_t>(opad)),
                       FastDiv(static_cast<uint32_t>(chunks)), part);
  });
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && partials) e = launch_finish(part, static_cast<int>(grid.x), a.amax_out, nullptr, st);
  return e;
}

hipError_t launch_gated_backward(const GatedArgs& a, hipStream_t st) {
  const int64_t octets = a.cols >> 3;
  // about two octets a thread; at most 2^20 workgroups (of at most 2^11 rows of 2^13 octets)
  const int64_t rows_per = std::max(ceil_div(512, octets), ceil_div(a.rows, int64_t(1) << 20));
  const int chunks = row_chunks(a.rows, rows_per, octets);
  const dim3 grid(static_cast<unsigned>(ceil_div(a.rows, rows_per) * chunks));
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, dim3(256), 0, st, a, static_cast<int>(rows_per), FastDiv(static_cast<uint32_t>(octets)),
                       FastDiv(static_cast<uint32_t>(chunks)));
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
