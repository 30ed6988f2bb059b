// expert_gemm.hip -- the experts' scaled products: rows of FP8 codes, gathered by the
// router's plan, against each expert's FP8 weights (one fragment-ordered image).
//
//   y[s,n] = s_a(r) s_b(e,n) sum_k dec(a[r,k]) dec(b[e,n,k]),   offsets[e] <= s < offsets[e+1]
#include <algorithm>

#include "device_common.h"
#include "internal.h"

namespace fp8rt {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

// A tile of up to TM consecutive slots of one expert.
struct Tile {
  int expert;
  int64_t row0, end;  // its first slot, the expert's end
};

// Slots [lo, hi) of expert e.
__device__ __forceinline__ void expert_slots(const ExpertGemmArgs& g, int e, int& lo, int& hi) {
  const int top = static_cast<int>(g.slots);
  lo = min(max(g.offsets[e], 0), top);
  hi = max(lo, min(g.offsets[e + 1], top));
}

// Tile `index` of all experts' tiles of TM slots, expert after expert; false past the last.  The whole wave calls
// it with one index.
template <int TM>
__device__ __forceinline__ bool find_tile(const ExpertGemmArgs& g, int index, Tile& t) {
  const int lane = threadIdx.x & 63, E = static_cast<int>(g.experts);
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    int lo = 0, hi = 0;
    if (e < E) expert_slots(g, e, lo, hi);
    const int n = (hi - lo + TM - 1) / TM;
    int s = n;  // inclusive sum over the lanes
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(s, o);
      if (lane >= o) s += up;
    }
    const uint64_t past = __ballot(before + s > index);
    if (past) {
      const int at = __ffsll(static_cast<unsigned long long>(past)) - 1;
      t.expert = e0 + at;
      const int first = before + __builtin_amdgcn_readlane(s, at) - __builtin_amdgcn_readlane(n, at);
      t.row0 = __builtin_amdgcn_readlane(lo, at) + static_cast<int64_t>(index - first) * TM;
      t.end = __builtin_amdgcn_readlane(hi, at);
      return true;
    }
    before += __builtin_amdgcn_readlane(s, 63);
  }
  return false;
}

// The row of a that slot s multiplies, or -1.
__device__ __forceinline__ int64_t row_of(const ExpertGemmArgs& g, const FastDiv& choices, int64_t s) {
  int64_t r = s;
  if (g.order) {
    const int32_t o = g.order[s];
    r = o < 0 ? -1 : static_cast<int64_t>(choices.div(static_cast<uint32_t>(o)));
  }
  return r < g.a_rows ? r : -1;
}

__device__ __forceinline__ i32x8 join(const u32x4& lo, const u32x4& hi) {
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// 4 consecutive columns of a row.
template <typename O>
__device__ __forceinline__ void store4(O* p, const f32x4& v) {
  if constexpr (sizeof(O) == 2)
    *reinterpret_cast<bf16x4*>(p) = __builtin_convertvector(v, bf16x4);
  else
    *reinterpret_cast<f32x4*>(p) = v;
}

// ---------------------------------------------------------------------------
// Few rows an expert: the weights are streamed straight into the matrix operands, once for each tile of 16 MT
// slots.  A workgroup of 8 waves: `ks` of them share the K steps of one set of 16 NT columns.
constexpr int kWaves = 8;

template <int FA, typename O, int MT, int NT>
__global__ void __launch_bounds__(kWaves * 64) k_expert_stream(ExpertGemmArgs g, FastDiv choices, int chunks, int ks) {
  __shared__ f32x4 red[kWaves][MT][NT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  Tile t;
  if (!find_tile<16 * MT>(g, blockIdx.x / chunks, t)) return;
  const int part = wave % ks;
  const int groups = static_cast<int>(g.N / 16);
  const int g0 = ((blockIdx.x % chunks) * (kWaves / ks) + wave / ks) * NT;  // first group of 16 columns
  const int steps = static_cast<int>(g.K / 128);
  const int s0 = steps * part / ks, s1 = steps * (part + 1) / ks;
  const uint8_t* arow[MT];
  float sa[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int64_t s = min(t.row0 + 16 * m + r, t.end - 1);
    const int64_t row = row_of(g, choices, s);
    arow[m] = g.a + max(row, int64_t(0)) * g.lda + 32 * q;
    sa[m] = g.sa[g.sa_rows ? max(row, int64_t(0)) : 0];
  }
  const uint8_t* bcol[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    bcol[n] = g.b + (static_cast<int64_t>(t.expert) * groups + min(g0 + n, groups - 1)) * steps * 2048 + lane * 16;
  f32x4 acc[MT][NT] = {};
  if (g0 < groups) {
    for (int s = s0; s < s1; ++s) {
      u32x4 b0[NT], b1[NT], a0[MT], a1[MT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        b0[n] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(bcol[n] + static_cast<int64_t>(s) * 2048));
        b1[n] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(bcol[n] + static_cast<int64_t>(s) * 2048 + 1024));
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        a0[m] = *reinterpret_cast<const u32x4*>(arow[m] + s * 128);
        a1[m] = *reinterpret_cast<const u32x4*>(arow[m] + s * 128 + 16);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          acc[m][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(b0[n], b1[n]), join(a0[m], a1[m]), acc[m][n],
                                                                      0, FA, 0, 0, 0, 0);
    }
  }
  if (ks > 1) {
    if (part > 0)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) red[wave][m][n][lane] = acc[m][n];
    __syncthreads();
    if (part > 0) return;
    for (int p = 1; p < ks; ++p)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n] += red[wave + p][m][n][lane];
  }
  // lane: slot row0 + 16 m + r, columns 16 (g0 + n) + 4 q ..
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (g0 + n >= groups) break;
    const int64_t col = static_cast<int64_t>(g0 + n) * 16 + 4 * q;
    f32x4 sb;
#pragma unroll
    for (int e = 0; e < 4; ++e) sb[e] = g.sb[t.expert * g.sb_expert + (col + e) * g.sb_col];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int64_t s = t.row0 + 16 * m + r;
      if (s >= t.end) continue;
      f32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = acc[m][n][e] * (sa[m] * sb[e]);
      if (row_of(g, choices, s) < 0) v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      store4(static_cast<O*>(g.y) + s * g.ldy + col, v);
    }
  }
}

}  // namespace

hipError_t launch_expert_gemm(const ExpertGemmArgs& g, hipStream_t st) {
  const FastDiv choices(static_cast<uint32_t>(g.choices));
  const int64_t avg = g.slots / g.experts;
  auto stream = [&](auto fa, auto o, auto mt, auto nt) {
    constexpr int FA = decltype(fa)::value, MT = decltype(mt)::value, NT = decltype(nt)::value;
    using O = decltype(o);
    const int64_t tiles = g.slots / (16 * MT) + std::min(g.experts, g.slots);
    const int64_t sets = ceil_div(g.N / 16, NT);
    int ks = 1;  // waves for each set of columns: 8 waves a CU at least, if the steps allow it
    while (ks < kWaves && tiles * sets * ks < int64_t(device_cus()) * 16 && g.K / 128 >= 4 * ks) ks <<= 1;
    const int64_t chunks = ceil_div(sets, kWaves / ks);
    hipLaunchKernelGGL((k_expert_stream<FA, O, MT, NT>), dim3(static_cast<unsigned>(tiles * chunks)), dim3(kWaves * 64), 0,
                       st, g, choices, static_cast<int>(chunks), ks);
  };
  auto by_rows = [&](auto fa, auto o) {
    if (avg <= 16) stream(fa, o, std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
    else if (avg <= 32) stream(fa, o, std::integral_constant<int, 2>{}, std::integral_constant<int, 2>{});
    else stream(fa, o, std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
  };
  auto by_out = [&](auto fa) { g.yt == FP8RT_BF16 ? by_rows(fa, uint16_t{}) : by_rows(fa, float{}); };
  g.fa == FP8RT_E4M3 ? by_out(std::integral_constant<int, kE4M3>{}) : by_out(std::integral_constant<int, kE5M2>{});
  return hipGetLastError();
}

}  // namespace fp8rt
