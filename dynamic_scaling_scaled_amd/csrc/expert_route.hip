// expert_route.hip -- the experts of each token: scores, biased and grouped choice of the
// k largest, weights, the plan that sorts the choices by expert; and the weights' gradient.
//
// A wave takes a token: lane l holds experts l NV .. l NV + NV - 1, so the lowest lane of a tie holds the lowest
// expert.  Keys are compared as integers that rise with them: the logit itself without a bias (softmax and sigmoid rise with
// it, so nothing is computed to choose), binary64 scores with one.
// The plan: a token chooses an expert at most once, so the tokens of one workgroup that chose expert e are
// a 64-bit mask; a choice's place among its expert's is the number of set bits below its token (stable and free of
// atomics on counters), and a workgroup's count is the mask's population.
#include <float.h>

#include <algorithm>

#include "device_common.h"
#include "internal.h"

namespace fp8rt {

namespace {

constexpr int kWaves = 16;
constexpr int kThreads = kWaves * 64;
constexpr int kMaxE = static_cast<int>(kRouteMaxExperts), kMaxK = static_cast<int>(kRouteMaxK);
constexpr int kMaxTokens = 64;  // of a workgroup

// Integers in the order of the numbers (0 is below all of them: an absent expert).
__device__ __forceinline__ uint64_t rising(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // (-0 and +0 are one key)
  return static_cast<uint64_t>((b & 0x80000000u) ? ~b : b | 0x80000000u) << 32;
}
__device__ __forceinline__ uint64_t rising(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  return (b >> 63) ? ~b : b | (uint64_t(1) << 63);
}
__device__ __forceinline__ double number(uint64_t r) {
  return __longlong_as_double(static_cast<long long>((r >> 63) ? r & ~(uint64_t(1) << 63) : ~r));
}

// Maximum over the wave, in every lane: row shifts, then the rows' last lanes.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define FP8RT_DPP_MAX(CTRL, ROWS) \
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(static_cast<int>(v), static_cast<int>(v), CTRL, ROWS, 0xF, false)))
  FP8RT_DPP_MAX(0x111, 0xF);  // row_shr 1, 2, 4, 8
  FP8RT_DPP_MAX(0x112, 0xF);
  FP8RT_DPP_MAX(0x114, 0xF);
  FP8RT_DPP_MAX(0x118, 0xF);
  FP8RT_DPP_MAX(0x142, 0xA);  // row_bcast 15, 31
  FP8RT_DPP_MAX(0x143, 0xC);
#undef FP8RT_DPP_MAX
  return __builtin_amdgcn_readlane(static_cast<int>(v), 63);
}
__device__ __forceinline__ float wave_max(float v) {  // (finite, or -Inf)
  const uint32_t b = __float_as_uint(v);
  const uint32_t m = wave_max((b & 0x80000000u) ? ~b : b | 0x80000000u);
  return __uint_as_float((m & 0x80000000u) ? m & 0x7FFFFFFFu : ~m);
}
template <typename V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// The lane of the largest key, the lowest of a tie (its key is returned; 0: no lane has one).  `low`: the
// keys' lower halves count.
__device__ __forceinline__ uint64_t wave_best(uint64_t key, bool low, int& lane) {
  const uint32_t hi = static_cast<uint32_t>(key >> 32), lo = static_cast<uint32_t>(key);
  const uint32_t mh = wave_max(hi);
  uint64_t who = __ballot(hi == mh);
  uint32_t ml = 0;
  if (low && __popcll(who) > 1) {
    ml = wave_max(hi == mh ? lo : 0u);
    who = __ballot(hi == mh && lo == ml);
  }
  lane = __ffsll(static_cast<unsigned long long>(who)) - 1;
  if (low) ml = __builtin_amdgcn_readlane(static_cast<int>(lo), lane);
  return (static_cast<uint64_t>(mh) << 32) | ml;
}

// A logit as it counts: NaN as -Inf (absent), +Inf as the largest finite value.
__device__ __forceinline__ float logit(float v) { return __builtin_isnan(v) ? -INFINITY : fminf(v, FLT_MAX); }
__device__ __forceinline__ float load_logit(const float* p) { return logit(*p); }
__device__ __forceinline__ float load_logit(const uint16_t* p) {
  return logit(__uint_as_float(static_cast<uint32_t>(*p) << 16));
}

// Chosen scores relative to their largest, q[j] proportional to p[j], finite and not all zero if one is present
// (p itself may underflow): e^(min(l,0) - M) / (1 + e^-|l|) for a sigmoid, e^(l - M) for a softmax.
__device__ __forceinline__ float relative(float l, bool there, int score) {
  const float a = there ? (score == FP8RT_SIGMOID ? fminf(l, 0.0f) : l) : -INFINITY;
  const float M = fmaxf(wave_max(a), -FLT_MAX);
  const float e = expf(a - M);
  return score == FP8RT_SIGMOID ? e / (1.0f + expf(-fabsf(l))) : e;
}

struct Plan {
  uint8_t* counts;      // [blocks][pitch]
  int pitch, tokens;    // bytes of a row; tokens of a block
  int blocks;
};

// Exclusive sum of n <= 1024 values over the workgroup's 1024 threads (thread t has value t), in place in `v`;
// returns the sum of all.  `part`: 16 words.
__device__ __forceinline__ uint32_t exclusive_sum(uint32_t& v, uint32_t* part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t s = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t up = __shfl_up(s, o);
    if (lane >= o) s += up;
  }
  if (lane == 63) part[wave] = s;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    before += w < wave ? part[w] : 0u;
    all += part[w];
  }
  v = before + s - v;
  return all;
}

// ---------------------------------------------------------------------------
// Forward.  Workgroup b takes tokens b plan.tokens ..; with one workgroup the plan is finished here.
template <typename T, int NV>
__global__ void __launch_bounds__(kThreads) k_route(RouteArgs a, Plan plan, FastDiv per_group) {
  __shared__ unsigned long long mask[kMaxE];
  __shared__ uint32_t base[kMaxE];
  __shared__ uint32_t part[kWaves];
  __shared__ int16_t chosen[kMaxTokens * kMaxK];
  extern __shared__ uint64_t members[];  // [waves][experts], where there are groups
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int E = a.experts, k = a.k;
  const int64_t t0 = int64_t(blockIdx.x) * plan.tokens;
  const bool planned = a.slots != nullptr;
  if (planned) {
    for (int e = threadIdx.x; e < E; e += kThreads) mask[e] = 0;
    __syncthreads();
  }
  const bool wide = a.bias || (a.groups > 1 && a.group_best == 2);  // binary64 scores are needed
  const T* logits = static_cast<const T*>(a.logits);
  for (int tt = wave; tt < plan.tokens; tt += kWaves) {
    const int64_t t = t0 + tt;
    if (t >= a.tokens) break;  // (uniform over the wave)
    float l[NV];
    uint64_t key[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = lane * NV + v;
      l[v] = e < E ? load_logit(logits + t * a.ld + e) : -INFINITY;
    }
    float top = l[0];
#pragma unroll
    for (int v = 1; v < NV; ++v) top = fmaxf(top, l[v]);
    const float m = fmaxf(wave_max(top), -FLT_MAX);
    uint64_t group[NV];  // what the groups are scored by
    if (wide) {
      double p[NV], sum = 0.0;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (a.score == FP8RT_SOFTMAX) {
          p[v] = exp(static_cast<double>(l[v]) - static_cast<double>(m));
          sum += p[v];
        } else {
          p[v] = 1.0 / (1.0 + exp(-static_cast<double>(l[v])));
        }
      }
      if (a.score == FP8RT_SOFTMAX) sum = wave_sum(sum);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int e = lane * NV + v;
        const bool there = l[v] > -INFINITY;
        if (a.score == FP8RT_SOFTMAX) p[v] /= sum;
        if (a.bias && there) p[v] += static_cast<double>(a.bias[e]);
        group[v] = there ? rising(p[v]) : 0;
        key[v] = a.bias ? group[v] : there ? rising(l[v]) : 0;
      }
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        key[v] = l[v] > -INFINITY ? rising(l[v]) : 0;
        group[v] = key[v];
      }
    }
    if (a.groups > 1) {
      // 64 / G' lanes a group (G' the next power of two) take its members in turn, then join
      uint64_t* mine = members + wave * E;
      int gp = 1;
      while (gp < a.groups) gp <<= 1;
      const int P = 64 / gp, g = lane / P, n = E / a.groups;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (lane * NV + v < E) mine[lane * NV + v] = group[v];
      __builtin_amdgcn_wave_barrier();
      uint64_t b1 = 0, b2 = 0;
      if (g < a.groups) {
        for (int i = lane - g * P; i < n; i += P) {
          const uint64_t x = mine[g * n + i];
          b2 = max(b2, min(b1, x));
          b1 = max(b1, x);
        }
      }
      for (int d = 1; d < P; d <<= 1) {
        const uint64_t c1 = __shfl_xor(static_cast<unsigned long long>(b1), d);
        const uint64_t c2 = __shfl_xor(static_cast<unsigned long long>(b2), d);
        b2 = max(max(b2, c2), min(b1, c1));
        b1 = max(b1, c1);
      }
      __builtin_amdgcn_wave_barrier();
      uint64_t score = b1;
      if (a.group_best == 2 && b1) score = rising(number(b1) + (b2 ? number(b2) : 0.0));
      if (lane != g * P) score = 0;
      uint64_t stay = 0;
      for (int i = 0; i < a.top_groups; ++i) {
        int at;
        if (wave_best(score, wide, at) == 0) break;
        stay |= uint64_t(1) << (at / P);
        if (lane == at) score = 0;
      }
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (!((stay >> per_group.div(min(lane * NV + v, E - 1))) & 1)) key[v] = 0;
    }
    // the lane's own best, and k rounds over the wave; lane j keeps choice j
    uint64_t best = 0;
    int bv = 0;
    float bl = 0.0f;
    auto own = [&] {
      best = 0;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (key[v] > best) {
          best = key[v];
          bv = v;
          bl = l[v];
        }
    };
    own();
    int id = -1;
    float chosen_l = 0.0f;
    for (int j = 0; j < k; ++j) {
      int at;
      if (wave_best(best, a.bias != nullptr, at) == 0) break;
      const int v = __builtin_amdgcn_readlane(bv, at);
      const float lv = __uint_as_float(__builtin_amdgcn_readlane(static_cast<int>(__float_as_uint(bl)), at));
      if (lane == j) {
        id = at * NV + v;
        chosen_l = lv;
      }
      if (lane == at) {
#pragma unroll
        for (int u = 0; u < NV; ++u)
          if (u == bv) key[u] = 0;
        own();
      }
    }
    const bool there = id >= 0;
    float w;
    if (a.renormalise) {
      const float q = relative(chosen_l, there, a.score);
      const float total = wave_sum(there ? q : 0.0f);
      w = q / total;
    } else if (a.score == FP8RT_SIGMOID) {
      w = 1.0f / (1.0f + expf(-chosen_l));
    } else {
      float sum = 0.0f;
#pragma unroll
      for (int v = 0; v < NV; ++v) sum += expf(l[v] - m);
      w = expf(chosen_l - m) / wave_sum(sum);
    }
    if (lane < k) {
      a.ids[t * k + lane] = id;
      a.weights[t * k + lane] = there ? a.scale * w : 0.0f;
      if (planned) {
        chosen[tt * k + lane] = static_cast<int16_t>(id);
        if (there) atomicOr(&mask[id], 1ull << tt);
      }
    }
  }
  if (!planned) return;
  __syncthreads();
  uint32_t n = static_cast<int>(threadIdx.x) < E ? __popcll(mask[threadIdx.x]) : 0u;
  if (plan.blocks == 1) {
    uint32_t at = n;
    const uint32_t all = exclusive_sum(at, part);
    if (static_cast<int>(threadIdx.x) < E) {
      base[threadIdx.x] = at;
      a.offsets[threadIdx.x] = static_cast<int32_t>(at);
    }
    if (threadIdx.x == 0) a.offsets[E] = static_cast<int32_t>(all);
    __syncthreads();
  } else if (static_cast<int>(threadIdx.x) < E) {
    plan.counts[int64_t(blockIdx.x) * plan.pitch + threadIdx.x] = static_cast<uint8_t>(n);
  }
  const int64_t here = min(static_cast<int64_t>(plan.tokens), a.tokens - t0);
  for (int i = threadIdx.x; i < here * k; i += kThreads) {
    const int e = chosen[i], tt = i / k;
    int32_t slot = -1;
    if (e >= 0) {
      slot = __popcll(mask[e] & ((1ull << tt) - 1));  // its place in this workgroup
      if (plan.blocks == 1) {
        slot += static_cast<int32_t>(base[e]);
        a.order[slot] = i;
      }
    }
    a.slots[t0 * k + i] = slot;
  }
}

// The plan over several blocks of tokens: each workgroup sums all blocks' counts (bytes, from the L2 cache) and those
// before its own blocks, and turns the places that k_route left in slots into slots.
__global__ void __launch_bounds__(kThreads) k_route_plan(RouteArgs a, Plan plan, int per_workgroup, int columns) {
  __shared__ uint32_t before[kMaxE], total[kMaxE];
  __shared__ uint32_t part[kWaves];
  const int E = a.experts, k = a.k, tid = threadIdx.x;
  const int b0 = blockIdx.x * per_workgroup;
  if (tid < E) before[tid] = total[tid] = 0;
  __syncthreads();
  const int c = tid & (columns - 1), slices = kThreads / columns;  // a thread: 4 experts of every slices-th block
  if (4 * c < plan.pitch) {
    uint32_t lo[4] = {}, sum[4] = {};
#pragma unroll 4
    for (int b = tid / columns; b < plan.blocks; b += slices) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(plan.counts + int64_t(b) * plan.pitch + 4 * c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x = (w >> (8 * i)) & 0xFFu;
        sum[i] += x;
        lo[i] += b < b0 ? x : 0u;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * c + i < E) {
        atomicAdd(&total[4 * c + i], sum[i]);
        atomicAdd(&before[4 * c + i], lo[i]);
      }
  }
  __syncthreads();
  uint32_t at = tid < E ? total[tid] : 0u;
  const uint32_t all = exclusive_sum(at, part);
  if (tid < E) {
    before[tid] += at;
    if (blockIdx.x == 0) a.offsets[tid] = static_cast<int32_t>(at);
  }
  if (blockIdx.x == 0 && tid == 0) a.offsets[E] = static_cast<int32_t>(all);
  __syncthreads();
  for (int b = b0; b < min(b0 + per_workgroup, plan.blocks); ++b) {
    const int64_t t0 = int64_t(b) * plan.tokens;
    const int64_t here = min(static_cast<int64_t>(plan.tokens), a.tokens - t0);
    for (int i = tid; i < here * k; i += kThreads) {
      const int64_t f = t0 * k + i;
      const int e = a.ids[f];
      if (e >= 0) {
        const int32_t slot = static_cast<int32_t>(before[e]) + a.slots[f];
        a.slots[f] = slot;
        a.order[slot] = static_cast<int32_t>(f);
      }
    }
    __syncthreads();
    if (tid < E) before[tid] += plan.counts[int64_t(b) * plan.pitch + tid];
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Gradient: a wave a token, lane j also choice j.
__device__ __forceinline__ void store_grad(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(uint16_t* p, float v) { *p = static_cast<uint16_t>(pack_bf16(v, v)); }

template <typename T, int NV>
__global__ void __launch_bounds__(256) k_route_backward(RouteArgs a) {
  const int lane = threadIdx.x & 63, E = a.experts;
  const T* logits = static_cast<const T*>(a.logits);
  T* out = static_cast<T*>(a.dlogits);
  const bool full = a.score == FP8RT_SOFTMAX && !a.renormalise;  // every expert's score has a gradient
  const int64_t waves = int64_t(gridDim.x) * 4;
  for (int64_t t = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); t < a.tokens; t += waves) {
    int id = lane < a.k ? a.ids[t * a.k + lane] : -1;
    if (id >= E) id = -1;
    const bool there = id >= 0;
    const float g = there ? a.scale * a.dweights[t * a.k + lane] : 0.0f;
    const float lj = there ? load_logit(logits + t * a.ld + id) : -INFINITY;
    float d[NV];
    float dj;  // choice j's gradient (full: what is added to the common term)
    if (full) {
      float m = -FLT_MAX, sum = 0.0f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int e = lane * NV + v;
        d[v] = e < E ? load_logit(logits + t * a.ld + e) : -INFINITY;
        m = fmaxf(m, d[v]);
      }
      m = wave_max(m);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        d[v] = expf(d[v] - m);
        sum += d[v];
      }
      sum = wave_sum(sum);
      const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
      dj = g * (expf(lj - m) * inv);
      const float dot = wave_sum(dj);
#pragma unroll
      for (int v = 0; v < NV; ++v) d[v] = -dot * (d[v] * inv);
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) d[v] = 0.0f;
      const bool present = lj > -INFINITY;
      const float c = expf(-fabsf(present ? lj : 0.0f));  // p = 1 / (1 + c) or c / (1 + c)
      if (a.renormalise) {
        // w = q / sum q: dq/q = (1 - p) dl for a sigmoid, dl for a softmax
        const float q = relative(present ? lj : 0.0f, present, a.score);
        const float total = wave_sum(present ? q : 0.0f);
        const float w = total > 0.0f && present ? q / total : 0.0f;
        dj = w * (g - wave_sum(w * g));
        if (a.score == FP8RT_SIGMOID) dj *= (lj > 0.0f ? c : 1.0f) / (1.0f + c);
      } else {
        dj = present ? g * (c / ((1.0f + c) * (1.0f + c))) : 0.0f;
      }
    }
    for (int j = 0; j < a.k; ++j) {
      const int e = __builtin_amdgcn_readlane(id, j);
      const float x = __uint_as_float(__builtin_amdgcn_readlane(static_cast<int>(__float_as_uint(dj)), j));
      if (e < 0) continue;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (e == lane * NV + v) d[v] += x;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = lane * NV + v;
      if (e < E) store_grad(out + t * a.lddl + e, d[v]);
    }
  }
}

template <typename F>
void by_width(int experts, F&& f) {
  if (experts <= 64) f(std::integral_constant<int, 1>{});
  else if (experts <= 128) f(std::integral_constant<int, 2>{});
  else if (experts <= 256) f(std::integral_constant<int, 4>{});
  else if (experts <= 512) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

}  // namespace

hipError_t launch_expert_route(const RouteArgs& a, hipStream_t st) {
  Plan plan{};
  // one workgroup finishes the plan of up to 64 tokens by itself
  plan.tokens = a.tokens <= kMaxTokens || a.tokens > 16384 ? kMaxTokens : 32;
  plan.blocks = static_cast<int>(ceil_div(a.tokens, plan.tokens));
  plan.pitch = (a.experts + 3) / 4 * 4;
  if (a.slots && plan.blocks > 1) {
    void* p = nullptr;
    const hipError_t e = get_scratch(st, size_t(plan.blocks) * plan.pitch, &p);
    if (e != hipSuccess) return e;
    plan.counts = static_cast<uint8_t*>(p);
  }
  const size_t lds = a.groups > 1 ? size_t(kWaves) * a.experts * sizeof(uint64_t) : 0;
  const FastDiv per_group(static_cast<uint32_t>(a.experts / a.groups));
  hipError_t e = hipSuccess;
  by_width(a.experts, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    auto go = [&](auto kern) {
      if (lds > 32768) {  // (beside the static arrays, past the default limit)
        e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
        if (e != hipSuccess) return;
      }
      hipLaunchKernelGGL(kern, dim3(plan.blocks), dim3(kThreads), lds, st, a, plan, per_group);
    };
    a.lt == FP8RT_BF16 ? go(k_route<uint16_t, NV>) : go(k_route<float, NV>);
  });
  if (e == hipSuccess) e = hipGetLastError();
  if (e == hipSuccess && a.slots && plan.blocks > 1) {
    int columns = 1;
    while (columns < plan.pitch / 4) columns <<= 1;
    const int per = static_cast<int>(ceil_div(plan.blocks, 256));
    hipLaunchKernelGGL(k_route_plan, dim3(ceil_div(plan.blocks, per)), dim3(kThreads), 0, st, a, plan, per, columns);
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_expert_route_backward(const RouteArgs& a, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(ceil_div(a.tokens, 4), int64_t(device_cus()) * 8)));
  by_width(a.experts, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, dim3(256), 0, st, a); };
    a.lt == FP8RT_BF16 ? go(k_route_backward<uint16_t, NV>) : go(k_route_backward<float, NV>);
  });
  return hipGetLastError();
}

}  // namespace fp8rt
