// expert_route.hip -- the experts of each token: scores, biased and grouped choice of the
// k largest, weights, the plan that sorts the choices by expert; and the weights' gradient.
//
// A wave takes a token: lane l holds experts l NV .. l NV + NV - 1, so the lowest lane of a tie holds the lowest
// expert.  Keys are compared as integers that rise with them.  Without a bias the logit itself is the key (softmax and
// sigmoid rise with it, so nothing is computed to choose); scores with a bias, and groups' sums of scores, are
// formed in binary32 first, with a bound of their error, and in binary64 for the tokens where that bound leaves the
// choice open.
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
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
// In binary32 by row shifts, as the maximum: 6 additions in a fixed order.
__device__ __forceinline__ float wave_sum(float v) {
#define FP8RT_DPP_ADD(CTRL, ROWS) \
  v += __uint_as_float(__builtin_amdgcn_update_dpp(0, static_cast<int>(__float_as_uint(v)), CTRL, ROWS, 0xF, false))
  FP8RT_DPP_ADD(0x111, 0xF);
  FP8RT_DPP_ADD(0x112, 0xF);
  FP8RT_DPP_ADD(0x114, 0xF);
  FP8RT_DPP_ADD(0x118, 0xF);
  FP8RT_DPP_ADD(0x142, 0xA);
  FP8RT_DPP_ADD(0x143, 0xC);
#undef FP8RT_DPP_ADD
  return __uint_as_float(__builtin_amdgcn_readlane(static_cast<int>(__float_as_uint(v)), 63));
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
// Forward.

// Keys as 32 bits: a binary32 value's.
__device__ __forceinline__ uint32_t rising32(float v) { return static_cast<uint32_t>(rising(v) >> 32); }
__device__ __forceinline__ float number32(uint32_t r) {
  return __uint_as_float((r & 0x80000000u) ? r & 0x7FFFFFFFu : ~r);
}

// The groups of a call: runs of n experts.
struct Groups {
  int n;              // experts of a group
  int lanes;          // lanes that hold one (n / NV, where that is a power of two), or 0
  FastDiv by_n;
};

// The two largest keys of every group, in all of its lanes: `lanes` lanes that hold its experts, or P lanes that read
// its members from `mine` (LDS of this wave).  Lane l belongs to group l / per (returned).
template <typename K, int NV>
__device__ __forceinline__ int group_tops(const RouteArgs& a, const Groups& gr, const K (&key)[NV], K* mine, K& b1, K& b2) {
  const int lane = threadIdx.x & 63;
  b1 = b2 = 0;
  int per = gr.lanes;
  if (per) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      b2 = max(b2, min(b1, key[v]));
      b1 = max(b1, key[v]);
    }
  } else {
    int gp = 1;
    while (gp < a.groups) gp <<= 1;
    per = 64 / gp;
    const int g = lane / per;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (lane * NV + v < a.experts) mine[lane * NV + v] = key[v];
    __builtin_amdgcn_wave_barrier();
    if (g < a.groups) {
      for (int i = lane - g * per; i < gr.n; i += per) {
        const K x = mine[g * gr.n + i];
        b2 = max(b2, min(b1, x));
        b1 = max(b1, x);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
  for (int d = 1; d < per; d <<= 1) {
    K c1, c2;
    if constexpr (sizeof(K) == 8) {
      c1 = __shfl_xor(static_cast<unsigned long long>(b1), d);
      c2 = __shfl_xor(static_cast<unsigned long long>(b2), d);
    } else {
      c1 = __shfl_xor(static_cast<int>(b1), d);
      c2 = __shfl_xor(static_cast<int>(b2), d);
    }
    b2 = max(max(b2, c2), min(b1, c1));
    b1 = max(b1, c1);
  }
  return per;
}

// Whether the lane's group is among the top_groups best by `score` (the same in a group's `per` lanes; equal scores go
// to the lower group): the groups ahead of it are counted.
template <typename K>
__device__ __forceinline__ bool group_stays(const RouteArgs& a, K score, int per) {
  const int g = (threadIdx.x & 63) / per;
  int ahead = 0;
  for (int o = 0; o < a.groups; ++o) {
    K s;
    if constexpr (sizeof(K) == 8)
      s = (static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(score >> 32), o * per))) << 32) |
          static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(score), o * per));
    else
      s = __builtin_amdgcn_readlane(static_cast<int>(score), o * per);
    ahead += (s > score || (s == score && o < g)) ? 1 : 0;
  }
  return g < a.groups && ahead < a.top_groups && score != 0;
}

// Takes the experts of groups that do not stay out of the keys.
template <typename K, int NV>
__device__ __forceinline__ void keep_groups(const RouteArgs& a, const Groups& gr, bool stays, int per, K (&key)[NV]) {
  const int lane = threadIdx.x & 63;
  if (gr.lanes) {
#pragma unroll
    for (int v = 0; v < NV; ++v) key[v] = stays ? key[v] : 0;
    return;
  }
  const uint64_t who = __ballot(stays);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int g = static_cast<int>(gr.by_n.div(min(lane * NV + v, a.experts - 1)));
    if (!((who >> (g * per)) & 1)) key[v] = 0;
  }
}

// Lane j's choice j in binary64: every score to 2^-50.
template <int NV>
__device__ __forceinline__ int choose_exactly(const RouteArgs& a, const Groups& gr, const float (&l)[NV], float m, uint64_t* mine) {
  const int lane = threadIdx.x & 63;
  double p[NV], sum = 0.0;
  uint64_t key[NV], group[NV];
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
    const bool there = l[v] > -INFINITY;
    if (a.score == FP8RT_SOFTMAX) p[v] /= sum;
    if (a.bias && there) p[v] += static_cast<double>(a.bias[lane * NV + v]);
    group[v] = there ? rising(p[v]) : 0;
    key[v] = a.bias ? group[v] : there ? rising(l[v]) : 0;
  }
  if (a.groups > 1) {
    uint64_t b1, b2;
    const int per = group_tops<uint64_t, NV>(a, gr, group, mine, b1, b2);
    uint64_t score = b1;
    if (a.group_best == 2 && b1) score = rising(number(b1) + (b2 ? number(b2) : 0.0));
    keep_groups<uint64_t, NV>(a, gr, group_stays<uint64_t>(a, score, per), per, key);
  }
  int id = -1;
  for (int j = 0; j < a.k; ++j) {
    uint64_t best = 0;
    int bv = 0, at;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (key[v] > best) {
        best = key[v];
        bv = v;
      }
    if (wave_best(best, true, at) == 0) break;
    const int v0 = __builtin_amdgcn_readlane(bv, at);  // (with all lanes on: inside the branch, bv would be computed there)
    if (lane == j) id = at * NV + v0;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (lane == at && v == bv) key[v] = 0;
  }
  return id;
}

// Lane j's choice j with 32-bit keys; `open` where their errors leave it undecided.  m: the largest logit; sum: of
// e^(l - m), for a softmax whose scores are needed.
template <int NV>
__device__ __forceinline__ int choose(const RouteArgs& a, const Groups& gr, const float (&l)[NV], float m, float sum,
                                      uint32_t* mine, bool& open) {
  const int lane = threadIdx.x & 63;
  const bool scores = a.bias || (a.groups > 1 && a.group_best == 2);
  uint32_t key[NV], group[NV];
  open = false;
  // A score's error: the exponential (2 u and u of its argument, which weighs p by at most 1 / e), sum or quotient,
  // product, 16 + 6 sums: 2^-19 of the largest score holds twice over, and the bias's sum adds u of the key.
  float err = 0.0f;
  if (scores) {
    float p[NV];
    const float inv = a.score == FP8RT_SOFTMAX ? __builtin_amdgcn_rcpf(sum) : 1.0f;
    err = 0x1p-18f * inv;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (a.score == FP8RT_SOFTMAX)
        p[v] = expf(l[v] - m) * inv;
      else
        p[v] = __builtin_amdgcn_rcpf(1.0f + expf(-l[v]));
      const bool there = l[v] > -INFINITY;
      if (a.bias && there) p[v] += a.bias[lane * NV + v];
      group[v] = there ? rising32(p[v]) : 0;
      key[v] = a.bias ? group[v] : there ? rising32(l[v]) : 0;
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) group[v] = key[v] = l[v] > -INFINITY ? rising32(l[v]) : 0;
  }
  if (a.groups > 1) {
    uint32_t b1, b2;
    const int per = group_tops<uint32_t, NV>(a, gr, group, mine, b1, b2);
    uint32_t score = b1;
    if (a.group_best == 2 && b1) score = rising32(number32(b1) + (b2 ? number32(b2) : 0.0f));
    const bool stays = group_stays<uint32_t>(a, score, per);
    if (scores && a.top_groups < a.groups) {  // the worst that stays against the best that goes
      const float in = number32(~wave_max(stays ? ~score : 0u));
      const uint32_t out = wave_max(stays || lane / per >= a.groups ? 0u : score);
      const float gap = in - number32(out);
      open = out != 0 && !(gap > 2.0f * err + 0x1p-20f * (fabsf(in) + fabsf(number32(b1)) + fabsf(number32(b2))));
      open = __ballot(open) != 0;
    }
    keep_groups<uint32_t, NV>(a, gr, stays, per, key);
  }
  // the lane's keys in falling order (neighbours change places, so equal ones keep theirs); a round takes a lane's first
  int at_v[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) at_v[v] = v;
#pragma unroll
  for (int r = 0; r < NV; ++r)
#pragma unroll
    for (int v = r & 1; v + 1 < NV; v += 2)
      if (key[v + 1] > key[v]) {
        const uint32_t x = key[v];
        key[v] = key[v + 1];
        key[v + 1] = x;
        const int y = at_v[v];
        at_v[v] = at_v[v + 1];
        at_v[v + 1] = y;
      }
  int id = -1;
  uint32_t last = 0;
  const bool check = a.bias != nullptr;  // (logits are exact keys)
  for (int j = 0; j < a.k + (check ? 1 : 0); ++j) {
    const uint32_t top = wave_max(key[0]);
    if (check && j > 0 && top != 0) {
      const float x = number32(last), y = number32(top);
      open = open || !(x - y > err + 0x1p-21f * (fabsf(x) + fabsf(y)));
    }
    last = top;
    if (top == 0 || j == a.k) break;
    const int at = __ffsll(static_cast<unsigned long long>(__ballot(key[0] == top))) - 1;
    const int v0 = __builtin_amdgcn_readlane(at_v[0], at);
    if (lane == j) id = at * NV + v0;
    if (lane == at) {
#pragma unroll
      for (int v = 0; v + 1 < NV; ++v) {
        key[v] = key[v + 1];
        at_v[v] = at_v[v + 1];
      }
      key[NV - 1] = 0;
    }
  }
  open = __ballot(open) != 0;
  return id;
}

// Workgroup b takes tokens b plan.tokens ..; with one workgroup the plan is finished here.
template <typename T, int NV>
__global__ void __launch_bounds__(kThreads) k_route(RouteArgs a, Plan plan, Groups gr) {
  __shared__ unsigned long long mask[kMaxE];
  __shared__ uint32_t base[kMaxE];
  __shared__ uint32_t part[kWaves];
  __shared__ int16_t chosen[kMaxTokens * kMaxK];
  extern __shared__ uint64_t members[];  // [waves][experts], where groups are not runs of lanes
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int E = a.experts, k = a.k;
  const int64_t t0 = int64_t(blockIdx.x) * plan.tokens;
  const bool planned = a.slots != nullptr;
  if (planned) {
    for (int e = threadIdx.x; e < E; e += kThreads) mask[e] = 0;
    __syncthreads();
  }
  uint64_t* mine = members + wave * E;
  const T* logits = static_cast<const T*>(a.logits);
  const bool summed = a.score == FP8RT_SOFTMAX && (a.bias || (a.groups > 1 && a.group_best == 2) || !a.renormalise);
  float next[NV];
  auto load = [&](int64_t t) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = lane * NV + v;
      next[v] = e < E && t < a.tokens ? load_logit(logits + t * a.ld + e) : -INFINITY;
    }
  };
  load(t0 + wave);
  for (int tt = wave; tt < plan.tokens; tt += kWaves) {
    const int64_t t = t0 + tt;
    if (t >= a.tokens) break;  // (uniform over the wave)
    float l[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) l[v] = next[v];
    if (tt + kWaves < plan.tokens) load(t + kWaves);  // in flight during this token's work
    float m = -FLT_MAX, sum = 0.0f;
    if (a.score == FP8RT_SOFTMAX) {
      float top = l[0];
#pragma unroll
      for (int v = 1; v < NV; ++v) top = fmaxf(top, l[v]);
      m = fmaxf(wave_max(top), -FLT_MAX);
      if (summed) {
#pragma unroll
        for (int v = 0; v < NV; ++v) sum += expf(l[v] - m);
        sum = wave_sum(sum);
      }
    }
    bool open;
    int id = choose<NV>(a, gr, l, m, sum, reinterpret_cast<uint32_t*>(mine), open);
    if (open) id = choose_exactly<NV>(a, gr, l, m, mine);
    const bool there = id >= 0;
    const float chosen_l = there ? load_logit(logits + t * a.ld + id) : 0.0f;
    float w;
    if (a.renormalise) {
      const float q = relative(chosen_l, there, a.score);
      const float total = wave_sum(there ? q : 0.0f);
      w = q / total;
    } else if (a.score == FP8RT_SIGMOID) {
      w = 1.0f / (1.0f + expf(-chosen_l));
    } else {
      w = expf(chosen_l - m) / sum;
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
  hipError_t e = hipSuccess;
  by_width(a.experts, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    Groups gr{};
    gr.n = a.experts / a.groups;
    gr.by_n = FastDiv(static_cast<uint32_t>(gr.n));
    gr.lanes = gr.n % NV == 0 ? gr.n / NV : 0;
    if (gr.lanes & (gr.lanes - 1)) gr.lanes = 0;
    const size_t lds = a.groups > 1 && !gr.lanes ? size_t(kWaves) * a.experts * sizeof(uint64_t) : 0;
    auto go = [&](auto kern) {
      if (lds > 32768) {  // (beside the static arrays, past the default limit)
        e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
        if (e != hipSuccess) return;
      }
      hipLaunchKernelGGL(kern, dim3(plan.blocks), dim3(kThreads), lds, st, a, plan, gr);
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
