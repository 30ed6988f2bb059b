// expert_route.hip -- the experts of each token: scores, biased and grouped choice of the
// k largest, weights, the plan that sorts the choices by expert; and the weights' gradient.
//
// L lanes of a wave take a token (16, 32 or 64: a reduction over 16 lanes is 4 steps and serves 4 tokens); lane l
// of them holds experts l NV .. l NV + NV - 1, so the lowest lane of a tie holds the lowest expert.  Keys are compared as
// integers that rise with them.  Without a bias the logit itself is the key (softmax and sigmoid rise with it, so nothing
// is computed to choose); scores with a bias, and groups' sums of scores, are formed in binary32 first, with a
// bound of their error, and in binary64 for the tokens where that bound leaves the choice open.
// The plan: a token chooses an expert at most once, so the tokens of one workgroup that chose expert e are
// a 64-bit mask; a choice's place among its expert's is the number of set bits below its token (stable and free of
// atomics on counters), and a workgroup's count is the mask's population.
//
// Measured (kernels alone): a token of 64 experts 4.6 us, of which a launch is 3; 16384 tokens of 64 (k 6, bf16) 7.5 us, their
// plan 4.2, the gradient 4.7; 8192 of 256 (k 8 of 4 of 8 groups, biased sigmoids) 19 us and the plan 5.8, of 512 35 and 9.  The
// bytes (8 MiB of logits there) would take 2 us: what bounds it is the chain of k + 2 rounds of a maximum over the token's lanes, of
// 10 to 14 dependent instructions each, hidden by the other waves of a SIMD.  The 64-bit path lives in the same kernel: it sets
// the registers (101 up to 4 experts a lane, so 4 waves a SIMD; bounds of 8 waves spill, 30 us) and 19 to 63 scalar ones are kept in
// vector lanes.  Past 512 experts (16 a lane) its arrays spill 159 vector registers: 8192 tokens of 1024 take 111 us with groups and
// bias and 72 with plain softmax (of 600 69), the plan 15.
#include <float.h>

#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "internal.h"

namespace fp8rt {

namespace {

constexpr int kThreads = 512;       // of k_route; up to 1024 where its 64-bit path has registers enough for them
constexpr int kPlanThreads = 1024;  // of k_route_plan
constexpr int kMaxE = static_cast<int>(kRouteMaxExperts), kMaxK = static_cast<int>(kRouteMaxK);
constexpr int kMaxTokens = 64;  // of a workgroup

// Integers in the order of the numbers (0 is below all of them: an absent expert).
__device__ __forceinline__ uint64_t rising(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  return (b >> 63) ? ~b : b | (uint64_t(1) << 63);
}
__device__ __forceinline__ double number(uint64_t r) {
  return __longlong_as_double(static_cast<long long>((r >> 63) ? r & ~(uint64_t(1) << 63) : ~r));
}

// Keys as 32 bits: a binary32 value's.
__device__ __forceinline__ uint32_t rising32(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // (-0 and +0 are one key)
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
// e^x of a score that only has to be compared: the hardware's exponential of the rounded product.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(1.44269504088896340736f * x); }
__device__ __forceinline__ float number32(uint32_t r) {
  return __uint_as_float((r & 0x80000000u) ? r & 0x7FFFFFFFu : ~r);
}

// Reductions over aligned runs of L lanes, in every lane: rotations within rows of 16, then halves exchanged.  Both
// sides of a step add the same two values, so all lanes hold the same bits.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), CTRL, 0xF, 0xF, true));
}
template <int L, typename F>
__device__ __forceinline__ uint32_t over(uint32_t v, F&& f) {
  v = f(v, dpp<0x128>(v));  // row_ror 8, 4, 2, 1
  v = f(v, dpp<0x124>(v));
  v = f(v, dpp<0x122>(v));
  v = f(v, dpp<0x121>(v));
  if constexpr (L >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = f(s[0], s[1]);
  }
  if constexpr (L >= 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = f(s[0], s[1]);
  }
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t run_max(uint32_t v) {
  return over<L>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int L>
__device__ __forceinline__ float run_max(float v) {  // (no NaN)
  return __uint_as_float(over<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int L>
__device__ __forceinline__ float run_sum(float v) {
  return __uint_as_float(over<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int L>
__device__ __forceinline__ double run_sum(double v) {
#pragma unroll
  for (int o = L / 2; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Whether the lane is the lowest of its run's with `on`.
template <int L>
__device__ __forceinline__ bool lowest(bool on) {
  const uint32_t lane = threadIdx.x & 63;
  const uint64_t who = __ballot(on);
  if constexpr (L == 64) return on && (who & ((uint64_t(1) << lane) - 1)) == 0;
  const uint32_t half = lane & 32 ? static_cast<uint32_t>(who >> 32) : static_cast<uint32_t>(who);
  const uint32_t below = (1u << (lane & 31)) - (1u << (lane & 31 & ~(L - 1)));
  return on && (half & below) == 0;
}

// A logit as it counts: NaN as -Inf (absent), +Inf as the largest finite value.
__device__ __forceinline__ float logit(float v) { return __builtin_isnan(v) ? -INFINITY : fminf(v, FLT_MAX); }
__device__ __forceinline__ float wide(float v) { return v; }
__device__ __forceinline__ float wide(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
template <typename T>
__device__ __forceinline__ float load_logit(const T* p) {
  return logit(wide(*p));
}
// The lane's NV logits of a row of E, absent past its end.  (Every load first, from addresses that are always there:
// a load under a condition would be waited for before the next.)
template <int NV, typename T>
__device__ __forceinline__ void load_logits(const T* row, int lane, int E, float (&l)[NV]) {
  T raw[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) raw[v] = row[min(lane * NV + v, E - 1)];
#pragma unroll
  for (int v = 0; v < NV; ++v) l[v] = lane * NV + v < E ? logit(wide(raw[v])) : -INFINITY;
}
// Whether an expert may be chosen.  A bias of -Inf or NaN switches it off: its key would be one of these, neither of which
// orders against an empty place.
__device__ __forceinline__ bool chosen_from(float l, float bias) { return l > -INFINITY && bias > -INFINITY; }
// The same of the bias as of the logits: 0 without one.
template <int NV>
__device__ __forceinline__ void load_bias(const float* bias, int lane, int E, float (&b)[NV]) {
#pragma unroll
  for (int v = 0; v < NV; ++v) b[v] = bias ? bias[min(lane * NV + v, E - 1)] : 0.0f;
}

// Chosen scores relative to their largest, q[j] proportional to p[j], finite and not all zero if one is present
// (p itself may underflow): e^(min(l,0) - M) / (1 + e^-|l|) for a sigmoid, e^(l - M) for a softmax.
template <int L>
__device__ __forceinline__ float relative(float l, bool there, int score) {
  const float a = there ? (score == FP8RT_SIGMOID ? fminf(l, 0.0f) : l) : -INFINITY;
  const float M = fmaxf(run_max<L>(a), -FLT_MAX);
  const float e = expf(a - M);
  return score == FP8RT_SIGMOID ? e / (1.0f + expf(-fabsf(l))) : e;
}

struct Plan {
  uint8_t* counts;      // [blocks][pitch]
  int pitch, tokens;    // bytes of a row; tokens of a block
  int blocks;
};

// Exclusive sum of one value a thread over a workgroup of THREADS, in place in `v`; returns the sum of all.  `part`:
// a word for each wave.
template <int THREADS>
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
  for (int w = 0; w < THREADS / 64; ++w) {
    before += w < wave ? part[w] : 0u;
    all += part[w];
  }
  v = before + s - v;
  return all;
}

// ---------------------------------------------------------------------------
// Forward.

// The groups of a call: runs of n experts.
struct Groups {
  int n;      // experts of a group
  int lanes;  // lanes that hold one (n / NV, where that is a power of two), or 0
  FastDiv by_n;
};

// The two largest keys of every group, in all of its lanes: `lanes` lanes that hold its experts, or a share of the token's
// lanes that read its members from `mine` (LDS of this token).  Returns the lanes per group.
template <typename K, int L, int NV, typename A>
__device__ __forceinline__ int group_tops(const A& a, const Groups& gr, const K (&key)[NV], K* mine, K& b1, K& b2) {
  const int lane = threadIdx.x & (L - 1);
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
    per = L / gp;
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
template <typename K, int L, typename A>
__device__ __forceinline__ bool group_stays(const A& a, K score, int per) {
  const int g = (threadIdx.x & (L - 1)) / per;
  int ahead = 0;
  for (int o = 0; o < a.groups; ++o) {
    K s;
    if constexpr (sizeof(K) == 8)
      s = __shfl(static_cast<unsigned long long>(score), o * per, L);
    else
      s = __shfl(static_cast<int>(score), o * per, L);
    ahead += (s > score || (s == score && o < g)) ? 1 : 0;
  }
  return g < a.groups && ahead < a.top_groups && score != 0;
}

// Takes the experts of groups that do not stay out of the keys.
template <typename K, int L, int NV, typename A>
__device__ __forceinline__ void keep_groups(const A& a, const Groups& gr, bool stays, int per, K (&key)[NV]) {
  const int lane = threadIdx.x & (L - 1);
  if (gr.lanes) {
#pragma unroll
    for (int v = 0; v < NV; ++v) key[v] = stays ? key[v] : 0;
    return;
  }
  const uint64_t who = __ballot(stays) >> (threadIdx.x & 63 & ~(L - 1));
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int g = static_cast<int>(gr.by_n.div(min(lane * NV + v, a.experts - 1)));
    if (!((who >> (g * per)) & 1)) key[v] = 0;
  }
}

// The choices of the tokens with `open` set in binary64 (every score to 2^-50), into `out` (k places of each token).
// (Its logits are loaded again: held over the common path they would cost it its registers.)
template <int L, int NV, typename T>
__device__ __forceinline__ void choose_exactly(const RouteArgs& a, const Groups& gr, const T* row, float m, uint64_t* mine,
                                               bool open, int16_t* out) {
  const int lane = threadIdx.x & (L - 1);
  float l[NV], bias[NV];
  load_logits<NV>(row, lane, a.experts, l);
  load_bias<NV>(a.bias, lane, a.experts, bias);
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
  if (a.score == FP8RT_SOFTMAX) sum = run_sum<L>(sum);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const bool there = chosen_from(l[v], bias[v]);
    if (a.score == FP8RT_SOFTMAX) p[v] /= sum;
    p[v] += static_cast<double>(bias[v]);
    group[v] = there ? rising(p[v]) : 0;
    key[v] = a.bias ? group[v] : there ? static_cast<uint64_t>(rising32(l[v])) << 32 : 0;
  }
  if (a.groups > 1) {
    uint64_t b1, b2;
    const int per = group_tops<uint64_t, L, NV>(a, gr, group, mine, b1, b2);
    uint64_t score = b1;
    if (a.group_best == 2 && b1) score = rising(number(b1) + (b2 ? number(b2) : 0.0));
    keep_groups<uint64_t, L, NV>(a, gr, group_stays<uint64_t, L>(a, score, per), per, key);
  }
  if (open && lane < a.k) out[lane] = -1;
  for (int j = 0; j < a.k; ++j) {
    uint64_t best = 0;
    int bv = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (key[v] > best) {
        best = key[v];
        bv = v;
      }
    const uint32_t hi = static_cast<uint32_t>(best >> 32), lo = static_cast<uint32_t>(best);
    const uint32_t mh = run_max<L>(hi);
    const uint32_t ml = run_max<L>(hi == mh ? lo : 0u);
    if (lowest<L>(best != 0 && hi == mh && lo == ml)) {
      if (open) out[j] = static_cast<int16_t>(lane * NV + bv);
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (v == bv) key[v] = 0;
    }
  }
}

// Puts the k + 1 best by their 32-bit keys in the order of their binary64 ones (lower experts first where equal), for tokens
// with `near` set: enough where the (k + 2)nd is certainly behind the k-th.
template <int L, int NV, typename T>
__device__ __forceinline__ void order_exactly(const RouteArgs& a, const T* row, float m, bool near, int16_t* out) {
  const int lane = threadIdx.x & (L - 1);
  double sum = 0.0;
  if (a.score == FP8RT_SOFTMAX) {
    float l[NV];
    load_logits<NV>(row, lane, a.experts, l);
#pragma unroll
    for (int v = 0; v < NV; ++v) sum += exp(static_cast<double>(l[v]) - static_cast<double>(m));
    sum = run_sum<L>(sum);
  }
  const int id = near && lane <= a.k ? out[lane] : -1;
  double key = -INFINITY;  // of an empty place: behind every expert's, whose bias is above it
  if (id >= 0) {
    const double l = load_logit(row + id);
    key = (a.score == FP8RT_SOFTMAX ? exp(l - static_cast<double>(m)) / sum : 1.0 / (1.0 + exp(-l))) +
          static_cast<double>(a.bias[id]);
  }
  int rank = 0;
  for (int j = 0; j <= a.k; ++j) {
    const double other = __shfl(key, j, L);
    const int oid = __shfl(id, j, L);
    rank += (other > key || (other == key && oid < id)) ? 1 : 0;
  }
  if (id >= 0 && rank < a.k) out[rank] = static_cast<int16_t>(id);
}

// How far the 32-bit keys settle a token's choice.
enum Settled { kSettled, kNear, kOpen };  // kNear: but for the order of the k + 1 best; kOpen: not at all

// The choices with 32-bit keys, into `out` (with a bias the next two as well).  m: the largest logit; sum: of e^(l - m),
// for a softmax whose scores are needed.
template <int L, int NV>
__device__ __forceinline__ Settled choose(const RouteArgs& a, const Groups& gr, const float (&l)[NV], const float (&bias)[NV],
                                          float m, float sum, uint32_t* mine, bool live, int16_t* out) {
  const int lane = threadIdx.x & (L - 1);
  const bool scores = a.bias || (a.groups > 1 && a.group_best == 2);
  uint32_t key[NV], group[NV];
  bool open = false, near = false;
  // Between two scores: a sigmoid's exponential (2 u, and u of its argument, at a slope of at most 1 / 4), sum and
  // reciprocal (2 u) leave 4 u each, 2^-21 in all; a softmax's exponential, product and sum of 16 + 6 terms 30 u of the
  // largest score each, 2^-18 of it.  The bias's sum adds u of a key.
  float err = 0.0f;
  if (scores) {
    float p[NV];
    const float inv = a.score == FP8RT_SOFTMAX ? __builtin_amdgcn_rcpf(sum) : 1.0f;
    err = a.score == FP8RT_SOFTMAX ? 0x1p-18f * inv : 0x1p-20f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (a.score == FP8RT_SOFTMAX)
        p[v] = fast_exp(l[v] - m) * inv;
      else
        p[v] = __builtin_amdgcn_rcpf(1.0f + fast_exp(-l[v]));
      const bool there = chosen_from(l[v], bias[v]);
      p[v] += bias[v];
      group[v] = there ? rising32(p[v]) : 0;
      key[v] = a.bias ? group[v] : there ? rising32(l[v]) : 0;
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) group[v] = key[v] = l[v] > -INFINITY ? rising32(l[v]) : 0;
  }
  if (a.groups > 1) {
    uint32_t b1, b2;
    const int per = group_tops<uint32_t, L, NV>(a, gr, group, mine, b1, b2);
    uint32_t score = b1;
    if (a.group_best == 2 && b1) score = rising32(number32(b1) + (b2 ? number32(b2) : 0.0f));
    const bool stays = group_stays<uint32_t, L>(a, score, per);
    if (scores && a.top_groups < a.groups) {  // the worst that stays against the best that goes
      const uint32_t in = ~run_max<L>(stays ? ~score : 0u), gone = run_max<L>(stays || lane / per >= a.groups ? 0u : score);
      const float size = run_max<L>((b1 ? fabsf(number32(b1)) : 0.0f) + (b2 ? fabsf(number32(b2)) : 0.0f));
      open = gone != 0 && !(number32(in) - number32(gone) > 2.0f * err + 0x1p-21f * size);
    }
    keep_groups<uint32_t, L, NV>(a, gr, stays, per, key);
  }
  // the lane's keys in falling order (neighbours change places, so equal ones keep theirs); a round takes a lane's first
  int at[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) at[v] = v;
#pragma unroll
  for (int r = 0; r < NV; ++r)
#pragma unroll
    for (int v = r & 1; v + 1 < NV; v += 2) {
      const bool swap = key[v + 1] > key[v];
      const uint32_t x = key[v], y = key[v + 1];
      key[v] = swap ? y : x;
      key[v + 1] = swap ? x : y;
      const int ax = at[v], ay = at[v + 1];
      at[v] = swap ? ay : ax;
      at[v + 1] = swap ? ax : ay;
    }
  typename std::conditional<NV <= 8, uint32_t, uint64_t>::type order = 0;  // the lane's experts, 4 bits each, the first lowest
#pragma unroll
  for (int v = 0; v < NV; ++v) order |= static_cast<decltype(order)>(at[v]) << (4 * v);
  const bool check = a.bias != nullptr;  // (logits are exact keys)
  const int rounds = check ? a.k + 2 : a.k;
  if (live && lane < rounds) out[lane] = -1;
  uint32_t got = 0;  // lane j: the j-th largest key
  for (int j = 0; j < rounds; ++j) {
    const uint32_t top = run_max<L>(key[0]);
    if (check) got = lane == j ? top : got;
    if (lowest<L>(key[0] == top && top != 0)) {
      if (live) out[j] = static_cast<int16_t>(lane * NV + static_cast<int>(order & 15));
      order >>= 4;
#pragma unroll
      for (int v = 0; v + 1 < NV; ++v) key[v] = key[v + 1];
      key[NV - 1] = 0;
    }
  }
  if (check) {  // lane j: its key against the next one's; lane k - 1 against the one after that as well
    const uint32_t next = __shfl_down(static_cast<int>(got), 1, L), after = __shfl_down(static_cast<int>(got), 2, L);
    const float x = number32(got), y = number32(next), z = number32(after);
    const bool close = lane < a.k && next != 0 && !(x - y > err + 0x1p-23f * (fabsf(x) + fabsf(y)));
    const bool far = lane == a.k - 1 && after != 0 && !(x - z > err + 0x1p-23f * (fabsf(x) + fabsf(z)));
    open = run_max<L>((open || far ? 2u : 0u)) != 0;
    near = run_max<L>(close ? 1u : 0u) != 0;
  }
  return open ? kOpen : near ? kNear : kSettled;
}

// Workgroup b takes tokens b plan.tokens ..; with one workgroup the plan is finished here.
template <typename T, int L, int NV>
__global__ void __launch_bounds__(NV <= 4 ? 2 * kThreads : kThreads) k_route(RouteArgs a, Plan plan, Groups gr) {
  __shared__ unsigned long long mask[kMaxE];
  __shared__ uint32_t base[kMaxE];
  __shared__ uint32_t part[kThreads / 64];
  __shared__ int16_t chosen[kMaxTokens * (kMaxK + 2)];
  extern __shared__ uint64_t members[];  // [runs of L lanes][experts], where groups are not runs of lanes
  const int lane = threadIdx.x & (L - 1), run = threadIdx.x / L;
  const int E = a.experts, k = a.k;
  const int64_t t0 = int64_t(blockIdx.x) * plan.tokens;
  const bool planned = a.slots != nullptr;
  if (planned) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) mask[e] = 0;
    __syncthreads();
  }
  uint64_t* mine = members + run * E;
  const T* logits = static_cast<const T*>(a.logits);
  const bool summed = a.score == FP8RT_SOFTMAX && (a.bias || (a.groups > 1 && a.group_best == 2) || !a.renormalise);
  for (int tt = run; tt < plan.tokens; tt += blockDim.x / L) {  // (the same rounds in every run)
    const int64_t t = t0 + tt;
    const bool live = t < a.tokens;
    if (__ballot(live) == 0) break;
    const T* row = logits + (live ? t : a.tokens - 1) * a.ld;
    int16_t* out = chosen + tt * (k + 2);
    float m = -FLT_MAX, sum = 0.0f;
    Settled how;
    {
      float l[NV], bias[NV];
      load_logits<NV>(row, lane, E, l);
      load_bias<NV>(a.bias, lane, E, bias);
      if (a.score == FP8RT_SOFTMAX) {
        float top = l[0];
#pragma unroll
        for (int v = 1; v < NV; ++v) top = fmaxf(top, l[v]);
        m = fmaxf(run_max<L>(top), -FLT_MAX);
        if (summed) {
#pragma unroll
          for (int v = 0; v < NV; ++v) sum += expf(l[v] - m);
          sum = run_sum<L>(sum);
        }
      }
      how = choose<L, NV>(a, gr, l, bias, m, sum, reinterpret_cast<uint32_t*>(mine), live, out);
    }
    if (!live) how = kSettled;
    __builtin_amdgcn_wave_barrier();
    if (__ballot(how == kNear) != 0) order_exactly<L, NV>(a, row, m, how == kNear, out);
    if (__ballot(how == kOpen) != 0)
      choose_exactly<L, NV>(a, gr, row, m, mine, how == kOpen, out);
    __builtin_amdgcn_wave_barrier();
    const int id = live && lane < k ? out[lane] : -1;  // lane j: choice j
    const bool there = id >= 0;
    const float cl = there ? load_logit(row + id) : 0.0f;
    float w;
    if (a.renormalise) {
      const float q = relative<L>(cl, there, a.score);
      const float total = run_sum<L>(there ? q : 0.0f);
      w = q / total;
    } else if (a.score == FP8RT_SIGMOID) {
      const float c = expf(-fabsf(cl));  // (e^-cl itself would overflow where the weight is still a number)
      w = (cl > 0.0f ? 1.0f : c) / (1.0f + c);
    } else {
      w = expf(cl - m) / sum;
    }
    if (live && lane < k) {
      a.ids[t * k + lane] = id;
      a.weights[t * k + lane] = there ? a.scale * w : 0.0f;
      if (planned && there) atomicOr(&mask[id], 1ull << tt);
    }
  }
  if (!planned) return;
  __syncthreads();
  if (plan.blocks == 1) {  // kThreads of them, thread t for experts 2 t and 2 t + 1
    static_assert(2 * kThreads >= kMaxE, "an expert for every half thread");
    const int e = 2 * threadIdx.x;
    const uint32_t n0 = e < E ? __popcll(mask[e]) : 0u, n1 = e + 1 < E ? __popcll(mask[e + 1]) : 0u;
    uint32_t at = n0 + n1;
    const uint32_t all = exclusive_sum<kThreads>(at, part);
    if (e < E) {
      base[e] = at;
      a.offsets[e] = static_cast<int32_t>(at);
    }
    if (e + 1 < E) {
      base[e + 1] = at + n0;
      a.offsets[e + 1] = static_cast<int32_t>(at + n0);
    }
    if (threadIdx.x == 0) a.offsets[E] = static_cast<int32_t>(all);
    __syncthreads();
  } else {
    for (int e = threadIdx.x; e < E; e += blockDim.x)
      plan.counts[int64_t(blockIdx.x) * plan.pitch + e] = static_cast<uint8_t>(__popcll(mask[e]));
  }
  const int64_t here = min(static_cast<int64_t>(plan.tokens), a.tokens - t0);
  for (int i = threadIdx.x; i < here * k; i += blockDim.x) {
    const int tt = i / k, e = chosen[i + 2 * tt];
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
__global__ void __launch_bounds__(kPlanThreads) k_route_plan(RouteArgs a, Plan plan, int per_workgroup, int columns) {
  __shared__ uint32_t before[kMaxE], total[kMaxE];
  __shared__ uint32_t part[kPlanThreads / 64];
  const int E = a.experts, k = a.k, tid = threadIdx.x;
  const int b0 = blockIdx.x * per_workgroup;
  if (tid < E) before[tid] = total[tid] = 0;
  __syncthreads();
  const int c = tid & (columns - 1), slices = kPlanThreads / columns;  // a thread: 4 experts of every slices-th block
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
  const uint32_t all = exclusive_sum<kPlanThreads>(at, part);
  if (tid < E) {
    before[tid] += at;
    if (blockIdx.x == 0) a.offsets[tid] = static_cast<int32_t>(at);
  }
  if (blockIdx.x == 0 && tid == 0) a.offsets[E] = static_cast<int32_t>(all);
  __syncthreads();
  for (int b = b0; b < min(b0 + per_workgroup, plan.blocks); ++b) {
    const int64_t t0 = int64_t(b) * plan.tokens;
    const int64_t here = min(static_cast<int64_t>(plan.tokens), a.tokens - t0);
    for (int i = tid; i < here * k; i += kPlanThreads) {
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
// Gradient: L lanes a token, lane j also choice j.  The row is put together in LDS: every expert's common term, then
// the chosen ones' own.
__device__ __forceinline__ void store_grad(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(uint16_t* p, float v) { *p = static_cast<uint16_t>(pack_bf16(v, v)); }

template <typename T, int L, int NV>
__global__ void __launch_bounds__(256) k_route_backward(RouteArgs a) {
  __shared__ float rows[256 * NV];
  const int lane = threadIdx.x & (L - 1), E = a.experts;
  float* row = rows + (threadIdx.x / L) * (L * NV);
  const T* logits = static_cast<const T*>(a.logits);
  T* out = static_cast<T*>(a.dlogits);
  const bool full = a.score == FP8RT_SOFTMAX && !a.renormalise;  // every expert's score has a gradient
  constexpr int kRuns = 256 / L;
  for (int64_t base = int64_t(blockIdx.x) * kRuns; base < a.tokens; base += int64_t(gridDim.x) * kRuns) {
    const bool live = base + threadIdx.x / L < a.tokens;
    const int64_t t = live ? base + threadIdx.x / L : a.tokens - 1;
    const T* lp = logits + t * a.ld;
    int id = lane < a.k ? a.ids[t * a.k + lane] : -1;
    if (id >= E) id = -1;
    const bool there = id >= 0;
    const float g = there ? a.scale * a.dweights[t * a.k + lane] : 0.0f;
    const float lj = there ? load_logit(lp + id) : -INFINITY;
    float d[NV];
    float dj;  // choice j's gradient (full: what is added to the common term)
    if (full) {
      float m = -FLT_MAX, sum = 0.0f;
      load_logits<NV>(lp, lane, E, d);
#pragma unroll
      for (int v = 0; v < NV; ++v) m = fmaxf(m, d[v]);
      m = run_max<L>(m);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        d[v] = expf(d[v] - m);
        sum += d[v];
      }
      sum = run_sum<L>(sum);
      const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
      dj = g * (expf(lj - m) * inv);
      const float dot = run_sum<L>(dj);
#pragma unroll
      for (int v = 0; v < NV; ++v) d[v] = -dot * (d[v] * inv);
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) d[v] = 0.0f;
      const bool present = lj > -INFINITY;
      const float c = expf(-fabsf(present ? lj : 0.0f));  // p = 1 / (1 + c) or c / (1 + c)
      if (a.renormalise) {
        // w = q / sum q: dq/q = (1 - p) dl for a sigmoid, dl for a softmax
        const float q = relative<L>(present ? lj : 0.0f, present, a.score);
        const float total = run_sum<L>(present ? q : 0.0f);
        const float w = total > 0.0f && present ? q / total : 0.0f;
        dj = w * (g - run_sum<L>(w * g));
        if (a.score == FP8RT_SIGMOID) dj *= (lj > 0.0f ? c : 1.0f) / (1.0f + c);
      } else {
        dj = present ? g * (c / ((1.0f + c) * (1.0f + c))) : 0.0f;
      }
    }
    // (one wave's LDS operations keep their order)
#pragma unroll
    for (int v = 0; v < NV; ++v) row[lane * NV + v] = d[v];
    __builtin_amdgcn_wave_barrier();
    if (there) atomicAdd(&row[id], dj);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = v * L + lane;  // (consecutive lanes, consecutive columns)
      if (live && e < E) store_grad(out + t * a.lddl + e, row[e]);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// Lanes of a token and experts of a lane: as few lanes as hold the experts 4 each, at least one for each group, choice
// and the two behind the choices.  (256 experts, 8 groups, 8192 tokens: 64 lanes of 4 take 18 us, 32 lanes of 8 23: they
// need half as many registers again.)
template <typename F>
void by_width(int experts, int k, int groups, F&& f) {
  using std::integral_constant;
  const int need = std::max(k + 2, groups);
  auto go = [&](auto l, auto nv) { f(l, nv); };
  if (experts <= 16 && need <= 16) go(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (experts <= 32 && need <= 16) go(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  else if (experts <= 64 && need <= 16) go(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  else if (experts <= 128 && need <= 32) go(integral_constant<int, 32>{}, integral_constant<int, 4>{});
  else if (experts <= 256) go(integral_constant<int, 64>{}, integral_constant<int, 4>{});
  else if (experts <= 512) go(integral_constant<int, 64>{}, integral_constant<int, 8>{});
  else go(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}

}  // namespace

hipError_t launch_expert_route(const RouteArgs& a, hipStream_t st) {
  Plan plan{};
  plan.pitch = (a.experts + 3) / 4 * 4;
  int groups_p2 = 1;  // (each group needs a lane of its own)
  while (groups_p2 < a.groups) groups_p2 <<= 1;
  hipError_t e = hipSuccess;
  by_width(a.experts, a.k, groups_p2, [&](auto l, auto nv) {
    constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
    // One workgroup finishes the plan by itself where its runs take at most two rounds (the plan's launch costs about as
    // much as a round).  Else about 256 workgroups, each of at least a round of kThreads (4096 tokens of 16 lanes in
    // 256 blocks of 16: 9.9 us and their plan 9.2, in 128 of 32: 7.6 and 6.4; both together in 128 of 32 9.3, in 64 of 64 10.1) and
    // of at most a mask's 64 tokens (16384 in 256 blocks of 64: 10.7 us with the plan, in 512 of 32 12.4).
    constexpr int kRuns = kThreads / L;
    if (a.tokens <= 2 * kRuns)
      plan.tokens = 2 * kRuns;
    else
      for (plan.tokens = kRuns; plan.tokens < kMaxTokens && plan.tokens * 256 < a.tokens;) plan.tokens *= 2;
    plan.blocks = static_cast<int>(ceil_div(a.tokens, plan.tokens));
    const int threads = plan.blocks == 1 ? kThreads : std::min(plan.tokens * L, NV <= 4 ? 2 * kThreads : kThreads);
    if (a.slots && plan.blocks > 1) {
      void* p = nullptr;
      e = get_scratch(st, size_t(plan.blocks) * plan.pitch, &p);
      if (e != hipSuccess) return;
      plan.counts = static_cast<uint8_t*>(p);
    }
    Groups gr{};
    gr.n = a.experts / a.groups;
    gr.by_n = FastDiv(static_cast<uint32_t>(gr.n));
    gr.lanes = gr.n % NV == 0 ? gr.n / NV : 0;
    if (gr.lanes & (gr.lanes - 1)) gr.lanes = 0;
    const size_t lds = a.groups > 1 && !gr.lanes ? size_t(threads / L) * a.experts * sizeof(uint64_t) : 0;
    auto go = [&](auto kern) {
      if (lds > 32768) {  // (beside the static arrays, past the default limit)
        e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
        if (e != hipSuccess) return;
      }
      hipLaunchKernelGGL(kern, dim3(plan.blocks), dim3(threads), lds, st, a, plan, gr);
    };
    a.lt == FP8RT_BF16 ? go(k_route<uint16_t, L, NV>) : go(k_route<float, L, NV>);
  });
  if (e == hipSuccess) e = hipGetLastError();
  if (e == hipSuccess && a.slots && plan.blocks > 1) {
    int columns = 1;
    while (columns < plan.pitch / 4) columns <<= 1;
    const int per = static_cast<int>(ceil_div(plan.blocks, 256));
    hipLaunchKernelGGL(k_route_plan, dim3(ceil_div(plan.blocks, per)), dim3(kPlanThreads), 0, st, a, plan, per, columns);
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_expert_route_backward(const RouteArgs& a, hipStream_t st) {
  by_width(a.experts, a.k, 1, [&](auto l, auto nv) {
    constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(ceil_div(a.tokens, 256 / L), int64_t(device_cus()) * 8)));
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, dim3(256), 0, st, a); };
    a.lt == FP8RT_BF16 ? go(k_route_backward<uint16_t, L, NV>) : go(k_route_backward<float, L, NV>);
  });
  return hipGetLastError();
}

}  // namespace fp8rt
