// paged_attention.hip -- attention over a paged cache of FP8 codes with one
// scale for each page and head.
//
// Mathematics.  With t_j = z_j log2(e) the scores of the visible positions and
// v_j = s_j dec(code_j) their values (s_j the page's v scale), the weight
//   w_j = 2^(t_j + log2 s_j - m + 8),   m at most 8 below the maximum of t_j + max(log2 s_j, -90),
// turns the output into  y = sum_j w_j dec(code_j) / sum_j (w_j / s_j):  the codes go
// into the second matrix product as they are, the weights stay within
// fp16 whatever the pages' scales, and the sums follow in one pass over the keys
// (when m moves, the sums so far are multiplied by 2^(m_old - m_new)).
// The denominator is kept as l = sum_j 2^(t_j - m), so m + log2 l is the log-sum-exp in base 2.
//
// Roundings.  Every FP8 code is a bf16 and an fp16 value, so q k multiplies exact
// operands (bf16 MFMA) and the codes enter the second product exactly (fp16 MFMA); the weights are
// rounded to fp16 (11 bits; bf16's 8 bits would add as much error as the bf16
// output itself has): from 2^-22 of the row's largest on they keep those bits, below they are rounded to
// multiples of 2^-32 of it.  Sums, maxima and accumulators are binary32.
//
// Orientation.  The scores are computed transposed, S^T = K Q^T: a lane then holds
// one query row's scores for several keys, which is the operand layout that the
// second product Y^T = V^T P^T wants, with the keys of a matrix instruction in the order in which
// the lane has them.  No score crosses lanes; a row's maximum and sum do only when they must.
//
// A query row is a (token, head of the group) pair: row r of a sequence and
// key / value head is token r / group, head r % group, so the heads that share keys share
// their loads.  Two kernels: k_attend_few for up to 16 rows (decode), each wave streaming its own
// keys from HBM; k_attend_many, 128 or 256 rows a workgroup, keys and values staged in LDS.
// Long key ranges are cut into chunks, whose unnormalised sums k_attend_join adds.
#include <algorithm>
#include <type_traits>

#include "paged_common.h"

namespace fp8rt {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// The reference m follows the running maximum only when weights grow too large for
// fp16: when a lane's weights of one 16-key part add up to its largest value.
constexpr float kFull = 65504.0f;
// When m has followed, the largest weight is 2^kLift: fp16 ends 2^-24 below 1, and where one key outweighs the rest (an
// attention sink, or a key in a page of large values) the small weights make the output.  The room left above sets how
// often m follows: a prompt of 8192 tokens takes 1096 us without a lift, 1105 with 6, 1108 with 8, 1124 with 10.
// Without a lift, 8192 keys 18 nats below one whose value is 0 come out as 0 (prompts) or 13% off (decode).
constexpr float kLift = 8.0f, kUnlift = 0x1p-8f;
// m stays within this of the scores however small the v scales are (2^-112 is the smallest that append writes): a term
// 2^(t - m) of the denominator is then at most 2^90, which leaves room for its sum, and the largest weight at least 2^-14.
constexpr float kReach = 90.0f;
// Before a row has seen a key, m is this: any score then gives an infinite
// weight, which makes m follow.
constexpr float kNoKey = -1e30f;
// Scales below the smallest normal count as that: log2 and 1 / s stay finite, and a score of -Inf
// times the k scale stays -Inf.
constexpr float kTinyScale = 0x1p-126f;

// Two codes (a half of a dword) as two bf16 / fp16 values, exactly.
template <int F, bool HI>
__device__ __forceinline__ uint32_t to_bf16(uint32_t w) {
  if constexpr (F == kE4M3)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, 1.0f, HI));
}
template <int F, bool HI>
__device__ __forceinline__ uint32_t to_f16(uint32_t w) {
  if constexpr (F == kE4M3)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(w, 1.0f, HI));
}
template <int F>
__device__ __forceinline__ u32x4 bf16_of(uint32_t a, uint32_t b) {
  return u32x4{to_bf16<F, false>(a), to_bf16<F, true>(a), to_bf16<F, false>(b), to_bf16<F, true>(b)};
}
template <int F>
__device__ __forceinline__ u32x4 f16_of(uint32_t a, uint32_t b) {
  return u32x4{to_f16<F, false>(a), to_f16<F, true>(a), to_f16<F, false>(b), to_f16<F, true>(b)};
}

// Whether any of four codes is a NaN or an infinity: the magnitude bits reach
// 0x7F (E4M3) or 0x7C (E5M2), so adding the rest to 0x80 carries into a byte's top bit.
template <int F>
__device__ __forceinline__ uint32_t non_finite(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + (F == kE4M3 ? 0x01010101u : 0x04040404u)) & 0x80808080u;
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), f16x2));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  bf16x2 v;
  v[0] = static_cast<__bf16>(a);
  v[1] = static_cast<__bf16>(b);
  return __builtin_bit_cast(uint32_t, v);
}
// A value that every lane has, in a scalar register.
__device__ __forceinline__ float uniform(float x) {
  return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x)));
}
// 0 in a vector register, of which the compiler knows only that it is an integer.
__device__ __forceinline__ int hidden_zero() {
  int z;
  asm("v_mov_b32 %0, 0" : "=v"(z));
  return z;
}
// Keeps the compiler from moving instructions across this point: the kernels' loops
// say themselves which work runs under which matrix instruction.
__device__ __forceinline__ void pin() { __builtin_amdgcn_sched_barrier(0); }
// This wave's priority among those of its SIMD.  A tile starts urgent and gets less so: the
// two waves of a SIMD drift apart, one feeding the matrix cores while the other widens and waits
// (8192-token prompt, 64 / 8 heads of 128: 1086 us, without 1130, urgent throughout 1227).
template <int P>
__device__ __forceinline__ void urgent() { __builtin_amdgcn_s_setprio(P); }
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_fast(float x) { return __builtin_amdgcn_logf(x); }

// Visible positions of one query: [lo, hi).
struct Range {
  int32_t lo, hi;
};

__device__ __forceinline__ Range visible(const AttendArgs& a, const SeqSpan& s, int64_t token) {
  const int64_t at = s.first + token;
  int64_t lo = 0, hi = s.len;
  if (a.causal && at + 1 < hi) hi = at + 1;
  if (a.window > 0 && at - a.window + 1 > 0) lo = at - a.window + 1;
  if (hi < 0) hi = 0;
  if (lo > hi) lo = hi;
  return Range{static_cast<int32_t>(lo), static_cast<int32_t>(hi)};
}

// What a tile of `rows` query rows from row r0 sees together (its first row
// starts first, its last row ends last), from a multiple of 64 on.
__device__ __forceinline__ Range tile_range(const AttendArgs& a, const SeqSpan& s, int32_t r0, int32_t rows,
                                            const FastDiv& group) {
  const Range x = visible(a, s, group.div(r0)), y = visible(a, s, group.div(r0 + rows - 1));
  return Range{x.lo & ~63, y.hi};
}

// How the keys of a tile are cut: `chunks` pieces of `len` keys (a multiple
// of 64), the last one open-ended.  And the divisors of the grid: a workgroup's
// start is dependent loads and index arithmetic, which the 64-bit quotients dominated.
struct Cut {
  int32_t chunks, len;
  int32_t ordered;  // decode: the longest of at most 64 sequences first
  int32_t mixed;    // both kernels run, each for the sequences that are its own (short: up to 16 rows)
  FastDiv by_heads, by_tiles, by_chunks, by_group;
};

// Workgroup -> (sequence, chunk, tile, head), head fastest: neighbours read
// neighbouring parts of the same pages, and with 8 heads each XCD's L2 keeps one of them.
struct Place {
  uint32_t head, tile, chunk, b;
};
__device__ __forceinline__ Place place_of(uint32_t blk, const Cut& c) {
  Place p;
  uint32_t x = c.by_heads.div(blk);
  p.head = blk - x * c.by_heads.d;
  uint32_t y = c.by_tiles.div(x);
  p.tile = x - y * c.by_tiles.d;
  p.b = c.by_chunks.div(y);
  p.chunk = y - p.b * c.by_chunks.d;
  return p;
}

__device__ __forceinline__ Range chunk_of(const Range& t, const Cut& c, int32_t i) {
  const int64_t lo = int64_t(t.lo) + int64_t(i) * c.len, hi = lo + c.len;
  return Range{lo < t.hi ? static_cast<int32_t>(lo) : t.hi,
               i == c.chunks - 1 || hi > t.hi ? t.hi : static_cast<int32_t>(hi)};
}

// The sequence of rank `slot` by falling length, of at most 64 (one a lane; larger batches run in their
// own order).  Where workgroups outnumber the places on the card, the long ones must not start last.
__device__ __forceinline__ int32_t by_length(const PagedArgs& p, int32_t slot) {
  const int32_t lane = threadIdx.x & 63, n = static_cast<int32_t>(p.seqs);
  const int32_t len = p.kv_len[lane < n ? lane : 0];
  int32_t rank = 0;
  for (int32_t j = 0; j < n; ++j) {
    const int32_t other = __builtin_amdgcn_readlane(len, j);
    rank += other > len || (other == len && j < lane);
  }
  return __builtin_ctzll(__ballot(lane < n && rank == slot));
}

// Partial results of cut tiles, in the stream's scratch.  Rows: (sequence, head, row of its
// tile) of k_attend_few, (token, query head) of k_attend_many.
struct Parts {
  float* o;      // [chunk][row][D], unnormalised
  float2* ml;    // [chunk][row]: m, sum of w / s
  int64_t rows;
};

// What one 16-key part of a step needs from its page: t = dot * c, log2 of the v scale with the lift, the factor that
// turns a weight into 2^(t - m).
// A page that is not there gives weights of 0 (its codes are staged as 0).  Scales that are not
// finite count as 1 here; the rows are done again by careful_row.
struct PartScale {
  float c, lv, inv;
};
__device__ __forceinline__ bool finite_scales(float ks, float vs) { return ks <= 3.4028235e38f && vs <= 3.4028235e38f; }
__device__ __forceinline__ PartScale part_scale(bool there, float ks, float vs, float sm) {
  const bool fine = finite_scales(ks, vs);
  const float c = fine ? ks * sm : 1.0f, v = fine && vs >= kTinyScale ? vs : fine ? kTinyScale : 1.0f;
  return PartScale{c < kTinyScale ? kTinyScale : c, there ? log2_fast(v) + kLift : -INFINITY,
                   there ? __builtin_amdgcn_rcpf(v) * kUnlift : 0.0f};  // (rcp: 1 ulp)
}

// log2 of a part's v scale (with the lift) as m follows it.  Absent pages stay at -Inf.
__device__ __forceinline__ float reached(float lv) { return lv > -INFINITY ? fmaxf(lv, kLift - kReach) : lv; }

// One query row over the keys [see.lo, see.hi), by one wave, without products that hidden keys take
// part in: m, l = sum 2^(t - m) and this lane's D/64 dimensions of sum 2^(t - m) v.  The matrix
// kernels multiply a hidden key's value by a weight of 0, which is not 0 for a NaN or an infinity; they
// notice such codes and scales and take this slow way for the rows concerned, after their loop
// (inside it, it would cost the registers that keep the accumulators out of memory).  A row takes about 16 us
// for 64 keys: with one NaN a prompt of 2048 tokens 17 ms instead of 0.16, two sequences of 131072 4 instead of 0.1.
template <int F, int D>
__device__ void careful_row(const AttendArgs& a, int64_t b, int32_t head, int64_t tok, int64_t qh, Range see, float& m,
                            float& l, float* y) {
  constexpr int E = D / 64;
  const int lane = threadIdx.x & 63;
  const int32_t page = a.p.page;
  const uint16_t* q = a.q + tok * a.ldq + qh * a.hdq;
  const float sm = a.sm_scale * kLog2e;
  m = kNoKey;
  l = 0.0f;
  for (int e = 0; e < E; ++e) y[e] = 0.0f;
  for (int32_t j0 = see.lo; j0 < see.hi; j0 += 64) {
    const int32_t j = j0 + lane;
    const int32_t pg = j < see.hi ? page_of(a.p, b, j / page) : -1;
    const int64_t at = int64_t(pg < 0 ? 0 : pg) * a.p.heads + head;
    const int64_t base = (at * page + j % page) * D;
    float t = -INFINITY;
    if (pg >= 0) {
      float dot = 0.0f;
      for (int d = 0; d < D; d += 4) {
        float v[4];
        decode4<F>(*reinterpret_cast<const uint32_t*>(a.kc + base + d), v);
        for (int i = 0; i < 4; ++i) dot = fmaf(v[i], __uint_as_float(static_cast<uint32_t>(q[d + i]) << 16), dot);
      }
      t = dot * (a.ks[at] * sm);
    }
    float top = t;
    for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    const float mn = fmaxf(m, top);
    const float fade = exp2_fast(m - mn), w = exp2_fast(t - mn);
    float sum = w;
    for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
    l = l * fade + sum;
    m = mn;
    for (int e = 0; e < E; ++e) y[e] *= fade;
    const float vs = a.vs[at];
    for (int k = 0; k < 64; ++k) {
      if (__shfl(pg, k) < 0) continue;
      const int64_t from = int64_t(__shfl(static_cast<int>(base >> 32), k)) << 32 |
                           static_cast<uint32_t>(__shfl(static_cast<int>(base), k));
      const float wk = __shfl(w, k), sk = __shfl(vs, k);
      for (int e = 0; e < E; ++e) {
        float v[4];
        decode4<F>(a.vc[from + lane * E + e], v);
        y[e] += wk * (sk * v[0]);
      }
    }
  }
}

// Writes such a row: the output (one chunk) or its part.
template <int D>
__device__ void careful_store(const AttendArgs& a, const Parts& parts, int32_t chunks, int64_t at, int64_t tok,
                              int64_t qh, float m, float l, const float* y) {
  constexpr int E = D / 64;
  const int lane = threadIdx.x & 63;
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
  for (int e = 0; e < E; ++e) {
    if (chunks == 1)
      a.y[tok * a.ldy + qh * a.hdy + lane * E + e] = static_cast<uint16_t>(pack_bf16(y[e] * inv, 0.0f));
    else
      parts.o[at * D + lane * E + e] = y[e];
  }
  if (lane == 0) {
    if (chunks > 1)
      parts.ml[at] = make_float2(m, l);
    else if (a.lse)
      a.lse[tok * a.q_heads + qh] = l != 0.0f ? (m + log2_fast(l)) * kLn2 : -INFINITY;
  }
}

// ---------------------------------------------------------------------------
// Up to 16 query rows: decode.  A workgroup takes one tile of 16 rows and one
// chunk of keys; its waves take 32-key steps in turn, each with its own reference and sums,
// joined through LDS at the end.  The keys of a step go from HBM to registers in operand order:
// lane l (c = l % 16, g = l / 16) loads 16-byte pieces of key c of each 16-key part, and for the keys
// {4g..4g+3, 16+4g..16+4g+3}, whose scores it will hold, D/16 bytes of the values; byte b of every
// key's dword w makes output tile 4w + b, so that two byte permutes a pair of codes transpose them.
// Bound by reading the codes: two sequences of 131072 tokens, 8 heads of 128, 90 us (6.0 TB/s, what a
// read-only pass reaches) and 5 us for the join; 64 ragged sequences of up to 8191 102 us (5.4 TB/s: the
// last workgroups end apart); one of 1001 tokens 11 us, a chain of launch, plan, table and 4 steps.
// 8 waves a workgroup: 64 ragged sequences of up to 8192 tokens, 8 heads, in one piece each,
// 114 us; 4 waves 124; 16 (which no longer fit the registers) 166.
constexpr int kFewWaves = 8;

template <int F, int D>
__global__ void __launch_bounds__(64 * kFewWaves) k_attend_few(AttendArgs a, Cut cut, Parts parts) {
  constexpr int W = kFewWaves;
  constexpr int KD = D / 64;      // 16-byte key pieces of a lane and part
  constexpr int VW = D / 64;      // dwords of a lane and key
  constexpr int DT = D / 16;      // 16-wide output tiles: tile 4w + b is byte b of dword w
  constexpr int LD = D + 4;
  __shared__ __align__(16) float sh_o[W][16][LD];
  __shared__ float2 sh_ml[W][16];
  __shared__ int sh_redo[W];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int32_t heads = a.p.heads, group = static_cast<int32_t>(cut.by_group.d);
  const Place place = place_of(blockIdx.x, cut);
  const int32_t head = place.head, chunk = place.chunk, r0 = place.tile * 16;
  const int64_t b = cut.ordered ? by_length(a.p, place.b) : static_cast<int32_t>(place.b);
  const SeqSpan s = seq_span(a.p, b);
  const int64_t all = int64_t(s.n) * group;
  if (r0 >= all || (cut.mixed && all > 16)) return;
  const int32_t rows = all - r0 < 16 ? static_cast<int32_t>(all - r0) : 16;
  const Range tile = tile_range(a, s, r0, rows, cut.by_group);
  const Range part = chunk_of(tile, cut, chunk);
  if (chunk > 0 && part.lo >= part.hi) return;  // (chunk 0 also writes the rows that see nothing)
  const int32_t page = a.p.page, shift = 31 - __builtin_clz(page);
  // this lane's query row
  const int32_t r = r0 + (c < rows ? c : 0);
  const int32_t ti = cut.by_group.div(r);
  const int64_t tok = s.tok0 + ti;
  const int64_t qh = int64_t(head) * group + (r - ti * group);
  Range see = visible(a, s, ti);
  see.hi = see.hi < part.hi ? see.hi : part.hi;
  if (c >= rows || see.hi < see.lo) see.hi = see.lo;
  // positions that every row sees, and that any row sees
  const Range first = visible(a, s, cut.by_group.div(r0)), last = visible(a, s, cut.by_group.div(r0 + rows - 1));
  const int32_t all_lo = last.lo, all_hi = first.hi, any_lo = first.lo;
  const float sm = fabsf(a.sm_scale) * kLog2e;
  const uint32_t flip = a.sm_scale < 0.0f ? 0x80008000u : 0u;  // a negative scale negates the query
  // q in key order: piece h, half u of a 16-byte piece -> dimensions 64 h + 16 g + 8 u ..
  u32x4 q[2 * KD];
#pragma unroll
  for (int h = 0; h < KD; ++h)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      q[2 * h + u] = *reinterpret_cast<const u32x4*>(a.q + tok * a.ldq + qh * a.hdq + 64 * h + 16 * g + 8 * u);
#pragma unroll
      for (int i = 0; i < 4; ++i) q[2 * h + u][i] ^= flip;
    }
  f32x4 o[DT] = {};
  float m = kNoKey, l = 0.0f;

  struct Step {
    u32x4 k[2][KD];
    uint32_t v[8][VW];
    int32_t pg[2];
    float ks[2], vs[2];
  };
  // Table entries are looked up a step before their keys are loaded, the keys a step
  // before they are used.  (Past the end the last page is looked up, and counts as absent.)
  const int32_t* table = a.p.table + b * a.p.ld_table;
  const uint32_t page_bytes = static_cast<uint32_t>(page) * D, pages = static_cast<uint32_t>(a.p.pages);
  const uint32_t k_at = c * D + 16 * g, v_at = 4 * g * D + c * (D / 16);
  int32_t entry[2];
  auto look_up = [&](int32_t k0) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int32_t j = k0 + 16 * t;
      entry[t] = table[(j < part.hi ? j : part.hi - 1) >> shift];
    }
  };
  auto load = [&](Step& st, int32_t k0) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int32_t p0 = k0 + 16 * t;
      const bool there = p0 < part.hi && static_cast<uint32_t>(entry[t]) < pages;
      st.pg[t] = there ? entry[t] : -1;
      const uint64_t ph = uint64_t(there ? static_cast<uint32_t>(entry[t]) : 0u) * static_cast<uint32_t>(heads) +
                          static_cast<uint32_t>(head);
      st.ks[t] = a.ks[ph];
      st.vs[t] = a.vs[ph];
      const uint64_t base = ph * page_bytes + static_cast<uint32_t>((p0 & (page - 1)) * D);
#pragma unroll
      for (int h = 0; h < KD; ++h) st.k[t][h] = *reinterpret_cast<const u32x4*>(a.kc + base + k_at + 64 * h);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint8_t* p = a.vc + base + v_at + j * D;
        if constexpr (VW == 2) {
          const u32x2 x = *reinterpret_cast<const u32x2*>(p);
          st.v[4 * t + j][0] = x[0];
          st.v[4 * t + j][1] = x[1];
        } else {
          st.v[4 * t + j][0] = *reinterpret_cast<const uint32_t*>(p);
        }
      }
    }
  };

  uint32_t redo = 0;  // a hidden value, or one under such a scale, may be no finite number
  const int32_t begin = part.lo + 32 * wave;
  Step cur;
  if (begin < part.hi) {
    look_up(begin);
    load(cur, begin);
    look_up(begin + 32 * W);
  }
  for (int32_t k0 = begin; k0 < part.hi; k0 += 32 * W) {
    Step next;
    load(next, k0 + 32 * W);
    look_up(k0 + 64 * W);
    f32x4 z[2];
    PartScale ps[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      z[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int h = 0; h < KD; ++h)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          z[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, bf16_of<F>(cur.k[t][h][2 * u], cur.k[t][h][2 * u + 1])),
              __builtin_bit_cast(bf16x8, q[2 * h + u]), z[t], 0, 0, 0);
      ps[t] = part_scale(cur.pg[t] >= 0, cur.ks[t], cur.vs[t], sm);
      redo |= cur.pg[t] >= 0 && !finite_scales(cur.ks[t], cur.vs[t]);
    }
    if (k0 < all_lo || k0 + 32 > all_hi || k0 + 32 > part.hi || cur.pg[0] < 0 || cur.pg[1] < 0) {
      // hidden keys score -Inf; values that no row sees are 0, the rest must be finite
      const int32_t from = see.lo - k0 - 4 * g;
      const uint32_t n = see.hi - see.lo;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int32_t j = k0 + 16 * t + 4 * g + i;
          const bool held = cur.pg[t] >= 0 && j >= any_lo && j < part.hi;
          z[t][i] = held && static_cast<uint32_t>(16 * t + i - from) < n ? z[t][i] : -INFINITY;
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            cur.v[4 * t + i][w] = held ? cur.v[4 * t + i][w] : 0u;
            redo |= non_finite<F>(cur.v[4 * t + i][w]);
          }
        }
    }
    float w[8], sum[2];
    auto weigh = [&] {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float lift = ps[t].lv - m;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 * t + i] = exp2_fast(fmaf(z[t][i], ps[t].c, lift));
        sum[t] = (w[4 * t] + w[4 * t + 1]) + (w[4 * t + 2] + w[4 * t + 3]);
      }
    };
    weigh();
    if (__any(!(fmaxf(sum[0], sum[1]) < kFull))) {
      float top = kNoKey;
#pragma unroll
      for (int t = 0; t < 2; ++t)
        top = fmaxf(top, fmaf(fmaxf(fmaxf(z[t][0], z[t][1]), fmaxf(z[t][2], z[t][3])), ps[t].c, reached(ps[t].lv)));
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float mn = fmaxf(m, top - kLift);
      const float fade = exp2_fast(m - mn);
      l *= fade;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] *= fade;
      m = mn;
      weigh();
    }
    l = fmaf(sum[0], ps[0].inv, l);
    l = fmaf(sum[1], ps[1].inv, l);
    const u32x4 pw = u32x4{pack_f16(w[0], w[1]), pack_f16(w[2], w[3]), pack_f16(w[4], w[5]), pack_f16(w[6], w[7])};
    const f16x8 pf = __builtin_bit_cast(f16x8, pw);
    // value operands of the 16-wide tiles of dword x: key pairs of each byte
    auto values = [&](int x, u32x4* out) {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const uint32_t a0 = to_f16<F, false>(cur.v[j][x]), a1 = to_f16<F, true>(cur.v[j][x]);
        const uint32_t b0 = to_f16<F, false>(cur.v[j + 1][x]), b1 = to_f16<F, true>(cur.v[j + 1][x]);
        out[0][j / 2] = __builtin_amdgcn_perm(b0, a0, 0x05040100u);
        out[1][j / 2] = __builtin_amdgcn_perm(b0, a0, 0x07060302u);
        out[2][j / 2] = __builtin_amdgcn_perm(b1, a1, 0x05040100u);
        out[3][j / 2] = __builtin_amdgcn_perm(b1, a1, 0x07060302u);
      }
    };
#pragma unroll
    for (int x = 0; x < VW; ++x) {
      u32x4 vf[4];
      values(x, vf);
#pragma unroll
      for (int d = 0; d < 4; ++d)
        o[4 * x + d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, vf[d]), pf, o[4 * x + d], 0, 0, 0);
    }
    cur = next;
  }
  // join the waves; o[4 x + d][i] is dimension (D/16) (4 g + i) + 4 x + d of row c
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (g == 0) sh_ml[wave][c] = make_float2(m, l);
  const bool wave_redo = __any(redo != 0);
  if (lane == 0) sh_redo[wave] = wave_redo;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int x = 0; x < VW; ++x)
      *reinterpret_cast<f32x4*>(&sh_o[wave][c][(D / 16) * (4 * g + i) + 4 * x]) =
          f32x4{o[4 * x][i], o[4 * x + 1][i], o[4 * x + 2][i], o[4 * x + 3][i]};
  __syncthreads();
  int any_redo = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) any_redo |= sh_redo[w];
  if (any_redo) {
    for (int row = wave; row < rows; row += W) {
      const int32_t rr = r0 + row;
      const int64_t t = s.tok0 + rr / group, h = int64_t(head) * group + rr % group;
      Range v = visible(a, s, rr / group);
      v = Range{v.lo > part.lo ? v.lo : part.lo, v.hi < part.hi ? v.hi : part.hi};
      float rm, rl, y[D / 64];
      careful_row<F, D>(a, b, head, t, h, v, rm, rl, y);
      careful_store<D>(a, parts, cut.chunks, chunk * parts.rows + (b * heads + head) * 16 + row, t, h, rm, rl, y);
    }
    return;
  }
  for (int e = threadIdx.x; e < rows * (D / 4); e += 64 * W) {
    const int row = e / (D / 4), d = e % (D / 4) * 4;
    float base = kNoKey;
#pragma unroll
    for (int w = 0; w < W; ++w) base = fmaxf(base, sh_ml[w][row].x);
    float lt = 0.0f;
    f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 ml = sh_ml[w][row];
      const float f = exp2_fast(ml.x - base);
      lt += ml.y * f;
      y += *reinterpret_cast<const f32x4*>(&sh_o[w][row][d]) * f;
    }
    const int32_t rr = r0 + row, ri = cut.by_group.div(rr);
    const int64_t t = s.tok0 + ri, h = int64_t(head) * group + (rr - ri * group);
    if (cut.chunks == 1) {
      const float inv = lt != 0.0f ? kUnlift / lt : 0.0f;
      *reinterpret_cast<u32x2*>(a.y + t * a.ldy + h * a.hdy + d) =
          u32x2{pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv)};
      if (a.lse && d == 0) a.lse[t * a.q_heads + h] = lt != 0.0f ? (base + log2_fast(lt)) * kLn2 : -INFINITY;
    } else {
      const int64_t at = chunk * parts.rows + (b * heads + head) * 16 + row;
      *reinterpret_cast<f32x4*>(parts.o + at * D + d) = y * kUnlift;
      if (d == 0) parts.ml[at] = make_float2(base, lt);
    }
  }
}

// ---------------------------------------------------------------------------
// 32 query rows a wave, 4 or 8 waves a workgroup: prompts and chunks of prompts.  Tiles of 64 keys
// are widened once into LDS (keys to bf16, values to fp16) while the tile before is computed
// from the other buffer, one barrier a tile.  Rows of 2 D bytes are
// stored with their 16-byte (keys) or 64-byte (values) pieces permuted by the key, so that the
// operand reads -- 16 bytes of 16 keys; 8 bytes of 4 keys, transposed by ds_read_b64_tr_b16 --
// touch every bank once.
// Bound by issue: a tile and wave are 32 matrix instructions (1024 cycles), about 235 vector
// instructions, 32 exponentials among them (1080 cycles), and LDS reads that a CU's waves
// share (a wave's 32 rows use each operand once).  Matrix cores busy 44% of the time, vector units 47%.  64 rows
// a wave would halve the LDS reads, but leave one wave a SIMD and move accumulators between register
// files: 1666 us against 1288 then.  8 waves share a tile's widening: 1131 us against 1228 with 4.
// An 8192-token prompt, 64 heads over 8 of 128: 1.08 to 1.15 ms between cards, 0.96 to 1.02 PFLOP/s, where a bf16
// library product of 8192^3 reaches 1.19.
constexpr int kBK = 64;

template <int D>
__device__ __forceinline__ int key_at(int key, int piece) {  // byte offset of a 16-byte piece of a key
  const int x = D == 128 ? (key & 15) : ((key >> 1) & 7);
  return key * (2 * D) + ((piece ^ x) << 4);
}
template <int D>
__device__ __forceinline__ int val_at(int key, int byte) {  // byte offset of a byte of a value row
  const int x = D == 128 ? (key & 3) : ((key >> 1) & 1);
  return key * (2 * D) + (byte ^ (x << 6));
}

__device__ __forceinline__ u32x2 read_tr(const uint8_t* p) {
  const i16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) i16x4*)(p));
  return __builtin_bit_cast(u32x2, v);
}

template <int F, int D, int NW>
__global__ void __launch_bounds__(64 * NW, 2) k_attend_many(AttendArgs a, Cut cut, Parts parts) {
  constexpr int NP = D / (16 * NW);  // 16-byte pieces of keys, and of values, that a thread stages
  constexpr int WG = 32 * NW;        // query rows
  constexpr int KS = D / 16;   // matrix steps along the dimensions
  constexpr int DT = D / 32;   // 32-wide output tiles
  constexpr int kBuf = kBK * D * 2;  // bytes of one buffer of keys, and of values
  __shared__ __align__(16) uint8_t sh[4 * kBuf];  // keys 0, keys 1, values 0, values 1
  __shared__ __align__(16) float4 sh_p[2][4];     // PartScale of the tile's 16-key parts; scales not finite
  __shared__ int sh_odd[2];                       // the last tile of this buffer with a value code that is not finite
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 31, h = lane >> 5;
  const int32_t heads = a.p.heads, group = static_cast<int32_t>(cut.by_group.d);
  const Place place = place_of(blockIdx.x, cut);
  const int32_t head = place.head, chunk = place.chunk;
  const int32_t r0 = (cut.by_tiles.d - 1 - place.tile) * WG;  // causal: the longest first
  const int64_t b = place.b;
  const SeqSpan s = seq_span(a.p, b);
  const int64_t all = int64_t(s.n) * group;
  if (r0 >= all || (cut.mixed && all <= 16)) return;
  const int32_t rows = all - r0 < WG ? static_cast<int32_t>(all - r0) : WG;
  const Range tile = tile_range(a, s, r0, rows, cut.by_group);
  const Range part = chunk_of(tile, cut, chunk);
  if (chunk > 0 && part.lo >= part.hi) return;
  const int32_t page = a.p.page, shift = 31 - __builtin_clz(page);
  // positions that some row of the workgroup sees, that all of them see; the same for this wave
  const int32_t wr = rows - 32 * wave < 32 ? rows - 32 * wave : 32;  // rows of this wave (may be <= 0)
  const Range wg_first = visible(a, s, cut.by_group.div(r0)), wg_last = visible(a, s, cut.by_group.div(r0 + rows - 1));
  const int32_t any_lo = wg_first.lo, all_lo = wg_last.lo, all_hi = wg_first.hi;
  const int32_t r = r0 + 32 * wave + (c < wr ? c : 0);  // this lane's query row
  const int32_t ti = wr > 0 ? cut.by_group.div(r) : 0;
  const int64_t tok = s.tok0 + ti;
  const int64_t qh = int64_t(head) * group + (wr > 0 ? r - ti * group : 0);
  Range see = {0, 0}, w_all = {0, 0}, w_any = {0, 0};
  if (wr > 0) {
    const Range f = visible(a, s, cut.by_group.div(r0 + 32 * wave)), e = visible(a, s, cut.by_group.div(r0 + 32 * wave + wr - 1));
    w_all = Range{e.lo, f.hi};
    w_any = Range{f.lo, e.hi};
    if (c < wr) see = visible(a, s, ti);
    if (wr < 32) w_all.hi = w_all.lo;  // idle rows see nothing: every tile is an edge
    see.hi = see.hi < part.hi ? see.hi : part.hi;
    see.hi = see.hi > see.lo ? see.hi : see.lo;
  }
  const float sm = fabsf(a.sm_scale) * kLog2e;
  const uint32_t flip = a.sm_scale < 0.0f ? 0x80008000u : 0u;
  u32x4 q[KS];
#pragma unroll
  for (int i = 0; i < KS; ++i) {
    q[i] = *reinterpret_cast<const u32x4*>(a.q + tok * a.ldq + qh * a.hdq + 16 * i + 8 * h);
#pragma unroll
    for (int j = 0; j < 4; ++j) q[i][j] ^= flip;
  }
  f32x16 o[DT] = {};
  float m = kNoKey, l = 0.0f;

  // operand addresses of this lane: the permuted pieces differ per dimension step,
  // everything else is an offset known when compiling
  uint32_t ka[KS], va[DT];
#pragma unroll
  for (int i = 0; i < KS; ++i) ka[i] = key_at<D>(c, 2 * i + h);
#pragma unroll
  for (int d = 0; d < DT; ++d)  // keys 4 h + (lane & 15) / 4, dimensions 32 d + 16 (lane / 16 & 1) + 4 (lane & 3)
    va[d] = 2 * kBuf + val_at<D>(4 * h + (lane & 15) / 4, 64 * d + 32 * ((lane >> 4) & 1) + 8 * (lane & 3));

  // staging: this thread's pieces are bytes [16 sp, 16 sp + 16) of keys sk + 64 / NP * i.  A wave's
  // keys of one piece lie in one 16-key part, so its page is the same for all lanes.
  constexpr int TK = D / 16;           // threads of a key
  constexpr int PK = kBK / NP;         // keys between a thread's pieces
  constexpr int WK = 64 / TK;          // keys of a wave's piece
  const int sk = threadIdx.x / TK, sp = threadIdx.x % TK;
  const uint32_t lane_at = (lane / TK) * D + 16 * sp;
  // the piece whose part's scales this wave takes, and the part (16 keys are one or two waves' pieces)
  const int mine = NP == 2 ? wave & 1 : 0;
  const int mine_part = NP == 2 ? (wave >> 1) + 2 * (wave & 1) : WK == 16 ? wave : wave >> 1;
  // looked up by vector loads, which retire in order with the tiles' (a scalar load
  // would make every wait for an LDS read wait for it too)
  const int32_t* table = a.p.table + b * a.p.ld_table + hidden_zero();
  const uint32_t page_bytes = static_cast<uint32_t>(page) * D, pages = static_cast<uint32_t>(a.p.pages);
  u32x4 kr[NP], vr[NP];
  int32_t entry[NP];   // table entries of the pieces fetched next
  bool there[NP];      // the page of the piece fetched last is present
  float ksr, vsr;
  // (positions past the end look up the last page: every load is of a page of the table)
  auto look_up = [&](int32_t k0) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int32_t j = k0 + WK * wave + PK * i;
      entry[i] = table[(j < part.hi ? j : part.hi - 1) >> shift];
    }
  };
  auto fetch = [&](int32_t k0) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int32_t j = k0 + WK * wave + PK * i;
      const uint32_t pg = __builtin_amdgcn_readfirstlane(entry[i]);
      there[i] = pg < pages;
      const uint64_t ph = uint64_t(there[i] ? pg : 0u) * static_cast<uint32_t>(heads) + static_cast<uint32_t>(head);
      const uint64_t at = ph * page_bytes + static_cast<uint32_t>((j & (page - 1)) * D);
      kr[i] = *reinterpret_cast<const u32x4*>(a.kc + at + lane_at);
      vr[i] = *reinterpret_cast<const u32x4*>(a.vc + at + lane_at);
      if (i == mine) {
        ksr = (a.ks + ph)[hidden_zero()];
        vsr = (a.vs + ph)[hidden_zero()];
      }
    }
  };
  // Before its codes are widened into LDS, a tile may need repairs: codes of 0 for pages that
  // are not there and for values that no row sees, a look at the values that some row does not
  // see; and its scales.  (Keys past the end need none: their scores are hidden.)
  auto repair = [&](int buf, int index) {
    const int32_t k0 = part.lo + kBK * index;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if (!there[i]) kr[i] = vr[i] = u32x4{0u, 0u, 0u, 0u};
      if (k0 < all_lo || k0 + kBK > all_hi || k0 + kBK > part.hi) {
        const int32_t key = k0 + sk + PK * i;
        uint32_t odd = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          vr[i][e] = key >= any_lo && key < part.hi ? vr[i][e] : 0u;
          odd |= non_finite<F>(vr[i][e]);
        }
        if (odd) sh_odd[buf] = index;
      }
    }
    const bool here = there[mine];
    const PartScale ps = part_scale(here, ksr, vsr, sm);
    if (lane == 0)
      sh_p[buf][mine_part] = make_float4(ps.c, ps.lv, ps.inv, here && !finite_scales(ksr, vsr) ? 1.0f : 0.0f);
  };
  const uint32_t kst0 = key_at<D>(sk, 2 * sp), kst1 = key_at<D>(sk, 2 * sp + 1), vst = 2 * kBuf + val_at<D>(sk, 32 * sp);
  auto stage = [&](int buf, int share, int shares) {  // one of `shares` equal shares of the widening
    const uint32_t at = buf * kBuf;
#pragma unroll
    for (int u = 4 * NP * share / shares; u < 4 * NP * (share + 1) / shares; ++u) {
      const int i = u / 4, x = u % 2 * 2;
      const uint32_t row = at + PK * i * (2 * D);
      if (u % 4 < 2)
        *reinterpret_cast<u32x4*>(sh + (x ? kst1 : kst0) + row) = bf16_of<F>(kr[i][x], kr[i][x + 1]);
      else
        *reinterpret_cast<u32x4*>(sh + vst + (row + 8 * x)) = f16_of<F>(vr[i][x], vr[i][x + 1]);
    }
  };
  const int32_t steps = (part.hi - part.lo + kBK - 1) / kBK;
  if (threadIdx.x < 2) sh_odd[threadIdx.x] = -1;
  __syncthreads();
  int redo = 0;
  if (steps > 0) {
    look_up(part.lo);
    fetch(part.lo);
    look_up(part.lo + kBK);
    repair(0, 0);
    stage(0, 0, 1);
  }
  __syncthreads();
  auto step = [&](int32_t t, auto which) {
    constexpr int buf = decltype(which)::value;
    const int32_t k0 = part.lo + kBK * t;
    if (t + 1 < steps) {
      fetch(k0 + kBK);
      look_up(k0 + 2 * kBK);
    }
    const bool more = t + 1 < steps;
    if (k0 < w_any.hi && k0 + kBK > w_any.lo) {
      constexpr uint32_t at = buf * kBuf;
      const bool edge = k0 < w_all.lo || k0 + kBK > w_all.hi || k0 + kBK > part.hi;
      auto key_of = [&](int kt, int i) {
        return *reinterpret_cast<const bf16x8*>(sh + ka[i] + (at + 32 * kt * (2 * D)));
      };
      // values of part e, output tile d: keys 16 e + {0..3, 8..11} + 4 h, dimension 32 d + c
      auto value_of = [&](int e, int d) {
        const uint8_t* v = sh + va[d];
        const u32x2 lo = read_tr(v + (at + 16 * e * (2 * D))), hi = read_tr(v + (at + (16 * e + 8) * (2 * D)));
        return __builtin_bit_cast(f16x8, (u32x4{lo[0], lo[1], hi[0], hi[1]}));
      };
      // register 8 e + i of part 2 kt + e is key 32 kt + 16 e + 8 (i / 4) + 4 h + i % 4
      f32x16 z[2] = {};
      auto hide = [&](int kt) {
        const int32_t from = see.lo - k0 - 4 * h;
        const uint32_t n = see.hi - see.lo;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          z[kt][i] = static_cast<uint32_t>(32 * kt + 8 * (i / 4) + i % 4 - from) < n ? z[kt][i] : -INFINITY;
      };
      float pc[4], plv[4], pinv[4];  // the scales of the tile's 16-key parts, the same in every lane
      u32x4 pw[4];   // weights of the parts
      float sum[4];  // this lane's sums of them
      auto weigh = [&](int kt, int i, int n) {  // scores i .. i + n of half kt
#pragma unroll
        for (int k = i; k < i + n; k += 2) {
          const int e = 2 * kt + k / 8;
          const float w0 = exp2_fast(fmaf(z[kt][k], pc[e], plv[e] - m)), w1 = exp2_fast(fmaf(z[kt][k + 1], pc[e], plv[e] - m));
          sum[e] = k % 8 == 0 ? w0 + w1 : sum[e] + (w0 + w1);
          pw[e][k % 8 / 2] = pack_f16(w0, w1);
        }
      };
      auto follow = [&](int kt) {  // too large for fp16: m follows the maximum
        if (__any(!(fmaxf(sum[2 * kt], sum[2 * kt + 1]) < kFull))) {
          float top = kNoKey;
#pragma unroll
          for (int e = 2 * kt; e < 2 * kt + 2; ++e) {
            float x = -INFINITY;
#pragma unroll
            for (int i = 0; i < 8; ++i) x = fmaxf(x, z[kt][8 * (e % 2) + i]);
            top = fmaxf(top, fmaf(x, pc[e], reached(plv[e])));
          }
          top = fmaxf(top, __shfl_xor(top, 32));
          const float mn = fmaxf(m, top - kLift);
          const float fade = exp2_fast(m - mn);
          l *= fade;
#pragma unroll
          for (int d = 0; d < DT; ++d) o[d] *= fade;
          m = mn;
          weigh(kt, 0, 16);
        }
        l = fmaf(sum[2 * kt], pinv[2 * kt], l);
        l = fmaf(sum[2 * kt + 1], pinv[2 * kt + 1], l);
      };
      // The matrix cores' work on one half of the tile runs under the exponentials of the
      // other, and the last products under the widening of the next tile: a matrix
      // instruction takes 8 passes of 4 cycles, in which this wave issues other work.
      constexpr int kAhead = 3;  // operands read ahead of their use
      bf16x8 kf[KS];
      auto scores = [&](int kt, auto&& under) {
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          if (i + kAhead < KS) kf[i + kAhead] = key_of(kt, i + kAhead);
          z[kt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[i], __builtin_bit_cast(bf16x8, q[i]), z[kt], 0, 0, 0);
          under(i);
          pin();
        }
      };
      f16x8 vf[2 * DT];
      auto add = [&](int kt, auto&& under) {
#pragma unroll
        for (int i = 0; i < 2 * DT; ++i) {
          if (i + kAhead < 2 * DT) vf[i + kAhead] = value_of(2 * kt + (i + kAhead) / DT, (i + kAhead) % DT);
          o[i % DT] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[i], __builtin_bit_cast(f16x8, pw[2 * kt + i / DT]),
                                                             o[i % DT], 0, 0, 0);
          under(i);
          pin();
        }
      };
      auto ahead_k = [&](int kt) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) kf[i] = key_of(kt, i);
      };
      auto ahead_v = [&](int kt) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) vf[i] = value_of(2 * kt + i / DT, i % DT);
      };
      ahead_k(0);
      float4 ps[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) ps[e] = sh_p[buf][e];
      pin();
      urgent<2>();
      scores(0, [&](int i) {
        if (i == KS - 1) ahead_k(1);
      });
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        pc[e] = uniform(ps[e].x);
        plv[e] = uniform(ps[e].y);
        pinv[e] = uniform(ps[e].z);
        redo |= __builtin_amdgcn_readfirstlane(__float_as_int(ps[e].w));
      }
      if (edge) {
        redo |= sh_odd[buf] == t;
        hide(0);
      }
      urgent<1>();
      scores(1, [&](int i) {
        weigh(0, 16 / KS * i, 16 / KS);
        if (i == KS - 1) ahead_v(0);
      });
      follow(0);
      if (edge) hide(1);
      add(0, [&](int i) {
        weigh(1, 16 / (2 * DT) * i, 16 / (2 * DT));
        if (i == 2 * DT - 1) ahead_v(1);
      });
      urgent<0>();
      follow(1);
      if (more) {
        repair(buf ^ 1, t + 1);
        add(1, [&](int i) { stage(buf ^ 1, i, 2 * DT); });
      } else {
        add(1, [](int) {});
      }
    } else if (more) {
      repair(buf ^ 1, t + 1);
      stage(buf ^ 1, 0, 1);
    }
    __syncthreads();
  };
  for (int32_t t = 0; t < steps; t += 2) {
    step(t, std::integral_constant<int, 0>{});
    if (t + 1 < steps) step(t + 1, std::integral_constant<int, 1>{});
  }
  if (redo) {
    for (int row = 0; row < wr; ++row) {
      const int32_t rr = r0 + 32 * wave + row;
      const int64_t ti = s.tok0 + rr / group, hi = int64_t(head) * group + rr % group;
      Range v = visible(a, s, rr / group);
      v = Range{v.lo > part.lo ? v.lo : part.lo, v.hi < part.hi ? v.hi : part.hi};
      float rm, rl, y[D / 64];
      careful_row<F, D>(a, b, head, ti, hi, v, rm, rl, y);
      careful_store<D>(a, parts, cut.chunks, chunk * parts.rows + ti * a.q_heads + hi, ti, hi, rm, rl, y);
    }
    return;
  }
  l += __shfl_xor(l, 32);
  if (c >= wr) return;
  const float inv = l != 0.0f ? kUnlift / l : 0.0f;
  const int64_t at = chunk * parts.rows + tok * a.q_heads + qh;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int dim = 32 * d + 8 * i + 4 * h;
      const f32x4 y = {o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
      if (cut.chunks == 1)
        *reinterpret_cast<u32x2*>(a.y + tok * a.ldy + qh * a.hdy + dim) =
            u32x2{pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv)};
      else
        *reinterpret_cast<f32x4*>(parts.o + at * D + dim) = y * kUnlift;
    }
  if (h == 0) {
    if (cut.chunks > 1)
      parts.ml[at] = make_float2(m, l);
    else if (a.lse)
      a.lse[tok * a.q_heads + qh] = l != 0.0f ? (m + log2_fast(l)) * kLn2 : -INFINITY;
  }
}

// ---------------------------------------------------------------------------
// Adds the chunks of a query row: with M = max m_i,
// y = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.  D / 4 threads take a chunk, `lanes` (a power of
// two, at most the 256 / (D / 4) chunks that a workgroup reads at once) groups of them a row, and a
// workgroup as many rows as that leaves room for: the kernel is a chain of loads, and its length is
// what it costs (32 chunks of 128 rows: 5 us; one wave a row took 10 to 29).
template <int D, bool FEW>
__global__ void __launch_bounds__(256) k_attend_join(AttendArgs a, Cut cut, int32_t tile_rows, int32_t lanes, Parts parts) {
  constexpr int T = D / 4, G = 256 / T;  // threads of a chunk, chunks at once
  __shared__ __align__(16) f32x4 sh_y[G][T];
  __shared__ float2 sh_ml[G];
  const int x = threadIdx.x % T, y = threadIdx.x / T, part = y & (lanes - 1);
  const int32_t group = static_cast<int32_t>(cut.by_group.d);
  const uint32_t r = blockIdx.x * (G / lanes) + y / lanes;  // row of the parts
  bool on = r < parts.rows;
  float m = kNoKey, l = 0.0f;
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  int64_t tok = 0, h = 0;
  if (on) {
    int64_t b, i;
    if (FEW) {  // (sequence, head, row)
      const uint32_t bh = r >> 4, row = r & 15;
      b = cut.by_heads.div(bh);
      i = cut.by_group.div(row);
      h = (bh - static_cast<uint32_t>(b) * cut.by_heads.d) * group + (row - i * group);
    } else {    // (token, query head): its sequence is the last that starts at or before it
      tok = cut.by_chunks.div(r);  // by_chunks: the query heads here
      h = r - static_cast<uint32_t>(tok) * cut.by_chunks.d;
      int64_t lo = 0, hi = a.p.seqs;
      while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if (a.p.seq_start[mid] <= tok) lo = mid;
        else hi = mid;
      }
      b = lo;
      i = 0;
    }
    const SeqSpan s = seq_span(a.p, b);
    if (!FEW) i = tok - s.tok0;
    const int64_t all = int64_t(s.n) * group;
    on = i >= 0 && i < s.n && (!cut.mixed || (all <= 16) == FEW);
    if (on) {
      tok = s.tok0 + i;
      const int32_t hg = static_cast<int32_t>(h) - static_cast<int32_t>(cut.by_group.div(static_cast<uint32_t>(h))) * group;
      const int32_t r0 = (static_cast<int32_t>(i) * group + hg) & ~(tile_rows - 1);
      const int64_t left = all - r0;
      const Range tile = tile_range(a, s, r0, left < tile_rows ? static_cast<int32_t>(left) : tile_rows, cut.by_group);
      int32_t n = (int64_t(tile.hi) - tile.lo + cut.len - 1) / cut.len;
      n = n < 1 ? 1 : n > cut.chunks ? cut.chunks : n;
#pragma unroll 4
      for (int32_t k = part; k < n; k += lanes) {
        const float2 ml = parts.ml[k * parts.rows + r];
        const f32x4 v = *reinterpret_cast<const f32x4*>(parts.o + (k * parts.rows + r) * D + 4 * x);
        const float mn = fmaxf(m, ml.x), fa = exp2_fast(m - mn), fb = exp2_fast(ml.x - mn);
        l = l * fa + ml.y * fb;
        o = o * fa + v * fb;
        m = mn;
      }
    }
  }
  sh_y[y][x] = o;
  if (x == 0) sh_ml[y] = make_float2(m, l);
  __syncthreads();
  if (!on || part != 0) return;
  float base = kNoKey;
  for (int k = 0; k < lanes; ++k) base = fmaxf(base, sh_ml[y + k].x);
  l = 0.0f;
  o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int k = 0; k < lanes; ++k) {
    const float f = exp2_fast(sh_ml[y + k].x - base);
    l += sh_ml[y + k].y * f;
    o += sh_y[y + k][x] * f;
  }
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
  *reinterpret_cast<u32x2*>(a.y + tok * a.ldy + h * a.hdy + 4 * x) =
      u32x2{pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
  if (a.lse && x == 0) a.lse[tok * a.q_heads + h] = l != 0.0f ? (base + log2_fast(l)) * kLn2 : -INFINITY;
}

}  // namespace

namespace {

// One kernel's share of a call: its tiles, how their keys are cut, its parts.
struct Plan {
  int64_t tile_rows, jobs;  // jobs: workgroups without a cut
  Cut cut;
  Parts parts;
};

// Cut the keys when the jobs alone do not fill the card.  Prompts: when they leave half of the
// workgroups that the CUs hold free.  Decode (1 a CU): a long stream per workgroup costs
// least (two sequences of 131072 tokens, 8 heads: 92 us in 256 chunks, 101 in 2048, and the parts'
// addition 5 and 7 us), so 1 a CU, and 2 from 8 sequences on, whose ragged lengths then even out; chunks of at
// least 1024 keys, below which the second launch costs more than the cut saves (1001 keys: 10.6 us
// uncut, 8.6 + 3.9 in halves).  Prompts' steps of 64 keys take 2 us each, so theirs may be shorter:
// 512 keys, 256 where they leave most CUs idle.  A window bounds what a causal tile can see.
// The host knows bounds only.  Sequences drawn evenly from 1 to 8192 tokens even out (64 / 96 / 128 of them, 8 heads: 107 / 157 /
// 190 us for 94 / 131 / 164 of reading); a single long one does not, since its workgroups are as many as a short one's (131072 tokens
// among 63 / 31 sequences of 1000: 724 / 369 us for 65 / 54 of reading).  A max_kv far above the lengths makes one chunk of
// each sequence and still pays for the join (8 of 2000 tokens: 17 us, under a bound of 131072 24).
Plan plan_for(const AttendArgs& a, bool few, bool mixed, int64_t tile_rows, int64_t tiles) {
  const int64_t group = a.q_heads / a.p.heads, cus = device_cus();
  Plan p;
  p.tile_rows = tile_rows;
  p.jobs = a.p.seqs * tiles * a.p.heads;
  int64_t span = a.max_kv, len = 0;
  if (a.causal && a.window > 0) span = std::min(span, a.window + tile_rows / group + 64);
  if (few) {
    const int64_t want = ceil_div((a.p.seqs < 8 ? 1 : 2) * cus, p.jobs);
    if (want > 1) len = std::max<int64_t>(1024, ceil_div(ceil_div(span, want), 64) * 64);
  } else {
    // tiles that the tokens can fill, and workgroups that fit at once (registers; of the widest only
    // half as many do, which then run in two rounds)
    const int64_t busy = std::min(p.jobs, (a.p.tokens * group / tile_rows + a.p.seqs) * a.p.heads);
    const int64_t fit = (a.p.dim == 64 ? 3 : 2) * cus;
    if (2 * busy <= fit)
      len = std::max<int64_t>(4 * busy > cus ? 512 : 256, ceil_div(ceil_div(span, ceil_div(fit, busy)), 64) * 64);
  }
  Cut& c = p.cut;
  c.chunks = len > 0 ? static_cast<int32_t>(ceil_div(span, len)) : 1;
  c.len = c.chunks > 1 ? static_cast<int32_t>(len) : 64;
  c.ordered = few && c.chunks == 1 && p.jobs > cus && a.p.seqs <= 64;
  c.mixed = mixed;
  c.by_heads = FastDiv(a.p.heads);
  c.by_tiles = FastDiv(static_cast<uint32_t>(tiles));
  c.by_chunks = FastDiv(c.chunks);
  c.by_group = FastDiv(static_cast<uint32_t>(group));
  p.parts = Parts{nullptr, nullptr, few ? a.p.seqs * a.p.heads * 16 : a.p.tokens * a.q_heads};
  return p;
}

size_t part_floats(const Plan& p, int dim) {
  return p.cut.chunks > 1 ? size_t(p.cut.chunks) * p.parts.rows * (dim + 2) : 0;
}

template <typename K>
hipError_t launch_tiles(K kern, const AttendArgs& a, const Plan& p, int waves, hipStream_t st) {
  hipLaunchKernelGGL(kern, dim3(p.jobs * p.cut.chunks), dim3(64 * waves), 0, st, a, p.cut, p.parts);
  return hipGetLastError();
}

template <bool FEW>
hipError_t launch_join(const AttendArgs& a, const Plan& p, hipStream_t st) {
  Cut cut = p.cut;
  if (!FEW) cut.by_chunks = FastDiv(static_cast<uint32_t>(a.q_heads));
  const int32_t at_once = 1024 / a.p.dim;
  int32_t lanes = 1;
  while (lanes < at_once && lanes < cut.chunks) lanes <<= 1;
  const dim3 grid(static_cast<uint32_t>(ceil_div(p.parts.rows, at_once / lanes)));
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, dim3(256), 0, st, a, cut, static_cast<int32_t>(p.tile_rows), lanes, p.parts);
  };
  a.p.dim == 128 ? go(k_attend_join<128, FEW>) : go(k_attend_join<64, FEW>);
  return hipGetLastError();
}

template <int F>
hipError_t launch_attention(const AttendArgs& a, hipStream_t st) {
  const int64_t rows = a.p.max_new * (a.q_heads / a.p.heads);
  // A batch whose sequences bring at most half of max_new on average may hold single tokens beside
  // prompts; a prompt's workgroup would read such a sequence at one wave's pace, so each kernel
  // then runs for its own (one prompt of 2000 tokens among 64 / 200 sequences of 4000, 64 / 8 heads: 229 / 501 us,
  // in one kernel 393 / 907; where no sequence is short the second launch costs 3.5).  Fewer single tokens than
  // prompts do not meet this: one prompt of 2000 tokens and one token behind 32768 take 848 us, in two calls 100 and 20.
  const bool few = rows <= 16;
  const bool mixed = !few && a.q_heads / a.p.heads <= 16 && 2 * a.p.tokens <= a.p.seqs * a.p.max_new;
  const bool wide = !few && a.p.dim == 128 && a.p.seqs * (rows / 256) * a.p.heads >= 2 * device_cus();
  const int64_t tile_rows = wide ? 256 : 128;
  Plan f = plan_for(a, true, mixed, 16, 1), m = plan_for(a, false, mixed, tile_rows, ceil_div(rows, tile_rows));
  const size_t nf = few || mixed ? part_floats(f, a.p.dim) : 0, nm = few ? 0 : part_floats(m, a.p.dim);
  if (nf + nm > 0) {
    void* mem = nullptr;
    const hipError_t e = get_scratch(st, (nf + nm) * sizeof(float), &mem);
    if (e != hipSuccess) return e;
    auto place = [&](Plan& p, float* at) {
      p.parts.o = at;
      p.parts.ml = reinterpret_cast<float2*>(at + size_t(p.cut.chunks) * p.parts.rows * a.p.dim);
    };
    place(f, static_cast<float*>(mem));
    place(m, static_cast<float*>(mem) + nf);
  }
  hipError_t e = hipSuccess;
  if (few || mixed) {
    e = a.p.dim == 128 ? launch_tiles(k_attend_few<F, 128>, a, f, kFewWaves, st)
                       : launch_tiles(k_attend_few<F, 64>, a, f, kFewWaves, st);
    if (e == hipSuccess && f.cut.chunks > 1) e = launch_join<true>(a, f, st);
  }
  if (!few && e == hipSuccess) {
    e = wide              ? launch_tiles(k_attend_many<F, 128, 8>, a, m, 8, st)
        : a.p.dim == 128 ? launch_tiles(k_attend_many<F, 128, 4>, a, m, 4, st)
                         : launch_tiles(k_attend_many<F, 64, 4>, a, m, 4, st);
    if (e == hipSuccess && m.cut.chunks > 1) e = launch_join<false>(a, m, st);
  }
  return e;
}

}  // namespace

hipError_t launch_paged_attention(const AttendArgs& a, hipStream_t st) {
  return a.p.fmt == FP8RT_E4M3 ? launch_attention<kE4M3>(a, st) : launch_attention<kE5M2>(a, st);
}

}  // namespace fp8rt
