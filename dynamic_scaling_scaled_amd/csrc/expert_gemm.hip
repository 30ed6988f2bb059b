// expert_gemm.hip -- the experts' scaled products: rows of FP8 codes, gathered by the
// router's plan, against each expert's FP8 weights (one fragment-ordered image).
//
//   y[s,n] = s_a(r) s_b(e,n) sum_k dec(a[r,k]) dec(b[e,n,k]),   offsets[e] <= s < offsets[e+1]
//
// Bounds: the weights of the experts that are used, read once (8 TB/s at most; a read-only pass over 4 GiB reaches 6.1), against
// 2 slots N K operations (5 PFLOP/s at most; the library product of 8192^3 reaches 3.15 and this library's large GEMM 2.3).
// Measured, 4096 x 7168 (N x K): one token of 8 experts 36.7 us (6.4 TB/s), a step of 64
// tokens, 8 of 128 experts, 498 us (6.3 TB/s), 1024 slots for each of 32 experts 775 to 810 us (2.38 to 2.48 PFLOP/s); 7168 x 2048,
// 2804 slots very unequally over 32 experts 106 us (4.2 TB/s: the few experts with hundreds of slots are bound by
// the matrix cores while the others' weights arrive, and a workgroup has 16 stages only).
#include <algorithm>

#include "gemm_tile.h"
#include "internal.h"

namespace fp8rt {

namespace {

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

// Work unit of workgroup b of the tile kernel: (row tile of TM slots, column tile).  Experts one after the other; inside an
// expert groups of 4 row tiles go through the column tiles together; each XCD (workgroups are dealt to the 8 in turn)
// gets a contiguous range of that order, so that its L2 serves what neighbours share.  False past the last.
template <int TM>
__device__ __forceinline__ bool find_unit(const ExpertGemmArgs& g, int b, int col_tiles, Tile& t, int& col) {
  const int lane = threadIdx.x & 63, E = static_cast<int>(g.experts);
  int lo0 = 0, hi0 = 0;  // the first 64 experts' slots are kept for the second pass
  if (lane < E) expert_slots(g, lane, lo0, hi0);
  int units = (hi0 - lo0 + TM - 1) / TM * col_tiles;
  for (int e = 64 + lane; e < E; e += 64) {
    int lo, hi;
    expert_slots(g, e, lo, hi);
    units += (hi - lo + TM - 1) / TM * col_tiles;
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) units += __shfl_xor(units, o);
  units = __builtin_amdgcn_readfirstlane(units);
  if (b >= units) return false;
  const int xcd = b & 7, per = units >> 3, more = units & 7;
  int index = xcd * per + min(xcd, more) + (b >> 3);
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    int lo = lo0, hi = hi0;
    if (e0 > 0) {
      lo = hi = 0;
      if (e < E) expert_slots(g, e, lo, hi);
    }
    const int n = (hi - lo + TM - 1) / TM;
    int s = n * col_tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(s, o);
      if (lane >= o) s += up;
    }
    const uint64_t past = __ballot(s > index);
    if (past) {
      const int at = __ffsll(static_cast<unsigned long long>(past)) - 1;
      const int rows = __builtin_amdgcn_readlane(n, at);
      index -= __builtin_amdgcn_readlane(s, at) - rows * col_tiles;
      // (Never so: of 1024 experts at most 512 can claim all slots, whose units stay below 2^31 by the host's bound on tiles.  A
      // unit outside its expert would be written outside y.)
      if (index < 0 || index >= rows * col_tiles) return false;
      const int first = index / (4 * col_tiles) * 4, in = index - first * col_tiles, m = min(4, rows - first);
      t.expert = e0 + at;
      t.row0 = __builtin_amdgcn_readlane(lo, at) + static_cast<int64_t>(first + in % m) * TM;
      t.end = __builtin_amdgcn_readlane(hi, at);
      col = in / m;
      return true;
    }
    index -= __builtin_amdgcn_readlane(s, 63);
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

// ---------------------------------------------------------------------------
// Many rows an expert: tiles of 256 slots by 256 columns, 4 waves of 64 columns each.
//  - B needs no LDS: the image holds matrix operands, and a wave is the only reader of its 64 columns.  Its 8 loads of a
//    128-deep stage (1 KB each) go to one of three register sets, two stages ahead.
//  - A is read by all four waves: its rows move to a ring of four 32 KB stages in LDS (direct loads, 16-byte chunks of a
//    row XOR-swizzled by row / 2 against bank conflicts), three stages ahead; one barrier a stage, halfway through,
//    where every wave's part of the next stage has landed and the stage before this one has been read by all.
//  - A wave's accumulators are 16 x 4 tiles of 16 x 16 (256 AGPRs, updated in place); each fragment of A is
//    read two row tiles before its 4 MFMAs.
//  - A tile of fewer slots runs the same loop over its blocks of 64 (NB = 1 .. 4).
constexpr int kTN = 256, kRing = 4;
constexpr int kTileThreads = 256;

// Waits until at most N of this wave's vector-memory operations are outstanding, then joins the workgroup's barrier; LDS
// reads and younger loads keep flying.
template <int N>
__device__ __forceinline__ void stage_barrier() {
  static_assert(N < 64, "vmcnt field");
  __builtin_amdgcn_sched_barrier(0);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(((N >> 4) << 14) | 0x0F70 | (N & 15));
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_sched_barrier(0);
}

// Wait states between VALU accesses of 16 accumulators and inline MFMAs: 24, more than the 8-pass MFMA's distances.
__device__ __forceinline__ void fence16(f32x4 (&a)[4][4]) {
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7"
               : "+a"(a[0][0]), "+a"(a[0][1]), "+a"(a[0][2]), "+a"(a[0][3]), "+a"(a[1][0]), "+a"(a[1][1]),
                 "+a"(a[1][2]), "+a"(a[1][3]), "+a"(a[2][0]), "+a"(a[2][1]), "+a"(a[2][2]), "+a"(a[2][3]),
                 "+a"(a[3][0]), "+a"(a[3][1]), "+a"(a[3][2]), "+a"(a[3][3]));
}

template <int BLOCKS>
struct TileShared {  // for tiles of up to BLOCKS blocks of 64 slots
  static constexpr int kSlot = BLOCKS * 64 * 128;
  __attribute__((aligned(16))) uint8_t ring[kRing * kSlot];
  int row[64 * BLOCKS];  // the row of a of each slot, -1: none
  float scale[64 * BLOCKS];
};

// The operands of one wave of a tile, fixed over its stages.
struct TileOperands {
  __amdgpu_buffer_rsrc_t a;
  uint32_t voa[8];        // offsets of the rows that this lane loads
  __amdgpu_buffer_rsrc_t b;
  int goff[4];            // offsets of its groups of 16 columns
  int lo, hi;             // offsets of the lane's two chunks of A in row tile 0 of a stage
  int wave, lane, last;   // last: the last stage
};

__device__ __forceinline__ i32x8 load_b(const TileOperands& p, int j, int s) {
  const int at = p.goff[j] + min(s, p.last) * 2048;
  return join(__builtin_amdgcn_raw_buffer_load_b128(p.b, p.lane * 16, at, 0),
              __builtin_amdgcn_raw_buffer_load_b128(p.b, p.lane * 16 + 1024, at, 0));
}
template <int BLOCKS>
__device__ __forceinline__ void load_a(const TileOperands& p, TileShared<BLOCKS>& sh, int j, int s) {
  dma1(p.a, min(s, p.last) * 128, p.voa[j], sh.ring + (s & (kRing - 1)) * sh.kSlot, 4 * j + p.wave);
}
template <int BLOCKS>
__device__ __forceinline__ i32x8 frag_a(const TileOperands& p, const TileShared<BLOCKS>& sh, int i, int s) {
  const uint8_t* at = sh.ring + (s & (kRing - 1)) * sh.kSlot + i * 2048;
  return join(*reinterpret_cast<const u32x4*>(at + p.lo), *reinterpret_cast<const u32x4*>(at + p.hi));
}

// As mfma16, with b in AGPRs: loads write them directly, and a wave of 256 registers has too few of the others for three
// sets of B beside A's fragments (a set that the compiler moved there by itself was waited for as soon as it was loaded).
template <int FA>
__device__ __forceinline__ void mfma16_ab(f32x4& acc, const i32x8& b, const i32x8& a) {
  if constexpr (FA == 0)
    asm volatile("v_mfma_f32_16x16x128_f8f6f4 %0, %1, %2, %0" : "+a"(acc) : "a"(b), "v"(a));
  else
    asm volatile("v_mfma_f32_16x16x128_f8f6f4 %0, %1, %2, %0 blgp:1" : "+a"(acc) : "a"(b), "v"(a));
}

// Stage s: B's fragments in bc (AB: in AGPRs).  kRound: the loads of stage s + 3 of A and s + 2 of B (to bn) are issued; kMore: all loads
// have been, a stage may follow; kEnd: none does.  (The barrier's count is that of the loads issued after those of stage
// s + 1 of A, which it waits for: a stage issues B's 8 before its barrier and A's 2 NB after it.)
enum StageKind { kRound, kMore, kEnd };
template <int FA, int NB, StageKind KIND, bool AB, int BLOCKS>
__device__ __forceinline__ void tile_stage(const TileOperands& p, TileShared<BLOCKS>& sh, int s, f32x4 (&acc)[NB][4][4],
                                           i32x8 (&af)[4], const i32x8 (&bc)[4], i32x8 (&bn)[4]) {
  constexpr int MI = 4 * NB;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    if (i == MI / 2 && KIND != kEnd) stage_barrier<(KIND == kRound ? 16 : 8) + 2 * NB>();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (AB)
        mfma16_ab<FA>(acc[i / 4][i & 3][j], bc[j], af[i & 3]);
      else
        mfma16<FA>(acc[i / 4][i & 3][j], bc[j], af[i & 3]);
      if (j == 0 && i + 2 < MI) af[(i + 2) & 3] = frag_a(p, sh, i + 2, s);
      if (j == 0 && i + 2 >= MI && KIND != kEnd) af[(i + 2) & 3] = frag_a(p, sh, i + 2 - MI, s + 1);
      if (KIND == kRound) {
        if (i < 2 && (j & 1)) bn[2 * i + j / 2] = load_b(p, 2 * i + j / 2, s + 2);
        const int d = 4 * (i - MI / 2) + j;
        if (d >= 0 && d < 2 * NB) load_a(p, sh, d, s + 3);
      }
    }
  }
}

template <int FA, int NB, typename O, int BLOCKS>
__device__ __forceinline__ void tile_body(const ExpertGemmArgs& g, TileShared<BLOCKS>& sh, TileOperands& p, const Tile& t,
                                          int64_t n0, i32x8 (&b0)[4], i32x8 (&b1)[4]) {
  f32x4 acc[NB][4][4];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[b][i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int b = 0; b < NB; ++b) fence16(acc[b]);
  i32x8 b2[4], af[4];
#pragma unroll
  for (int s = 0; s < 3; ++s)
#pragma unroll
    for (int j = 0; j < 2 * NB; ++j) load_a(p, sh, j, s);
  stage_barrier<2 * NB>();  // stages 0 and 1 of A have landed
  af[0] = frag_a(p, sh, 0, 0);
  af[1] = frag_a(p, sh, 1, 0);
  // (whole rounds of the register sets, then what is left: a loop with exits between them made the compiler wait
  // for younger loads at its head)
  const int ns = p.last + 1;
  int s = 0;
  for (; s + 3 <= ns; s += 3) {
    tile_stage<FA, NB, kRound, false>(p, sh, s, acc, af, b0, b2);
    tile_stage<FA, NB, kRound, false>(p, sh, s + 1, acc, af, b1, b0);
    tile_stage<FA, NB, kRound, BLOCKS == 1>(p, sh, s + 2, acc, af, b2, b1);
  }
  if (s < ns) tile_stage<FA, NB, kMore, false>(p, sh, s, acc, af, b0, b2);
  if (s + 1 < ns) tile_stage<FA, NB, kEnd, false>(p, sh, s + 1, acc, af, b1, b0);
#pragma unroll
  for (int b = 0; b < NB; ++b) fence16(acc[b]);
  step_barrier<0>();  // every load has landed and every fragment is read: the ring is free

  // Lane: slots 16 i + fr, columns 16 j + 4 q .. of the wave's 64.  Rows go through the wave's quarter of the ring
  // (16-byte chunks XOR-swizzled by row) to stores of whole 16-byte chunks.
  const int fr = p.lane & 15, q = p.lane >> 4;
  const int64_t col0 = n0 + 64 * p.wave;
  float sb[4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      sb[j][e] = g.sb[t.expert * g.sb_expert + min(col0 + 16 * j + 4 * q + e, g.N - 1) * g.sb_col];
  constexpr int kRowBytes = 64 * sizeof(O), kChunks = kRowBytes / 16;
  constexpr int kSlot = TileShared<BLOCKS>::kSlot;
  constexpr int kRows = 64 * NB < kSlot / kRowBytes ? 64 * NB : kSlot / kRowBytes;  // rows of one pass, the last may have fewer
  static_assert(kRows % 16 == 0, "whole row tiles");
  uint8_t* mine = sh.ring + p.wave * kSlot;
#pragma unroll
  for (int r0 = 0; r0 < 64 * NB; r0 += kRows) {
    const int rows = 64 * NB - r0 < kRows ? 64 * NB - r0 : kRows;  // (192 fp32 rows: 128 and 64)
#pragma unroll
    for (int i = r0 / 16; i < (r0 + rows) / 16; ++i) {
      const int r = 16 * i + fr;
      const float sa = sh.scale[r];
      const bool none = sh.row[r] < 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = none ? 0.0f : acc[i / 4][i & 3][j][e] * (sa * sb[j][e]);
        const int byte = (16 * j + 4 * q) * static_cast<int>(sizeof(O));
        uint8_t* dst = mine + (r - r0) * kRowBytes + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15);
        store4(reinterpret_cast<O*>(dst), v);
      }
    }
    for (int c = p.lane; c < rows * kChunks; c += 64) {
      const int r = c / kChunks, k = c % kChunks;
      const int64_t s = t.row0 + r0 + r, col = col0 + k * (16 / static_cast<int>(sizeof(O)));
      const u32x4 v = *reinterpret_cast<const u32x4*>(mine + r * kRowBytes + ((k ^ (r & 7)) << 4));
      if (s < t.end && col < g.N) *reinterpret_cast<u32x4*>(static_cast<O*>(g.y) + s * g.ldy + col) = v;
    }
  }
}

// Tiles of up to BLOCKS blocks of 64 slots.  Four blocks take most of the registers and the LDS (one workgroup a CU); with
// one block a second workgroup fills the first one's start, end and barriers.
template <int FA, typename O, int BLOCKS>
__global__ void __launch_bounds__(kTileThreads, BLOCKS == 4 ? 1 : 2) k_expert_tile(ExpertGemmArgs g, FastDiv choices, int col_tiles) {
  __shared__ TileShared<BLOCKS> sh;
  constexpr int TM = 64 * BLOCKS;
  Tile t;
  int col;
  if (!find_unit<TM>(g, blockIdx.x, col_tiles, t, col)) return;
  const int tid = threadIdx.x;
  TileOperands p;
  p.lane = tid & 63;
  p.wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int groups = static_cast<int>(g.N / 16);
  const int64_t steps = g.K / 128;
  p.last = static_cast<int>(steps) - 1;
  const int g0 = min(col * (kTN / 16) + p.wave * 4, groups - 1);  // (waves past the last column repeat it)
  p.b = __builtin_amdgcn_make_buffer_rsrc(
      uniform_ptr(g.b + (static_cast<int64_t>(t.expert) * groups + g0) * steps * 2048), 0, -1, 0x00020000);
#pragma unroll
  for (int j = 0; j < 4; ++j) p.goff[j] = __builtin_amdgcn_readfirstlane(static_cast<int>(min(j, groups - 1 - g0) * steps * 2048));
  i32x8 b0[4], b1[4];  // the first loads of B fly while the rows of a are looked up
#pragma unroll
  for (int j = 0; j < 4; ++j) b0[j] = load_b(p, j, 0);
#pragma unroll
  for (int j = 0; j < 4; ++j) b1[j] = load_b(p, j, 1);
  if (tid < TM) {
    const int64_t row = row_of(g, choices, min(t.row0 + tid, t.end - 1));
    sh.row[tid] = static_cast<int>(row);
    sh.scale[tid] = g.sa[g.sa_rows ? max(row, int64_t(0)) : 0];
  }
  lds_barrier();
  const int nb = static_cast<int>((min(t.end - t.row0, int64_t(TM)) + 63) / 64);
#pragma unroll
  for (int j = 0; j < 2 * BLOCKS; ++j) {
    const int r = (4 * j + p.wave) * 8 + (p.lane >> 3);
    const int c = (p.lane & 7) ^ ((r >> 1) & 7);
    p.voa[j] = static_cast<uint32_t>(static_cast<int64_t>(max(sh.row[r], 0)) * g.lda + c * 16);
  }
  p.a = __builtin_amdgcn_make_buffer_rsrc(uniform_ptr(g.a), 0, -1, 0x00020000);
  const int fr = p.lane & 15, q = p.lane >> 4, sw = (fr >> 1) & 7;
  p.lo = fr * 128 + (((2 * q) ^ sw) << 4);
  p.hi = fr * 128 + (((2 * q + 1) ^ sw) << 4);
  const int64_t n0 = static_cast<int64_t>(col) * kTN;
  if constexpr (BLOCKS == 1) {
    tile_body<FA, 1, O>(g, sh, p, t, n0, b0, b1);
  } else {
    switch (nb) {
      case 1: tile_body<FA, 1, O>(g, sh, p, t, n0, b0, b1); break;
      case 2: tile_body<FA, 2, O>(g, sh, p, t, n0, b0, b1); break;
      case 3: tile_body<FA, 3, O>(g, sh, p, t, n0, b0, b1); break;
      default: tile_body<FA, 4, O>(g, sh, p, t, n0, b0, b1); break;
    }
  }
}

}  // namespace

// Which kernel.  The host knows the slots and the experts, not how the plan shares them out, so the rule goes by the
// average a = slots / experts and by the units that the tile kernel would have at least.  Measured, experts x slots of each,
// us (in brackets the weights alone at the 6.1 TB/s of a read-only pass):
//   stream of 16 slots / of 32, tiles of 64 / of 256
//     4096 x 7168:  32 x 4 139 / 144, 159 / 160 (154);  32 x 16 169 / 153, 161 / 163;  8 x 16 44 / 44, 52 / 53 (38);
//                   8 x 32 67 / 54, 54 / 55;  2 x 16 14 / 16, 27 / 27 (10);  2 x 32 25 / 17, 27 / 27
//                   32 x 8 142 / 144, 159 / 161;  of 32 with 8 on average, one has 64: 166 / 195, 159 / 161, one has 200: 184 / 196,
//                   182 / 171;  with 16, one has 300: 239 / 200, 184 / 210;  with 32, one has 700: 347 / 258, 183 / 203
//     7168 x 2048:  32 x 8 88 / 98, 88 / 92 (77), one has 200: 100 / 108, 86 / 95;  32 x 32 170 / 110, 92 / 98, one has 700:
//                   176 / 138, 99 / 111
//   tiles of 64 / of 256
//     4096 x 7168:  32 x 64 169 / 171, 32 x 128 213 / 190;  8 x 64 58 / 59, 8 x 128 59 / 67, 8 x 160 84 / 73
//     4096 x 4096:  32 x 88 121 / 107, of 32 with 96 on average but unequal 131 / 139;  8 x 88 30 / 37
//     7168 x 2048:  32 x 88 112 / 116, of 88 on average but unequal 124 / 142;  32 x 128 118 / 121, 32 x 256 182 / 154
//     4096 x 1024:  32 x 128 43 / 48, 32 x 192 59 / 58, of 178 on average but unequal 58 / 68
// A few slots an expert are streamed, up to 32 where tiles would not fill the CUs (also where one expert has most of them: up to
// 17% slower than tiles of 64 at an average of 8, which the host cannot see).  Tiles of 256 read the weights
// from the L2 cache a quarter as often; those of 64, two workgroups a CU, waste less of a CU on starts, ends, partial tiles and
// uneven shares.  So the latter take up to 64 slots, more the shorter their loops (a K up to 2^18) and up to 128 where all of
// them run at once.
hipError_t launch_expert_gemm(const ExpertGemmArgs& g, hipStream_t st) {
  const FastDiv choices(static_cast<uint32_t>(g.choices));
  const int64_t a = ceil_div(g.slots, g.experts), col_tiles = ceil_div(g.N, kTN), cus = device_cus();
  auto stream = [&](auto fa, auto o, auto mt, auto nt) {
    constexpr int FA = decltype(fa)::value, MT = decltype(mt)::value, NT = decltype(nt)::value;
    using O = decltype(o);
    const int64_t tiles = g.slots / (16 * MT) + std::min(g.experts, g.slots);
    const int64_t sets = ceil_div(g.N / 16, NT);
    int ks = 1;  // waves for each set of columns: 16 waves a CU, if the steps allow it
    while (ks < kWaves && tiles * sets * ks < cus * 16 && g.K / 128 >= 4 * ks) ks <<= 1;
    const int64_t chunks = ceil_div(sets, kWaves / ks);
    hipLaunchKernelGGL((k_expert_stream<FA, O, MT, NT>), dim3(static_cast<unsigned>(tiles * chunks)), dim3(kWaves * 64), 0,
                       st, g, choices, static_cast<int>(chunks), ks);
  };
  auto tile = [&](auto fa, auto o, auto blocks) {
    constexpr int FA = decltype(fa)::value, BLOCKS = decltype(blocks)::value;
    using O = decltype(o);
    const int64_t rows = g.slots / (64 * BLOCKS) + std::min(g.experts, g.slots);
    hipLaunchKernelGGL((k_expert_tile<FA, O, BLOCKS>), dim3(static_cast<unsigned>(rows * col_tiles)), dim3(kTileThreads), 0,
                       st, g, choices, static_cast<int>(col_tiles));
  };
  auto by_rows = [&](auto fa, auto o) {
    using std::integral_constant;
    const int64_t units = std::min(g.experts, g.slots) * col_tiles;
    if (a <= 8 || (a <= 16 && units < cus)) return stream(fa, o, integral_constant<int, 1>{}, integral_constant<int, 1>{});
    if (a <= 32 && units < cus) return stream(fa, o, integral_constant<int, 2>{}, integral_constant<int, 2>{});
    if (a <= 64 || a * g.K <= (int64_t(1) << 18) || (a <= 128 && units <= cus)) return tile(fa, o, integral_constant<int, 1>{});
    tile(fa, o, integral_constant<int, 4>{});
  };
  auto by_out = [&](auto fa) { g.yt == FP8RT_BF16 ? by_rows(fa, uint16_t{}) : by_rows(fa, float{}); };
  g.fa == FP8RT_E4M3 ? by_out(std::integral_constant<int, kE4M3>{}) : by_out(std::integral_constant<int, kE5M2>{});
  return hipGetLastError();
}

}  // namespace fp8rt
