// gemm_tile.h -- pieces that the large GEMM and the experts' GEMM share: operand types,
// buffer-to-LDS loads, the barriers and the 16x16x128 MFMA.
#pragma once

#include "device_common.h"

namespace fp8rt {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void gbl_void;

__device__ __forceinline__ void* uniform_ptr(const void* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<void*>((static_cast<uint64_t>(hi) << 32) | lo);
}

// Wait until at most N of this wave's vector-memory operations (the loads of
// the younger stage) are outstanding and all its LDS operations are done,
// then join the workgroup barrier.  No memory fence: younger loads keep
// flying across the barrier.
template <int N>
__device__ __forceinline__ void step_barrier() {
  static_assert(N < 64, "vmcnt field");
  __builtin_amdgcn_sched_barrier(0);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(((N >> 4) << 14) | 0x0070 | (N & 15));
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_sched_barrier(0);
}

// Wait for this wave's LDS operations (its vector-memory loads keep flying) and
// join the workgroup barrier.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0), vmcnt and expcnt at their maximum
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_sched_barrier(0);
}

// One 16x16x128 MFMA, acc += B-fragment x A-fragment (the transposed tile),
// written inline with the accumulator as one tied operand, so it stays in
// the same AGPRs from stage to stage (the builtin's untied form made the
// register allocator rotate the 64 accumulators between the two unrolled
// stages and copy them back, about 100 moves per stage).  A E5M2 (FA = 1) is
// the instruction's second source: blgp:1.
template <int FA>
__device__ __forceinline__ void mfma16(f32x4& acc, const i32x8& b, const i32x8& a) {
  if constexpr (FA == 0)
    asm volatile("v_mfma_f32_16x16x128_f8f6f4 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
  else
    asm volatile("v_mfma_f32_16x16x128_f8f6f4 %0, %1, %2, %0 blgp:1" : "+a"(acc) : "v"(b), "v"(a));
}

// One DMA instruction of a stage: 1 KB (8 rows of 128 bytes) into slot k.
__device__ __forceinline__ void dma1(__amdgpu_buffer_rsrc_t rs, int soff, uint32_t voff, uint8_t* lds, int k) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(lds + k * 1024), 16, static_cast<int>(voff), soff, 0, 0);
}

}  // namespace

}  // namespace fp8rt
