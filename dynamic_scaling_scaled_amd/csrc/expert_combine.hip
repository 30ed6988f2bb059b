// expert_combine.hip -- the weighted sum of a token's experts on its residual, and its
// gradient: rows are gathered (scattered) by the router's slots.
//
//   y[t] = residual[t] + sum_j w[t,j] x[slot(t,j)];   dx[slot(t,j)] = w[t,j] dy[t],   dw[t,j] = <dy[t], x[slot(t,j)]>
//
// Bound by memory: every row once (4096 tokens of 8 x 7168 bf16: 587 MB forward, 998 back).  Measured: 126 us (4.7 TB/s)
// and 201 us (5.0 TB/s; a large copy reaches 4.8); a step of 64 tokens 4.9 us, of which a launch is 3.  1365 tokens of 24
// experts, bf16: 115 and 276 us (4.4 and 3.5 TB/s: 32 partial products a thread leave fewer waves); fp32, 1024 of 16 117 and 203
// (4.5 and 4.8), 512 of 32 114 and 217 (4.4 and 4.4, 12 registers spilled).
#include <algorithm>

#include "device_common.h"
#include "internal.h"

namespace fp8rt {

namespace {

constexpr int64_t kMaxGrid = int64_t(1) << 20;  // workgroups loop past it

// Forward: a thread takes 8 columns of a token; the loads of 8 experts' rows are in flight together.
template <typename T>
__device__ __forceinline__ void combine8(const CombineArgs& a, int64_t t, int64_t c) {
  const T* x = static_cast<const T*>(a.x);
  float y[8] = {};
  if (a.res) {
    Octet<T> o;
    o.load_nt(static_cast<const T*>(a.res) + t * a.ldr + c);
    widen(o, y);
  }
  const int32_t* slots = a.slots + t * a.k;
  const float* w = a.weights + t * a.k;
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    Octet<T> o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t s = j0 + j < a.k ? slots[j0 + j] : -1;
      if (s >= 0 && s < a.x_rows) o[j].load_nt(x + s * a.ldx + c);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t s = j0 + j < a.k ? slots[j0 + j] : -1;
      if (s >= 0 && s < a.x_rows) {
        const float wj = w[j0 + j];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] += wj * o[j].get(i);
      }
    }
  }
  store8(static_cast<T*>(a.y) + t * a.ldy + c, y);
}
template <typename T>
__global__ void __launch_bounds__(64) k_combine(CombineArgs a, int64_t chunks) {
  for (int64_t i = blockIdx.x; i < a.tokens * chunks; i += gridDim.x) {
    const int64_t t = i / chunks, c = ((i - t * chunks) * blockDim.x + threadIdx.x) * 8;
    if (c < a.cols) combine8<T>(a, t, c);
  }
}

// Gradient: a workgroup takes a token; its threads keep the k partial products.
template <typename T, int K>
__global__ void __launch_bounds__(1024) k_combine_backward(CombineArgs a) {
  __shared__ float sh[16][K];
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const T* x = static_cast<const T*>(a.x);
    const T* dy = static_cast<const T*>(a.dy) + t * a.lddy;
    T* dx = static_cast<T*>(a.dx);
    const int32_t* slots = a.slots + t * a.k;
    const float* w = a.weights + t * a.k;
    float dot[K] = {};
    for (int64_t c = threadIdx.x * 8; c < a.cols; c += blockDim.x * 8) {
      Octet<T> g;
      g.load_nt(dy + c);
#pragma unroll
      for (int j0 = 0; j0 < K; j0 += 8) {
        if (j0 >= a.k) break;
        Octet<T> o[8];  // (all loads before the stores, which they might otherwise have to wait for: dx may be x)
        int64_t s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s[j] = j0 + j < a.k ? slots[j0 + j] : -1;
          if (s[j] >= a.x_rows) s[j] = -1;
          if (s[j] >= 0) o[j].load_nt(x + s[j] * a.ldx + c);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (s[j] < 0) continue;
          const float wj = w[j0 + j];
          float d[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[j0 + j] += g.get(i) * o[j].get(i);
            d[i] = wj * g.get(i);
          }
          store8(dx + s[j] * a.lddx + c, d);
        }
      }
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
#pragma unroll
    for (int j = 0; j < K; ++j) {
      for (int o = 32; o >= 1; o >>= 1) dot[j] += __shfl_xor(dot[j], o);
      if (lane == 0) sh[wave][j] = dot[j];
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < a.k) {
      float s = 0.0f;
      for (int i = 0; i < nw; ++i) s += sh[i][threadIdx.x];
      a.dw[t * a.k + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_expert_combine(const CombineArgs& a, hipStream_t st) {
  const int64_t octets = a.cols >> 3;
  const int threads = 64;  // (workgroups of one wave: 120 us where 128 / 256 / 512 threads took 122 / 130 / 127)
  const int64_t chunks = ceil_div(octets, threads);
  const dim3 grid(static_cast<unsigned>(std::min(a.tokens * chunks, kMaxGrid)));
  if (a.xt == FP8RT_BF16)
    hipLaunchKernelGGL(k_combine<uint16_t>, grid, dim3(threads), 0, st, a, chunks);
  else
    hipLaunchKernelGGL(k_combine<float>, grid, dim3(threads), 0, st, a, chunks);
  return hipGetLastError();
}

hipError_t launch_expert_combine_backward(const CombineArgs& a, hipStream_t st) {
  const int64_t octets = a.cols >> 3;
  // many tokens: a quarter of 1024 threads each, so that several workgroups a CU overlap loads and sums (4096 tokens of
  // 7168: 204 us, 64 / 128 / 1024 threads 207 / 222 / 211); few: one round of columns (64 tokens: 11 us against 20)
  const int64_t most = a.tokens >= 2 * device_cus() ? 256 : 1024;
  const int threads = static_cast<int>(ceil_div(ceil_div(octets, ceil_div(octets, most)), 64) * 64);
  const dim3 grid(static_cast<unsigned>(std::min(a.tokens, kMaxGrid)));
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, dim3(threads), 0, st, a); };
  auto by_k = [&](auto t) {
    using T = decltype(t);
    if (a.k <= 8) go(k_combine_backward<T, 8>);
    else if (a.k <= 16) go(k_combine_backward<T, 16>);
    else go(k_combine_backward<T, 32>);
  };
  a.xt == FP8RT_BF16 ? by_k(uint16_t{}) : by_k(float{});
  return hipGetLastError();
}

}  // namespace fp8rt
