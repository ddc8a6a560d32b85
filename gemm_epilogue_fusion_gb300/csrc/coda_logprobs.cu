// Log probabilities of given tokens from logits, with entropy and the best
// alternatives, and their gradient:
//   lse = log sum_j exp x_j,  logp = x_t - lse,  H = lse - sum_j p_j x_j
//   dx_j = dlogp ([j = t] - p_j) - dH p_j (x_j - lse + H),  p_j = exp(x_j - lse)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "coda_internal.h"
#include "sm103_ptx.cuh"

namespace coda {
namespace {

__device__ unsigned g_logprobs_status;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

constexpr int kThreads = 256;

__device__ __forceinline__ float block_sum(float v) {
  __shared__ float red[32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
  for (int w = 0; w < kThreads / 32; ++w) v += red[w];
  return v;
}

// Order of two candidates: the larger value first, then the lower index; NaN
// counts as the largest value.  64-bit keys that compare the same way.
__device__ __forceinline__ uint64_t order_key(float x, uint32_t j) {
  uint32_t b = __float_as_uint(x + 0.0f);
  b = x != x ? 0xffffffffu : (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return (static_cast<uint64_t>(b) << 32) | (~j);
}

__device__ __forceinline__ uint64_t block_max_key(uint64_t v) {
  __shared__ uint64_t red[32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t u = __shfl_xor_sync(0xffffffffu, v, o);
    v = u > v ? u : v;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  for (int w = 0; w < kThreads / 32; ++w) v = red[w] > v ? red[w] : v;
  return v;
}

// One block per row: the maximum, then the sums, then the alternatives one by one.
template <class T>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const __grid_constant__ LogprobsParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t i = blockIdx.x;
  const T* x = static_cast<const T*>(p.logits) + i * p.ld;
  uint64_t best = 0;
  for (int j = threadIdx.x; j < p.V; j += kThreads) {
    const uint64_t k = order_key(to_f32(x[j]), j);
    best = k > best ? k : best;
  }
  best = block_max_key(best);
  const float m = to_f32(x[~static_cast<uint32_t>(best)]);
  float s = 0.0f, t = 0.0f;
  if (m != -INFINITY) {
    for (int j = threadIdx.x; j < p.V; j += kThreads) {
      const float d = to_f32(x[j]) - m, e = expf(d);
      s += e;
      t += e == 0.0f ? 0.0f : e * d;
    }
    s = block_sum(s);
    t = block_sum(t);
  }
  const float lse = s == 0.0f ? -INFINITY : m + logf(s);
  if (threadIdx.x == 0) {
    const int tgt = p.targets[i];
    float lp = 0.0f;
    if (tgt >= p.V)
      atomicOr(&g_logprobs_status, kDevBadIndex);
    else if (tgt >= 0)
      lp = s == 0.0f ? -INFINITY : (to_f32(x[tgt]) - m) - logf(s);
    p.logp[i] = lp;
    if (p.entropy) p.entropy[i] = s == 0.0f ? 0.0f : logf(s) - t / s;
    if (p.lse) p.lse[i] = lse;
  }
  for (int k = 0; k < p.top; ++k) {
    if (threadIdx.x == 0) {
      const uint32_t j = ~static_cast<uint32_t>(best);
      p.top_ids[i * p.top + k] = static_cast<int>(j);
      p.top_logp[i * p.top + k] = s == 0.0f ? -INFINITY : (to_f32(x[j]) - m) - logf(s);
    }
    uint64_t next = 0;
    for (int j = threadIdx.x; j < p.V; j += kThreads) {
      const uint64_t key = order_key(to_f32(x[j]), j);
      next = key < best && key > next ? key : next;
    }
    best = block_max_key(next);
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads) logprobs_backward_kernel(const __grid_constant__ LogprobsGradParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t i = blockIdx.x;
  const T* x = static_cast<const T*>(p.logits) + i * p.ld;
  T* dx = static_cast<T*>(p.dlogits) + i * p.ldd;
  int tgt = p.targets[i];
  if (tgt >= p.V) {
    if (threadIdx.x == 0) atomicOr(&g_logprobs_status, kDevBadIndex);
    tgt = -1;
  }
  const float lse = p.lse[i], H = p.entropy ? p.entropy[i] : 0.0f;
  const float dl = p.dlogp && tgt >= 0 ? p.dlogp[i] : 0.0f, dh = p.dentropy ? p.dentropy[i] : 0.0f;
  for (int j = threadIdx.x; j < p.V; j += kThreads) {
    const float lp = to_f32(x[j]) - lse, e = lse == -INFINITY ? 0.0f : expf(lp);
    float g = e == 0.0f ? 0.0f : -e * (dl + dh * (lp + H));
    if (j == tgt) g += dl;
    if (lse == -INFINITY) g = 0.0f;
    if constexpr (sizeof(T) == 4)
      dx[j] = g;
    else
      dx[j] = __float2bfloat16_rn(g);
  }
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsParams& p, int64_t M, bool f32, cudaStream_t s, bool pdl) {
  const void* k = f32 ? reinterpret_cast<const void*>(logprobs_kernel<float>)
                      : reinterpret_cast<const void*>(logprobs_kernel<__nv_bfloat16>);
  void* args[] = {const_cast<LogprobsParams*>(&p)};
  return launch_ex(k, dim3(static_cast<unsigned>(M)), dim3(kThreads), 0, s, pdl, args);
}

cudaError_t launch_logprobs_backward(const LogprobsGradParams& p, int64_t M, bool f32, cudaStream_t s, bool pdl) {
  const void* k = f32 ? reinterpret_cast<const void*>(logprobs_backward_kernel<float>)
                      : reinterpret_cast<const void*>(logprobs_backward_kernel<__nv_bfloat16>);
  void* args[] = {const_cast<LogprobsGradParams*>(&p)};
  return launch_ex(k, dim3(static_cast<unsigned>(M)), dim3(kThreads), 0, s, pdl, args);
}

unsigned read_clear_status_logprobs() {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_logprobs_status, sizeof(v)) != cudaSuccess) return ~0u;
  if (cudaMemcpyToSymbol(g_logprobs_status, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace coda
