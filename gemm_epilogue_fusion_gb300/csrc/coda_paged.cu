// Paged key/value cache of the decode step around the block tail:
//   append     rows of a QKV product -> rotated Q, and K (rotated) and V into
//              the cache's pages
//   attention  one new token per row over the cached keys and values
// Cache layout: [num_pages, kv_heads, page_size, head_dim], so that a page's
// rows of one head are contiguous.  Nothing here waits on another block.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "coda_internal.h"
#include "fp8_e4m3.cuh"
#include "sm103_ptx.cuh"

namespace coda {
namespace {

// Status word of this translation unit (kDevBadIndex), read back and cleared
// by read_clear_status_paged().
__device__ unsigned g_paged_status;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__nv_fp8_e4m3 x) { return static_cast<float>(x); }
template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// One thread per pair of a row's columns.
template <class T, class C>
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ AppendParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int half = p.head_dim / 2, heads = p.q_heads + 2 * p.kv_heads;
  const int64_t i = blockIdx.x;
  const int pos = p.positions[i];
  if (pos < 0) return;
  const int seq = p.row_seq ? p.row_seq[i] : static_cast<int>(i);
  int page = -1;
  if (seq >= 0 && seq < p.num_seqs && pos / p.page_size < p.max_pages)
    page = p.page_table[static_cast<int64_t>(seq) * p.max_pages + pos / p.page_size];
  if (page < 0 || page >= p.num_pages) {
    if (threadIdx.x == 0) atomicOr(&g_paged_status, kDevBadIndex);
    return;
  }
  const T* z = static_cast<const T*>(p.Z) + i * heads * p.head_dim;
  for (int e = threadIdx.x; e < heads * half; e += blockDim.x) {
    const int h = e / half, j = e % half;
    float a = to_f32(z[h * p.head_dim + 2 * j]), b = to_f32(z[h * p.head_dim + 2 * j + 1]);
    if (p.rotate && h < p.q_heads + p.kv_heads) {
      const int turn = static_cast<int>((p.turn[j] * static_cast<uint64_t>(pos)) >> 32);
      float s, c;
      sincospif(static_cast<float>(turn) * 0x1p-31f, &s, &c);
      const float x = a;
      a = x * c - b * s;
      b = x * s + b * c;
    }
    if (h < p.q_heads) {
      if (p.Q == nullptr) continue;
      T* q = static_cast<T*>(p.Q) + (i * p.q_heads + h) * p.head_dim + 2 * j;
      q[0] = from_f32<T>(a);
      q[1] = from_f32<T>(b);
      continue;
    }
    const bool is_v = h >= p.q_heads + p.kv_heads;
    const int hk = h - p.q_heads - (is_v ? p.kv_heads : 0);
    const int64_t at = ((static_cast<int64_t>(page) * p.kv_heads + hk) * p.page_size + pos % p.page_size) *
                           p.head_dim + 2 * j;
    C* c = static_cast<C*>(is_v ? p.Vc : p.Kc) + at;
    if constexpr (sizeof(C) == 1) {
      const float s = is_v ? *p.scale_v : *p.scale_k;
      *reinterpret_cast<uint16_t*>(c) = to_e4m3x2<false>(a, b, s, 0.0f);
    } else {
      c[0] = from_f32<C>(a);
      c[1] = from_f32<C>(b);
    }
  }
}

constexpr int kAttnWarps = 4;
constexpr int kAttnGroup = 8;  // query heads per block

// One block per row, key/value head and group of up to 8 of its query heads.
// Each warp takes every fourth key with its own running maximum and sum; the
// warps are joined at the end.
template <class T, class C>
__global__ void __launch_bounds__(32 * kAttnWarps) attention_kernel(const __grid_constant__ AttnParams p) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int NE = 8;  // head_dim <= 256
  __shared__ float s_m[kAttnWarps][kAttnGroup], s_l[kAttnWarps][kAttnGroup];
  __shared__ float s_o[kAttnWarps][256];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int G = p.q_heads / p.kv_heads, chunks = (G + kAttnGroup - 1) / kAttnGroup;
  const int64_t item = blockIdx.x;
  const int chunk = static_cast<int>(item % chunks), hk = static_cast<int>(item / chunks % p.kv_heads);
  const int64_t row = item / chunks / p.kv_heads;
  const int g0 = chunk * kAttnGroup, ng = min(kAttnGroup, G - g0);
  const int seq = p.row_seq ? p.row_seq[row] : static_cast<int>(row);
  int64_t len = p.lengths[row];
  bool bad = false;
  if (len > static_cast<int64_t>(p.max_pages) * p.page_size) {
    len = static_cast<int64_t>(p.max_pages) * p.page_size;
    bad = true;
  }
  if (len > 0 && (seq < 0 || seq >= p.num_seqs)) {
    len = 0;
    bad = true;
  }
  float q[kAttnGroup][NE], o[kAttnGroup][NE], m[kAttnGroup], l[kAttnGroup];
#pragma unroll
  for (int g = 0; g < kAttnGroup; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.0f;
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      const int d = lane + 32 * e;
      o[g][e] = 0.0f;
      q[g][e] = g < ng && d < p.head_dim
                    ? to_f32(static_cast<const T*>(p.Q)[row * p.ldq + static_cast<int64_t>(hk * G + g0 + g) * p.head_dim + d])
                    : 0.0f;
    }
  }
  const float sk = sizeof(C) == 1 ? p.scale * *p.scale_k : p.scale;
  for (int64_t t = w; t < len; t += kAttnWarps) {
    const int page = p.page_table[static_cast<int64_t>(seq) * p.max_pages + t / p.page_size];
    if (page < 0 || page >= p.num_pages) {
      bad = true;
      continue;
    }
    const int64_t at = ((static_cast<int64_t>(page) * p.kv_heads + hk) * p.page_size + t % p.page_size) * p.head_dim;
    float k[NE], v[NE];
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      const int d = lane + 32 * e;
      k[e] = d < p.head_dim ? to_f32(static_cast<const C*>(p.Kc)[at + d]) : 0.0f;
      v[e] = d < p.head_dim ? to_f32(static_cast<const C*>(p.Vc)[at + d]) : 0.0f;
    }
#pragma unroll
    for (int g = 0; g < kAttnGroup; ++g) {
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < NE; ++e) s += q[g][e] * k[e];
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= sk;
      const float m2 = fmaxf(m[g], s);
      const float base = m2 == -INFINITY ? 0.0f : m2;
      const float c = expf(m[g] - base), pr = expf(s - base);
      m[g] = m2;
      l[g] = l[g] * c + pr;
#pragma unroll
      for (int e = 0; e < NE; ++e) o[g][e] = o[g][e] * c + pr * v[e];
    }
  }
  if (bad) atomicOr(&g_paged_status, kDevBadIndex);
#pragma unroll
  for (int g = 0; g < kAttnGroup; ++g)
    if (lane == 0) {
      s_m[w][g] = m[g];
      s_l[w][g] = l[g];
    }
  const float sv = sizeof(C) == 1 ? *p.scale_v : 1.0f;
#pragma unroll
  for (int g = 0; g < kAttnGroup; ++g) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < NE; ++e) s_o[w][lane + 32 * e] = o[g][e];
    __syncthreads();
    if (g >= ng) continue;
    float mm = -INFINITY;
    for (int x = 0; x < kAttnWarps; ++x) mm = fmaxf(mm, s_m[x][g]);
    const float base = mm == -INFINITY ? 0.0f : mm;
    float ll = 0.0f;
    for (int x = 0; x < kAttnWarps; ++x) ll += s_l[x][g] * expf(s_m[x][g] - base);
    const int64_t head = static_cast<int64_t>(hk) * G + g0 + g;
    for (int d = threadIdx.x; d < p.head_dim; d += blockDim.x) {
      float oo = 0.0f;
      for (int x = 0; x < kAttnWarps; ++x) oo += s_o[x][d] * expf(s_m[x][g] - base);
      static_cast<T*>(p.O)[(row * p.q_heads + head) * p.head_dim + d] =
          from_f32<T>(ll == 0.0f ? 0.0f : oo / ll * sv);
    }
    if (p.lse && threadIdx.x == 0) p.lse[row * p.q_heads + head] = ll == 0.0f ? -INFINITY : mm + logf(ll);
  }
}

}  // namespace

cudaError_t launch_paged_append(const AppendParams& p, int64_t M, bool f32, bool e4m3, cudaStream_t s, bool pdl) {
  const void* k = f32    ? reinterpret_cast<const void*>(append_kernel<float, float>)
                  : e4m3 ? reinterpret_cast<const void*>(append_kernel<__nv_bfloat16, __nv_fp8_e4m3>)
                         : reinterpret_cast<const void*>(append_kernel<__nv_bfloat16, __nv_bfloat16>);
  void* args[] = {const_cast<AppendParams*>(&p)};
  return launch_ex(k, dim3(static_cast<unsigned>(M)), dim3(256), 0, s, pdl, args);
}

cudaError_t launch_paged_attention(const AttnParams& p, bool f32, bool e4m3, cudaStream_t s, bool pdl) {
  const int G = p.q_heads / p.kv_heads;
  const int64_t items = static_cast<int64_t>(p.M) * p.kv_heads * ((G + kAttnGroup - 1) / kAttnGroup);
  const void* k = f32    ? reinterpret_cast<const void*>(attention_kernel<float, float>)
                  : e4m3 ? reinterpret_cast<const void*>(attention_kernel<__nv_bfloat16, __nv_fp8_e4m3>)
                         : reinterpret_cast<const void*>(attention_kernel<__nv_bfloat16, __nv_bfloat16>);
  void* args[] = {const_cast<AttnParams*>(&p)};
  return launch_ex(k, dim3(static_cast<unsigned>(items)), dim3(32 * kAttnWarps), 0, s, pdl, args);
}

int64_t paged_attention_workspace_bytes(int q_heads, int kv_heads, int head_dim) { return 16; }

unsigned read_clear_status_paged() {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_paged_status, sizeof(v)) != cudaSuccess) return ~0u;
  if (cudaMemcpyToSymbol(g_paged_status, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace coda
