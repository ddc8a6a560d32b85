// RMSNorm as a pass of its own, with the residual's addition before it and, on
// request, its result in e4m3 with a scale for each row; and its gradient.
//   h = round(x + R);  r = 1 / sqrt(mean h^2 + eps);  y = h r gamma
//   s = max_j |y_j| / 448 (1 for a row of zeros, rounded up if subnormal);  q = e4m3(y / s)
// Without gamma the row x itself is quantised.  Everything between the loads
// and the stores is fp32; y is rounded once, to the output type or to a code.
//
// Bound by memory traffic: a row stays in registers between its two passes
// (sum of squares, largest |y|), so each input is read once and each output
// written once.  A row is taken by 32 to 1024 threads.  16384 rows of 4096 with a
// residual, bf16 to e4m3: 79.4 us, 5.9 TB/s, with 128 threads of 4 vectors a row
// (256 of 2: 86, 512 of 1: 129, 64 of 8: 84, streaming stores 80).
//
// Gradient, with dy the gradient of y and dR that of h from elsewhere:
//   dh = r (gamma dy - z mean_j gamma_j dy_j z_j) + dR,  z = r h
//   dgamma = sum over the rows of dy z
// A block walks rows, keeping its threads' columns of dgamma in registers; a
// second kernel adds the blocks' sums in the blocks' order.  These sums are fp32:
// dgamma of 16384 rows of 4096 is 1.7e-7 off the 64-bit one (2-norm), where a sum
// in 64 bits, rounded, is 3.6e-8 off.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "coda_experts.h"
#include "fp8_e4m3.cuh"
#include "sm103_ptx.cuh"

namespace coda {
namespace {

template <bool F32>
struct Vec {
  static constexpr int N = F32 ? 4 : 8;  // columns of a 16-byte vector
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[N]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F32) {
        f[i] = __uint_as_float(w[i]);
      } else {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[N]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F32) {
        w[i] = __float_as_uint(f[i]);
      } else {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&p);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// gamma of a vector's columns.
template <int N>
__device__ __forceinline__ void load_gamma(const float* gamma, int col, float (&g)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const float4 v = *reinterpret_cast<const float4*>(gamma + col + 4 * i);
    g[4 * i] = v.x, g[4 * i + 1] = v.y, g[4 * i + 2] = v.z, g[4 * i + 3] = v.w;
  }
}

// Sum or maximum over the TPR threads of a row, in a fixed order; `red` is
// used once per row and kind.  A maximum passes a NaN on.
template <int TPR, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* red) {
  auto join = [](float a, float b) { return MAX ? (a > b || a != a ? a : b) : a + b; };
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, o));
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < TPR / 32; ++i) v = join(v, red[i]);
  }
  return v;
}

// A row's scale: its largest value over 448 (1 for zeros).  A subnormal one is rounded up: rounded to nearest, its
// coarse steps would leave values above 448 of them, or it would be 0, and a zero over it NaN.
__device__ __forceinline__ float row_scale(float amax) {
  const float s = e4m3_scale(amax);
  return s < 0x1p-126f ? __fdiv_ru(amax, 448.0f) : s;
}

template <int N, bool FAST>
__device__ __forceinline__ void store_codes(uint8_t* q, const float (&y)[N], float s, float inv) {
  uint32_t w[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    w[i] = static_cast<uint32_t>(to_e4m3x2<FAST>(y[4 * i], y[4 * i + 1], s, inv)) |
           (static_cast<uint32_t>(to_e4m3x2<FAST>(y[4 * i + 2], y[4 * i + 3], s, inv)) << 16);
  if constexpr (N == 8) *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(q) = w[0];
}

// TPR threads take a row, NV vectors each, TPR vectors apart.
template <bool F32, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) norm_kernel(const __grid_constant__ NormParams p) {
  using V = Vec<F32>;
  constexpr int kRows = TPR < 128 ? 128 / TPR : 1;  // rows of a block
  __shared__ float red_sum[32], red_again[32], red_max[32];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + (kRows > 1 ? threadIdx.x / TPR : 0);
  const int t = kRows > 1 ? threadIdx.x % TPR : threadIdx.x;
  const int vecs = p.N / V::N;
  pdl_wait();
  pdl_launch_dependents();
  if (kRows > 1 && row >= p.M) return;  // whole warps; no barrier follows where kRows > 1
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const char*>(p.X) + row * p.ldx * (F32 ? 4 : 2));
  uint4 h[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = t + i * TPR;
    h[i] = v < vecs ? __ldcs(x + v) : make_uint4(0, 0, 0, 0);
  }
  // one vector a thread: its gamma comes along with the row instead of after the sum
  float g1[NV == 1 ? V::N : 1];
  if constexpr (NV == 1)
    if (p.gamma != nullptr && t < vecs) load_gamma<V::N>(p.gamma, t * V::N, g1);
  if (p.R != nullptr) {
    const uint4* res = reinterpret_cast<const uint4*>(static_cast<const char*>(p.R) + row * p.ldr * (F32 ? 4 : 2));
    uint4 b[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * TPR;
      b[i] = v < vecs ? __ldcs(res + v) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float fa[V::N], fb[V::N];
      V::unpack(h[i], fa);
      V::unpack(b[i], fb);
#pragma unroll
      for (int e = 0; e < V::N; ++e) fa[e] += fb[e];
      h[i] = V::pack(fa);  // the norm is that of the stored stream
    }
  }
  if (p.H != nullptr) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * TPR;
      if (v < vecs) static_cast<uint4*>(p.H)[row * vecs + v] = h[i];
    }
  }
  float r = 1.0f;
  if (p.gamma != nullptr) {
    auto squares = [&](float f2, float* red) {  // sum of (f2 h)^2
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[V::N];
        V::unpack(h[i], f);
#pragma unroll
        for (int e = 0; e < V::N; ++e) ss = fmaf(f[e] * f2, f[e] * f2, ss);
      }
      return row_reduce<TPR, false>(ss, red);
    };
    const float n = static_cast<float>(p.N);
    const float ss = squares(1.0f, red_sum), size = ss + p.eps;
    if (size > 0x1p126f || size < 0x1p-80f) {
      // the squares of finite values leave fp32's range, or lose their low bits at its end, beside no larger eps: summed
      // again 2^75 times smaller or larger, which 32768 of the largest, or the smallest normal ones, do not leave
      // (uniform over the row)
      const float f2 = size > 1.0f ? 0x1p-75f : 0x1p75f;
      r = f2 / sqrtf(squares(f2, red_again) / n + p.eps * f2 * f2);
    } else {
      r = 1.0f / sqrtf(ss / n + p.eps);
    }
    if (p.r != nullptr && t == 0) p.r[row] = r;
  }
  // y of vector i, once for each of the two passes that want it
  auto y_of = [&](int i, int v, float (&y)[V::N]) {
    V::unpack(h[i], y);
    if (p.gamma != nullptr && v < vecs) {
      if constexpr (NV == 1) {
#pragma unroll
        for (int e = 0; e < V::N; ++e) y[e] = y[e] * r * g1[e];
      } else {
        float g[V::N];
        load_gamma<V::N>(p.gamma, v * V::N, g);
#pragma unroll
        for (int e = 0; e < V::N; ++e) y[e] = y[e] * r * g[e];
      }
    }
  };
  float amax = 0.0f;
  if (p.Y != nullptr || p.Yq != nullptr) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * TPR;
      float y[V::N];
      y_of(i, v, y);
      if (p.Y != nullptr && v < vecs) static_cast<uint4*>(p.Y)[row * vecs + v] = V::pack(y);
#pragma unroll
      for (int e = 0; e < V::N; ++e) amax = (fabsf(y[e]) > amax || y[e] != y[e]) ? fabsf(y[e]) : amax;
    }
  }
  if (p.Yq != nullptr) {
    amax = row_reduce<TPR, true>(amax, red_max);
    const float s = row_scale(amax);
    if (t == 0) p.scale[row] = s;
    const bool fast = e4m3_fast_scale(s);
    const float inv = fast ? __frcp_rn(s) : 0.0f;
    uint8_t* q = p.Yq + row * p.N;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * TPR;
      float y[V::N];
      y_of(i, v, y);
      if (v >= vecs) continue;
      if (fast) store_codes<V::N, true>(q + v * V::N, y, s, inv);
      else store_codes<V::N, false>(q + v * V::N, y, s, inv);
    }
  }
}

// The gradient's first kernel.  TPR threads take a row, NV vectors each, and
// ROWS rows are side by side in a block (a warp each, where a row is short
// enough for that).  Each thread copies its own vectors of the rows to come into
// shared memory, STAGES rows deep, so no barrier stands between the copies and
// their use, and no registers are held for them; r h and gamma dy stay in
// registers for the outputs.  What is left to hide is the row's sum, so blocks
// side by side on an SM matter more than depth: 16384 rows of 4096, bf16, dR
// given, take 103 us with loads into registers and two blocks an SM, 106 and
// 101 with 4 stages (without and with the held products), 92 with three blocks
// of 3 stages and 88.6 with three of 2 (6.06 TB/s of the inputs and outputs).
__device__ __forceinline__ void copy16_async(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {  // for all but the N latest groups
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int TPR, int NV, int ROWS, int STAGES>
struct NormBwdShape {
  static constexpr int kThreads = TPR * ROWS;
  static constexpr int kStage = 3 * NV * kThreads;  // 16-byte vectors: dy, h, dR
  static constexpr int kSmem = STAGES * kStage * 16;
  static_assert(ROWS == 1 || TPR == 32, "rows side by side are a warp each");
  static_assert(kSmem <= 196608, "a block's share of the shared memory");
};

template <bool F32, int TPR, int NV, int ROWS, int STAGES, int PER_SM>
__global__ void __launch_bounds__(TPR* ROWS, PER_SM) norm_backward_kernel(const __grid_constant__ NormGradParams p) {
  using V = Vec<F32>;
  using S = NormBwdShape<TPR, NV, ROWS, STAGES>;
  extern __shared__ uint4 staged[];
  __shared__ float red[2][32];
  const int t = ROWS > 1 ? threadIdx.x % TPR : threadIdx.x;
  const int vecs = p.N / V::N;
  const auto* DY = static_cast<const uint4*>(p.dY);
  const auto* H = static_cast<const uint4*>(p.H);
  const auto* DR = static_cast<const uint4*>(p.dH_in);
  auto* DH = static_cast<uint4*>(p.dH);
  // this thread's vectors of a stage: which = 0 dy, 1 h, 2 dR
  auto at = [&](int stage, int which, int i) -> uint4& {
    return staged[stage * S::kStage + (which * NV + i) * S::kThreads + threadIdx.x];
  };
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int k = 0; k < STAGES; ++k)
#pragma unroll
    for (int i = 0; i < NV; ++i)  // vectors behind the row, and dR where there is none
#pragma unroll
      for (int w = 0; w < 3; ++w) at(k, w, i) = zero;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * ROWS + (ROWS > 1 ? threadIdx.x / TPR : 0);
  auto fetch = [&](int64_t row, int stage) {
    if (row < p.M) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = t + i * TPR;
        if (v >= vecs) continue;
        copy16_async(&at(stage, 0, i), DY + row * vecs + v);
        copy16_async(&at(stage, 1, i), H + row * vecs + v);
        if (DR != nullptr) copy16_async(&at(stage, 2, i), DR + row * vecs + v);
      }
    }
    copy_commit();
  };
#pragma unroll
  for (int k = 0; k < STAGES - 1; ++k) fetch(row0 + k * step, k);
  float dg[NV][V::N];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < V::N; ++e) dg[i][e] = 0.0f;
  int stage = 0, flip = 0;
  for (int64_t row = row0; row < p.M; row += step, flip ^= 1) {
    const float r = p.r[row];
    copy_wait<STAGES - 2>();
    float dot = 0.0f;
    float z[NV][V::N], gy[NV][V::N];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * TPR;
      if (v >= vecs) continue;
      float y[V::N], h[V::N], g[V::N];
      V::unpack(at(stage, 0, i), y);
      V::unpack(at(stage, 1, i), h);
      load_gamma<V::N>(p.gamma, v * V::N, g);
#pragma unroll
      for (int e = 0; e < V::N; ++e) {
        z[i][e] = r * h[e];  // the normed value: no size of h leaves fp32's range
        gy[i][e] = g[e] * y[e];
        dot = fmaf(gy[i][e], z[i][e], dot);
        dg[i][e] = fmaf(y[e], z[i][e], dg[i][e]);
      }
    }
    // the stage before this one has been used up by this thread
    fetch(row + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
    dot = row_reduce<TPR, false>(dot, red[flip]);
    const float c = dot / static_cast<float>(p.N);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * TPR;
      if (v >= vecs) continue;
      float x[V::N];
      V::unpack(at(stage, 2, i), x);
#pragma unroll
      for (int e = 0; e < V::N; ++e) x[e] = fmaf(r, fmaf(-c, z[i][e], gy[i][e]), x[e]);
      DH[row * vecs + v] = V::pack(x);
    }
    stage = stage + 1 == STAGES ? 0 : stage + 1;
  }
  copy_wait<0>();
  float* part = p.part + static_cast<int64_t>(blockIdx.x) * p.N;
  if constexpr (ROWS > 1) {
    // the warps' sums, in the warps' order
    float* sums = reinterpret_cast<float*>(staged);  // [ROWS][NV TPR V::N]
    __syncthreads();
    constexpr int kWidth = NV * TPR * V::N;
    static_assert(ROWS * kWidth * 4 <= S::kSmem, "the staged rows' place holds the sums");
    float* own = sums + threadIdx.x / TPR * kWidth;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < V::N; e += 4)
        *reinterpret_cast<float4*>(own + (t + i * TPR) * V::N + e) =
            make_float4(dg[i][e], dg[i][e + 1], dg[i][e + 2], dg[i][e + 3]);
    __syncthreads();
    for (int j = threadIdx.x; j < p.N; j += S::kThreads) {
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < ROWS; ++k) sum += sums[k * kWidth + j];
      part[j] = sum;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * TPR;
      if (v >= vecs) continue;
#pragma unroll
      for (int e = 0; e < V::N; e += 4)
        *reinterpret_cast<float4*>(part + v * V::N + e) =
            make_float4(dg[i][e], dg[i][e + 1], dg[i][e + 2], dg[i][e + 3]);
    }
  }
}

// Rows too wide for stages in shared memory (more than 2048 vectors): loaded
// for the sum and, from L2, once more for the outputs.
template <bool F32, int NV>
__global__ void __launch_bounds__(1024) norm_backward_wide_kernel(const __grid_constant__ NormGradParams p) {
  using V = Vec<F32>;
  __shared__ float red[2][32];
  const int t = threadIdx.x;
  const int vecs = p.N / V::N;
  const auto* DY = static_cast<const uint4*>(p.dY);
  const auto* H = static_cast<const uint4*>(p.H);
  const auto* DR = static_cast<const uint4*>(p.dH_in);
  pdl_wait();
  pdl_launch_dependents();
  float dg[NV][V::N];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < V::N; ++e) dg[i][e] = 0.0f;
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, flip ^= 1) {
    const float r = p.r[row];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * 1024;
      if (v >= vecs) continue;
      float y[V::N], h[V::N], g[V::N];
      V::unpack(DY[row * vecs + v], y);
      V::unpack(H[row * vecs + v], h);
      load_gamma<V::N>(p.gamma, v * V::N, g);
#pragma unroll
      for (int e = 0; e < V::N; ++e) {
        const float yz = y[e] * (r * h[e]);
        dot = fmaf(g[e], yz, dot);
        dg[i][e] += yz;
      }
    }
    dot = row_reduce<1024, false>(dot, red[flip]);
    const float c = dot / static_cast<float>(p.N);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * 1024;
      if (v >= vecs) continue;
      float y[V::N], h[V::N], x[V::N], g[V::N];
      V::unpack(DY[row * vecs + v], y);
      V::unpack(H[row * vecs + v], h);
      V::unpack(DR != nullptr ? __ldcs(DR + row * vecs + v) : make_uint4(0, 0, 0, 0), x);
      load_gamma<V::N>(p.gamma, v * V::N, g);
#pragma unroll
      for (int e = 0; e < V::N; ++e) x[e] = fmaf(r, fmaf(-c, r * h[e], g[e] * y[e]), x[e]);
      static_cast<uint4*>(p.dH)[row * vecs + v] = V::pack(x);
    }
  }
  float* part = p.part + static_cast<int64_t>(blockIdx.x) * p.N;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = t + i * 1024;
    if (v >= vecs) continue;
#pragma unroll
    for (int e = 0; e < V::N; e += 4)
      *reinterpret_cast<float4*>(part + v * V::N + e) = make_float4(dg[i][e], dg[i][e + 1], dg[i][e + 2], dg[i][e + 3]);
  }
}

// dgamma[j] = sum over the blocks of part[block, j].  A block takes 32 columns:
// a warp reads four of the rows at a time, eight lanes four columns each; the
// lanes' sums are joined by shuffles and the 32 warps' in the warps' order.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps) norm_column_sum_kernel(const float* part, int blocks, int N,
                                                                        float* out) {
  __shared__ float4 s[kSumWarps][8];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + lane % 8 * 4;  // N is a multiple of four
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (j < N) {
#pragma unroll 4
    for (int b = w * 4 + lane / 8; b < blocks; b += 4 * kSumWarps) {
      const float4 v = *reinterpret_cast<const float4*>(part + static_cast<int64_t>(b) * N + j);
      acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
    }
  }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
  }
  if (lane < 8) s[w][lane] = acc;
  __syncthreads();
  const int c = blockIdx.x * 32 + lane;
  if (w == 0 && c < N) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kSumWarps; ++i) sum += reinterpret_cast<const float*>(&s[i][0])[lane];
    out[c] = sum;
  }
}

template <bool F32, int TPR, int NV>
cudaError_t norm_launch(const NormParams& p, cudaStream_t s, bool pdl) {
  NormParams q = p;
  void* args[] = {&q};
  constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
  return launch_ex(reinterpret_cast<const void*>(norm_kernel<F32, TPR, NV>),
                   dim3(static_cast<unsigned>((static_cast<int64_t>(p.M) + kRows - 1) / kRows)),
                   dim3(TPR < 128 ? 128 : TPR), 0, s, pdl, args);
}

// Threads of a row by its vectors: a warp up to 128 (no barrier), then up to
// four vectors a thread, with as few threads as that allows (more rows of loads
// in flight on an SM).
template <bool F32>
cudaError_t norm_pick(const NormParams& p, cudaStream_t s, bool pdl) {
  const int vecs = p.N / Vec<F32>::N;
  if (vecs <= 32) return norm_launch<F32, 32, 1>(p, s, pdl);
  if (vecs <= 64) return norm_launch<F32, 32, 2>(p, s, pdl);
  if (vecs <= 128) return norm_launch<F32, 32, 4>(p, s, pdl);
  if (vecs <= 256) return norm_launch<F32, 128, 2>(p, s, pdl);
  // few rows: latency, a vector a thread
  if (p.M <= device_sm_count() && vecs <= 512) return norm_launch<F32, 512, 1>(p, s, pdl);
  if (vecs <= 512) return norm_launch<F32, 128, 4>(p, s, pdl);
  if (vecs <= 1024) return norm_launch<F32, 256, 4>(p, s, pdl);
  if (vecs <= 2048) return norm_launch<F32, 512, 4>(p, s, pdl);
  if constexpr (F32)  // a row of kMaxNormWidth has 4096 vectors in bf16, 8192 in fp32
    if (vecs > 4096) return norm_launch<F32, 1024, 8>(p, s, pdl);
  return norm_launch<F32, 1024, 4>(p, s, pdl);
}

// Blocks of the gradient's first kernel, `rows` rows side by side in each: what
// runs at once, but six rows for each at least where that leaves every SM one
// (the second kernel reads all their sums: 1003 rows of 2060 fp32 columns, 152
// blocks 14.1 us, 304 14.6, 456 17.0).
// GB300's SMs, not asked of the device: the workspace's size is told without one.
constexpr int kNormBwdSms = 152, kNormBwdMost = 3 * kNormBwdSms;
int norm_backward_blocks(int64_t M, int rows, int most) {
  const int64_t all = (M + rows - 1) / rows, few = all < kNormBwdSms ? all : kNormBwdSms;
  const int64_t n = all / 6 > few ? all / 6 : few;
  return static_cast<int>(n < most ? n : most);
}

cudaError_t norm_backward_launch(const void* kernel, int threads, int smem, int rows, int most,
                                 const NormGradParams& p, cudaStream_t s, bool pdl) {
  NormGradParams q = p;
  const int blocks = norm_backward_blocks(p.M, rows, most);
  if (blocks == 1) q.part = p.dgamma;  // its share is the sum
  void* args[] = {&q};
  cudaError_t e = launch_ex(kernel, dim3(blocks), dim3(threads), smem, s, pdl, args);
  if (e != cudaSuccess || blocks == 1) return e;
  const float* part = p.part;
  int nb = blocks, N = p.N;
  float* out = p.dgamma;
  void* sum_args[] = {&part, &nb, &N, &out};
  return launch_ex(reinterpret_cast<const void*>(norm_column_sum_kernel), dim3((N + 31) / 32), dim3(32 * kSumWarps), 0,
                   s, pdl, sum_args);
}

template <bool F32, int TPR, int NV, int ROWS, int STAGES, int PER_SM>
cudaError_t norm_backward_shape(const NormGradParams& p, cudaStream_t s, bool pdl) {
  using S = NormBwdShape<TPR, NV, ROWS, STAGES>;
  const void* kernel = reinterpret_cast<const void*>(norm_backward_kernel<F32, TPR, NV, ROWS, STAGES, PER_SM>);
  static std::atomic<unsigned> opted{0};  // devices with the shared-memory opt-in
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 32 || !(opted.load(std::memory_order_relaxed) >> dev & 1u)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 32) opted.fetch_or(1u << dev, std::memory_order_relaxed);
  }
  return norm_backward_launch(kernel, S::kThreads, S::kSmem, ROWS, PER_SM * kNormBwdSms, p, s, pdl);
}

template <bool F32>
cudaError_t norm_backward_pick(const NormGradParams& p, cudaStream_t s, bool pdl) {
  const int vecs = p.N / Vec<F32>::N;
  if (vecs <= 32) return norm_backward_shape<F32, 32, 1, 8, 3, 3>(p, s, pdl);
  if (vecs <= 64) return norm_backward_shape<F32, 32, 2, 8, 3, 3>(p, s, pdl);
  if (vecs <= 128) return norm_backward_shape<F32, 32, 4, 8, 2, 2>(p, s, pdl);
  if (vecs <= 256) return norm_backward_shape<F32, 256, 1, 1, 3, 3>(p, s, pdl);
  if (vecs <= 512) return norm_backward_shape<F32, 256, 2, 1, 2, 3>(p, s, pdl);
  if (vecs <= 1024) return norm_backward_shape<F32, 512, 2, 1, 2, 2>(p, s, pdl);
  if (vecs <= 2048) return norm_backward_shape<F32, 1024, 2, 1, 2, 1>(p, s, pdl);
  const void* wide = reinterpret_cast<const void*>(norm_backward_wide_kernel<F32, 4>);
  if constexpr (F32)
    if (vecs > 4096) wide = reinterpret_cast<const void*>(norm_backward_wide_kernel<F32, 8>);
  return norm_backward_launch(wide, 1024, 0, 1, kNormBwdSms, p, s, pdl);
}

}  // namespace

int64_t norm_backward_workspace_bytes(int64_t M, int64_t N) { return norm_backward_blocks(M, 1, kNormBwdMost) * N * 4; }

cudaError_t launch_norm(const NormParams& p, bool f32, cudaStream_t s, bool pdl) {
  return f32 ? norm_pick<true>(p, s, pdl) : norm_pick<false>(p, s, pdl);
}

cudaError_t launch_norm_backward(const NormGradParams& p, bool f32, cudaStream_t s, bool pdl) {
  return f32 ? norm_backward_pick<true>(p, s, pdl) : norm_backward_pick<false>(p, s, pdl);
}

}  // namespace coda
