// The router of a mixture of experts, and the rows' way into expert order and
// back.
//   route             the k largest logits of each row, their weights, and each
//                     (row, choice) pair's place when pairs are sorted by expert
//   route_backward    gradient of the weights with respect to the logits
//   dispatch          Xs[slots[i, j]] = X[i]
//   combine           H[i] = R[i] + sum_j w_ij Y[slots[i, j]], and H's partial
//                     sums of squares for the norm that follows
//   combine_backward  dY[slots[i, j]] = w_ij dH[i], dw_ij = <dH[i], Y[slots[i, j]]>
// None of them waits on another block, so none can time out.
//
// The router is bound by latency: 8192 rows of 128 experts are 2 MB of logits,
// 0.3 us of copying.  32 rows take one launch and 7.5 us, 16384 rows two
// launches and 20 us (8.6 and 9.1 us of the GPU for half as many: a load and the
// picks one after the other, then every block's sum over all counts).  The other
// kernels are bound by HBM: 8192 rows of 2048, 8 choices each, bf16, dispatch 49
// us (6.1 TB/s of what it has to move), combine 51 us (6.6), its gradient 86 us
// (6.6).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "coda_experts.h"
#include "sm103_ptx.cuh"

namespace coda {
namespace {

__device__ unsigned g_status;  // kDevBadIndex: a slot or an expert's number was out of range

constexpr float kInf = __builtin_huge_valf();

// A plain load: what an earlier kernel of the stream wrote is not read through
// the non-coherent path, whose loads may move above the wait for that kernel.
template <class T>
__device__ __forceinline__ T ldv(const T* p) {
  return *p;
}
__device__ __forceinline__ float bf16_bits(uint32_t h) { return __uint_as_float(h << 16); }
__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// ------------------------------------------------------------------ router ----
// A warp takes a row: lane l holds the VPL consecutive logits from l VPL on.

constexpr int kRouteThreads = 1024;
constexpr int kRouteWarps = kRouteThreads / 32;
static_assert(kRouteThreads >= kMaxExperts && kRouteWarps == 32, "a thread for each expert, a lane for each warp");
// Pairs that one block takes through the whole router in one launch.
constexpr int kRouteOneBlock = 1024;
// Blocks of the two-launch form: the second launch's blocks each read all counts.  Fixed, not asked of the device: the
// workspace's size is told without one (GB300 has 152 SMs; 16384 rows of 128 on 76, 216 and 288 blocks: 26.6, 22.6 and
// 20.5 us, 20.5 on these).
constexpr int kRouteBlocks = 144;

template <bool F32, int VPL>
__device__ __forceinline__ void load_logits(const void* logits, int64_t ld, int row, int E, float (&x)[VPL]) {
  const int e0 = (threadIdx.x & 31) * VPL;
  if constexpr (F32) {
    const float* p = static_cast<const float*>(logits) + row * ld + e0;
    if (VPL % 4 == 0 && e0 + VPL <= E) {
#pragma unroll
      for (int i = 0; i < VPL / 4; ++i) {
        const float4 v = ldv(reinterpret_cast<const float4*>(p) + i);
        x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) x[i] = e0 + i < E ? ldv(p + i) : -kInf;
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(logits) + row * ld + e0;
    if (VPL % 8 == 0 && e0 + VPL <= E) {
#pragma unroll
      for (int i = 0; i < VPL / 8; ++i) {
        const uint4 v = ldv(reinterpret_cast<const uint4*>(p) + i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[8 * i + 2 * j] = bf16_bits(w[j] & 0xFFFFu);
          x[8 * i + 2 * j + 1] = bf16_bits(w[j] >> 16);
        }
      }
      return;
    }
    if (VPL == 4 && e0 + VPL <= E) {
      const uint2 v = ldv(reinterpret_cast<const uint2*>(p));
      x[0] = bf16_bits(v.x & 0xFFFFu);
      if constexpr (VPL == 4) x[1] = bf16_bits(v.x >> 16), x[2] = bf16_bits(v.y & 0xFFFFu), x[3] = bf16_bits(v.y >> 16);
      return;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) x[i] = e0 + i < E ? bf16_bits(ldv(p + i)) : -kInf;
  }
}

// Whole numbers that order like the floats (both zeros alike); 0 for what is never chosen: -inf and NaN.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (!(x > -kInf)) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}
// e^(x - m) for m the row's largest: 1 at the largest itself, an infinite one too.
__device__ __forceinline__ float exp_below(float x, float m) { return x == m ? 1.0f : expf(x - m); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The row's choices: lane j < k gets the j-th one's expert (-1: none left) and
// weight.  x: the row's logits.  A choice is a maximum over the warp and, for
// fp32, a minimum over the experts that reach it; a bf16 value leaves room for
// the expert in its key's low half, so there one maximum gives both.  A lane
// sorts its few keys first (32 rows of 128 experts 8.2 -> 7.5 us), so that a
// choice is taken off their front; many keys are searched for it instead.
template <bool F32, int VPL>
__device__ __forceinline__ void route_row(const RouteParams& p, const float (&x)[VPL], int& id, float& w) {
  const int lane = threadIdx.x & 31;
  constexpr uint32_t kLow = F32 ? 0u : 0xFFFFu;
  constexpr bool kSorted = VPL <= 8;
  uint32_t key[VPL], best = 0;
  [[maybe_unused]] uint32_t expert[F32 ? VPL : 1];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    key[i] = order_key(x[i]);
    if constexpr (F32) expert[i] = lane * VPL + i;
    else if (key[i]) key[i] = (key[i] & ~kLow) | (kLow - (lane * VPL + i));
    best = max(best, key[i]);
  }
  // a bf16 value's key has zeros (or, below zero, ones) in its low half
  const auto value = [](uint32_t k) { return key_value(F32 ? k : (k & 0x80000000u) ? k & ~kLow : k | kLow); };
  uint32_t b = __reduce_max_sync(0xffffffffu, best), mine = 0;
  const float m = value(b);
  float total = 0.0f;
  if (!p.renormalize && b != 0u) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) total += key[i] ? exp_below(value(key[i]), m) : 0.0f;
    total = warp_sum(total);
  }
  if constexpr (kSorted) {  // in falling order, equal ones by the lower expert (only neighbours out of order change)
#pragma unroll
    for (int i = 1; i < VPL; ++i)
#pragma unroll
      for (int j = i; j > 0; --j) {
        const bool swap = key[j] > key[j - 1];
        const uint32_t hi = swap ? key[j] : key[j - 1], lo = swap ? key[j - 1] : key[j];
        key[j - 1] = hi, key[j] = lo;
        if constexpr (F32) {
          const uint32_t a = swap ? expert[j] : expert[j - 1], c = swap ? expert[j - 1] : expert[j];
          expert[j - 1] = a, expert[j] = c;
        }
      }
  }
  id = -1;
  for (int j = 0; j < p.k && b != 0u; ++j) {  // uniform: at 0 the rest of the row takes no expert
    uint32_t at;
    if constexpr (F32) {
      at = ~0u;
#pragma unroll
      for (int i = kSorted ? 0 : VPL - 1; i >= 0; --i) at = key[i] == b ? expert[i] : at;
      at = __reduce_min_sync(0xffffffffu, at);  // ties: the lowest expert
    } else {
      at = kLow - (b & kLow);
    }
    if (lane == j) mine = b, id = static_cast<int>(at);
    if constexpr (kSorted) {
      bool taken = key[0] == b;
      if constexpr (F32) taken = taken && expert[0] == at;
#pragma unroll
      for (int i = 0; i + 1 < VPL; ++i) {
        key[i] = taken ? key[i + 1] : key[i];
        if constexpr (F32) expert[i] = taken ? expert[i + 1] : expert[i];
      }
      key[VPL - 1] = taken ? 0u : key[VPL - 1];
      best = key[0];
    } else {
      best = 0u;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (F32 ? at == static_cast<uint32_t>(lane * VPL + i) : key[i] == b) key[i] = 0u;
        best = max(best, key[i]);
      }
    }
    b = __reduce_max_sync(0xffffffffu, best);
  }
  const float e = mine ? exp_below(value(mine), m) : 0.0f;
  if (p.renormalize) total = warp_sum(e);
  w = mine ? e / total : 0.0f;
}

// Rows [row0, row1): choices to global memory, and (SH) each pair's expert to
// shared memory; the choices of each expert are counted in `hist`.
template <bool F32, int VPL, bool SH>
__device__ __forceinline__ void route_rows(const RouteParams& p, int row0, int row1, int* hist, int* pair_ids) {
  const int lane = threadIdx.x & 31;
  int row = row0 + (threadIdx.x >> 5);
  constexpr bool kAhead = VPL <= 8;  // registers for the next row's logits
  float x[VPL], next[kAhead ? VPL : 1];
  if constexpr (kAhead)
    if (row < row1) load_logits<F32, VPL>(p.logits, p.ld, row, p.E, next);
  for (; row < row1; row += kRouteWarps) {
    if constexpr (kAhead) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) x[i] = next[i];
      if (row + kRouteWarps < row1) load_logits<F32, VPL>(p.logits, p.ld, row + kRouteWarps, p.E, next);
    } else {
      load_logits<F32, VPL>(p.logits, p.ld, row, p.E, x);
    }
    int id;
    float w;
    route_row<F32, VPL>(p, x, id, w);
    if (lane < p.k) {
      const int64_t at = static_cast<int64_t>(row) * p.k + lane;
      p.ids[at] = id;
      p.weights[at] = w;
      if (SH) pair_ids[(row - row0) * p.k + lane] = id;
      if (id >= 0) atomicAdd(&hist[id], 1);
    }
  }
}

// Exclusive scan of counts[0 .. E) over the block (E <= kRouteThreads), in place; returns the total.
__device__ __forceinline__ int scan_counts(int* counts, int E, int* warp_sums) {
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  const int mine = t < E ? counts[t] : 0;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) warp_sums[w] = incl;
  __syncthreads();
  // every warp scans the warps' sums
  int sums = warp_sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, sums, o);
    if (lane >= o) sums += up;
  }
  const int before = w > 0 ? __shfl_sync(0xffffffffu, sums, w - 1) : 0;
  if (t < E) counts[t] = before + incl - mine;
  __syncthreads();
  return __shfl_sync(0xffffffffu, sums, 31);
}

// Places of n pairs in their order, base[e] being the first free place of
// expert e (moved on).  A pass takes a pair per thread: its rank among the
// warp's pairs of the same expert, behind the pairs of the warps before.
// `table`: kRouteWarps x E counts, zero on entry.
template <class IdOf>
__device__ __forceinline__ void place_pairs(int n, int E, IdOf&& id_of, int32_t* slots, int* base, uint8_t* table) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  for (int p0 = 0; p0 < n; p0 += kRouteThreads) {
    const int at = p0 + static_cast<int>(threadIdx.x);
    const int id = at < n ? id_of(at) : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (id >= 0 && rank == 0) table[w * E + id] = static_cast<uint8_t>(__popc(same));
    __syncthreads();
    if (id >= 0) {
      int place = base[id] + rank;
#pragma unroll 8
      for (int i = 0; i < w; ++i) place += table[i * E + id];
      slots[at] = place;
    } else if (at < n) {
      slots[at] = -1;
    }
    __syncthreads();
    if (p0 + kRouteThreads < n) {  // the next pass: bases moved on, the table zero again
      if (id >= 0 && rank == 0) {
        atomicAdd(&base[id], __popc(same));
        table[w * E + id] = 0;
      }
      __syncthreads();
    }
  }
}

// The whole router in one block, for up to kRouteOneBlock pairs: latency is
// one launch, one round of loads, k picks of each of a warp's rows, and a scan.
template <bool F32, int VPL>
__global__ void __launch_bounds__(kRouteThreads) route_one_block_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ uint8_t table[];  // kRouteWarps x E
  __shared__ int hist[kMaxExperts], pair_ids[kRouteOneBlock], warp_sums[kRouteWarps];
  for (int i = threadIdx.x; i < p.E; i += kRouteThreads) hist[i] = 0;
  for (int i = threadIdx.x; i < kRouteWarps / 4 * p.E; i += kRouteThreads) reinterpret_cast<uint32_t*>(table)[i] = 0;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  route_rows<F32, VPL, true>(p, 0, p.M, hist, pair_ids);
  __syncthreads();
  const int total = scan_counts(hist, p.E, warp_sums);
  for (int i = threadIdx.x; i < p.E; i += kRouteThreads) p.offsets[i] = hist[i];
  if (threadIdx.x == 0) p.offsets[p.E] = total;
  __syncthreads();
  place_pairs(p.M * p.k, p.E, [&](int i) { return pair_ids[i]; }, p.slots, hist, table);
}

// First launch of the two: rows_per_block rows of each block, and its counts.
// A row is latency (a load, k picks one after the other), so many warps and the
// next row's logits on their way.
template <bool F32, int VPL>
__global__ void __launch_bounds__(kRouteThreads) route_choose_kernel(const __grid_constant__ RouteParams p) {
  __shared__ int hist[kMaxExperts];
  for (int i = threadIdx.x; i < p.E; i += kRouteThreads) hist[i] = 0;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  const int row0 = blockIdx.x * p.rows_per_block;
  route_rows<F32, VPL, false>(p, row0, min(p.M, row0 + p.rows_per_block), hist, nullptr);
  __syncthreads();
  for (int i = threadIdx.x; i < p.E; i += kRouteThreads) p.counts[static_cast<int64_t>(blockIdx.x) * p.E + i] = hist[i];
}

// Second launch: every block sums all blocks' counts (its threads share an
// expert's column of them), scans the totals over the experts, and places its
// own pairs behind those of the blocks before it.
__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ uint8_t table[];
  __shared__ int totals[kMaxExperts], before[kMaxExperts], warp_sums[kRouteWarps];
  for (int i = threadIdx.x; i < p.E; i += kRouteThreads) totals[i] = before[i] = 0;
  for (int i = threadIdx.x; i < kRouteWarps / 4 * p.E; i += kRouteThreads) reinterpret_cast<uint32_t*>(table)[i] = 0;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  const int nb = gridDim.x, mine = blockIdx.x;
  // kRouteThreads / E threads share a column
  const int share = kRouteThreads / p.E, e = static_cast<int>(threadIdx.x) % p.E;
  const int g = static_cast<int>(threadIdx.x) / p.E;
  if (g < share) {
    int all = 0, first = 0;
#pragma unroll 16
    for (int b = g; b < nb; b += share) {
      const int c = ldv(p.counts + static_cast<int64_t>(b) * p.E + e);
      all += c;
      if (b < mine) first += c;
    }
    atomicAdd(&totals[e], all);  // whole numbers: the order does not matter
    atomicAdd(&before[e], first);
  }
  __syncthreads();
  const int total = scan_counts(totals, p.E, warp_sums);
  if (mine == 0) {
    for (int i = threadIdx.x; i < p.E; i += kRouteThreads) p.offsets[i] = totals[i];
    if (threadIdx.x == 0) p.offsets[p.E] = total;
  }
  for (int i = threadIdx.x; i < p.E; i += kRouteThreads) before[i] += totals[i];
  __syncthreads();
  const int row0 = mine * p.rows_per_block;
  const int64_t pair0 = static_cast<int64_t>(row0) * p.k;
  place_pairs((min(p.M, row0 + p.rows_per_block) - row0) * p.k, p.E,
              [&](int i) { return ldv(p.ids + pair0 + i); }, p.slots + pair0, before, table);
}

// A warp takes a row.  With g_j = w_j dw_j and G their sum: softmax over the
// chosen, dx = g_j - w_j G at the chosen ones and 0 elsewhere; over all
// experts, dx_e = [e chosen] g_j - p_e G with p recomputed from the logits.
template <bool F32, int VPL>
__global__ void __launch_bounds__(256) route_backward_kernel(const __grid_constant__ RouteGradParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  for (int row = blockIdx.x * 8 + (threadIdx.x >> 5); row < p.M; row += gridDim.x * 8) {
    int id = -1;
    float w = 0.0f, g = 0.0f;
    if (lane < p.k) {
      const int64_t at = static_cast<int64_t>(row) * p.k + lane;
      id = ldv(p.ids + at);
      if (id >= p.E || id < -1) {
        atomicOr(&g_status, kDevBadIndex);
        id = -1;
      }
      if (id >= 0) {
        w = ldv(p.weights + at);
        g = w * ldv(p.dweights + at);
      }
    }
    const float G = warp_sum(g);
    float d[VPL];
    if (p.renormalize) {
      g = fmaf(-w, G, g);
#pragma unroll
      for (int i = 0; i < VPL; ++i) d[i] = 0.0f;
    } else {
      float x[VPL];
      load_logits<F32, VPL>(p.logits, p.ld, row, p.E, x);
      float m = -kInf, total = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) m = x[i] > m ? x[i] : m;  // NaN never
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        d[i] = x[i] > -kInf ? exp_below(x[i], m) : 0.0f;
        total += d[i];
      }
      total = warp_sum(total);
      const float f = total > 0.0f ? -G / total : 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) d[i] *= f;
    }
    for (int j = 0; j < p.k; ++j) {
      const int e = __shfl_sync(0xffffffffu, id, j);
      const float v = __shfl_sync(0xffffffffu, g, j);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (e == lane * VPL + i) d[i] += v;
    }
    const int e0 = lane * VPL;
    if constexpr (F32) {
      float* o = static_cast<float*>(p.dlogits) + row * p.ldd + e0;
      if (VPL % 4 == 0 && e0 + VPL <= p.E) {
#pragma unroll
        for (int i = 0; i < VPL / 4; ++i)
          reinterpret_cast<float4*>(o)[i] = make_float4(d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (e0 + i < p.E) o[i] = d[i];
      }
    } else {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.dlogits) + row * p.ldd + e0;
      if (VPL % 8 == 0 && e0 + VPL <= p.E) {
#pragma unroll
        for (int i = 0; i < VPL / 8; ++i)
          reinterpret_cast<uint4*>(o)[i] =
              make_uint4(bf16x2_rn(d[8 * i], d[8 * i + 1]), bf16x2_rn(d[8 * i + 2], d[8 * i + 3]),
                         bf16x2_rn(d[8 * i + 4], d[8 * i + 5]), bf16x2_rn(d[8 * i + 6], d[8 * i + 7]));
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (e0 + i < p.E) o[i] = __float2bfloat16_rn(d[i]);
      }
    }
  }
}

// ------------------------------------------------- to and from the experts ----

// A slot of a pair, or -1; one out of range is reported and left out.
__device__ __forceinline__ int slot_of(const int32_t* slots, int64_t at, int T) {
  const int s = ldv(slots + at);
  if (s >= T || s < -1) {
    atomicOr(&g_status, kDevBadIndex);
    return -1;
  }
  return s;
}

// A block copies kCopyVecs 16-byte vectors of a row to the row's k places: the
// row is read once.  Bound by the k-fold writes.
constexpr int kCopyThreads = 128;
constexpr int kCopyVecs = 4 * kCopyThreads;

__global__ void __launch_bounds__(kCopyThreads) dispatch_kernel(const __grid_constant__ DispatchParams p, int segs) {
  __shared__ int places[kMaxChoices];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t vecs = p.row_bytes / 16, items = static_cast<int64_t>(p.M) * segs;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t row = it / segs;
    const int v0 = static_cast<int>(it - row * segs) * kCopyVecs + threadIdx.x;
    const uint4* src = static_cast<const uint4*>(p.X) + row * vecs;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (v0 + i * kCopyThreads < vecs) v[i] = __ldcs(src + v0 + i * kCopyThreads);
    if (threadIdx.x < p.k) places[threadIdx.x] = slot_of(p.slots, row * p.k + threadIdx.x, p.T);
    __syncthreads();
    for (int j = 0; j < p.k; ++j) {
      const int s = places[j];
      if (s < 0) continue;
      uint4* dst = static_cast<uint4*>(p.Xs) + s * vecs;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (v0 + i * kCopyThreads < vecs) dst[v0 + i * kCopyThreads] = v[i];
      if (p.scale != nullptr && v0 == 0) p.scale_s[s] = ldv(p.scale + row);
    }
    __syncthreads();
  }
}

// Eight columns (bf16) or four (fp32) of a row as floats, and back.
template <bool F32>
struct Vec {
  static constexpr int N = F32 ? 4 : 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[N]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F32) {
        f[i] = __uint_as_float(w[i]);
      } else {
        f[2 * i] = bf16_bits(w[i] & 0xFFFFu);
        f[2 * i + 1] = bf16_bits(w[i] >> 16);
      }
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[N]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F32) w[i] = __float_as_uint(f[i]);
      else w[i] = bf16x2_rn(f[2 * i], f[2 * i + 1]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// A thread owns one 16-byte vector of a row of H and adds the k rows in the
// choices' order, in fp32, eight loads in flight.  A 128-column group of the
// partial sums is 16 threads (bf16) or a warp (fp32).
constexpr int kCombineThreads = 128;

template <bool F32>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const __grid_constant__ CombineParams p, int segs) {
  using V = Vec<F32>;
  pdl_wait();
  pdl_launch_dependents();
  const int vecs = p.N / V::N;
  const int64_t row = blockIdx.x / segs;
  const int v0 = static_cast<int>(blockIdx.x % segs) * kCombineThreads + threadIdx.x;
  const bool in = v0 < vecs;
  float acc[V::N];
  uint4 res = make_uint4(0, 0, 0, 0);
  if (in && p.R != nullptr) res = __ldcs(static_cast<const uint4*>(p.R) + row * vecs + v0);
  V::unpack(res, acc);
  for (int j0 = 0; j0 < p.k; j0 += 8) {
    uint4 y[8];
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int s = j0 + j < p.k ? slot_of(p.slots, row * p.k + j0 + j, p.T) : -1;
      w[j] = s < 0 ? 0.0f : p.weights != nullptr ? ldv(p.weights + row * p.k + j0 + j) : 1.0f;
      // a missing row adds 0 times 0
      y[j] = s >= 0 && in ? __ldcs(static_cast<const uint4*>(p.Y) + static_cast<int64_t>(s) * vecs + v0)
                          : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j0 + j >= p.k) break;
      float f[V::N];
      V::unpack(y[j], f);
#pragma unroll
      for (int i = 0; i < V::N; ++i) acc[i] = fmaf(w[j], f[i], acc[i]);
    }
  }
  const uint4 out = V::pack(acc);
  if (in) static_cast<uint4*>(p.H)[row * vecs + v0] = out;
  if (p.P != nullptr) {
    float f[V::N], ss = 0.0f;
    V::unpack(out, f);  // of the stored values
#pragma unroll
    for (int i = 0; i < V::N; ++i) ss += in ? f[i] * f[i] : 0.0f;
    constexpr int G = kPartialCols / V::N;  // threads of a group
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (in && threadIdx.x % G == 0) p.P[row * ((p.N + kPartialCols - 1) / kPartialCols) + v0 / G] = ss;
  }
}

// A block takes a row of dH, kept in registers (NV vectors a thread; a row too
// long for that in pieces), and goes through its k rows of Y, J at a time: the
// weighted copy and the dot product, joined over the block in the threads' order.
// The copy is rounded to the rows' type: the experts' products take it as an
// operand.  Left unweighted, with the weight in the epilogue of dY . Wd, dG and dU
// would lie behind one rounding less, but dW_d = dY' act needs the weighted rows
// too: another T x N write, half as much traffic again.
constexpr int kCombineBwdThreads = 256;

template <bool F32, int NV, int J>
__global__ void __launch_bounds__(kCombineBwdThreads)
    combine_backward_kernel(const __grid_constant__ CombineGradParams p) {
  using V = Vec<F32>;
  constexpr int kWarps = kCombineBwdThreads / 32;
  __shared__ float part[kWarps][kMaxChoices];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int vecs = p.N / V::N;
  const int64_t row = blockIdx.x;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int c0 = 0; c0 < vecs; c0 += NV * kCombineBwdThreads) {
    uint4 g[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = c0 + i * kCombineBwdThreads + threadIdx.x;
      g[i] = v < vecs ? __ldcs(static_cast<const uint4*>(p.dH) + row * vecs + v) : zero;
    }
    for (int j0 = 0; j0 < p.k; j0 += J) {
      uint4 t[J][NV];
      int s[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        s[j] = j0 + j < p.k ? slot_of(p.slots, row * p.k + j0 + j, p.T) : -1;
        const uint4* y = static_cast<const uint4*>(p.Y) + static_cast<int64_t>(s[j]) * vecs;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int v = c0 + i * kCombineBwdThreads + threadIdx.x;
          t[j][i] = s[j] >= 0 && v < vecs ? __ldcs(y + v) : zero;
        }
      }
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (j0 + j >= p.k) break;
        const float wj = s[j] >= 0 ? ldv(p.weights + row * p.k + j0 + j) : 0.0f;
        uint4* dy = static_cast<uint4*>(p.dY) + static_cast<int64_t>(s[j]) * vecs;
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int v = c0 + i * kCombineBwdThreads + threadIdx.x;
          float a[V::N], b[V::N];
          V::unpack(g[i], a);
          V::unpack(t[j][i], b);
#pragma unroll
          for (int e = 0; e < V::N; ++e) {
            dot = fmaf(a[e], b[e], dot);
            a[e] *= wj;
          }
          if (s[j] >= 0 && v < vecs) dy[v] = V::pack(a);
        }
        if (s[j] < 0) dot = 0.0f;  // of a row with infinities too
        dot = warp_sum(dot);
        if (lane == 0) part[w][j0 + j] = c0 == 0 ? dot : part[w][j0 + j] + dot;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < p.k) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) sum += part[i][threadIdx.x];
    p.dweights[row * p.k + threadIdx.x] = sum;
  }
}

template <bool F32, int VPL>
cudaError_t route_launch(const RouteParams& p, cudaStream_t s, bool pdl) {
  RouteParams q = p;
  void* args[] = {&q};
  const int64_t pairs = static_cast<int64_t>(p.M) * p.k;
  const size_t table = kRouteWarps * static_cast<size_t>(p.E);
  if (pairs <= kRouteOneBlock)
    return launch_ex(reinterpret_cast<const void*>(route_one_block_kernel<F32, VPL>), dim3(1), dim3(kRouteThreads),
                     table, s, pdl, args);
  q.rows_per_block = (p.M + kRouteBlocks - 1) / kRouteBlocks;
  const int blocks = (p.M + q.rows_per_block - 1) / q.rows_per_block;
  cudaError_t e = launch_ex(reinterpret_cast<const void*>(route_choose_kernel<F32, VPL>), dim3(blocks),
                            dim3(kRouteThreads), 0, s, pdl, args);
  if (e != cudaSuccess) return e;
  return launch_ex(reinterpret_cast<const void*>(route_place_kernel), dim3(blocks), dim3(kRouteThreads), table, s, pdl,
                   args);
}

template <bool F32, int VPL>
cudaError_t route_backward_launch(const RouteGradParams& p, cudaStream_t s, bool pdl) {
  RouteGradParams q = p;
  void* args[] = {&q};
  const int64_t blocks = (static_cast<int64_t>(p.M) + 7) / 8, cap = 8 * static_cast<int64_t>(device_sm_count());
  return launch_ex(reinterpret_cast<const void*>(route_backward_kernel<F32, VPL>),
                   dim3(static_cast<unsigned>(blocks < cap ? blocks : cap)), dim3(256), 0, s, pdl, args);
}

// f(std::integral_constant<int, VPL>) for the logits a lane holds of E.
template <class F>
cudaError_t with_vpl(int E, F&& f) {
  if (E <= 32) return f(std::integral_constant<int, 1>{});
  if (E <= 64) return f(std::integral_constant<int, 2>{});
  if (E <= 128) return f(std::integral_constant<int, 4>{});
  if (E <= 256) return f(std::integral_constant<int, 8>{});
  if (E <= 512) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

unsigned row_grid(int64_t items) {
  const int64_t cap = 16 * static_cast<int64_t>(device_sm_count());
  return static_cast<unsigned>(items < cap ? items : cap);
}

}  // namespace

int64_t route_workspace_bytes(int64_t M, int64_t E, int64_t k) {
  return M * k <= kRouteOneBlock ? 0 : static_cast<int64_t>(kRouteBlocks) * E * 4;
}

cudaError_t launch_route(const RouteParams& p, bool f32, cudaStream_t s, bool pdl) {
  return with_vpl(p.E, [&](auto vpl) {
    return f32 ? route_launch<true, decltype(vpl)::value>(p, s, pdl)
               : route_launch<false, decltype(vpl)::value>(p, s, pdl);
  });
}

cudaError_t launch_route_backward(const RouteGradParams& p, bool f32, cudaStream_t s, bool pdl) {
  return with_vpl(p.E, [&](auto vpl) {
    return f32 ? route_backward_launch<true, decltype(vpl)::value>(p, s, pdl)
               : route_backward_launch<false, decltype(vpl)::value>(p, s, pdl);
  });
}

cudaError_t launch_dispatch(const DispatchParams& p, cudaStream_t s, bool pdl) {
  DispatchParams q = p;
  int segs = static_cast<int>((p.row_bytes / 16 + kCopyVecs - 1) / kCopyVecs);
  void* args[] = {&q, &segs};
  return launch_ex(reinterpret_cast<const void*>(dispatch_kernel), dim3(row_grid(static_cast<int64_t>(p.M) * segs)),
                   dim3(kCopyThreads), 0, s, pdl, args);
}

cudaError_t launch_combine(const CombineParams& p, bool f32, cudaStream_t s, bool pdl) {
  CombineParams q = p;
  int segs = combine_blocks(p.N, f32);
  void* args[] = {&q, &segs};
  const void* k = f32 ? reinterpret_cast<const void*>(combine_kernel<true>)
                      : reinterpret_cast<const void*>(combine_kernel<false>);
  return launch_ex(k, dim3(static_cast<unsigned>(static_cast<int64_t>(p.M) * segs)), dim3(kCombineThreads), 0, s, pdl,
                   args);
}

int combine_blocks(int64_t N, bool f32) {
  return static_cast<int>((N / (f32 ? 4 : 8) + kCombineThreads - 1) / kCombineThreads);
}

// Vectors a thread holds of a row, and rows of Y on their way with it: 16 loads in flight at most.
template <bool F32>
static const void* combine_backward_pick(int N) {
  const int vecs = N / Vec<F32>::N;
  if (vecs <= kCombineBwdThreads) return reinterpret_cast<const void*>(combine_backward_kernel<F32, 1, 4>);
  if (vecs <= 2 * kCombineBwdThreads) return reinterpret_cast<const void*>(combine_backward_kernel<F32, 2, 4>);
  return reinterpret_cast<const void*>(combine_backward_kernel<F32, 4, 2>);
}

cudaError_t launch_combine_backward(const CombineGradParams& p, bool f32, cudaStream_t s, bool pdl) {
  CombineGradParams q = p;
  void* args[] = {&q};
  return launch_ex(f32 ? combine_backward_pick<true>(p.N) : combine_backward_pick<false>(p.N),
                   dim3(static_cast<unsigned>(p.M)), dim3(kCombineBwdThreads), 0, s, pdl, args);
}

unsigned read_clear_status_experts() {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_status, sizeof(v)) != cudaSuccess) return ~0u;
  if (cudaMemcpyToSymbol(g_status, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace coda
