// Log probabilities of given tokens from logits, with entropy and the best
// alternatives, and their gradient:
//   lse = log sum_j exp x_j,  logp = x_t - lse,  H = lse - sum_j p_j x_j
//   dx_j = dlogp ([j = t] - p_j) - dH p_j (x_j - lse + H),  p_j = exp(x_j - lse)
// Nothing here waits on another block, but for the blocks of one cluster.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "coda_decode.h"
#include "coda_internal.h"
#include "sm103_ptx.cuh"

namespace coda {
namespace {

// Status word of this translation unit (kDevBadIndex), read back and cleared
// by read_clear_status_logprobs().
__device__ unsigned g_logprobs_status;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// The two halves of cluster_sync, for work between them.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The larger of two values, NaN if one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// 16 bytes of logits as pairs of fp32 values.
template <class E>
__device__ __forceinline__ void pairs(const uint4& w, float2 (&f)[8 / sizeof(E)]) {
  if constexpr (sizeof(E) == 4) {
    f[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    f[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
  } else {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = __bfloat1622float2(h[e]);
  }
}

// The largest of N times 16 bytes of logits.
template <class E, int N>
__device__ __forceinline__ float largest(const uint4 (&w)[N]) {
  if constexpr (sizeof(E) == 4) {
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < N; ++u)
      m = max_nan(m, max_nan(max_nan(__uint_as_float(w[u].x), __uint_as_float(w[u].y)),
                             max_nan(__uint_as_float(w[u].z), __uint_as_float(w[u].w))));
    return m;
  } else {
    __nv_bfloat162 m[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w[u]);
      m[u] = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
      if (u > 0) m[0] = __hmax2_nan(m[0], m[u]);
    }
    return max_nan(__low2float(m[0]), __high2float(m[0]));
  }
}

// The pass takes x log2 e relative to a rounded base, whose rounding is at most
// 1 while |x| < 2^24 (its weights are off by a factor within [1/2, 2], which is
// taken out at the end) and grows with |x| without bound.  So
//   - logits below -kLift are taken as -kLift;
//   - a thread whose largest logit is kFar or more in size leaves its sums out;
//   - a row (or a block's part of it) whose largest logit is kCareful or more in
//     size is summed once more from the differences to it.
// The steps between the three are far more than the 150 beyond which a weight
// is 0, so what is lifted or left out has no weight beside a largest logit above
// -kCareful.  Powers of two that bf16 holds.
constexpr float kCareful = 0x1p23f, kFar = 0x1p24f, kLift = 0x1p25f;

// 16 bytes of logits, none below -kLift (NaN stays).
template <class E>
__device__ __forceinline__ uint4 lifted(const uint4& w) {
  uint4 o;
  if constexpr (sizeof(E) == 4) {
    o = make_uint4(__float_as_uint(max_nan(__uint_as_float(w.x), -kLift)), __float_as_uint(max_nan(__uint_as_float(w.y), -kLift)),
                   __float_as_uint(max_nan(__uint_as_float(w.z), -kLift)), __float_as_uint(max_nan(__uint_as_float(w.w), -kLift)));
  } else {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
    __nv_bfloat162* r = reinterpret_cast<__nv_bfloat162*>(&o);
    const __nv_bfloat162 low = __floats2bfloat162_rn(-kLift, -kLift);
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = __hmax2_nan(h[e], low);
  }
  return o;
}

// Vector v of a row of V logits; elements behind the row are -inf.
template <class E>
__device__ __forceinline__ uint4 load_vec(const E* x, int v, int V) {
  constexpr int VEC = 16 / sizeof(E);
  if ((v + 1) * VEC <= V) return __ldg(reinterpret_cast<const uint4*>(x) + v);
  uint4 w;
  E* e = reinterpret_cast<E*>(&w);
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    const int j = v * VEC + k;
    if constexpr (sizeof(E) == 4)
      e[k] = j < V ? x[j] : -INFINITY;
    else
      e[k] = j < V ? x[j] : __ushort_as_bfloat16(0xFF80);
  }
  return w;
}

// Order of the alternatives: the larger value first (NaN counts as the
// largest), then the lower index.  32-bit keys order the values; 64-bit keys
// with the index's complement below are distinct.  No value has the key 0.
__device__ __forceinline__ uint32_t value_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);  // -0 is 0
  return x != x ? 0xffffffffu : (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k == 0xffffffffu ? 0x7fffffffu : (k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// Partial sums of a set of logits relative to their largest m: s = sum 2^d,
// t = sum d 2^d with d = (x - m) log2 e.  -inf has no part in either.
struct Sums {
  float m, s, t;
  // the same sums relative to a larger (or NaN) maximum
  __device__ __forceinline__ void raise(float mn) {
    if (s != 0.0f) {
      const float d = (m - mn) * kLog2e, c = ex2_approx(d);
      t = c == 0.0f ? 0.0f : (t + s * d) * c;
      s *= c;
    }
    m = mn;
  }
};

constexpr int kRowVecs = 4;  // vectors of a thread in flight (figures below)
constexpr int kCandidates = 1024;
constexpr int kMaxCluster = 8;

template <int NT>
struct LogprobsShared {
  Sums warp[NT / 32];
  __align__(16) uint32_t tops[128];  // each warp's largest thread maxima
  uint32_t bound;
  int owner[NT];          // threads whose largest value reaches the bound
  int owners, found;
  __align__(16) uint64_t cand[kCandidates];
  uint64_t red[NT / 32];
  // what the cluster's first block collects
  Sums part;
  uint64_t best[kMaxTop];
};

// One pass over a row (or, in a cluster, over a part of it) with a running
// maximum, sum and sum of d 2^d per thread, joined at the end.
//
// The alternatives cost the pass nothing: each thread knows its own largest
// value, and the top-th largest of those is a bound that at least `top`
// elements reach (a slightly lower one is quicker to find).  Only threads whose
// largest value reaches it can hold an alternative, each with 1 / NT of the
// row, so their elements are read once more, from L2 as a rule: 20 of 512
// threads are 4% of the row.  The few elements that reach the bound are ranked
// by counting.  If ties leave more than kCandidates of them (512 to 2048 make
// no difference otherwise), those at the bound are taken in the order of the
// row, and if more than that are above it, one by one.
//
// Bound by the row's bytes.  bf16 costs about 5 issue slots an element (the
// arithmetic is packed in pairs) of the 11 that the HBM rate leaves.  2048 rows
// of 128256 bf16 logits take 82 us without alternatives (6.4 TB/s), 92 with 8
// (5.7 TB/s), 101 with 20 and 128 with 64: the end of a row costs its block
// about as long as 1 / 8 of the row.  kRowVecs of 2 / 3 / 4 / 6 made that
// 102 / 98 / 92 / 103; a ring of cp.async stages that ran across the rows 130;
// the bound found by bits over all warps 106.
template <class E, int NT, bool CLUSTER>
__global__ void __launch_bounds__(NT, CLUSTER ? 2 : 1536 / NT) logprobs_kernel(const __grid_constant__ LogprobsParams p) {
  constexpr int VEC = 16 / sizeof(E), U = kRowVecs;
  __shared__ LogprobsShared<NT> sh;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int rank = CLUSTER ? static_cast<int>(cluster_ctarank()) : 0, ranks = CLUSTER ? p.ranks : 1;
  const int64_t i = blockIdx.x / ranks;
  pdl_wait();
  pdl_launch_dependents();
  const E* x = static_cast<const E*>(p.logits) + i * p.ld;
  const int vecs = (p.V + VEC - 1) / VEC, per = (vecs + ranks - 1) / ranks;
  const int v0 = min(rank * per, vecs), v1 = min(v0 + per, vecs);

  // the row's token: fetched now, its logit behind the loop, both used at the end
  const int tgt = tid == 0 && rank == 0 ? p.targets[i] : -1;

  // This thread's running maximum m and sums relative to base = m log2 e, two of each side by side: d = x log2 e - base
  // is one operation for two elements.  -inf and huge negative logits are lifted to -kLift, whose weight is 0 as well.
  float m = -INFINITY, base = 0.0f;
  float2 s2 = make_float2(0.0f, 0.0f), t2 = s2;
  const int whole = min(v1, p.V / VEC);  // vectors without an end of the row inside
  uint4 q[U];
  for (int v = v0 + tid; v < v1; v += U * NT) {
    if (v + (U - 1) * NT < whole) {
#pragma unroll
      for (int u = 0; u < U; ++u) q[u] = __ldg(reinterpret_cast<const uint4*>(x) + v + u * NT);
    } else {
      // the last round: what lies behind the row or this block's part of it is -inf
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (v + u * NT < whole)
          q[u] = __ldg(reinterpret_cast<const uint4*>(x) + v + u * NT);
        else
          q[u] = load_vec<E>(x, v + u * NT < v1 ? v + u * NT : vecs, p.V);
      }
    }
    const float big = largest<E, U>(q);
    if (!(big <= m)) {
      m = max_nan(m, big);
      const float to = fminf(fmaxf(m, -kLift), kLift) * kLog2e, d = base - to, c = ex2_approx(d);
      // the first time there is nothing to scale (and c may be infinite); a weight of 0 ends what was summed
      const bool none = c == 0.0f || s2.x + s2.y == 0.0f;
      t2 = none ? make_float2(0.0f, 0.0f) : fmul2(ffma2(s2, make_float2(d, d), t2), make_float2(c, c));
      s2 = none ? make_float2(0.0f, 0.0f) : fmul2(s2, make_float2(c, c));
      base = to;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 f[8 / sizeof(E)];
      pairs<E>(lifted<E>(q[u]), f);
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) {
        const float2 d = ffma2(f[e], make_float2(kLog2e, kLog2e), make_float2(-base, -base));
        const float2 g = make_float2(ex2_approx(d.x), ex2_approx(d.y));
        s2 = fadd2(s2, g);
        t2 = ffma2(g, d, t2);
      }
    }
  }
  E at_tgt = {};
  if (tgt >= 0 && tgt < p.V) at_tgt = x[tgt];
  // the sums relative to m itself: base was rounded by `off`
  Sums a = {m, s2.x + s2.y, t2.x + t2.y};
  if (!(m < INFINITY)) {
    a.s = a.t = NAN;  // +inf or NaN
  } else if (fabsf(m) >= kFar) {
    a.s = a.t = 0.0f;  // no weight beside an ordinary logit (and see `careful`)
  } else {
    const float off = fmaf(m, kLog2e, -base), c = ex2_approx(-off);
    a.t = (a.t - off * a.s) * c;
    a.s *= c;
  }
  const uint32_t key = v0 + tid < v1 ? value_key(m) : 0u;
  if (tid == 0) {
    sh.owners = 0;
    sh.found = 0;
  }
  // sums of a warp relative to its largest m
  auto warp_sums = [&]() {
    a.raise(key_value(__reduce_max_sync(0xffffffffu, value_key(a.m))));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
      a.t += __shfl_xor_sync(0xffffffffu, a.t, o);
    }
  };

  // ---- the bound of the alternatives: each warp's `each` largest keys (taken out one by one), of all of those the
  // top-th.  top threads reach it, and with one or two more a warp than top needs few others do.  (A last warp with few
  // elements counts as a whole one: from 30 alternatives on, rows of 1025 to 1552 bf16 logits may gather fewer than top
  // keys.  The bound is 0 then and every element reaches it: 300 rows of 1032 with 50 take 100 us, of 1000 8 us.)
  if (p.top > 0) {
    const int warps = max(min(NT / 32, (v1 - v0 + 31) / 32), 1);  // that have elements
    const int each = min(warps == NT / 32 ? (p.top + NT / 32 - 1) / (NT / 32) + 1 : (p.top + warps - 1) / warps + 1, 32);
    const int n = warps * each, n4 = (n + 3) & ~3;
    if (w < warps) {
      uint32_t k = key;
#pragma unroll 1
      for (int e = 0; e < each; ++e) {
        const uint32_t best = __reduce_max_sync(0xffffffffu, k);
        if (lane == 0) sh.tops[e * warps + w] = best;
        if (lane == __ffs(__ballot_sync(0xffffffffu, k == best)) - 1) k = 0;
      }
    }
    if (tid < n4 - n) sh.tops[n + tid] = 0;
    if (tid == 0) sh.bound = 0;
    __syncthreads();
    // how many are above a key, and how many reach it: up to 32 keys lie in a warp's lanes, else a thread counts for each
    if (n <= 32) {
      const uint32_t all = lane < n4 ? sh.tops[lane] : 0u;
#pragma unroll 1
      for (int c = w; c < n; c += NT / 32) {
        const uint32_t mine = __shfl_sync(0xffffffffu, all, c);
        const int above = __popc(__ballot_sync(0xffffffffu, all > mine)), reach = __popc(__ballot_sync(0xffffffffu, all >= mine));
        if (above < p.top && reach >= p.top) sh.bound = mine;  // the same value from all that write it
      }
    } else {
#pragma unroll 1
      for (int c = tid; c < n; c += NT) {
        const uint32_t mine = sh.tops[c];
        int above = 0, reach = 0;
#pragma unroll 2
        for (int o = 0; o < n4; o += 4) {
          const uint4 t = *reinterpret_cast<const uint4*>(sh.tops + o);
          above += (t.x > mine) + (t.y > mine) + (t.z > mine) + (t.w > mine);
          reach += (t.x >= mine) + (t.y >= mine) + (t.z >= mine) + (t.w >= mine);
        }
        if (above < p.top && reach >= p.top) sh.bound = mine;
      }
    }
    __syncthreads();
  }
  // ---- the elements that reach it, and the row's sums meanwhile
  int local = 0;  // alternatives this block has: min(top, its elements)
  bool sums_done = false;
  if (p.top > 0) {
    const int64_t first = static_cast<int64_t>(v0) * VEC, last = min(static_cast<int64_t>(v1) * VEC, static_cast<int64_t>(p.V));
    local = static_cast<int>(min(static_cast<int64_t>(p.top), max(last - first, static_cast<int64_t>(0))));
    const uint32_t bound = sh.bound;
    const bool owner = v0 + tid < v1 && key >= bound;
    auto collect = [&](const uint4& vec, int u) {
      const E* e = reinterpret_cast<const E*>(&vec);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const uint32_t j = u * VEC + k, val = value_key(to_f32(e[k]));
        if (val >= bound && j < static_cast<uint32_t>(p.V)) {
          const int at = atomicAdd(&sh.found, 1);
          if (at < kCandidates) sh.cand[at] = (static_cast<uint64_t>(val) << 32) | static_cast<uint32_t>(~j);
        }
      }
    };
    const uint32_t mask = __ballot_sync(0xffffffffu, owner);
    int at = 0;
    if (lane == 0 && mask != 0) at = atomicAdd(&sh.owners, __popc(mask));
    at = __shfl_sync(0xffffffffu, at, 0) + __popc(mask & ((1u << lane) - 1u));
    if (owner) sh.owner[at] = tid;
    __syncthreads();
    // the owners' vectors dealt to the threads, 2^shift an owner (a few more than it has)
    const int mine = (v1 - v0 + NT - 1) / NT, shift = mine > 1 ? 32 - __clz(mine - 1) : 0, all = sh.owners << shift;
    auto place = [&](int k) { return k < all ? v0 + sh.owner[k >> shift] + (k & ((1 << shift) - 1)) * NT : v1; };
    int u = place(tid);
    uint4 vec;
    if (u < v1) vec = load_vec<E>(x, u, p.V);
    warp_sums();  // while the elements are on their way
    sums_done = true;
#pragma unroll 1
    for (int k = tid; k < all; k += NT) {
      if (u < v1) collect(vec, u);
      u = place(k + NT);
      if (u < v1) vec = load_vec<E>(x, u, p.V);
    }
  }
  if (!sums_done) warp_sums();
  if (lane == 0) sh.warp[w] = a;
  __syncthreads();
  if (w == 0) {
    a = lane < NT / 32 ? sh.warp[lane] : Sums{-INFINITY, 0.0f, 0.0f};
    warp_sums();
    if (lane == 0) sh.part = a;
  }
  if (p.top > 0) {
    int n = sh.found;
    if (__builtin_expect(n > kCandidates, 0)) {
      // many equal elements at the bound: those above it once more, then as many of the equal ones as are missing, in
      // the order of the row
      const uint32_t bound = sh.bound;
      __syncthreads();
      if (tid == 0) sh.found = 0;
      __syncthreads();
#pragma unroll 1
      for (int u = v0 + tid; u < v1; u += NT) {
        const uint4 vec = load_vec<E>(x, u, p.V);
        const E* e = reinterpret_cast<const E*>(&vec);
#pragma unroll
        for (int z = 0; z < VEC; ++z) {
          const uint32_t j = u * VEC + z, val = value_key(to_f32(e[z]));
          if (val > bound && j < static_cast<uint32_t>(p.V)) {
            const int at = atomicAdd(&sh.found, 1);
            if (at < kCandidates) sh.cand[at] = (static_cast<uint64_t>(val) << 32) | static_cast<uint32_t>(~j);
          }
        }
      }
      __syncthreads();
      n = sh.found;
#pragma unroll 1
      for (int first = v0; first < v1 && n < local; first += NT) {
        const int u = first + tid;
        uint4 vec;
        uint32_t equal = 0;  // a bit for each
        if (u < v1) {
          vec = load_vec<E>(x, u, p.V);
          const E* e = reinterpret_cast<const E*>(&vec);
#pragma unroll
          for (int z = 0; z < VEC; ++z)
            equal |= (value_key(to_f32(e[z])) == bound && u * VEC + z < p.V ? 1u : 0u) << z;
        }
        int upto = __popc(equal);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += t;
        }
        if (lane == 31) sh.red[w] = upto;
        __syncthreads();
        int at = n + upto - __popc(equal), all = 0;
        for (int o = 0; o < NT / 32; ++o) {
          if (o < w) at += static_cast<int>(sh.red[o]);
          all += static_cast<int>(sh.red[o]);
        }
        for (; equal != 0 && at < local; ++at, equal &= equal - 1)
          sh.cand[at] = (static_cast<uint64_t>(bound) << 32) | static_cast<uint32_t>(~(u * VEC + __ffs(equal) - 1));
        n = min(n + all, local);
        __syncthreads();
      }
    }
    if (__builtin_expect(n <= kCandidates, 1)) {
      if (n <= 32) {
        const uint64_t all = lane < n ? sh.cand[lane] : 0u;
#pragma unroll 1
        for (int c = w; c < n; c += NT / 32) {
          const uint64_t mine = sh.cand[c];
          const int before = __popc(__ballot_sync(0xffffffffu, all > mine));
          if (before < local) sh.best[before] = mine;
        }
      } else {
#pragma unroll 1
        for (int c = tid; c < n; c += NT) {  // a thread for each counts those above it
          const uint64_t mine = sh.cand[c];
          int before = n & 1 ? sh.cand[n - 1] > mine : 0;
#pragma unroll 2
          for (int o = 0; o + 1 < n; o += 2) {
            const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(sh.cand + o);
            before += (t.x > mine) + (t.y > mine);
          }
          if (before < local) sh.best[before] = mine;
        }
      }
    } else {
      uint64_t below = ~0ull;
#pragma unroll 1
      for (int k = 0; k < local; ++k) {
        uint64_t best = 0;
#pragma unroll 1
        for (int u = v0 + tid; u < v1; u += NT) {
          const uint4 q = load_vec<E>(x, u, p.V);
          const E* e = reinterpret_cast<const E*>(&q);
#pragma unroll
          for (int z = 0; z < VEC; ++z) {
            const uint32_t j = u * VEC + z;
            const uint64_t key = (static_cast<uint64_t>(value_key(to_f32(e[z]))) << 32) | static_cast<uint32_t>(~j);
            if (j < static_cast<uint32_t>(p.V) && key < below && key > best) best = key;
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const uint64_t b = __shfl_xor_sync(0xffffffffu, best, o);
          best = b > best ? b : best;
        }
        if (lane == 0) sh.red[w] = best;
        __syncthreads();
        for (int o = 0; o < NT / 32; ++o) best = sh.red[o] > best ? sh.red[o] : best;
        if (tid == 0) sh.best[k] = best;
        below = best;
        __syncthreads();
      }
    }
  }
  __syncthreads();
  if (__builtin_expect(fabsf(sh.part.m) >= kCareful && fabsf(sh.part.m) < INFINITY, 0)) {
    // careful: the largest logit is huge (a row of the type's lowest value), so d is taken from the difference
    const float top = sh.part.m;
    a = {top, 0.0f, 0.0f};
#pragma unroll 1
    for (int v = v0 + tid; v < v1; v += NT) {
      float2 f[8 / sizeof(E)];
      pairs<E>(load_vec<E>(x, v, p.V), f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = fmaxf(((e & 1 ? f[e / 2].y : f[e / 2].x) - top) * kLog2e, -200.0f), g = ex2_approx(d);
        a.s += g;
        a.t += g * d;
      }
    }
    warp_sums();
    if (lane == 0) sh.warp[w] = a;
    __syncthreads();  // and every thread has read sh.part
    if (w == 0) {
      a = lane < NT / 32 ? sh.warp[lane] : Sums{-INFINITY, 0.0f, 0.0f};
      warp_sums();
      if (lane == 0) sh.part = a;
    }
    __syncthreads();
  }

  // ---- the cluster's parts, collected by its first block
  Sums row = sh.part;
  if constexpr (CLUSTER) {
    cluster_sync();
    if (rank == 0) {
      if (w == 0) {  // a lane for each block
        a = Sums{-INFINITY, 0.0f, 0.0f};
        if (lane < ranks) {
          const uint32_t at = mapa_shared(smem_u32(&sh.part), lane);
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(a.m) : "r"(at) : "memory");
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(a.s) : "r"(at + 4) : "memory");
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(a.t) : "r"(at + 8) : "memory");
        }
        warp_sums();
        row = a;  // lane 0's is handed on below
      }
      // every block's alternatives side by side; a block with fewer has the key 0 in their place
      static_assert(kMaxCluster * kMaxTop <= kCandidates, "the cluster's alternatives fit the candidates");
      for (int c = tid; c < ranks * p.top; c += NT) {
        const int r = c / p.top, k = c % p.top;
        const int r0 = min(r * per, vecs), r1 = min(r0 + per, vecs);
        const int64_t have = min(static_cast<int64_t>(r1) * VEC, static_cast<int64_t>(p.V)) - static_cast<int64_t>(r0) * VEC;
        uint64_t key = 0;
        if (k < have) {
          const uint32_t at = mapa_shared(smem_u32(&sh.best[k]), r);
          asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(key) : "r"(at) : "memory");
        }
        sh.cand[c] = key;
      }
    }
    __syncwarp();
    cluster_arrive();
    if (rank != 0) {
      cluster_wait();  // this block's shared memory was read
      return;
    }
    __syncthreads();
    if (tid == 0) sh.part = row;
    if (p.top > 0) {
      // an alternative's rank: those above it in each block's list, found by bisection by a lane for each list (the
      // lists' number is a power of two), two alternatives at a time
      constexpr int SIDE = 2;
      const int n = ranks * p.top * ranks, log2_ranks = 31 - __clz(ranks), half = 1 << (31 - __clz(p.top));
#pragma unroll 1
      for (int c0 = tid; c0 < ((n + 31) & ~31); c0 += SIDE * NT) {
        uint64_t mine[SIDE];
        int list[SIDE], lo[SIDE];
#pragma unroll
        for (int j = 0; j < SIDE; ++j) {
          const int from = min(c0 + j * NT, n - 1);
          mine[j] = sh.cand[from >> log2_ranks];
          list[j] = (from & (ranks - 1)) * p.top - 1;
          lo[j] = 0;
        }
#pragma unroll 1
        for (int step = half; step > 0; step >>= 1)
#pragma unroll
          for (int j = 0; j < SIDE; ++j)
            if (lo[j] + step <= p.top && sh.cand[list[j] + lo[j] + step] > mine[j]) lo[j] += step;
#pragma unroll
        for (int j = 0; j < SIDE; ++j) {
          for (int o = 1; o < ranks; o <<= 1) lo[j] += __shfl_xor_sync(0xffffffffu, lo[j], o);
          if (c0 + j * NT < n && (c0 & (ranks - 1)) == 0 && lo[j] < p.top && mine[j] != 0) sh.best[lo[j]] = mine[j];
        }
      }
    }
    __syncthreads();
    row = sh.part;
  }

  // ---- results
  const bool empty = row.s == 0.0f;  // nothing but -inf
  const float log_s = tid == 0 || tid < p.top ? logf(row.s) : 0.0f;
  if (tid == 0) {
    float lp = 0.0f;
    if (tgt >= p.V)
      atomicOr(&g_logprobs_status, kDevBadIndex);
    else if (tgt >= 0)
      lp = empty ? -INFINITY : (to_f32(at_tgt) - row.m) - log_s;
    p.logp[i] = lp;
    if (p.entropy) p.entropy[i] = empty ? 0.0f : log_s - row.t / row.s * kLn2;
    if (p.lse) p.lse[i] = empty ? -INFINITY : row.m + log_s;
  }
  for (int k = tid; k < p.top; k += NT) {
    const uint64_t key = sh.best[k];
    p.top_ids[i * p.top + k] = static_cast<int>(~static_cast<uint32_t>(key));
    p.top_logp[i * p.top + k] = empty ? -INFINITY : (key_value(static_cast<uint32_t>(key >> 32)) - row.m) - log_s;
  }
  if constexpr (CLUSTER) {
    __syncwarp();
    cluster_wait();
  }
}

// Gradient: element by element, bound by reading the logits and writing the
// gradient.  A block takes kGradVecs vectors a thread of one row, so the row's
// statistics are read once for 8 KB and the loads are in flight meanwhile.
// 4096 rows of 128256 bf16 logits take 320 us (6.6 TB/s); blocks of 256 threads
// 321, of 512 453; 2 vectors a thread 392, 8 325.
//   dx = 2^(lp log2 e) (A + B lp),  lp = x - lse, A = -(dlogp + dH H), B = -dH
// From kFarLse on, fp32 rounds lse by more than 2^-10 and in the end loses log V
// altogether (a row of the type's lowest value), and p with it.  Such a row's
// blocks each sum its exp(x - lse), whose differences are exact, and write their
// part once more with the logarithm `rest` off lp as well.  That comes behind
// the ordinary pass, which it costs 1%: with `rest` in the pass, or the choice
// ahead of it, 4096 rows took 326 to 338 us.
constexpr int kGradThreads = 128, kGradVecs = 4;
constexpr float kFarLse = 0x1p15f;

template <class E>
__global__ void __launch_bounds__(kGradThreads) logprobs_backward_kernel(const __grid_constant__ LogprobsGradParams p) {
  constexpr int VEC = 16 / sizeof(E);
  const int64_t i = blockIdx.x / p.blocks;
  const int v0 = static_cast<int>(blockIdx.x % p.blocks) * kGradThreads * kGradVecs + threadIdx.x;
  const E* x = static_cast<const E*>(p.logits) + i * p.ld;
  E* dx = static_cast<E*>(p.dlogits) + i * p.ldd;
  const int vecs = (p.V + VEC - 1) / VEC;
  pdl_wait();
  pdl_launch_dependents();
  uint4 q[kGradVecs];
#pragma unroll
  for (int u = 0; u < kGradVecs; ++u)
    if (v0 + u * kGradThreads < vecs) q[u] = load_vec<E>(x, v0 + u * kGradThreads, p.V);
  int tgt = p.targets[i];
  if (tgt >= p.V) {
    if (v0 == 0) atomicOr(&g_logprobs_status, kDevBadIndex);
    tgt = -1;
  }
  const float lse = p.lse[i], H = p.entropy ? p.entropy[i] : 0.0f;
  const bool empty = lse == -INFINITY;
  const float dl = p.dlogp && tgt >= 0 && !empty ? p.dlogp[i] : 0.0f, dh = p.dentropy && !empty ? p.dentropy[i] : 0.0f;
  const float B = -dh;
  // the gradient of vector v with its logits; far: with `rest`
  auto put = [&](auto far, int v, const uint4& logits, float A, float rest) {
    float2 f[8 / sizeof(E)];
    pairs<E>(logits, f);
    float g[VEC];
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) {
      const float2 lp = fadd2(f[e], make_float2(-lse, -lse));
      float2 pr;
      if constexpr (sizeof(E) == 4) {
        pr = decltype(far)::value ? make_float2(expf(lp.x - rest), expf(lp.y - rest)) : make_float2(expf(lp.x), expf(lp.y));
      } else {
        float2 d;
        if constexpr (decltype(far)::value)
          d = ffma2(lp, make_float2(kLog2e, kLog2e), make_float2(-rest * kLog2e, -rest * kLog2e));
        else
          d = fmul2(lp, make_float2(kLog2e, kLog2e));
        pr = make_float2(ex2_approx(d.x), ex2_approx(d.y));
      }
      const float2 r = fmul2(pr, ffma2(make_float2(B, B), lp, make_float2(A, A)));
      // no probability, no gradient: x = -inf would give 0 * inf, and so would an empty row
      g[2 * e] = pr.x == 0.0f || empty ? 0.0f : r.x;
      g[2 * e + 1] = pr.y == 0.0f || empty ? 0.0f : r.y;
    }
    const int at = tgt - v * VEC;
    if (at >= 0 && at < VEC) {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e == at) g[e] += dl;
    }
    uint4 o;
    E* oe = reinterpret_cast<E*>(&o);
    if constexpr (sizeof(E) == 4) {
      o = make_uint4(__float_as_uint(g[0]), __float_as_uint(g[1]), __float_as_uint(g[2]), __float_as_uint(g[3]));
    } else {
      __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&o);
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(g[2 * e], g[2 * e + 1]);
    }
    if ((v + 1) * VEC <= p.V) {
      __stcs(reinterpret_cast<uint4*>(dx) + v, o);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (v * VEC + e < p.V) dx[v * VEC + e] = oe[e];
    }
  };
#pragma unroll
  for (int u = 0; u < kGradVecs; ++u) {
    if (v0 + u * kGradThreads >= vecs) break;
    put(std::false_type(), v0 + u * kGradThreads, q[u], -(dl + dh * H), 0.0f);
  }
  if (__builtin_expect(fabsf(lse) >= kFarLse && fabsf(lse) < INFINITY, 0)) {
    __shared__ float sums[kGradThreads / 32];
    float sum = 0.0f;
#pragma unroll 1
    for (int v = threadIdx.x; v < vecs; v += kGradThreads) {
      float2 f[8 / sizeof(E)];
      pairs<E>(load_vec<E>(x, v, p.V), f);
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) sum += ex2_approx((f[e].x - lse) * kLog2e) + ex2_approx((f[e].y - lse) * kLog2e);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x / 32] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kGradThreads / 32; ++w) sum += sums[w];
    // no more than a rounding may lack; an lse of other logits than this row's is taken as it is
    const float lacks = logf(sum), rest = fabsf(lacks) <= fabsf(lse) * 0x1p-23f ? lacks : 0.0f;
#pragma unroll 1
    for (int u = 0; u < kGradVecs; ++u)
      if (v0 + u * kGradThreads < vecs)
        put(std::true_type(), v0 + u * kGradThreads, load_vec<E>(x, v0 + u * kGradThreads, p.V), dh * rest - (dl + dh * H), rest);
  }
}

template <class E, int NT, bool CLUSTER>
cudaError_t run_logprobs(LogprobsParams p, int64_t M, int c, cudaStream_t s, bool pdl) {
  p.ranks = c;
  void* args[] = {&p};
  return launch_ex(reinterpret_cast<const void*>(logprobs_kernel<E, NT, CLUSTER>), dim3(static_cast<unsigned>(M * c)),
                   dim3(NT), 0, s, pdl, args, c);
}

// How many threads take a row (us for M rows of V bf16 logits with 8 alternatives, by 128 / 256 / 512 threads):
//   many rows   4096 x 1000: 17 / 24 / 41    4096 x 16000: 32 / 36 / 51   4096 x 32000: 56 / 53 / 68
//               4096 x 50264: 89 / 80 / 93   2048 x 65536: 63 / 53 / 54   2048 x 128256: 131 / 100 / 92
//   few rows    64 x 16000: 6.0 / 4.7 / 4.7  200 x 16000: 6.4 / 5.3 / 5.9  400 x 8192: 5.3 / 5.4 / 7.9
// so rows that leave SMs idle take 512 threads, many rows fewer while they are short: a row's serial end, which finds
// its alternatives, then leaves more of the SM to other rows.
// One row or a few that are long take a cluster (us by 1 / 2 / 4 / 8 blocks of 512, for 0, 8 and 50 alternatives):
//   1 x 50264    4.6 / 4.7 / 4.0 / 4.0   6.1 / 6.9 / 6.3 / 6.7    8.2 / 8.3 / 7.8 / 9.8
//   1 x 70000    5.5 / 5.2 / 4.5 / 4.0   7.1 / 7.4 / 6.7 / 6.6   10.1 / 9.4 / 8.3 / 9.8
//   1 x 128256   7.3 / 5.9 / 4.6 / 4.0   8.8 / 8.0 / 6.9 / 6.6   12.1 / 10.0 / 8.5 / 9.7
//   1 x 200000   10.5 / 7.7 / 5.8 / 4.8  12.2 / 9.8 / 8.0 / 7.3  16.8 / 12.9 / 10.2 / 10.6
// and 76 x 128256 takes 9.4 by one and 8.8 by two (8 alternatives).  So from 3.5 rounds of loads a row is split until a
// block has one round, or the blocks fill the SMs, by at most 8, or 4 where many alternatives have to be merged.
template <class E>
cudaError_t pick_logprobs(const LogprobsParams& p, int64_t M, cudaStream_t s, bool pdl) {
  constexpr int64_t ROUND = 512 * kRowVecs * (16 / sizeof(E));
  const int sms = device_sm_count();
  int c = 1;
  if (p.V * 2 >= ROUND * 7)
    while (c < (p.top > 16 ? kMaxCluster / 2 : kMaxCluster) && M * c * 2 <= sms && p.V > ROUND * c) c *= 2;
  if (c > 1) return run_logprobs<E, 512, true>(p, M, c, s, pdl);
  const int64_t bytes = static_cast<int64_t>(p.V) * sizeof(E);
  if (M <= 2 * sms || bytes > 128 * 1024) return run_logprobs<E, 512, false>(p, M, 1, s, pdl);
  return bytes > 48 * 1024 ? run_logprobs<E, 256, false>(p, M, 1, s, pdl) : run_logprobs<E, 128, false>(p, M, 1, s, pdl);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsParams& p, int64_t M, bool f32, cudaStream_t s, bool pdl) {
  return f32 ? pick_logprobs<float>(p, M, s, pdl) : pick_logprobs<__nv_bfloat16>(p, M, s, pdl);
}

int64_t logprobs_backward_blocks(int64_t V, bool f32) {
  const int64_t per = static_cast<int64_t>(kGradThreads) * kGradVecs * (f32 ? 4 : 8);
  return (V + per - 1) / per;
}

cudaError_t launch_logprobs_backward(const LogprobsGradParams& q, int64_t M, bool f32, cudaStream_t s, bool pdl) {
  LogprobsGradParams p = q;
  p.blocks = static_cast<int>(logprobs_backward_blocks(p.V, f32));
  const void* k = f32 ? reinterpret_cast<const void*>(logprobs_backward_kernel<float>)
                      : reinterpret_cast<const void*>(logprobs_backward_kernel<__nv_bfloat16>);
  void* args[] = {&p};
  return launch_ex(k, dim3(static_cast<unsigned>(M * p.blocks)), dim3(kGradThreads), 0, s, pdl, args);
}

unsigned read_clear_status_logprobs() {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_logprobs_status, sizeof(v)) != cudaSuccess) return ~0u;
  if (cudaMemcpyToSymbol(g_logprobs_status, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace coda
