// Paged key/value cache of the decode step around the block tail:
//   append     rows of a QKV product -> rotated Q, and K (rotated) and V into
//              the cache's pages
//   attention  one new token per row over the cached keys and values
// Cache layout: [num_pages, kv_heads, page_size, head_dim], so that a page's
// rows of one head are contiguous.  Nothing here waits on another block.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "coda_decode.h"
#include "coda_internal.h"
#include "fp8_e4m3.cuh"
#include "sm103_ptx.cuh"

namespace coda {
namespace {

// Status word of this translation unit (kDevBadIndex), read back and cleared
// by read_clear_status_paged().
__device__ unsigned g_paged_status;

// 16 bytes of a row as fp32 values, and back.
template <class E>
__device__ __forceinline__ void unpack(const uint4& w, float (&f)[16 / sizeof(E)]) {
  if constexpr (sizeof(E) == 4) {
    f[0] = __uint_as_float(w.x);
    f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z);
    f[3] = __uint_as_float(w.w);
  } else {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 t = __bfloat1622float2(h[e]);
      f[2 * e] = t.x;
      f[2 * e + 1] = t.y;
    }
  }
}
template <class E>
__device__ __forceinline__ uint4 pack(const float (&f)[16 / sizeof(E)]) {
  uint4 w;
  if constexpr (sizeof(E) == 4) {
    w = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  } else {
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
  }
  return w;
}

// ------------------------------------------------------------------- append ----
// A block takes rows in turn, one thread per 16-byte chunk of a head: a thread
// keeps its chunk's columns for all the heads it takes, so the sines and
// cosines of its pairs are computed once a row.  The angle of pair j at
// position pos is the fraction of a turn turn[j] * pos / 2^64, an exact product
// that wraps by whole turns by itself; its upper 32 bits go to fp32 (2^-25 of
// half a turn).  Rows stored in bf16 take the sine and cosine of the
// special-function unit (2^-21 of 1 on this range; the output's rounding is
// 2^-9), fp32 the accurate ones, and so do e4m3 caches: an error that moves a
// value over the middle of two codes costs a whole step, and the fast ones moved
// 82 of 10^7 keys, these 13 (exact angles in fp32 arithmetic: 11).
// Bound by the bytes of Z, Q and the new slots: a row's heads are loaded while
// its angles are computed, and its position and page are read a row ahead.
// 16384 rows of 32 and 8 heads of 128 take 66 us in bf16 (6.1 TB/s; the accurate
// sines would make it 70), 74 with an e4m3 cache (70 with the fast ones), whose
// conversions and sines cost registers (6 blocks an SM, not 8), 126 in fp32.  One
// block a row took 71; 6 heads in flight and 7 blocks an SM 85, 2 heads 71,
// blocks of 256 threads 86 and more; prefetching the next row to L2 82.  A
// single row takes 2.6 us, a launch's own.
constexpr int kAppendThreads = 128, kAppendHeads = 3;  // heads of a thread in flight

// What a row needs to know: its position (< 0: left out) and page.
struct AppendRow {
  int pos, page;
};
__device__ __forceinline__ AppendRow append_row(const AppendParams& p, uint32_t i, uint32_t M) {
  AppendRow r = {-1, -1};
  if (i >= M) return r;
  r.pos = __ldg(p.positions + i);
  const int seq = p.row_seq ? __ldg(p.row_seq + i) : static_cast<int>(i);
  if (r.pos < 0) return r;
  const int at = p.page_shift >= 0 ? r.pos >> p.page_shift : r.pos / p.page_size;
  if (seq >= 0 && seq < p.num_seqs && at < p.max_pages)
    r.page = __ldg(p.page_table + static_cast<int64_t>(seq) * p.max_pages + at);
  return r;
}

template <class E, class C>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int VEC = 16 / sizeof(E);
  const int chunks = p.head_dim / VEC, heads = p.q_heads + 2 * p.kv_heads, lanes = p.lanes;
  const int c = threadIdx.x % chunks, group = threadIdx.x / chunks, r0 = group / lanes;
  const int turn_of = blockIdx.x / p.parts, h0 = group - r0 * lanes + (blockIdx.x - turn_of * p.parts) * (lanes * kAppendHeads);
  uint64_t turn[VEC / 2];
  if (p.rotate) {
    // by its generic address: the threads' chunks differ, and the constant cache serves one address at a time
    const uint64_t* t = p.turn + c * (VEC / 2);
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) asm volatile("ld.u64 %0, [%1];" : "=l"(turn[e]) : "l"(t + e));
  }
  pdl_wait();
  pdl_launch_dependents();
  if (r0 >= p.rows) return;
  float inv_k = 0.0f, inv_v = 0.0f, sk = 1.0f, sv = 1.0f;
  bool fast = true;
  if constexpr (sizeof(C) == 1) {
    sk = *p.scale_k;
    sv = *p.scale_v;
    fast = e4m3_fast_scale(sk) && e4m3_fast_scale(sv);
    inv_k = __frcp_rn(sk);
    inv_v = __frcp_rn(sv);
  }
  const uint32_t M = static_cast<uint32_t>(p.M), first = turn_of * p.rows + r0, step = gridDim.x / p.parts * p.rows;  // below 2^31, as a step is
  AppendRow next = append_row(p, first, M);
  for (uint32_t i = first; i < M; i += step) {
    const AppendRow row = next;
    next = append_row(p, i + step, M);
    if (row.pos < 0) continue;
    if (row.page < 0 || row.page >= p.num_pages) {
      if (c == 0 && h0 == 0) atomicOr(&g_paged_status, kDevBadIndex);
      continue;
    }
    const int in_page = p.page_shift >= 0 ? row.pos & (p.page_size - 1) : row.pos % p.page_size;
    const uint4* z = reinterpret_cast<const uint4*>(static_cast<const E*>(p.Z) + static_cast<int64_t>(i) * heads * p.head_dim) + c;
    E* const q = static_cast<E*>(p.Q) + (p.Q ? static_cast<int64_t>(i) * p.q_heads * p.head_dim + c * VEC : 0);
    // elements of the caches before this row's slot of head 0
    const int64_t slot = (static_cast<int64_t>(row.page) * p.kv_heads * p.page_size + in_page) * p.head_dim + c * VEC;
    float s[VEC / 2], co[VEC / 2];
    for (int hb = h0; hb < heads; hb += lanes * kAppendHeads * p.parts) {
      uint4 w[kAppendHeads];
#pragma unroll
      for (int u = 0; u < kAppendHeads; ++u)
        if (hb + u * lanes < heads) w[u] = __ldcs(z + (hb + u * lanes) * chunks);
      if (p.rotate && hb == h0) {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
          const int t = static_cast<int>((turn[e] * static_cast<uint64_t>(row.pos)) >> 32);
          const float half_turns = static_cast<float>(t) * 0x1p-31f;
          if constexpr (sizeof(E) == 4 || sizeof(C) == 1)
            sincospif(half_turns, &s[e], &co[e]);
          else
            __sincosf(half_turns * 3.14159265358979f, &s[e], &co[e]);
        }
      }
#pragma unroll
      for (int u = 0; u < kAppendHeads; ++u) {
        const int h = hb + u * lanes;
        if (h >= heads) break;
        if (h < p.q_heads && p.Q == nullptr) continue;
        const int hv = h - p.q_heads - p.kv_heads;  // >= 0: a value head
        if (hv >= 0 && sizeof(C) == sizeof(E)) {    // values are only laid out
          *reinterpret_cast<uint4*>(static_cast<C*>(p.Vc) + slot + hv * p.page_size * static_cast<int64_t>(p.head_dim)) = w[u];
          continue;
        }
        float f[VEC];
        unpack<E>(w[u], f);
        if (p.rotate && hv < 0) {
#pragma unroll
          for (int e = 0; e < VEC / 2; ++e) {
            const float a = f[2 * e], b = f[2 * e + 1];
            f[2 * e] = a * co[e] - b * s[e];
            f[2 * e + 1] = a * s[e] + b * co[e];
          }
        }
        if (h < p.q_heads) {
          *reinterpret_cast<uint4*>(q + h * p.head_dim) = pack<E>(f);
          continue;
        }
        const int hk = hv >= 0 ? hv : h - p.q_heads;
        C* dst = static_cast<C*>(hv >= 0 ? p.Vc : p.Kc) + slot + hk * p.page_size * static_cast<int64_t>(p.head_dim);
        if constexpr (sizeof(C) == 1) {
          const float sc = hv >= 0 ? sv : sk, inv = hv >= 0 ? inv_v : inv_k;
          uint32_t o[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t lo = fast ? to_e4m3x2<true>(f[4 * j], f[4 * j + 1], sc, inv)
                                     : to_e4m3x2<false>(f[4 * j], f[4 * j + 1], sc, inv);
            const uint32_t hi = fast ? to_e4m3x2<true>(f[4 * j + 2], f[4 * j + 3], sc, inv)
                                     : to_e4m3x2<false>(f[4 * j + 2], f[4 * j + 3], sc, inv);
            o[j] = lo | (hi << 16);
          }
          *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
        } else {
          *reinterpret_cast<uint4*>(dst) = pack<C>(f);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- attention ----
// One new token per row: o = sum_t p_t v_t / sum_t p_t,
// p_t = 2^(s_t - m), with the running maximum m, the sum and o kept in fp32 and
// every key and value read once.
//
// What bounds it: a key of G query heads is 4 G D operations on 2 D e bytes, so
// for any G up to 16 the bytes of the cache decide.  Everything serves the loads:
//   - the work is cut into tiles of kAttnWarps * KT keys of one row and key/value
//     head, and each block of a grid that fills the GPU takes an equal run of
//     consecutive tiles, whatever the rows' lengths (the lengths are on the
//     device: every block computes the same partition from them);
//   - each warp has its own keys of a tile, its own ring of ST stages filled with
//     cp.async and its own running m, sum and o: no barrier in the loop.  Page
//     numbers are read a tile ahead of the loads that need them;
//   - a row and head whose tiles lie in one block is finished there; otherwise
//     each block leaves (m, sum, o) in the workspace and the block that comes
//     last joins them in the order of the keys, so the bits do not depend on
//     which one it was.  No block waits for another.
// The products run on mma.sync with keys (then columns of v) as the 16 rows of
// the instruction and query heads as its 8 columns: heads as the 16 rows did
// twice the work for 8 heads (443 us for 380, see below).  tcgen05's smallest
// tile has 64 rows, and its operands would have to be rearranged in shared
// memory page by page; at the full HBM rate mma.sync keeps the tensor pipe busy
// for 9% (bf16) and 28% (e4m3) of the time.  fp32 runs on the FMA pipe.
//
// Measured, of heads of 128 (share of a plain copy's 6.77 TB/s):
//   64 rows of 17 to 8192 keys, 32 query and 8 key heads, bf16    162 us   98%
//   128 rows of 4000 to 16000 keys, 64 and 8 heads, e4m3 cache    387 us  100%
//   one row of 131071 keys, 32 and 8 heads, bf16                   88 us   90%
//   one row of 1900 keys, 32 and 8 heads, bf16                    10.0 us
// The last is latency: 1.3 us until a block knows its run, 1.5 until its first
// page and keys are there, about 4 for the join.  Other choices, in the first
// two and the last of these (when they took 160, 380 and 10.0): 2 blocks an SM 171 / 401, 4 (that spill) 232 / 560;
// stages of 16 KB (bf16, KT = 32) 183, of 4 KB (e4m3, KT = 16) 475; 1, 2 or 3
// tiles a block at least 11.2 / 10.0 / 10.6; the next tile's loads before the
// wait for this one's 169 / 406; every part joined at once 93 in the third.
constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kMaxWorkers = 512;  // blocks of a grid: bounds the workspace
constexpr int kMinTiles = 2;      // tiles a block takes at least
constexpr int kFlatJoin = 24;     // parts of an item joined at once (see the kernel's end)
constexpr int kJoinBatch = 16;    // parts fetched at a time
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// What a block does with a key/value head's query heads at a time:
//   kFew   up to 4 (fp32: 1);  kSome  up to 8 (fp32: 4);  kMany  up to 16 (fp32: 8)
// Each takes what the next larger could take as well, for its registers and its
// products (us, for 32 rows of 4096 keys of 8 heads of 128):
//   4 query heads each   bf16 kFew 86.0, kSome 86.1, kMany 92.7;  e4m3 50.4, 50.8, 62.6
//   8                    bf16 kSome 87.0, kMany 94.2;  e4m3 52.5, 63.9
//   16                   bf16 kMany 96.8;  e4m3 68.7
//   fp32, 1 and 4        kFew 157, as kSome 161;  kSome 163, kMany 207
// More than 16 heads take the keys once for each 16: 32 heads of one key head
// run at 44% of the copy rate, 33% with an e4m3 cache.
enum Heads { kFew, kSome, kMany };

template <class T, class C, int DP_, Heads HEADS_>
struct AttnShape {
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr bool E4M3 = sizeof(C) == 1;
  static constexpr Heads HEADS = HEADS_;
  static constexpr int DP = DP_;                              // head_dim rounded up
  static constexpr int NH = HEADS == kMany ? 2 : 1;           // mma: tiles of 8 heads
  static constexpr int RG = F32 ? (HEADS == kFew ? 1 : HEADS == kSome ? 4 : 8) : 8 * NH;   // rows of state
  static constexpr int MAXG = F32 ? RG : HEADS == kFew ? 4 : RG;      // query heads of a block
  static constexpr int PITCH = DP * static_cast<int>(sizeof(C));      // bytes of a staged row
  static constexpr int KT0 = 4096 / PITCH;
  // keys of a warp's tile: 8 KB a stage where the products allow it (16 to 32 keys)
  static constexpr int KT = F32 ? 1024 / DP : KT0 > 32 || (E4M3 && NH == 2) ? 32 : KT0 < 16 ? 16 : KT0;
  static constexpr int CT = KT * kAttnWarps;
  static constexpr int STAGE = 2 * KT * PITCH;
  // stages of a ring: one more tile in flight made 162 us 169 (64 ragged rows); where one block fills an SM's shared
  // memory, 179 became 174 (32 rows of 4096 keys of 8 heads of 256)
  static constexpr int ST = DP == 256 && sizeof(C) == 2 ? 3 : 2;
  static constexpr int CPR = PITCH / 16;  // 16-byte chunks of a row
  static constexpr int RING = kAttnWarps * ST * STAGE;
  // the widest shape keeps its queries in shared memory, 64 registers a thread that o needs (329 us became 190)
  static constexpr bool Q_SMEM = !F32 && NH == 2 && DP == 256;
  static constexpr int QBYTES = F32 ? RG * DP * 4 + kAttnWarps * KT * RG * 4 : Q_SMEM ? DP / 16 * 32 * 16 : 0;
  static constexpr int SMEM = RING + QBYTES;
  static_assert(RG * DP * 4 <= STAGE, "a warp's part of o fits a stage of its ring");
  static constexpr int REGS = F32 ? 128 : NH * (DP / 4 + (Q_SMEM ? 0 : DP / 8)) + 80;  // about what a thread needs
  static constexpr int BY_SMEM = 233472 / (SMEM + 1024 + 1024), BY_REGS = 65536 / (kAttnThreads * REGS);
  static constexpr int CTAS0 = BY_SMEM < BY_REGS ? BY_SMEM : BY_REGS;
  static constexpr int MOST = NH == 2 && DP > 64 ? 2 : 3;
  static constexpr int CTAS = CTAS0 < 1 ? 1 : CTAS0 > MOST ? MOST : CTAS0;  // blocks on an SM
};

// Chunk c of staged row `row`: 16-byte chunks are permuted within 128 bytes so
// that eight rows' equal chunks lie in different banks.
template <int PITCH>
__device__ __forceinline__ int staged(int row, int c) {
  constexpr int GROUP = PITCH >= 128 ? 8 : PITCH / 16, STEP = PITCH >= 128 ? 1 : 128 / PITCH;
  return row * PITCH + ((c ^ ((row / STEP) & (GROUP - 1))) << 4);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t a) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
// c [16 x 8] += a [16 x 16] b [16 x 8], f16 or bf16 operands, fp32 sums.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two e4m3 codes (the low 16 bits) as f16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t codes) {
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(d) : "r"(codes));
  return d;
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2_hi(uint32_t codes) {  // ... of the high 16 bits
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(d) : "r"(codes));
  return d;
}
// An 8 x 8 matrix of 16-bit values, transposed across the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  if constexpr (F16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ unsigned atom_add_acq_rel_gpu(unsigned* p, unsigned v) {
  unsigned old;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

// What the kernel knows of a row: keys that count, and its sequence.
struct RowInfo {
  int len, seq;
};
__device__ __forceinline__ RowInfo row_info(const AttnParams& p, int row, bool& bad) {
  RowInfo r;
  r.len = max(p.lengths[row], 0);
  r.seq = p.row_seq ? p.row_seq[row] : row;
  const int64_t room = static_cast<int64_t>(p.max_pages) * p.page_size;
  if (r.len > room) {
    r.len = static_cast<int>(room);
    bad = true;
  }
  if (r.len > 0 && (r.seq < 0 || r.seq >= p.num_seqs)) {
    r.len = 0;
    bad = true;
  }
  return r;
}

// Tiles of a row: one at least, so that a row without keys is written too.
__device__ __forceinline__ int tiles_of(int len, int CT) { return len > 0 ? (len - 1) / CT + 1 : 1; }

// A tile in a block's run: tile t of nt of row `row` and head unit h (a
// key/value head and a group of its query heads).
struct Cursor {
  int row, h, t, nt, len, seq;
  __device__ __forceinline__ void enter(const AttnParams& p, int CT) {
    bool bad = false;
    const RowInfo r = row_info(p, row, bad);
    len = r.len;
    seq = r.seq;
    nt = tiles_of(len, CT);
  }
  __device__ __forceinline__ void next(const AttnParams& p, int units, int CT) {
    if (++t < nt) return;
    t = 0;
    if (++h < units) return;
    h = 0;
    if (++row < p.M) enter(p, CT);
  }
};

// a / b; the 64-bit division is a long subroutine, so numbers that fit take the 32-bit one.
__device__ __forceinline__ int64_t div_small(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// T tiles dealt to the blocks that take part: runs of `per` tiles, the first `more` runs one longer.
struct Runs {
  int64_t T, per;
  int workers, more;
  __device__ __forceinline__ void set(int64_t tiles, int grid) {
    T = tiles;
    workers = static_cast<int>(min(static_cast<int64_t>(grid), max(T / kMinTiles, static_cast<int64_t>(1))));
    per = div_small(T, workers);
    more = static_cast<int>(T - per * workers);
  }
  __device__ __forceinline__ int64_t first(int c) const { return per * c + min(c, more); }
  __device__ __forceinline__ int owner(int64_t i) const {  // the block of tile i
    const int64_t longer = (per + 1) * more;
    return static_cast<int>(i < longer ? div_small(i, per + 1) : more + div_small(i - longer, per));
  }
};

// Four columns of o of a part of an item, with its row's m and l.
struct Part {
  float m, l;
  float4 v;
};

template <class E, class C, int DP, Heads HEADS>
__global__ void __launch_bounds__(kAttnThreads, AttnShape<E, C, DP, HEADS>::CTAS)
    attention_kernel(const __grid_constant__ AttnParams p) {
  using S = AttnShape<E, C, DP, HEADS>;
  constexpr int KT = S::KT, CT = S::CT, ST = S::ST, PITCH = S::PITCH, CPR = S::CPR, RG = S::RG, NH = S::NH;
  constexpr bool F16 = S::E4M3;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_scan[kAttnWarps];
  __shared__ int s_start[5], s_last;
  __shared__ uint32_t s_mask[kAttnWarps][ST];
  __shared__ float2 s_ml[kAttnWarps][RG];  // (m, l) of the warps' parts of an item
  // the blocks' parts of an item as they are joined: (m, l), weight and weighted l, running m, next m and old weight
  __shared__ float2 s_joined[kJoinBatch][RG], s_weight[kJoinBatch][RG], s_next[RG];
  __shared__ float s_run[RG];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int G = p.q_heads / p.kv_heads, groups = (G + S::MAXG - 1) / S::MAXG, gsize = (G + groups - 1) / groups;
  const int units = p.kv_heads * groups;
  const int chunks = p.head_dim * static_cast<int>(sizeof(C)) / 16;
  const uint32_t ring = smem_u32(smem) + w * ST * S::STAGE;

  // columns [head_dim, DP) of the ring are never loaded: zero once
  if (chunks < CPR)
    for (int i = tid; i < S::RING / 16; i += kAttnThreads) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
  pdl_wait();
  pdl_launch_dependents();

  // ---- this block's run of tiles: [i0, i1) of T, in the order (row, unit, tile)
  Runs run;
  int64_t i0, i1;
  {
    const int per = (p.M + kAttnThreads - 1) / kAttnThreads;
    const int r0 = min(tid * per, p.M), r1 = min(r0 + per, p.M);
    int64_t sum = 0;
    bool bad = false;
    RowInfo info = {0, 0};
#pragma unroll 4
    for (int r = r0; r < r1; ++r) {
      info = row_info(p, r, bad);
      sum += tiles_of(info.len, CT);
    }
    if (bad && blockIdx.x == 0) atomicOr(&g_paged_status, kDevBadIndex);
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) s_scan[w] = incl;
    __syncthreads();
    int64_t before = 0, total = 0;
#pragma unroll
    for (int x = 0; x < kAttnWarps; ++x) {
      if (x < w) before += s_scan[x];
      total += s_scan[x];
    }
    run.set(total * units, gridDim.x);
    if (static_cast<int>(blockIdx.x) >= run.workers) return;
    i0 = run.first(blockIdx.x);
    i1 = run.first(blockIdx.x + 1);
    int64_t at = (before + incl - sum) * units;  // first tile of this thread's rows
    if (i0 >= at && i0 < at + sum * units) {
      for (int r = r0; r < r1; ++r) {
        if (per > 1) info = row_info(p, r, bad);  // else it is still here
        const int nt = tiles_of(info.len, CT);
        if (i0 < at + static_cast<int64_t>(nt) * units) {
          s_start[0] = r;
          s_start[3] = info.len;
          s_start[4] = info.seq;
          s_start[1] = static_cast<int>(div_small(i0 - at, nt));
          s_start[2] = static_cast<int>(i0 - at - static_cast<int64_t>(s_start[1]) * nt);
          break;
        }
        at += static_cast<int64_t>(nt) * units;
      }
    }
    __syncthreads();
  }
  const int64_t n = i1 - i0;

  // ---- the loads: page numbers one tile ahead, rows ST - 1 tiles ahead
  Cursor in;
  in.row = s_start[0];
  in.h = s_start[1];
  in.t = s_start[2];
  in.len = s_start[3];
  in.seq = s_start[4];
  in.nt = tiles_of(in.len, CT);
  Cursor at = in;
  int pg, slot;
  bool bad_page = false;
  auto look_up = [&]() {
    const int key = in.t * CT + w * KT + lane;
    pg = -1;
    slot = -1;  // no such key
    if (lane < KT && key < in.len) {
      const int q = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
      slot = key - q * p.page_size;
      pg = __ldg(p.page_table + static_cast<int64_t>(in.seq) * p.max_pages + q);
    }
  };
  const int row_bytes = p.head_dim * static_cast<int>(sizeof(C));
  constexpr int LPR = (CPR & -CPR) < 32 ? CPR & -CPR : 32;  // lanes of a row: a power of two
  const char* const k_src = static_cast<const char*>(p.Kc) + (lane % LPR) * 16;
  const char* const v_src = static_cast<const char*>(p.Vc) + (lane % LPR) * 16;
  auto issue = [&](int stage) {
    if (in.t == 0 && w == 0) {
      // a new item: its queries start their way to L2 (the products need them as soon as these keys are there)
      const int g0 = (in.h % groups) * gsize, bytes = min(gsize, G - g0) * p.head_dim * static_cast<int>(sizeof(E));
      const char* src = reinterpret_cast<const char*>(static_cast<const E*>(p.Q) + in.row * p.ldq +
                                                      static_cast<int64_t>(in.h / groups * G + g0) * p.head_dim);
      for (int b = lane * 128; b < bytes; b += 32 * 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + b));
    }
    const bool ok = pg >= 0 && pg < p.num_pages && slot >= 0;
    bad_page |= !ok && slot >= 0;
    // row of the caches (fewer than 2^31); -1: filled with zeros
    const int mine = ok ? (pg * p.kv_heads + in.h / groups) * p.page_size + slot : -1;
    const uint32_t mask = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) s_mask[w][stage] = mask;
    const uint32_t dst = ring + stage * S::STAGE;
#pragma unroll
    for (int r0 = 0; r0 < KT; r0 += 32 / LPR) {
      const int row = r0 + lane / LPR;
      const int from = __shfl_sync(0xffffffffu, mine, row);
      const int64_t off = static_cast<int64_t>(max(from, 0)) * row_bytes;
#pragma unroll
      for (int c0 = 0; c0 < CPR; c0 += LPR) {
        const int c = c0 + lane % LPR;
        if (c < chunks) {
          const int to = staged<PITCH>(row, c);
          cp_async16(dst + to, k_src + off + c0 * 16, from >= 0);
          cp_async16(dst + KT * PITCH + to, v_src + off + c0 * 16, from >= 0);
        }
      }
    }
  };
  look_up();
#pragma unroll
  for (int s = 0; s < ST - 1; ++s) {
    if (s < n) {
      issue(s);
      in.next(p, units, CT);
      if (s + 1 < n) look_up();
    }
    cp_async_commit();
  }

  // ---- per-warp state.  mma: the keys (then the columns) are the 16 rows of the
  // instruction and the heads its 8 columns, so a lane holds heads 2 (lane % 4)
  // and the next one of each tile of 8; fp32: all heads, some columns.
  constexpr int OW = S::F32 ? RG * DP / 32 : NH * DP / 4;
  constexpr int NR = S::F32 ? RG : 2 * NH;
  constexpr int KS = DP / 16;
  // kFew: columns 4 to 7 repeat the heads and take what the weights lose when they are rounded to 16 bits; kSome and
  // kMany: a second product does.
  // f16 weights (e4m3 caches) are taken 2^15 times as large: 2^-29 of the largest is still a normal number, and what
  // vanishes below 2^-40 of it is no 2^-20 of a row's sum in 10^6 keys.
  constexpr float UP = F16 ? 15.0f : 0.0f;
  constexpr bool LOW_COLS = !S::F32 && HEADS == kFew, LOW_MMA = !S::F32 && HEADS != kFew;
  float o[OW], m[NR], l[NR];
  uint32_t q[S::F32 ? 1 : NH * KS * 2] = {};
  float s2[NR];  // scale log2 e (and the scales of an e4m3 cache's keys and of q)
  float* s_q = reinterpret_cast<float*>(smem + S::RING);  // fp32: [RG][DP]
  float* s_p = s_q + RG * DP + w * KT * RG;                         // fp32: [KT][RG] of this warp
  uint4* s_frag = reinterpret_cast<uint4*>(s_q);                    // Q_SMEM: [KS][32]
  const float sk = S::E4M3 ? p.scale * *p.scale_k : p.scale;
  const float sv = S::E4M3 ? *p.scale_v : 1.0f;

  auto begin_item = [&]() {
    const int hk = at.h / groups, g0 = (at.h % groups) * gsize, ng = min(gsize, G - g0);
    const E* src = static_cast<const E*>(p.Q) + at.row * p.ldq + static_cast<int64_t>(hk * G + g0) * p.head_dim;
#pragma unroll
    for (int i = 0; i < OW; ++i) o[i] = 0.0f;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.0f;
      s2[r] = sk * kLog2e;
    }
    if constexpr (S::F32) {
      __syncthreads();
      for (int i = tid; i < RG * DP; i += kAttnThreads) {
        const int g = i / DP, d = i % DP;
        s_q[i] = g < ng && d < p.head_dim ? src[g * p.head_dim + d] : 0.0f;
      }
      __syncthreads();
    } else {
      const int c4 = lane & 3;
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) {
        const int g = LOW_COLS ? (lane >> 2) & 3 : (lane >> 2) + 8 * nh;
        const uint32_t* row = reinterpret_cast<const uint32_t*>(src + static_cast<int64_t>(g) * p.head_dim);
        float big = 0.0f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            // e4m3: the 16 columns of a step in the order of the staged bytes (see the products)
            const int d = ks * 16 + (S::E4M3 ? 4 * c4 + 2 * x : 2 * c4 + 8 * x);
            const uint32_t v = g < ng && d < p.head_dim ? __ldg(row + d / 2) : 0u;
            q[(nh * KS + ks) * 2 + x] = v;
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
            big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        if constexpr (S::E4M3) {
          // q in f16 beside the keys' exact f16 values: each head's q is scaled by a power of two to a largest
          // value in [2^14, 2^15), so what f16 cannot hold lies 2^-28 and more below it
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
          const int ex = big > 0.0f ? min(max(14 - (static_cast<int>(__float_as_uint(big) >> 23) - 127), -112), 126) : 0;
          const float up = __uint_as_float(static_cast<uint32_t>(ex + 127) << 23);
#pragma unroll
          for (int i = 0; i < 2 * KS; ++i) {
            uint32_t& v = q[nh * KS * 2 + i];
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
            v = pack2<true>(f.x * up, f.y * up);
          }
          const float down = sk * kLog2e * __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
#pragma unroll
          for (int x = 0; x < 2; ++x) s2[2 * nh + x] = __shfl_sync(0xffffffffu, down, (2 * c4 + x) * 4);
        }
      }
      if constexpr (S::Q_SMEM) {
        // every warp has the same fragments: one writes them, [step][lane] of both heads' tiles
        __syncthreads();
        if (w == 0) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
            s_frag[ks * 32 + lane] = make_uint4(q[ks * 2], q[ks * 2 + 1], q[(KS + ks) * 2], q[(KS + ks) * 2 + 1]);
        }
        __syncthreads();
      }
    }
  };

  // One tile of the products on the tensor cores.
  auto tile_mma = [&](int stage, uint32_t mask) {
    constexpr int MT = KT < 16 ? 1 : KT / 16;
    const uint32_t kb = ring + stage * S::STAGE, vb = kb + KT * PITCH;
    // s^T = k q^T: 16 keys by 8 heads a tile
    auto query = [&](int ks, uint32_t (&b)[2 * NH]) {
      if constexpr (S::Q_SMEM) {
        const uint4 v = s_frag[ks * 32 + lane];
        b[0] = v.x;
        b[1] = v.y;
        b[2 * NH - 2] = v.z;
        b[2 * NH - 1] = v.w;
      } else {
#pragma unroll
        for (int i = 0; i < 2 * NH; ++i) b[i] = q[((i >> 1) * KS + ks) * 2 + (i & 1)];
      }
    };
    float s[NH][MT][4];
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[nh][t][x] = 0.0f;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int row = t * 16 + (lane & 15);
      if constexpr (!S::E4M3) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t a[4], b[2 * NH];
          ldmatrix4<false>(a, kb + staged<PITCH>(row, ks * 2 + (lane >> 4)));
          query(ks, b);
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) mma16816<F16>(s[nh][t], a[0], a[1], a[2], a[3], b[2 * nh], b[2 * nh + 1]);
        }
      } else {
        // a lane's 4 bytes are 4 consecutive columns: the pairs (0, 1) and (2, 3) are taken as the instruction's
        // columns 2 c4 and 2 c4 + 8, for q and k alike
#pragma unroll
        for (int ks = 0; ks < KS; ks += 2) {
          uint32_t a[4];
          ldmatrix4<false>(a, kb + staged<PITCH>(row, ks + (lane >> 4)));
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t a0 = e4m3x2_f16x2(a[2 * u]), a1 = e4m3x2_f16x2(a[2 * u + 1]);
            const uint32_t a2 = e4m3x2_f16x2_hi(a[2 * u]), a3 = e4m3x2_f16x2_hi(a[2 * u + 1]);
            uint32_t b[2 * NH];
            query(ks + u, b);
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) mma16816<F16>(s[nh][t], a0, a1, a2, a3, b[2 * nh], b[2 * nh + 1]);
          }
        }
      }
    }
    // weights 2^(s2 s - m).  The product is rounded before m is taken off it, so that the largest weight is 2^0: relative to
    // a rounded m, one multiply-add would make it 2^(m's rounding), which scores of 10^7 and more carry out of range
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int x = 0; x < 4; x += 2) {
          const float2 v = fmul2(make_float2(s[nh][t][x], s[nh][t][x + 1]), make_float2(s2[2 * nh], s2[2 * nh + 1]));
          s[nh][t][x] = v.x;
          s[nh][t][x + 1] = v.y;
        }
    if (mask != (KT == 32 ? 0xffffffffu : (1u << (KT & 31)) - 1u)) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
          if (!((mask >> (t * 16 + hf * 8 + (lane >> 2))) & 1u))
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) s[nh][t][2 * hf] = s[nh][t][2 * hf + 1] = -INFINITY;
    }
    float big[NR];
    bool more = false;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      big[r] = -INFINITY;
#pragma unroll
      for (int t = 0; t < MT; ++t) big[r] = fmaxf(big[r], fmaxf(s[r >> 1][t][r & 1], s[r >> 1][t][2 + (r & 1)]));
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) big[r] = fmaxf(big[r], __shfl_xor_sync(0xffffffffu, big[r], x));
      more |= big[r] > m[r];
    }
    if (__any_sync(0xffffffffu, more)) {
      float c[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float mn = fmaxf(m[r], big[r]);
        c[r] = mn == -INFINITY ? 1.0f : ex2_approx(m[r] - mn);
        m[r] = mn;
        l[r] *= c[r];
      }
#pragma unroll
      for (int i = 0; i < OW; ++i) o[i] *= c[i / (DP / 4) * 2 + (i & 1)];
    }
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
      const float2 off = make_float2(m[2 * nh] == -INFINITY ? 0.0f : -m[2 * nh], m[2 * nh + 1] == -INFINITY ? 0.0f : -m[2 * nh + 1]);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int x = 0; x < 4; x += 2) {
          float2 v = fadd2(make_float2(s[nh][t][x], s[nh][t][x + 1]), off);
          if constexpr (F16) v = fadd2(v, make_float2(UP, UP));
          v = make_float2(ex2_approx(v.x), ex2_approx(v.y));
          s[nh][t][x] = v.x;
          s[nh][t][x + 1] = v.y;
          l[2 * nh] += v.x;
          l[2 * nh + 1] += v.y;
        }
    }
    // o^T += v^T p^T: 16 columns by 8 heads a tile, 16 keys at a time
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      uint32_t b[NH][2], low[NH][2];
#pragma unroll
      for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float p0 = s[nh][t][2 * hf], p1 = s[nh][t][2 * hf + 1];
          uint32_t hi = pack2<F16>(p0, p1);
          if constexpr (LOW_COLS || LOW_MMA) {
            const float2 f = F16 ? __half22float2(*reinterpret_cast<const __half2*>(&hi))
                                 : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&hi));
            const uint32_t lo = pack2<F16>(p0 - f.x, p1 - f.y);
            if constexpr (LOW_COLS)
              hi = lane & 2 ? lo : hi;
            else
              low[nh][hf] = transpose8x8(lo);
          }
          b[nh][hf] = transpose8x8(hi);
        }
      const int row = t * 16 + (lane & 7) + ((lane >> 4) << 3);
      if constexpr (!S::E4M3) {
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
          uint32_t a[4];
          ldmatrix4<true>(a, vb + staged<PITCH>(row, d * 2 + ((lane >> 3) & 1)));
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) {
            float(&acc)[4] = *reinterpret_cast<float(*)[4]>(o + (nh * (DP / 16) + d) * 4);
            mma16816<F16>(acc, a[0], a[1], a[2], a[3], b[nh][0], b[nh][1]);
            if constexpr (LOW_MMA) mma16816<F16>(acc, a[0], a[1], a[2], a[3], low[nh][0], low[nh][1]);
          }
        }
      } else {
        // a transposed pair of bytes is two columns of one key: the even columns of 16 are the upper rows of a
        // tile, the odd ones the lower
#pragma unroll
        for (int d = 0; d < DP / 16; d += 2) {
          uint32_t a[4];
          ldmatrix4<true>(a, vb + staged<PITCH>(row, d + ((lane >> 3) & 1)));
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t x0 = e4m3x2_f16x2(a[u]), x1 = e4m3x2_f16x2_hi(a[u]);
            const uint32_t y0 = e4m3x2_f16x2(a[u + 2]), y1 = e4m3x2_f16x2_hi(a[u + 2]);
            const uint32_t a0 = __byte_perm(x0, x1, 0x5410), a1 = __byte_perm(x0, x1, 0x7632);
            const uint32_t a2 = __byte_perm(y0, y1, 0x5410), a3 = __byte_perm(y0, y1, 0x7632);
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) {
              float(&acc)[4] = *reinterpret_cast<float(*)[4]>(o + (nh * (DP / 16) + d + u) * 4);
              mma16816<F16>(acc, a0, a1, a2, a3, b[nh][0], b[nh][1]);
              if constexpr (LOW_MMA) mma16816<F16>(acc, a0, a1, a2, a3, low[nh][0], low[nh][1]);
            }
          }
        }
      }
    }
  };

  // One tile in fp32: 32 / KT lanes share a key's columns, then each lane takes DP / 32 columns of o.
  auto tile_f32 = [&](int stage, uint32_t mask) {
    constexpr int PARTS = 32 / (KT < 32 ? KT : 32), NC = DP / 32;
    const uint8_t* kb = smem + w * ST * S::STAGE + stage * S::STAGE;
    const uint8_t* vb = kb + KT * PITCH;
    const int key = lane % KT, part = lane / KT;
    float s[RG];
    float2 s2v[RG];
#pragma unroll
    for (int g = 0; g < RG; ++g) s2v[g] = make_float2(0.0f, 0.0f);
#pragma unroll 4
    for (int c = part; c < chunks; c += PARTS) {
      const float4 k = *reinterpret_cast<const float4*>(kb + staged<PITCH>(key, c));
#pragma unroll
      for (int g = 0; g < RG; ++g) {
        const float4 x = *reinterpret_cast<const float4*>(s_q + g * DP + 4 * c);
        s2v[g] = ffma2(make_float2(k.x, k.y), make_float2(x.x, x.y), s2v[g]);
        s2v[g] = ffma2(make_float2(k.z, k.w), make_float2(x.z, x.w), s2v[g]);
      }
    }
    const bool there = (mask >> key) & 1u;
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      s[g] = s2v[g].x + s2v[g].y;
#pragma unroll
      for (int x = KT; x < 32; x <<= 1) s[g] += __shfl_xor_sync(0xffffffffu, s[g], x);
      s[g] = there ? s[g] * s2[g] : -INFINITY;
      float big = s[g];
#pragma unroll
      for (int x = 1; x < KT; x <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, x));
      if (big > m[g]) {  // the same in every lane
        const float c = ex2_approx(m[g] - big);
        m[g] = big;
        l[g] *= c;
#pragma unroll
        for (int i = 0; i < NC; ++i) o[g * NC + i] *= c;
      }
      s[g] = ex2_approx(s[g] - (m[g] == -INFINITY ? 0.0f : m[g]));
      if (part == 0) {
        l[g] += s[g];
        s_p[key * RG + g] = s[g];
      }
    }
    __syncwarp();
#pragma unroll 4
    for (int t = 0; t < KT; ++t) {
      float v[NC];
      if constexpr (NC == 2) {
        const float2 x = *reinterpret_cast<const float2*>(vb + staged<PITCH>(t, lane / 2) + (lane & 1) * 8);
        v[0] = x.x;
        v[1] = x.y;
      } else {
#pragma unroll
        for (int i = 0; i < NC / 4; ++i) {
          const float4 x = *reinterpret_cast<const float4*>(vb + staged<PITCH>(t, lane + 32 * i));
          v[4 * i] = x.x;
          v[4 * i + 1] = x.y;
          v[4 * i + 2] = x.z;
          v[4 * i + 3] = x.w;
        }
      }
#pragma unroll
      for (int g = 0; g < RG; ++g) {
        const float pr = s_p[t * RG + g];
#pragma unroll
        for (int i = 0; i < NC; i += 2) {
          const float2 r = ffma2(make_float2(pr, pr), make_float2(v[i], v[i + 1]),
                                 make_float2(o[g * NC + i], o[g * NC + i + 1]));
          o[g * NC + i] = r.x;
          o[g * NC + i + 1] = r.y;
        }
      }
    }
    __syncwarp();
  };

  // o of a warp's part of an item lies in the stage of its ring that was just used up: element (row, d) at
  // [row][d ^ 8 (row / 2 mod 4)], so that the four lanes of two rows each write to different banks.
  auto part_at = [&](int warp, int st, int row, int d) {
    return reinterpret_cast<float*>(smem + (warp * ST + st) * S::STAGE) + row * DP + (d ^ ((row & 6) << 2));
  };
  auto put = [&](int st) {
    if constexpr (S::F32) {
      constexpr int NC = DP / 32;
#pragma unroll
      for (int g = 0; g < RG; ++g) {
        if (lane == 0) s_ml[w][g] = make_float2(m[g], l[g]);
        if constexpr (NC == 2) {
          *reinterpret_cast<float2*>(part_at(w, st, g, 2 * lane)) = make_float2(o[g * 2], o[g * 2 + 1]);
        } else {
#pragma unroll
          for (int i = 0; i < NC; i += 4)
            *reinterpret_cast<float4*>(part_at(w, st, g, 4 * lane + 32 * i)) =
                make_float4(o[g * NC + i], o[g * NC + i + 1], o[g * NC + i + 2], o[g * NC + i + 3]);
        }
      }
    } else if (!LOW_COLS || (lane & 2) == 0) {
#pragma unroll
      for (int r = 0; r < NR; ++r)
        if (lane < 4) s_ml[w][(r >> 1) * 8 + 2 * lane + (r & 1)] = make_float2(m[r], l[r]);
#pragma unroll
      for (int i = 0; i < OW; ++i) {
        const int nh = i / (DP / 4), d = i % (DP / 4) / 4 * 16, hf = (i >> 1) & 1;
        *part_at(w, st, nh * 8 + 2 * (lane & 3) + (i & 1), d + (S::E4M3 ? 2 * (lane >> 2) + hf : 8 * hf + (lane >> 2))) =
            o[i];
      }
    }
  };

  // Counters [2][kMaxWorkers], then per block two parts of o [gsize][head_dim] and (m, l) [gsize], in 16-byte units
  unsigned* counters = static_cast<unsigned*>(p.workspace);
  const int part_floats = gsize * p.head_dim + ((gsize + 1) & ~1) * 2;
  float* parts = reinterpret_cast<float*>(counters + 2 * kMaxWorkers);

  auto write_row = [&](int r, int d, float4 v, float mm, float ll) {
    const int hk = at.h / groups, g0 = (at.h % groups) * gsize;
    const int64_t head = static_cast<int64_t>(at.row) * p.q_heads + hk * G + g0 + r;
    const float inv = ll == 0.0f ? 0.0f : sv / ll;
    v.x = ll == 0.0f ? 0.0f : v.x * inv;
    v.y = ll == 0.0f ? 0.0f : v.y * inv;
    v.z = ll == 0.0f ? 0.0f : v.z * inv;
    v.w = ll == 0.0f ? 0.0f : v.w * inv;
    E* dst = static_cast<E*>(p.O) + head * p.head_dim + d;
    if constexpr (S::F32) {
      *reinterpret_cast<float4*>(dst) = v;
    } else {
      uint2 u = make_uint2(pack2<false>(v.x, v.y), pack2<false>(v.z, v.w));
      *reinterpret_cast<uint2*>(dst) = u;
    }
    if (p.lse && d == 0) p.lse[head] = ll == 0.0f ? -INFINITY : (mm - UP + log2f(ll)) * kLn2;
  };

  // The warps' parts of the item at `at` joined, and written out or left for the last block.  first_tile, last_tile: of
  // the whole item, among all T; st: the stage that was just used up.
  auto end_item = [&](int64_t first_tile, int64_t last_tile, int st) {
    if constexpr (!S::F32) {
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
      if constexpr (LOW_COLS) {
#pragma unroll
        for (int i = 0; i < OW; ++i) o[i] += __shfl_xor_sync(0xffffffffu, o[i], 2);
      }
    } else {
#pragma unroll
      for (int g = 0; g < RG; ++g)
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) l[g] += __shfl_xor_sync(0xffffffffu, l[g], x);
    }
    const int ng = min(gsize, G - (at.h % groups) * gsize), vecs = p.head_dim / 4;
    __syncwarp();  // every lane has read this stage
    put(st);
    __syncthreads();
    auto both = [&](int r, int d, float& mm, float& ll) {
      float2 ml[kAttnWarps];
      mm = -INFINITY;
#pragma unroll
      for (int x = 0; x < kAttnWarps; ++x) {
        ml[x] = s_ml[x][r];
        mm = fmaxf(mm, ml[x].x);
      }
      const float base = mm == -INFINITY ? 0.0f : mm;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      ll = 0.0f;
#pragma unroll
      for (int x = 0; x < kAttnWarps; ++x) {
        const float c = ex2_approx(ml[x].x - base);
        const float4 a = *reinterpret_cast<const float4*>(part_at(x, st, r, d));
        ll += ml[x].y * c;
        v = make_float4(v.x + a.x * c, v.y + a.y * c, v.z + a.z * c, v.w + a.w * c);
      }
      return v;
    };
    auto row_of = [&](int i) { return p.head_dim == DP ? i / (DP / 4) : i / vecs; };
    const bool whole = first_tile >= i0 && last_tile < i1;
    if (whole) {
      for (int i = tid; i < ng * vecs; i += kAttnThreads) {
        const int r = row_of(i), d = (i - r * vecs) * 4;
        float mm, ll;
        const float4 v = both(r, d, mm, ll);
        write_row(r, d, v, mm, ll);
      }
    } else {
      // blocks that share the item; one begun in block wf behind its first tile is that block's second part
      const int wf = run.owner(first_tile), wl = run.owner(last_tile);
      const int second = first_tile > run.first(wf);
      auto part_of = [&](int c) { return parts + (2 * c + (c == wf ? second : 0)) * static_cast<int64_t>(part_floats); };
      float* mine = part_of(blockIdx.x);
      for (int i = tid; i < ng * vecs; i += kAttnThreads) {
        const int r = row_of(i), d = (i - r * vecs) * 4;
        float mm, ll;
        const float4 v = both(r, d, mm, ll);
        __stcg(reinterpret_cast<float4*>(mine + r * p.head_dim + d), v);
        if (d == 0) __stcg(reinterpret_cast<float2*>(mine + gsize * p.head_dim + r * 2), make_float2(mm, ll));
      }
      // The block that comes last of `others` + 1: its parts released (ordered before by the barrier), theirs acquired.
      auto comes_last = [&](unsigned* counter, int others) {
        __syncthreads();
        if (tid == 0) {
          s_last = atom_add_acq_rel_gpu(counter, 1u) == static_cast<unsigned>(others);
          if (s_last) *counter = 0;  // ready for the next call
        }
        __syncthreads();
        return s_last != 0;
      };
      // Parts c, c + step, ... (`more` of them behind c) joined in the order of the keys: f(row, column, result).  They
      // are copied into the used stages, as many at a time as fit: what a batch costs is a trip to L2, about 1 us.
      auto join = [&](int c, int step, int more, auto&& f) {
        constexpr int VECS = (S::MAXG * DP / 4 + kAttnThreads - 1) / kAttnThreads;  // of a thread, at most
        const int size = ng * vecs, fit = S::STAGE / (size * 16), batch = min(kJoinBatch, kAttnWarps * fit);
        Part acc[VECS];
#pragma unroll
        for (int k = 0; k < VECS; ++k) acc[k] = {0.0f, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
        if (tid < RG) s_run[tid] = -INFINITY;
        // part u of a batch lies in the stage of warp u mod 4, behind u / 4 others
        const uint32_t to = smem_u32(smem) + st * S::STAGE + tid * 16;
        const uint8_t* from = smem + st * S::STAGE + tid * 16;
#pragma unroll 1
        for (int c0 = 0; c0 <= more; c0 += batch) {
          const int here = min(batch, more + 1 - c0);
#pragma unroll 4
          for (int u = 0; u < here; ++u) {
            const float* part = part_of(c + (c0 + u) * step) + tid * 4;
            const uint32_t at_u = to + (u & 3) * ST * S::STAGE + (u >> 2) * size * 16;
#pragma unroll
            for (int k = 0; k < VECS; ++k)
              if (tid + k * kAttnThreads < size)
                cp_async16(at_u + k * kAttnThreads * 16, part + k * kAttnThreads * 4, true);
          }
          cp_async_commit();
          for (int x = tid; x < here * ng; x += kAttnThreads) {
            const int u = x / ng, r = x - u * ng;
            s_joined[u][r] = __ldcg(reinterpret_cast<const float2*>(part_of(c + (c0 + u) * step) + gsize * p.head_dim + r * 2));
          }
          cp_async_wait<0>();
          __syncthreads();
          // the parts' weights, once for each part and row
          for (int x = tid; x < here * ng; x += kAttnThreads) {
            const int u = x / ng, r = x - u * ng;
            const float old = s_run[r];
            float mn = old;
#pragma unroll 4
            for (int y = 0; y < here; ++y) mn = fmaxf(mn, s_joined[y][r].x);
            const float base = mn == -INFINITY ? 0.0f : mn, w1 = ex2_approx(s_joined[u][r].x - base);
            s_weight[u][r] = make_float2(w1, s_joined[u][r].y * w1);
            if (u == 0) s_next[r] = make_float2(mn, ex2_approx(old - base));
          }
          __syncthreads();
          if (tid < ng) s_run[tid] = s_next[tid].x;
#pragma unroll
          for (int k = 0; k < VECS; ++k) {
            const int i = tid + k * kAttnThreads;
            if (i < size) {
              const int r = row_of(i);
              const float old = s_next[r].y;
              acc[k].m = s_next[r].x;
              float l2 = acc[k].l * old;
              float4 v = make_float4(acc[k].v.x * old, acc[k].v.y * old, acc[k].v.z * old, acc[k].v.w * old);
#pragma unroll 4
              for (int u = 0; u < here; ++u) {
                const float2 wl = s_weight[u][r];
                const float4 x = *reinterpret_cast<const float4*>(from + (u & 3) * ST * S::STAGE + (u >> 2) * size * 16 +
                                                                  k * kAttnThreads * 16);
                l2 += wl.y;
                v = make_float4(v.x + x.x * wl.x, v.y + x.y * wl.x, v.z + x.z * wl.x, v.w + x.w * wl.x);
              }
              acc[k].l = l2;
              acc[k].v = v;
            }
          }
          __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < VECS; ++k) {
          const int i = tid + k * kAttnThreads;
          if (i < size) f(row_of(i), (i - row_of(i) * vecs) * 4, acc[k]);
        }
      };
      const int count = wl - wf + 1;
      int step = 1;
      bool mine_last = true;
      if (count > kFlatJoin) {
        // many parts: groups of neighbours first, each joined into its first part, most of them long before the end
        step = count <= 8 * kFlatJoin / 3 ? 8 : 16;
        const int c = wf + (static_cast<int>(blockIdx.x) - wf) / step * step, more = min(step - 1, wl - c);
        if (more > 0) {
          mine_last = comes_last(counters + kMaxWorkers + c, more);
          if (mine_last) {
            float* to = part_of(c);
            join(c, 1, more, [&](int r, int d, const Part& j) {
              __stcg(reinterpret_cast<float4*>(to + r * p.head_dim + d), j.v);
              if (d == 0) {
                s_ml[0][r] = make_float2(j.m, j.l);
              }
            });
            __syncthreads();
            if (tid < ng) __stcg(reinterpret_cast<float2*>(to + gsize * p.head_dim + tid * 2), s_ml[0][tid]);
          }
        }
      }
      const int groups_of = (count + step - 1) / step;
      if (mine_last && comes_last(counters + wf, groups_of - 1))
        join(wf, step, groups_of - 1, [&](int r, int d, const Part& j) { write_row(r, d, j.v, j.m, j.l); });
    }
    __syncthreads();  // the stages are free again
    if (chunks < CPR) {
      // the columns of the keys behind head_dim are zeros once more
      for (int i = lane; i < KT * (CPR - chunks); i += 32)
        *reinterpret_cast<uint4*>(smem + (w * ST + st) * S::STAGE +
                                  staged<PITCH>(i / (CPR - chunks), chunks + i % (CPR - chunks))) = make_uint4(0, 0, 0, 0);
      __syncwarp();
    }
  };

  int64_t item = i0 - at.t;  // first tile, among all T, of the item at `at`
  begin_item();
  int stage = 0;
  for (int64_t i = 0; i < n; ++i) {
    cp_async_wait<ST - 2>();
    __syncwarp();
    if (i + ST - 1 < n) {
      issue(stage == 0 ? ST - 1 : stage - 1);
      in.next(p, units, CT);
      if (i + ST < n) look_up();
    }
    cp_async_commit();
    const uint32_t mask = s_mask[w][stage];
    if (mask != 0u) {
      if constexpr (S::F32)
        tile_f32(stage, mask);
      else
        tile_mma(stage, mask);
    }
    if (at.t + 1 == at.nt || i + 1 == n) {
      end_item(item, item + at.nt - 1, stage);
      item += at.nt;
      at.next(p, units, CT);
      if (i + 1 < n) begin_item();
    } else {
      ++at.t;
    }
    if (++stage == ST) stage = 0;
  }
  cp_async_wait<0>();
  if (bad_page) atomicOr(&g_paged_status, kDevBadIndex);
}

template <class T, class C, int DP, Heads HEADS>
cudaError_t run_attention(const AttnParams& p, cudaStream_t s, bool pdl) {
  using S = AttnShape<T, C, DP, HEADS>;
  const void* k = reinterpret_cast<const void*>(attention_kernel<T, C, DP, HEADS>);
  static std::atomic<uint64_t> configured{0};  // a bit for each device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(configured.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  const int G = p.q_heads / p.kv_heads;
  const int64_t units = static_cast<int64_t>(p.kv_heads) * ((G + S::MAXG - 1) / S::MAXG);
  const int64_t tiles = (static_cast<int64_t>(p.max_pages) * p.page_size + S::CT - 1) / S::CT;
  int64_t grid = static_cast<int64_t>(device_sm_count()) * S::CTAS;
  if (grid > kMaxWorkers) grid = kMaxWorkers;
  // no more blocks than the page table has room for
  if (tiles < grid && p.M * units < grid && tiles * p.M * units < grid) grid = tiles * p.M * units;
  void* args[] = {const_cast<AttnParams*>(&p)};
  return launch_ex(k, dim3(static_cast<unsigned>(grid)), dim3(kAttnThreads), S::SMEM, s, pdl, args);
}

template <class T, class C, Heads HEADS>
cudaError_t pick_width(const AttnParams& p, cudaStream_t s, bool pdl) {
  if (p.head_dim <= 64) return run_attention<T, C, 64, HEADS>(p, s, pdl);
  if (p.head_dim <= 128) return run_attention<T, C, 128, HEADS>(p, s, pdl);
  // 192 in the shape of 256 took 164 us instead of 125 (32 rows of 4096 keys, 32 and 8 heads): one block an SM, not two
  if constexpr (sizeof(C) == 2)
    if (p.head_dim <= 192) return run_attention<T, C, 192, HEADS>(p, s, pdl);
  return run_attention<T, C, 256, HEADS>(p, s, pdl);
}

template <class T, class C>
cudaError_t pick_attention(const AttnParams& p, cudaStream_t s, bool pdl) {
  const int G = p.q_heads / p.kv_heads;
  if constexpr (sizeof(T) == 4) {
    if (G == 1) return pick_width<T, C, kFew>(p, s, pdl);
    return G <= 4 ? pick_width<T, C, kSome>(p, s, pdl) : pick_width<T, C, kMany>(p, s, pdl);
  } else {
    if (G <= 4) return pick_width<T, C, kFew>(p, s, pdl);
    return G <= 8 ? pick_width<T, C, kSome>(p, s, pdl) : pick_width<T, C, kMany>(p, s, pdl);
  }
}

}  // namespace

cudaError_t launch_paged_append(const AppendParams& p, bool f32, bool e4m3, cudaStream_t s, bool pdl) {
  const void* k = f32    ? reinterpret_cast<const void*>(append_kernel<float, float>)
                  : e4m3 ? reinterpret_cast<const void*>(append_kernel<__nv_bfloat16, __nv_fp8_e4m3>)
                         : reinterpret_cast<const void*>(append_kernel<__nv_bfloat16, __nv_bfloat16>);
  static std::atomic<int> fits[3];  // blocks that fit an SM, by type: 6 to 9
  std::atomic<int>& fit = fits[f32 ? 2 : e4m3];
  int blocks = fit.load(std::memory_order_relaxed);
  if (blocks == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, k, kAppendThreads, 0);
    if (e != cudaSuccess) return e;
    if (blocks < 1) blocks = 1;
    fit.store(blocks, std::memory_order_relaxed);
  }
  // Rows that are short lie side by side in a block (16384 rows of 8 and 2 heads of 64: 11 us, 20.6 one by one), and
  // there are no more blocks than fit the GPU at once, each with its share of the rows (one an SM more, for an e4m3 cache:
  // 92 us, not 70).
  AppendParams a = p;
  const int heads = p.q_heads + 2 * p.kv_heads;
  a.lanes = kAppendThreads / (p.head_dim / (f32 ? 4 : 8));
  a.rows = 1;
  while (a.lanes % 2 == 0 && heads * 2 <= a.lanes * kAppendHeads) {
    a.lanes /= 2;
    a.rows *= 2;
  }
  // few rows of many heads: a block for each round of loads (250 rows of 64 and 8 heads of 128: 5.0 us, 6.0 with one)
  const int64_t most = static_cast<int64_t>(device_sm_count()) * blocks, all = (p.M + a.rows - 1) / a.rows;
  const int64_t turns = (all + most - 1) / most, grid = (all + turns - 1) / turns;
  const int round = a.lanes * kAppendHeads;
  a.parts = static_cast<int>(std::min<int64_t>((heads + round - 1) / round, most / grid));
  void* args[] = {&a};
  return launch_ex(k, dim3(static_cast<unsigned>(grid * a.parts)), dim3(kAppendThreads), 0, s, pdl, args);
}

cudaError_t launch_paged_attention(const AttnParams& p, bool f32, bool e4m3, cudaStream_t s, bool pdl) {
  return f32    ? pick_attention<float, float>(p, s, pdl)
         : e4m3 ? pick_attention<__nv_bfloat16, __nv_fp8_e4m3>(p, s, pdl)
                : pick_attention<__nv_bfloat16, __nv_bfloat16>(p, s, pdl);
}

// Counters and two parts of at most min(G, 16) heads for each block.
int64_t paged_attention_workspace_bytes(int q_heads, int kv_heads, int head_dim) {
  const int G = q_heads / kv_heads, rows = G < 16 ? G : 16;
  return kMaxWorkers * (8 + 2 * static_cast<int64_t>(rows) * (head_dim + 4) * 4);
}

unsigned read_clear_status_paged() {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_paged_status, sizeof(v)) != cudaSuccess) return ~0u;
  if (cudaMemcpyToSymbol(g_paged_status, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace coda
