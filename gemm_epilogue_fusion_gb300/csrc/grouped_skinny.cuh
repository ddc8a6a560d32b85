// Products of rows grouped by expert where an expert has few rows: the weights
// of the experts that are hit stream through the GPU once, and nothing else
// matters (grouped_gemm.cuh is for the rest).
//
// A tile is 32 rows of an expert by 256 accumulator columns.  The MMA still has
// 128 rows, but the 96 behind the tile's are never loaded: a row of the
// accumulator depends on its own row of A alone, so whatever lies in shared
// memory there (the next k-block's rows, weights) gives accumulator rows that
// nobody reads.  A k-block of A is then 4 KB instead of 16.
//
// A k-block costs its waits, signals and issues however few its columns (0.17 us
// and more), so narrower tiles do not spread a product over more SMs without
// slowing each.  Instead a cluster of CL CTAs splits a tile's contraction: each CTA runs its share of the k-blocks
// into its own TMEM, sends every other CTA the columns that this one finishes
// (fp32, through distributed shared memory), and adds what it receives in the
// CTAs' order, so results do not depend on timing.  64 rows of 8 experts of 4096
// x 4096, SwiGLU: 88 us, the 537 MB of weights at 6.1 TB/s.
//
// Roles: warp 0 epilogue (the 32 TMEM lanes of the tile's rows; each thread
// stores its own row), warp 1 TMEM owner and MMA issuer, warp 2 producer.
#pragma once
#include <cmath>
#include <cstring>

#include "grouped_gemm.cuh"
#include "grouped_wide.cuh"

namespace coda {

template <int KIND, int PROG, int CL_>
struct SkinnyCfg {
  static constexpr int kKind = KIND;
  static constexpr int kProg = PROG;
  static constexpr bool SWIGLU = PROG == kGroupSwiGLU || PROG == kGroupSwiGLUSave;
  static constexpr bool SAVE = PROG == kGroupSwiGLUSave;
  static constexpr bool BWD = PROG == kGroupSwiGLUBwd;
  static constexpr bool WGRAD = false;
  static constexpr bool EVEN = false;
  static constexpr bool B_MN = BWD || PROG == kGroupPlainMN;
  static constexpr int CL = CL_;
  static constexpr int TILE_M = 32;
  static constexpr int BAND_ROWS = 0;  // all: further row tiles follow the first one column by column, weights from L2
  static constexpr int BN = 256;
  static constexpr int STAGES = CL == 1 ? 6 : 5;
  static constexpr int ELEM = KIND == kKindBF16 ? 2 : 1;
  static constexpr int BK = 128 / ELEM;
  static constexpr int UMMA_K = 32 / ELEM;
  static constexpr int K_STEPS = BK / UMMA_K;
  static constexpr int A_BYTES = TILE_M * 128;
  static constexpr int B_BYTES = BN * 128;
  static constexpr int OUT_COLS = SWIGLU ? BN / 2 : BN;
  static constexpr int B_BOX = SWIGLU ? BN / 2 : BN;
  static constexpr int MINE = OUT_COLS / CL;        // output columns that a CTA finishes
  static constexpr int CHUNK = MINE < 32 ? MINE : 32;  // of them at a time
  static constexpr int TMEM_COLS = 2 * BN;
  static constexpr int NUM_THREADS = 96;
  static constexpr int MN_BOX_BYTES = 64 * 128;
  // shared memory: [A stages][B stages][partial sums, one set a CTA][barriers][TMEM slot, abort flag]
  static constexpr int OFF_B = STAGES * A_BYTES;
  static constexpr int OFF_PART = OFF_B + STAGES * B_BYTES;
  static constexpr int PART_BYTES = CL == 1 ? 0 : TILE_M * (BN / CL) * 4;  // from one CTA
  static constexpr int OFF_BARS = OFF_PART + CL * PART_BYTES;
  static constexpr int NUM_BARS = 2 * STAGES + 4 + 2 + 1;
  static constexpr int SMEM_BYTES = OFF_BARS + NUM_BARS * 8 + 16 + 1024;
  static constexpr uint32_t FMT = KIND == kKindBF16 ? 1u : 0u;
  static constexpr uint32_t IDESC = make_idesc(FMT, FMT, 128, BN, false, B_MN);
  static_assert(KIND == kKindBF16 || !B_MN, "MN-major operands are bf16");
  static_assert(MINE % 16 == 0, "whole 16-column pieces");
  // the MMA reads 128 rows from a k-block's A: 96 past it, into what follows
  static_assert(STAGES * B_BYTES >= 96 * 128, "reads past A stay in the tile buffers");
  static_assert(SMEM_BYTES <= 232448, "exceeds 227 KB of shared memory");
};

// Load of 16 fp32 accumulator columns of this warp's 32 TMEM lanes; valid after tmem_wait_ld16().
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, const uint32_t* v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3])
               : "memory");
}

template <class C>
__global__ void __launch_bounds__(C::NUM_THREADS, 1)
    grouped_skinny_kernel(const __grid_constant__ GroupMaps maps, const __grid_constant__ GroupArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + C::OFF_B;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* part_full = acc_empty + 2;   // every CTA's share of this CTA's columns has arrived
  uint64_t* part_free = part_full + 1;   // every CTA has read what this CTA sent it
  uint64_t* mma_drain = part_free + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = C::CL > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = blockIdx.x / C::CL, n_units = gridDim.x / C::CL;
  // this CTA's k-blocks
  const int k_blocks = (args.K + C::BK - 1) / C::BK;
  const int kb0 = k_blocks * rank / C::CL, kb1 = k_blocks * (rank + 1) / C::CL;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 1);
    }
    mbar_init(part_full, C::CL);
    mbar_init(part_free, C::CL);
    mbar_init(mma_drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 2 && elect_one()) {
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b);
    if constexpr (C::SWIGLU) tma_prefetch_desc(&maps.b2);
  }
  if (warp == 1) {
    tmem_alloc<1>(tmem_slot, C::TMEM_COLS);
    tmem_relinquish<1>();
  }
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (C::CL > 1) cluster_sync();  // the peers' barriers exist before anyone signals them
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;

  pdl_wait();
  pdl_launch_dependents();

  GroupWalk<C> walk(args);
  GroupTile tl;
  if (warp == 2) {
    // ------------------------------------------------------- TMA producer ----
    const uint64_t pol_a = l2_policy_evict_last();
    const uint64_t pol_w = args.stream_w ? l2_policy_evict_first() : l2_policy_evict_last();
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!walk.find(unit + k * n_units, tl)) break;
      if (elect_one()) {
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, &g_status)) {
            ok = false;
            break;
          }
          uint8_t* b = sB + stage * C::B_BYTES;
          uint64_t* bar = &full[stage];
          const int kx = kb * C::BK;
          mbar_arrive_expect_tx(bar, C::A_BYTES + C::B_BYTES);
          tma_load_2d(sA + stage * C::A_BYTES, &maps.a, bar, kx, tl.row0, pol_a);
          if constexpr (C::B_MN) {
#pragma unroll
            for (int i = 0; i < C::BN / 64; ++i)
              tma_load_3d(b + i * C::MN_BOX_BYTES, &maps.b, bar, tl.n * C::BN + i * 64, kx, tl.e, pol_w);
          } else {
            tma_load_3d(b, &maps.b, bar, kx, tl.n * C::B_BOX, tl.e, pol_w);
            if constexpr (C::SWIGLU)  // gate rows, then up rows
              tma_load_3d(b + C::B_BOX * 128, &maps.b2, bar, kx, tl.n * C::B_BOX, tl.e, pol_w);
          }
          ++issued;
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (elect_one()) drain_ring(full, C::STAGES, issued, abort_flag);
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer ----
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      if (!walk.find(unit + it * n_units, tl)) break;
      if (elect_one()) {
        const int buf = it & 1;
        const uint32_t use = static_cast<uint32_t>(it >> 1) & 1u;
        ok = mbar_wait(&acc_empty[buf], use ^ 1u, abort_flag, &g_status);
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * C::BN);
        for (int kb = kb0; ok && kb < kb1; ++kb) {
          if (!mbar_wait(&full[stage], phase, abort_flag, &g_status)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint64_t adesc = sdesc_kmajor_sw128(smem_u32(sA + stage * C::A_BYTES));
          const uint32_t b_s = smem_u32(sB + stage * C::B_BYTES);
          const uint64_t bdesc = C::B_MN ? sdesc_mnmajor_sw128(b_s, C::MN_BOX_BYTES) : sdesc_kmajor_sw128(b_s);
          constexpr uint64_t b_step = C::B_MN ? C::UMMA_K * 8u : 2u;
#pragma unroll
          for (int s = 0; s < C::K_STEPS; ++s)
            tc_mma<C::kKind, 1>(d_tmem, adesc + 2u * s, bdesc + b_step * s, C::IDESC, kb != kb0 || s != 0);
          tc_commit<1>(&empty[stage]);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) tc_commit<1>(&acc_full[buf]);
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (elect_one()) {
      tc_commit<1>(mma_drain);
      (void)mbar_wait(mma_drain, 0, abort_flag, &g_status, false);
    }
  } else {
    // ----------------------------------------------------------- epilogue ----
    const int64_t N = args.N;
    uint32_t peer_part[C::CL], peer_full[C::CL], peer_free[C::CL];
    if constexpr (C::CL > 1) {
#pragma unroll
      for (int r = 0; r < C::CL; ++r) {
        peer_part[r] = mapa_shared(smem_u32(smem + C::OFF_PART + rank * C::PART_BYTES), r);
        peer_full[r] = mapa_shared(smem_u32(part_full), r);
        peer_free[r] = mapa_shared(smem_u32(part_free), r);
      }
    }
    const bool none = kb0 == kb1;  // fewer k-blocks than CTAs: nothing was multiplied here
    for (int it = 0;; ++it) {
      if (!walk.find(unit + it * n_units, tl)) break;
      const int buf = it & 1;
      const uint32_t use = static_cast<uint32_t>(it >> 1) & 1u;
      const int64_t row = tl.row0 + lane;
      const bool mine = row < tl.row_end;
      float sc = 1.0f;
      if constexpr (!C::BWD) {
        if (args.row_scale != nullptr && mine) sc = args.row_scale[row];
        if (args.w_scale != nullptr) sc *= args.w_scale[tl.e];
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[buf], use, abort_flag, &g_status))) break;
      tc_fence_after_sync();
      const uint32_t t_row = tmem_base + static_cast<uint32_t>(buf * C::BN);
      auto release_acc = [&]() {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[buf]);
      };
      if constexpr (C::CL > 1) {
        // every CTA's columns to it: its BN / CL columns are MINE output columns
        // (SwiGLU: of the gate, then of the up product), four to a vector, the
        // vectors of a warp side by side
        if (!__all_sync(0xffffffffu, mbar_wait_cluster(part_free, (it & 1) ^ 1u, abort_flag, &g_status))) break;
#pragma unroll
        for (int c0 = 0; c0 < C::BN; c0 += 16) {
          uint32_t g[16];
          tmem_ld16(t_row + c0, g);
          tmem_wait_ld16(g);
          const int half = c0 / C::OUT_COLS, to = c0 % C::OUT_COLS / C::MINE;
          const int at = half * C::MINE + c0 % C::MINE;  // column among those of CTA `to`
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            if (none) g[4 * v] = g[4 * v + 1] = g[4 * v + 2] = g[4 * v + 3] = 0u;
            st_cluster_v4(peer_part[to] + static_cast<uint32_t>(((at / 4 + v) * 32 + lane) * 16), g + 4 * v);
          }
        }
        release_acc();
        // each lane's vectors, ordered by the warp's barrier before the arrivals
        __syncwarp();
        if (lane < C::CL) {
          uint32_t bar = 0;
#pragma unroll
          for (int r = 0; r < C::CL; ++r) bar = lane == r ? peer_full[r] : bar;
          mbar_arrive_cluster(bar);
        }
        if (!__all_sync(0xffffffffu, mbar_wait_cluster(part_full, it & 1, abort_flag, &g_status))) break;
      }
      // 16 or 32 output columns at a time
#pragma unroll 1
      for (int b = 0; b < C::MINE; b += C::CHUNK) {
        const int col0 = tl.n * C::OUT_COLS + rank * C::MINE + b;
        float g[C::CHUNK], u[C::SWIGLU ? C::CHUNK : 1];
        if constexpr (C::CL == 1) {
          uint32_t t[32], t2[C::SWIGLU ? 32 : 1];
          tmem_ld32(t_row + b, t);
          if constexpr (C::SWIGLU) tmem_ld32(t_row + C::BN / 2 + b, t2);
          tmem_wait_ld(t);
          if constexpr (C::SWIGLU) tmem_touch(t2);
#pragma unroll
          for (int i = 0; i < C::CHUNK; ++i) {
            g[i] = __uint_as_float(t[i]);
            if constexpr (C::SWIGLU) u[i] = __uint_as_float(t2[i]);
          }
          if (b + C::CHUNK == C::MINE) release_acc();
        } else {
          auto gather = [&](int at, float* out) {
#pragma unroll
            for (int i = 0; i < C::CHUNK; ++i) out[i] = 0.0f;
#pragma unroll
            for (int r = 0; r < C::CL; ++r) {
              const float4* src = reinterpret_cast<const float4*>(smem + C::OFF_PART + r * C::PART_BYTES) + at / 4 * 32;
#pragma unroll
              for (int v = 0; v < C::CHUNK / 4; ++v) {
                const float4 x = src[v * 32 + lane];
                out[4 * v] += x.x;
                out[4 * v + 1] += x.y;
                out[4 * v + 2] += x.z;
                out[4 * v + 3] += x.w;
              }
            }
          };
          gather(b, g);
          if constexpr (C::SWIGLU) gather(C::MINE + b, u);
        }
#pragma unroll
        for (int c = 0; c < C::CHUNK / 8; ++c) {
          const int col = col0 + c * 8;
          if (!mine || col >= args.N) continue;
          uint32_t w[4];
          [[maybe_unused]] uint32_t wg[4], wu[4], gin[4], uin[4];
          if constexpr (C::BWD) {
            const uint4 gv = *reinterpret_cast<const uint4*>(args.GU + row * 2 * N + col);
            const uint4 uv = *reinterpret_cast<const uint4*>(args.GU + row * 2 * N + N + col);
            gin[0] = gv.x, gin[1] = gv.y, gin[2] = gv.z, gin[3] = gv.w;
            uin[0] = uv.x, uin[1] = uv.y, uin[2] = uv.z, uin[3] = uv.w;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = c * 8 + 2 * e;
            const float2 x = make_float2(g[j], g[j + 1]);
            if constexpr (C::BWD) {
              group_swiglu_grad(x, gin[e], uin[e], wg[e], wu[e]);
            } else if constexpr (C::SWIGLU) {
              const float2 s2 = make_float2(sc, sc);
              const float2 G = fmul2(x, s2);
              const float2 U = fmul2(make_float2(u[j], u[j + 1]), s2);
              const float2 o = fmul2(silu2(G), U);
              w[e] = pack_bf16x2(o.x, o.y);
              if constexpr (C::SAVE) {
                wg[e] = pack_bf16x2(G.x, G.y);
                wu[e] = pack_bf16x2(U.x, U.y);
              }
            } else {
              w[e] = pack_bf16x2(x.x * sc, x.y * sc);
            }
          }
          if constexpr (!C::BWD)
            *reinterpret_cast<uint4*>(args.D + row * N + col) = make_uint4(w[0], w[1], w[2], w[3]);
          if constexpr (C::BWD || C::SAVE) {
            __nv_bfloat16* gu = (C::BWD ? args.D : args.GU) + row * 2 * N + col;
            *reinterpret_cast<uint4*>(gu) = make_uint4(wg[0], wg[1], wg[2], wg[3]);
            *reinterpret_cast<uint4*>(gu + N) = make_uint4(wu[0], wu[1], wu[2], wu[3]);
          }
        }
      }
      if constexpr (C::CL > 1) {
        // the partial sums are read: every CTA may send the next tile's
        __syncwarp();
        if (lane < C::CL) {
          uint32_t bar = 0;
#pragma unroll
          for (int r = 0; r < C::CL; ++r) bar = lane == r ? peer_free[r] : bar;
          mbar_arrive_cluster(bar);
        }
      }
    }
  }

  // --------------------------------------------------------------- teardown ----
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (C::CL > 1) cluster_sync();  // no CTA leaves while others may write to it or signal it
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc<1>(tmem_base, C::TMEM_COLS);
}

template <class C>
cudaError_t launch_skinny_cfg(const GroupProblem& p, const char** msg) {
  constexpr CUtensorMapDataType in =
      C::kKind == kKindBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const uint64_t T = p.T, K = p.K, el = C::ELEM;
  GroupMaps m = {};
  CUresult e = encode_tmap_2d(&m.a, in, p.A, K, T, K * el, C::BK, C::TILE_M);
  if (e == CUDA_SUCCESS) e = encode_group_weights<C>(&m, in, p);
  if (e != CUDA_SUCCESS) {
    *msg = "cuTensorMapEncodeTiled rejected an operand (pointer, stride or extent)";
    return cudaErrorInvalidValue;
  }
  auto kernel = grouped_skinny_kernel<C>;
  int units = 0;
  cudaError_t ce = group_units<C, C::CL>(reinterpret_cast<const void*>(kernel), &units, msg);
  if (ce != cudaSuccess) return ce;
  const int64_t bound = group_tile_bound<C>(p);
  GroupArgs a = group_args<C>(p);
  a.stream_w = p.T <= C::TILE_M;
  void* kargs[] = {&m, &a};
  ce = launch_ex(reinterpret_cast<const void*>(kernel),
                 dim3(static_cast<unsigned>(C::CL * (bound < units ? bound : units))), dim3(C::NUM_THREADS),
                 C::SMEM_BYTES, p.stream, p.pdl, kargs, C::CL, false);
  if (ce != cudaSuccess) *msg = "grouped GEMM kernel launch failed";
  return ce;
}

// The form of a product: CTA pairs (grouped_wide.cuh), lone CTAs with 128-row
// tiles (grouped_gemm.cuh), or 32-row tiles whose contraction 1, 2, 4 or 8 CTAs
// split.
enum GroupForm { kFormPair = -2, kFormLone = -1 };

// The form with the least time: rounds of tiles over what runs at once, each the
// k-blocks' time and some for the tile's ends, or the weights' way from HBM where
// that is longer.  The experts hit are as many as T rows hit when all are as
// likely.  The constants fit 720 bf16 measurements (4 to 128 experts, of 4096 x
// 14336 to 1024 x 512 and 456 x 3712, 1 to 51200 rows, every form) to 10% on
// average.  With every form of the 120 cases timed again, the one chosen takes
// 1.7% more than the best on average, 8% or more in 9 (28% in one: 512 rows of 4
// experts, 456 x 3712, SwiGLU).  e4m3 was not in the fit: 5.3%, 8% or more in 19
// of 120, up to 49% where a contraction is 4 to 16 of its k-blocks long, and lone
// CTAs often do better than the pairs taken.  The 0.21 us of a pair's k-block fits
// tiles of few rows (their heights are not in the model); at 160 and 256 rows it
// is 0.30 and 0.37 (grouped_wide.cuh), where pairs are the best form anyway.
// Measured, in us, pairs, lone CTAs, and 32 rows split by 1, 2, 4 and 8: 2 rows,
// K = 14336, N = 4096: 53, 84, 65, 43, 37, 42; 640 rows of 16 experts, 1024 x 512,
// SwiGLU: 8.4, 10.4, 10.5, 12.5, 17, 28; 768 rows of 8 experts of 4096 x 14336,
// SwiGLU: 287, 279, 438, 492, 601, 878, 2048 rows: 377, 459, 1173 and more; 1024
// rows of 4 experts, 456 x 3712, SwiGLU: 19.3, 15.5, 31 and more.
// CODA_GROUP_SPLIT=1|2|4|8 forces 32-row tiles split by that many CTAs,
// CODA_CTA_GROUP=1|2 lone CTAs or pairs (read on every call).
template <class Lone>
int group_form(const GroupProblem& p) {
  const char* split = getenv("CODA_GROUP_SPLIT");
  if (split && split[0] && !split[1] && strchr("1248", split[0])) return split[0] - '0';
  const char* force = getenv("CODA_CTA_GROUP");
  if (force && force[0] == '1') return kFormLone;
  if (force && force[0] == '2') return kFormPair;
  const int sms = device_sm_count();
  const double n_tiles = (p.N + Lone::OUT_COLS - 1) / Lone::OUT_COLS;
  const double hit = p.E * (1.0 - std::pow(1.0 - 1.0 / p.E, p.T));
  const double k_blocks = (p.K + Lone::BK - 1) / Lone::BK;
  const double weights = hit * p.N * p.K * Lone::ELEM * (Lone::SWIGLU ? 2 : 1) / 6.5e6;  // us
  const auto rounds = [&](int rows, double units) {
    return std::ceil(hit * std::fmax(1.0, p.T / hit / rows + 0.5) * n_tiles / units);
  };
  int form = kFormPair;
  double least = 1e30;
  const auto consider = [&](int f, double tiles, double stream, double begin) {
    const double t = std::fmax(stream, tiles) + 0.1 * std::fmin(stream, tiles) + begin;
    if (t < least) {
      least = t;
      form = f;
    }
  };
  consider(kFormPair, rounds(256, sms / 2) * (k_blocks * 0.21 + 1.8), weights * 1.02, 2.7);
  consider(kFormLone, rounds(128, sms) * (k_blocks * 0.38 + 1.0), weights * 1.01, 3.2);
  consider(1, rounds(32, sms) * std::fmax(k_blocks * 0.33, 1.5), weights * 1.01, 4.4);
  for (int split = 2; split <= 8; split *= 2)  // an epilogue with the others' sums takes 3.8 us
    consider(split, rounds(32, static_cast<double>(sms) / split) * std::fmax(k_blocks / split * 0.33, 3.8), weights, 4.1);
  return form;
}

template <int KIND, int PROG, class Lone>
cudaError_t launch_group(const GroupProblem& p, const char** msg) {
  switch (group_form<Lone>(p)) {
    case kFormPair: return launch_wide_cfg<WideCfg<KIND, PROG>>(p, msg);
    case kFormLone: return launch_group_cfg<Lone>(p, msg);
    case 8: return launch_skinny_cfg<SkinnyCfg<KIND, PROG, 8>>(p, msg);
    case 4: return launch_skinny_cfg<SkinnyCfg<KIND, PROG, 4>>(p, msg);
    case 2: return launch_skinny_cfg<SkinnyCfg<KIND, PROG, 2>>(p, msg);
    default: return launch_skinny_cfg<SkinnyCfg<KIND, PROG, 1>>(p, msg);
  }
}

}  // namespace coda
