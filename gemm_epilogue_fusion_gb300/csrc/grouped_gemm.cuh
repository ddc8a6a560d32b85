// Persistent tcgen05 GEMM over rows grouped by expert, with ragged group sizes.
//
// Rows [offsets[e], offsets[e + 1]) of A [T, K] are multiplied with expert e's
// weight W_e; one launch covers all experts.  The offsets stay on the device:
// the grid is fixed by bounds that the host knows (T and E), and every warp
// role of every CTA derives the same tile sequence from them (GroupWalk).
//
// The kernel of this file works in lone CTAs: 128 rows of an expert by 256
// accumulator columns, or (weight gradient, dW_e = dY_e' X_e) 128 x 256 of dW.
// grouped_wide.cuh and grouped_wgrad.cuh have the CTA pairs for experts of many
// rows, grouped_skinny.cuh the 32-row tiles for few.  The tiles of all experts
// form one sequence, dealt round robin, so that an expert's last, part-filled
// round is filled by the next expert's tiles.  Roles of the warps as in
// gemm_epilogue.cuh: 0 TMA producer, 1 TMEM owner and MMA issuer, 2..5 epilogue
// (weight gradient: and 8..11), 6 loader of G and U boxes (SwiGLU backward) or
// fixer of last k-blocks (weight gradient).
//
// Where an expert's rows end inside a tile:
//   - the A box reads on into the next expert's rows (or zeros behind T): a row
//     of the accumulator depends on its own row of A alone, and those rows are
//     not stored;
//   - a tile's rows go from the staging slot to global memory with ordinary
//     16-byte stores, eight threads a row, that stop at the expert's last row;
//     whole tiles go through TMA stores (8% of the weight gradient of 448 rows);
//   - the weight gradient sums over rows, so there both operands' rows behind
//     the last one must be zero, not merely one of them (0 * inf): the last
//     k-block's copies are counted on a barrier of their own, on which warp 6
//     waits and then overwrites the rows that the MMA's groups of 16 would read
//     behind the expert's (copies in boxes of 8 rows and of single rows, the
//     missing ones from beyond the tensor, cost 60% of the whole gradient:
//     up to 60 copies for a k-block).
// Weights are 3-D tensors for TMA ([E][rows][cols]): a box never reads across
// the end of an expert's matrix, so widths need not be multiples of a tile.
#pragma once
#include "coda_experts.h"
#include "gemm_epilogue.cuh"

namespace coda {

namespace {
__device__ unsigned g_index_status;
}

// True in one lane of a converged warp, the same one every time.  Where one lane
// of a warp issues MMAs, commits and TMA copies, the branch is taken by this and
// not by a lane number: the compiler then knows that one lane is active, and
// passes their operands on without a loop over lanes (a k-block of four MMAs
// of a CTA pair took 0.32 us to issue, 0.19 this way).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* m, uint64_t* bar, int32_t x, int32_t y,
                                            int32_t z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* m, uint32_t bar_cluster, int32_t x,
                                                 int32_t y, int32_t z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar_cluster), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, const void* src, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(x), "r"(y), "r"(z), "r"(smem_u32(src))
               : "memory");
}

// Wait for an mbarrier's phase that other CTAs of the cluster arrive on, with
// their writes acquired; bounded like mbar_wait.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                                  unsigned* status) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(a), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((it & 63u) == 0) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > CODA_WAIT_TIMEOUT_NS) {
        *abort_flag = 1;
        atomicOr(status, kDevTimeout);
        return false;
      }
    }
  }
}

// Tensor maps of a launch; each program uses some of them.
struct GroupMaps {
  CUtensorMap a;       // A; weight gradient: dY, 64-row boxes
  CUtensorMap b;       // W (SwiGLU: gate rows); weight gradient: X, 64-row boxes
  CUtensorMap b2;      // SwiGLU: up rows
  CUtensorMap d;       // D
  CUtensorMap g, u;    // SwiGLU backward: G and U
};

struct GroupArgs {
  const int32_t* offsets;
  const float* row_scale;
  const float* w_scale;
  __nv_bfloat16* D;
  __nv_bfloat16* GU;
  int T, E, N, K;
  int m_tiles, n_tiles;  // n_tiles: tiles of N (weight gradient: of K); m_tiles: weight gradient, of N
  int group;             // M-tiles of a band
  int stream_w;          // weights are loaded evict-first
};

template <int KIND, int PROG, int STAGES_, int NSLOTS_>
struct GroupCfg {
  static constexpr int kKind = KIND;
  static constexpr int kProg = PROG;
  static constexpr bool SWIGLU = PROG == kGroupSwiGLU || PROG == kGroupSwiGLUSave;
  static constexpr bool SAVE = PROG == kGroupSwiGLUSave;
  static constexpr bool BWD = PROG == kGroupSwiGLUBwd;
  static constexpr bool WGRAD = PROG == kGroupWgrad;
  static constexpr bool EVEN = false;
  static constexpr bool A_MN = WGRAD;
  static constexpr bool B_MN = WGRAD || BWD || PROG == kGroupPlainMN;
  static constexpr int BM = 128;
  static constexpr int TILE_M = BM;
  static constexpr int BAND_ROWS = SWIGLU ? CODA_RASTER_ROWS_SWIGLU : CODA_RASTER_ROWS;
  static constexpr int BN = 256;
  static constexpr int STAGES = STAGES_;
  static constexpr int NSLOTS = NSLOTS_;
  static constexpr int SPB = BWD ? 2 : (SAVE ? 3 : 1);  // slots of a box of 64 output columns
  static constexpr int ELEM = KIND == kKindBF16 ? 2 : 1;
  static constexpr int BK = 128 / ELEM;
  static constexpr int UMMA_K = 32 / ELEM;
  static constexpr int K_STEPS = BK / UMMA_K;
  static constexpr int A_BYTES = BM * 128;
  static constexpr int B_BYTES = BN * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int OUT_COLS = SWIGLU ? BN / 2 : BN;
  static constexpr int B_BOX = SWIGLU ? BN / 2 : BN;  // weight rows of a K-major box
  static constexpr int A_BOX = 32;  // rows of an A box: those past the expert's end are not loaded
  static constexpr int BOX_COLS = 64;
  static constexpr int NUM_BOXES = OUT_COLS / BOX_COLS / (WGRAD ? 2 : 1);  // of a group of epilogue warps
  static constexpr int SLOT_BYTES = BM * 128;
  static constexpr int TMEM_COLS = 2 * BN;
  static constexpr int NUM_EPI_THREADS = 128;  // of a group of epilogue warps
  // The weight gradient's tiles sum over few k-blocks (8 for 512 rows): two groups of epilogue warps (2..5 and 8..11)
  // take two boxes of a tile each.
  static constexpr int EPI_GROUPS = WGRAD ? 2 : 1;
  static constexpr int GROUP_BOXES = NSLOTS / SPB / EPI_GROUPS;  // boxes of slots that a group of epilogue warps has
  static constexpr bool TMA_OUT = !SAVE && !BWD;  // whole tiles are stored by TMA
  static constexpr int NUM_THREADS = WGRAD ? 384 : (BWD ? 224 : 192);
  static constexpr int OFF_B = STAGES * A_BYTES;
  static constexpr int OFF_SLOTS = OFF_B + STAGES * B_BYTES;
  static constexpr int OFF_BARS = OFF_SLOTS + NSLOTS * SLOT_BYTES;
  static constexpr int NUM_BARS = 4 * STAGES + 4 + 2 * NSLOTS + 1;
  static constexpr int SMEM_BYTES = OFF_BARS + NUM_BARS * 8 + 16 + 1024;
  static constexpr uint32_t FMT = KIND == kKindBF16 ? 1u : 0u;
  static constexpr uint32_t IDESC = make_idesc(FMT, FMT, TILE_M, BN, A_MN, B_MN);
  static constexpr int MN_BOX = 64;
  static constexpr int MN_BOX_BYTES = MN_BOX * 128;
  static_assert(KIND == kKindBF16 || !(A_MN || B_MN), "MN-major operands are bf16");
  static_assert(!TMA_OUT || GROUP_BOXES == 2, "a box is stored while the next one is written");
  static_assert(GROUP_BOXES >= 1 && NSLOTS % (SPB * EPI_GROUPS) == 0, "slot ring");
  static_assert(SMEM_BYTES <= 232448, "exceeds 227 KB of shared memory");
};

// One tile: the first row of its expert's A rows (of dW for the weight
// gradient) that it covers and their end, its column tile, and the expert.
struct GroupTile {
  int e, row0, row_end, n;
  int k0, k1;  // weight gradient: the expert's rows, summed over
};

// The tile sequence, walked by a whole warp.  Tiles of expert e follow those
// of the experts before it; within an expert, bands of `group` M-tiles walk
// down a column of tiles before moving right.  Lane l of the warp looks at
// expert base + l: its tile count, and the scan of the 32 counts, say where
// tile t lies.  t never decreases, so experts already passed are not looked
// at again.
template <class C>
struct GroupWalk {
  const GroupArgs& a;
  int base = -32, before = 0, total = 0;  // first expert of the 32, tiles before them, tiles of them
  int reach = 0;                          // where the rows of all experts before them end
  int start = 0, count = 0, incl = 0, tiles = 0;  // of this lane's expert

  __device__ __forceinline__ explicit GroupWalk(const GroupArgs& args) : a(args) {}

  __device__ __forceinline__ int rows_of(int e, int& first) const {
    const int o0 = a.offsets[e], o1 = a.offsets[e + 1];
    first = o0;
    if (o0 < 0 || o1 < o0 || o1 > a.T) {
      atomicOr(&g_index_status, kDevBadIndex);  // such an expert is left out
      first = 0;
      return 0;
    }
    return o1 - o0;
  }

  __device__ __forceinline__ bool find(int t, GroupTile& tl) {
    if constexpr (C::WGRAD) {  // as many tiles for every expert
      const int per = a.m_tiles * a.n_tiles;
      if (base < 0 || t >= before + per) {
        base = base < 0 ? 0 : base;
        while (t >= before + per) before += per, ++base;
        if (base >= a.E) return false;
        count = rows_of(base, start);
      }
      const TileCoord c = tile_coord(t - before, a.m_tiles, a.n_tiles, a.group);
      tl = {base, c.m * C::TILE_M, a.N, c.n, start, start + count};
      return true;
    }
    const int lane = threadIdx.x & 31;
    while (t >= before + total) {
      before += total;
      base += 32;
      total = 0;
      if (base >= a.E) return false;
      const int e = base + lane;
      count = e < a.E ? rows_of(e, start) : 0;
      // two experts never share a row: one that begins before another's end is left out too
      int end = count > 0 ? start + count : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end = max(end, up);
      }
      const int earlier = max(reach, __shfl_up_sync(0xffffffffu, end, 1));
      if (count > 0 && start < (lane > 0 ? earlier : reach)) {
        atomicOr(&g_index_status, kDevBadIndex);
        count = 0;
      }
      reach = max(reach, __shfl_sync(0xffffffffu, end, 31));
      tiles = (count + C::TILE_M - 1) / C::TILE_M * a.n_tiles;
      incl = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      total = __shfl_sync(0xffffffffu, incl, 31);
    }
    const int local = t - before;
    const int src = __ffs(__ballot_sync(0xffffffffu, local < incl)) - 1;
    const int t0 = __shfl_sync(0xffffffffu, incl - tiles, src);
    const int first = __shfl_sync(0xffffffffu, start, src);
    const int n = __shfl_sync(0xffffffffu, count, src);
    const int m_tiles = (n + C::TILE_M - 1) / C::TILE_M;
    const TileCoord c = tile_coord(local - t0, m_tiles, a.n_tiles, a.group);
    if constexpr (C::EVEN) {  // equal heights, whole 32 rows; none is empty, as all but the last tile hold 256 at most
      const int h = ((n + m_tiles - 1) / m_tiles + 31) & ~31;
      tl = {base + src, first + c.m * h, first + min(n, (c.m + 1) * h), c.n, 0, 0};
    } else {
      tl = {base + src, first + c.m * C::TILE_M, first + n, c.n, 0, 0};
    }
    return true;
  }
};

// Two columns of the SwiGLU backward, act = silu(G) U: dG = dAct U silu'(G) and
// dU = dAct silu(G), with s = sigmoid(G) and silu'(G) = s + silu(G) (1 - s).
// All in fp32 (the sigmoid's exponential and reciprocal are approximate, 2^-20,
// as in the dense kernels) and rounded once, to the 16 bits that the products
// behind it take as operands.
__device__ __forceinline__ void group_swiglu_grad(float2 dact, uint32_t g2, uint32_t u2, uint32_t& dg2, uint32_t& du2) {
  const float2 G = make_float2(bf16_lo(g2), bf16_hi(g2));
  const float2 U = make_float2(bf16_lo(u2), bf16_hi(u2));
  const float2 s = sigmoid2(G);
  const float2 gs = fmul2(G, s);
  const float2 rest = ffma2(s, make_float2(-1.0f, -1.0f), make_float2(1.0f, 1.0f));
  const float2 dg = fmul2(fmul2(dact, U), ffma2(gs, rest, s));
  const float2 du = fmul2(dact, gs);
  dg2 = pack_bf16x2(dg.x, dg.y);
  du2 = pack_bf16x2(du.x, du.y);
}

template <class C>
__global__ void __launch_bounds__(C::NUM_THREADS, 1)
    grouped_gemm_kernel(const __grid_constant__ GroupMaps maps, const __grid_constant__ GroupArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + C::OFF_B;
  uint8_t* slots = smem + C::OFF_SLOTS;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* r_full = acc_empty + 2;
  uint64_t* r_empty = r_full + C::NSLOTS;
  uint64_t* tail_full = r_empty + C::NSLOTS;     // weight gradient: a last k-block's copies have landed
  uint64_t* tail_ready = tail_full + C::STAGES;  // and its rows behind the expert's are zero
  uint64_t* mma_drain = tail_ready + C::STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int unit = blockIdx.x;
  const int n_units = gridDim.x;
  const int k_blocks = (args.K + C::BK - 1) / C::BK;  // the contraction of all programs but the weight gradient's

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&tail_full[s], 1);
      mbar_init(&tail_ready[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], C::EPI_GROUPS * C::NUM_EPI_THREADS / 32);
    }
    for (int s = 0; s < C::NSLOTS; ++s) {
      mbar_init(&r_full[s], 1);
      mbar_init(&r_empty[s], 1);
    }
    mbar_init(mma_drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && elect_one()) {
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b);
    if constexpr (C::SWIGLU) tma_prefetch_desc(&maps.b2);
    if constexpr (C::TMA_OUT) tma_prefetch_desc(&maps.d);
    if constexpr (C::BWD) {
      tma_prefetch_desc(&maps.g);
      tma_prefetch_desc(&maps.u);
    }
  }
  if (warp == 1) {
    tmem_alloc<1>(tmem_slot, C::TMEM_COLS);
    tmem_relinquish<1>();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;

  pdl_wait();
  pdl_launch_dependents();

  GroupWalk<C> walk(args);
  GroupTile tl;
  if (warp == 0) {
    // ------------------------------------------------------- TMA producer ----
    const uint64_t pol_a = l2_policy_evict_last();
    const uint64_t pol_w = args.stream_w ? l2_policy_evict_first() : l2_policy_evict_last();
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    [[maybe_unused]] uint32_t tails = 0, tail_uses = 0;  // parity of each stage's next tail, stages that had one
    bool ok = true;
    auto load2 = [&](void* dst, const CUtensorMap* m, int x, int y, uint64_t pol) {
      tma_load_2d(dst, m, &full[stage], x, y, pol);
    };
    auto load3 = [&](void* dst, const CUtensorMap* m, int x, int y, int z) {
      tma_load_3d(dst, m, &full[stage], x, y, z, pol_w);
    };
    for (int k = 0; ok; ++k) {
      if (!walk.find(unit + k * n_units, tl)) break;
      if (elect_one()) {
        const int num_kb = C::WGRAD ? (tl.k1 - tl.k0 + C::BK - 1) / C::BK : k_blocks;
        const int a_boxes = min(C::BM, tl.row_end - tl.row0 + C::A_BOX - 1) / C::A_BOX;  // with rows of the expert in them
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, &g_status)) {
            ok = false;
            break;
          }
          uint8_t* a = sA + stage * C::A_BYTES;
          uint8_t* b = sB + stage * C::B_BYTES;
          const int kx = kb * C::BK;
          if constexpr (C::WGRAD) {
            const int y0 = tl.k0 + kx;
            auto columns = [&](auto&& load) {
#pragma unroll
              for (int i = 0; i < C::BM / C::MN_BOX; ++i)
                load(a + i * C::MN_BOX_BYTES, &maps.a, tl.row0 + i * C::MN_BOX);
#pragma unroll
              for (int i = 0; i < C::BN / C::MN_BOX; ++i)
                load(b + i * C::MN_BOX_BYTES, &maps.b, tl.n * C::BN + i * C::MN_BOX);
            };
            if (tl.k1 - y0 >= C::BK) {
              mbar_arrive_expect_tx(&full[stage], C::STAGE_BYTES);
              columns([&](uint8_t* dst, const CUtensorMap* m, int x) { load2(dst, m, x, y0, pol_a); });
            } else {
              // rows of the next expert come along; warp 6 overwrites them before the MMA reads the stage
              mbar_arrive(&full[stage]);
              mbar_arrive_expect_tx(&tail_full[stage], C::STAGE_BYTES);
              tails ^= 1u << stage;
              tail_uses |= 1u << stage;
              columns([&](uint8_t* dst, const CUtensorMap* m, int x) {
                tma_load_2d(dst, m, &tail_full[stage], x, y0, pol_a);
              });
            }
          } else {
            mbar_arrive_expect_tx(&full[stage], a_boxes * C::A_BOX * 128 + C::B_BYTES);
            for (int i = 0; i < a_boxes; ++i)
              load2(a + i * (C::A_BOX * 128), &maps.a, kx, tl.row0 + i * C::A_BOX, pol_a);
            if constexpr (C::B_MN) {
#pragma unroll
              for (int i = 0; i < C::BN / C::MN_BOX; ++i)
                load3(b + i * C::MN_BOX_BYTES, &maps.b, tl.n * C::BN + i * C::MN_BOX, kx, tl.e);
            } else {
              load3(b, &maps.b, kx, tl.n * C::B_BOX, tl.e);
              if constexpr (C::SWIGLU) load3(b + C::B_BOX * 128, &maps.b2, kx, tl.n * C::B_BOX, tl.e);  // up rows
            }
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
    if constexpr (C::WGRAD)  // and the last k-blocks' copies
      if (elect_one())
        for (int s = 0; s < C::STAGES; ++s)
          if (tail_uses >> s & 1u) (void)mbar_wait(&tail_full[s], (tails >> s & 1u) ^ 1u, abort_flag, &g_status, false);
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer ----
    int stage = 0;
    uint32_t phase = 0;
    [[maybe_unused]] uint32_t tails = 0;  // parity of each stage's tail barriers
    bool ok = true;
    for (int it = 0; ok; ++it) {
      if (!walk.find(unit + it * n_units, tl)) break;
      if (elect_one()) {
        const int num_kb = C::WGRAD ? (tl.k1 - tl.k0 + C::BK - 1) / C::BK : k_blocks;
        const int buf = it & 1;
        const uint32_t use = static_cast<uint32_t>(it >> 1) & 1u;
        ok = mbar_wait(&acc_empty[buf], use ^ 1u, abort_flag, &g_status);
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * C::BN);
        for (int kb = 0; ok && kb < num_kb; ++kb) {
          if (!mbar_wait(&full[stage], phase, abort_flag, &g_status)) {
            ok = false;
            break;
          }
          if constexpr (C::WGRAD) {
            if (tl.k1 - tl.k0 - kb * C::BK < C::BK) {
              if (!mbar_wait(&tail_ready[stage], tails >> stage & 1u, abort_flag, &g_status)) {
                ok = false;
                break;
              }
              tails ^= 1u << stage;
            }
          }
          tc_fence_after_sync();
          const uint32_t a_s = smem_u32(sA + stage * C::A_BYTES), b_s = smem_u32(sB + stage * C::B_BYTES);
          const uint64_t adesc = C::A_MN ? sdesc_mnmajor_sw128(a_s, C::MN_BOX_BYTES) : sdesc_kmajor_sw128(a_s);
          const uint64_t bdesc = C::B_MN ? sdesc_mnmajor_sw128(b_s, C::MN_BOX_BYTES) : sdesc_kmajor_sw128(b_s);
          constexpr uint64_t a_step = C::A_MN ? C::UMMA_K * 8u : 2u;
          constexpr uint64_t b_step = C::B_MN ? C::UMMA_K * 8u : 2u;
          // the weight gradient's last k-block: the groups of 16 rows with rows of the expert
          const int steps =
              C::WGRAD ? min(C::K_STEPS, (tl.k1 - tl.k0 - kb * C::BK + C::UMMA_K - 1) / C::UMMA_K) : C::K_STEPS;
#pragma unroll
          for (int s = 0; s < C::K_STEPS; ++s)
            if (!C::WGRAD || s < steps)
              tc_mma<C::kKind, 1>(d_tmem, adesc + a_step * s, bdesc + b_step * s, C::IDESC, (kb | s) != 0);
          tc_commit<1>(&empty[stage], 1);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) tc_commit<1>(&acc_full[buf], 1);
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (elect_one()) {
      tc_commit<1>(mma_drain, 1);
      (void)mbar_wait(mma_drain, 0, abort_flag, &g_status, false);
    }
  } else if (warp == 6) {
    // ------------------------------------------ loader of G and U boxes ----
    if constexpr (C::BWD) {
      const uint64_t pol = l2_policy_evict_first();
      int slot = 0;
      uint32_t phase = 0, used = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (!walk.find(unit + k * n_units, tl)) break;
        if (elect_one()) {
          for (int b = 0; b < C::NUM_BOXES && ok; ++b) {
            const int col0 = tl.n * C::OUT_COLS + b * C::BOX_COLS;
            if (col0 >= args.N) break;
            for (int sb = 0; sb < 2; ++sb) {
              if (!mbar_wait(&r_empty[slot], phase ^ 1u, abort_flag, &g_status)) {
                ok = false;
                break;
              }
              mbar_arrive_expect_tx(&r_full[slot], C::SLOT_BYTES);
              tma_load_2d(slots + slot * C::SLOT_BYTES, sb == 0 ? &maps.g : &maps.u, &r_full[slot], col0, tl.row0, pol);
              ++used;
              if (++slot == C::NSLOTS) {
                slot = 0;
                phase ^= 1u;
              }
            }
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      if (elect_one()) drain_ring(r_full, C::NSLOTS, used, abort_flag);
    }
    if constexpr (C::WGRAD) {
      // ------------- zeros behind an expert's last row, up to the MMA's 16 ----
      int stage = 0;
      uint32_t tails = 0;
      for (int k = 0;; ++k) {
        if (!walk.find(unit + k * n_units, tl)) break;
        const int n = tl.k1 - tl.k0, valid = n % C::BK;
        stage = (stage + (n + C::BK - 1) / C::BK) % C::STAGES;
        if (valid == 0) continue;
        const int s = (stage + C::STAGES - 1) % C::STAGES;  // of the tile's last k-block
        // every lane waits, so every lane's writes follow the copies (an abort ends all lanes' waits)
        if (!__all_sync(0xffffffffu, mbar_wait(&tail_full[s], tails >> s & 1u, abort_flag, &g_status))) break;
        tails ^= 1u << s;
        // at most 15 rows of each box, 128 bytes each and side by side
        const int chunks = ((valid + C::UMMA_K - 1) / C::UMMA_K * C::UMMA_K - valid) * 8;
        auto clear = [&](uint8_t* box) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (lane + 32 * i < chunks)
              *reinterpret_cast<uint4*>(box + valid * 128 + (lane + 32 * i) * 16) = make_uint4(0, 0, 0, 0);
        };
#pragma unroll
        for (int i = 0; i < C::BM / C::MN_BOX; ++i) clear(sA + s * C::A_BYTES + i * C::MN_BOX_BYTES);
#pragma unroll
        for (int i = 0; i < C::BN / C::MN_BOX; ++i) clear(sB + s * C::B_BYTES + i * C::MN_BOX_BYTES);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail_ready[s]);
      }
    }
  } else if (C::EPI_GROUPS == 2 ? warp != 7 : true) {
    // ----------------------------------------------------------- epilogue ----
    const int q = warp & 3;
    const int row_in_tile = q * 32 + lane;
    const int group = C::EPI_GROUPS == 2 && warp >= 8 ? 1 : 0;
    const int tid = static_cast<int>(threadIdx.x) - (group ? 256 : 64);  // 0..127
    const uint32_t bar_id = 1 + group;
    const bool store_warp = tid < 32;  // the group's warp with the lane that stores and signals
    constexpr int kSlots = C::NSLOTS / C::EPI_GROUPS;  // of this group, from slot0 on
    const int slot0 = group * kSlots;
    int slot = 0;
    uint32_t sphase = 0;
    bool ok = true;

    // Rows [row0, row0 + rows) of a staged box to global memory, 8 threads a row.
    auto copy_rows = [&](const uint8_t* sp, __nv_bfloat16* dst, int64_t ld, int row0, int rows, int col0, int cols) {
      const int c = tid & 7;
      if (col0 + c * 8 >= cols) return;
      __nv_bfloat16* to = dst + static_cast<int64_t>(row0 + (tid >> 3)) * ld + col0 + c * 8;
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const uint4*>(sp + swz((tid >> 3) + 16 * i, c));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((tid >> 3) + 16 * i < rows) *reinterpret_cast<uint4*>(to + 16 * i * ld) = v[i];
    };

    for (int it = 0; ok; ++it) {
      if (!walk.find(unit + it * n_units, tl)) break;
      const int buf = it & 1;
      const uint32_t use = static_cast<uint32_t>(it >> 1) & 1u;
      if (!named_bar_and(bar_id, C::NUM_EPI_THREADS, mbar_wait(&acc_full[buf], use, abort_flag, &g_status))) break;
      tc_fence_after_sync();
      const int row0 = tl.row0;
      const int rows = min(C::BM, tl.row_end - row0);
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(buf * C::BN);
      auto release_acc = [&]() {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[buf]);
      };
      const bool some = !C::WGRAD || tl.k1 > tl.k0;  // an expert without rows has a zero gradient
      float sc = 1.0f;
      if constexpr (!C::WGRAD && !C::BWD) {
        if (args.row_scale != nullptr && row_in_tile < rows) sc = args.row_scale[row0 + row_in_tile];
        if (args.w_scale != nullptr) sc *= args.w_scale[tl.e];
      }
#pragma unroll 1
      for (int box = 0; box < C::NUM_BOXES; ++box) {
        const int b = group * C::NUM_BOXES + box;
        const int col0 = tl.n * C::OUT_COLS + b * C::BOX_COLS;
        const int n_cols = C::WGRAD ? args.K : args.N;
        if (col0 >= n_cols) {
          if (box == 0) release_acc();  // the second group's columns lie beyond the matrix
          break;
        }
        uint32_t g[2][32];
        uint32_t u[C::SWIGLU ? 2 : 1][32];
#pragma unroll
        for (int i = 0; i < 2; ++i) tmem_ld32(t_row + b * C::BOX_COLS + 32 * i, g[i]);
        if constexpr (C::SWIGLU) {
#pragma unroll
          for (int i = 0; i < 2; ++i) tmem_ld32(t_row + C::BN / 2 + b * C::BOX_COLS + 32 * i, u[i]);
        }
        tmem_wait_ld(g[0]);
#pragma unroll
        for (int i = 1; i < 2; ++i) tmem_touch(g[i]);
        if constexpr (C::SWIGLU) {
#pragma unroll
          for (int i = 0; i < 2; ++i) tmem_touch(u[i]);
        }
        if (box == C::NUM_BOXES - 1 || col0 + C::BOX_COLS >= n_cols) release_acc();
        bool got = true;
        if constexpr (C::BWD) {
#pragma unroll
          for (int sb = 0; sb < 2; ++sb) got = got && mbar_wait(&r_full[slot + sb], sphase, abort_flag, &g_status);
        }
        uint8_t* sp = slots + (slot0 + slot) * C::SLOT_BYTES;
        if (got) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t w[4];
            [[maybe_unused]] uint32_t wg[4], wu[4];
            uint8_t* p = sp + swz(row_in_tile, c);
            [[maybe_unused]] uint32_t gin[4], uin[4];
            if constexpr (C::BWD) {
              const uint4 gv = *reinterpret_cast<const uint4*>(p);
              const uint4 uv = *reinterpret_cast<const uint4*>(p + C::SLOT_BYTES);
              gin[0] = gv.x, gin[1] = gv.y, gin[2] = gv.z, gin[3] = gv.w;
              uin[0] = uv.x, uin[1] = uv.y, uin[2] = uv.z, uin[3] = uv.w;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = c * 8 + 2 * e;
              float2 x = make_float2(__uint_as_float(g[j >> 5][j & 31]), __uint_as_float(g[(j + 1) >> 5][(j + 1) & 31]));
              if constexpr (C::BWD) {
                group_swiglu_grad(x, gin[e], uin[e], wg[e], wu[e]);
              } else if constexpr (C::SWIGLU) {
                const float2 s2 = make_float2(sc, sc);
                const float2 G = fmul2(x, s2);
                const float2 U = fmul2(make_float2(__uint_as_float(u[j >> 5][j & 31]),
                                                   __uint_as_float(u[(j + 1) >> 5][(j + 1) & 31])),
                                       s2);
                const float2 o = fmul2(silu2(G), U);
                w[e] = pack_bf16x2(o.x, o.y);
                if constexpr (C::SAVE) {
                  wg[e] = pack_bf16x2(G.x, G.y);
                  wu[e] = pack_bf16x2(U.x, U.y);
                }
              } else {
                w[e] = some ? pack_bf16x2(x.x * sc, x.y * sc) : 0u;
              }
            }
            if constexpr (C::BWD) {
              *reinterpret_cast<uint4*>(p) = make_uint4(wg[0], wg[1], wg[2], wg[3]);
              *reinterpret_cast<uint4*>(p + C::SLOT_BYTES) = make_uint4(wu[0], wu[1], wu[2], wu[3]);
            } else {
              *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
              if constexpr (C::SAVE) {
                *reinterpret_cast<uint4*>(p + C::SLOT_BYTES) = make_uint4(wg[0], wg[1], wg[2], wg[3]);
                *reinterpret_cast<uint4*>(p + 2 * C::SLOT_BYTES) = make_uint4(wu[0], wu[1], wu[2], wu[3]);
              }
            }
          }
        }
        // the weight gradient's map ends with the matrix, the others' with the last expert
        const bool by_tma = C::WGRAD || (C::TMA_OUT && rows == C::BM);
        if (by_tma) fence_proxy_async_smem();
        if (!named_bar_and(bar_id, C::NUM_EPI_THREADS, got)) {
          ok = false;
          break;
        }
        const int64_t N = args.N;
        if (by_tma) {
          if (store_warp && elect_one()) {
            if constexpr (C::WGRAD) tma_store_3d(&maps.d, sp, col0, row0, tl.e);
            else tma_store_2d(&maps.d, sp, col0, row0);
            tma_store_commit();
            tma_store_wait_read_all();  // before the next box's barrier, after which this slot may be written again
          }
        } else if constexpr (C::BWD) {
          copy_rows(sp, args.D, 2 * N, row0, rows, col0, n_cols);
          copy_rows(sp + C::SLOT_BYTES, args.D + N, 2 * N, row0, rows, col0, n_cols);
        } else {
          copy_rows(sp, args.D, N, row0, rows, col0, n_cols);
          if constexpr (C::SAVE) {
            copy_rows(sp + C::SLOT_BYTES, args.GU, 2 * N, row0, rows, col0, n_cols);
            copy_rows(sp + 2 * C::SLOT_BYTES, args.GU + N, 2 * N, row0, rows, col0, n_cols);
          }
        }
        // with two boxes of slots the next box's barrier comes before anyone writes these again
        if constexpr (C::BWD || C::GROUP_BOXES == 1) named_bar_sync(bar_id, C::NUM_EPI_THREADS);
        if constexpr (C::BWD) {
          if (store_warp && elect_one()) {  // every thread has read the slots: the loader may fill them
            mbar_arrive(&r_empty[slot]);
            mbar_arrive(&r_empty[slot + 1]);
          }
        }
        slot += C::SPB;
        if (slot == kSlots) {
          slot = 0;
          sphase ^= 1u;
        }
      }
    }
    if (C::TMA_OUT && store_warp && elect_one()) tma_store_wait_all();
  }

  // --------------------------------------------------------------- teardown ----
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc<1>(tmem_base, C::TMEM_COLS);
}

// ------------------------------------------------------------------ host ----

// Output tiles that a launch can have, for any offsets: an expert's last tile
// may be part-filled.
template <class C>
int64_t group_tile_bound(const GroupProblem& p) {
  const auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  if constexpr (C::WGRAD) {
    return p.E * up(p.N, C::TILE_M) * up(p.K, C::BN);
  } else {
    const int64_t experts = p.E < p.T ? p.E : p.T;
    return (p.T / C::TILE_M + experts) * up(p.N, C::OUT_COLS);
  }
}

// Tensor maps of the weights [E, N, K], [E, 2 N, K] or (MN-major) [E, K, N].
template <class C, class Maps>
CUresult encode_group_weights(Maps* m, CUtensorMapDataType in, const GroupProblem& p) {
  const uint64_t E = p.E, N = p.N, K = p.K, el = C::ELEM;
  if (C::B_MN) return encode_tmap_3d(&m->b, in, p.W, N, K, E, N * el, N * K * el, 64, C::BK);
  if (!C::SWIGLU) return encode_tmap_3d(&m->b, in, p.W, K, N, E, K * el, N * K * el, C::BK, C::B_BOX);
  const auto* up = static_cast<const uint8_t*>(p.W) + N * K * el;
  const CUresult e = encode_tmap_3d(&m->b, in, p.W, K, N, E, K * el, 2 * N * K * el, C::BK, C::B_BOX);
  return e != CUDA_SUCCESS ? e : encode_tmap_3d(&m->b2, in, up, K, N, E, K * el, 2 * N * K * el, C::BK, C::B_BOX);
}

// Units (clusters of CL CTAs) of a kernel that run at once on the current
// device; with the shared-memory opt-in, once a device.
template <class C, int CL>
cudaError_t group_units(const void* kernel, int* units, const char** msg) {
  static std::mutex mu;
  static int known[32] = {0};
  int dev = 0;
  cudaError_t ce = cudaGetDevice(&dev);
  if (ce != cudaSuccess) return ce;
  std::lock_guard<std::mutex> lock(mu);
  *units = dev < 32 ? known[dev] : 0;
  if (*units > 0) return cudaSuccess;
  ce = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (ce != cudaSuccess) {
    *msg = "cudaFuncSetAttribute(MaxDynamicSharedMemorySize) failed";
    return ce;
  }
  int n = device_sm_count();
  if (CL > 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CL * n);
    cfg.blockDim = dim3(C::NUM_THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CL;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    ce = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (ce != cudaSuccess || n <= 0) {
      *msg = "cudaOccupancyMaxActiveClusters failed for the grouped GEMM";
      return ce != cudaSuccess ? ce : cudaErrorInvalidConfiguration;
    }
  }
  if (dev < 32) known[dev] = n;
  *units = n;
  return cudaSuccess;
}

// What a form's kernel is told of a problem: the operands, and the grid of its
// tiles with the bands they are walked in.
template <class C>
GroupArgs group_args(const GroupProblem& p) {
  GroupArgs a = {};
  a.offsets = p.offsets;
  a.row_scale = p.row_scale;
  a.w_scale = p.w_scale;
  a.D = static_cast<__nv_bfloat16*>(p.D);
  a.GU = static_cast<__nv_bfloat16*>(p.GU);
  a.T = p.T;
  a.E = p.E;
  a.N = p.N;
  a.K = p.K;
  if constexpr (C::WGRAD) {
    a.m_tiles = (p.N + C::TILE_M - 1) / C::TILE_M;
    a.n_tiles = (p.K + C::BN - 1) / C::BN;
  } else {
    a.n_tiles = (p.N + C::OUT_COLS - 1) / C::OUT_COLS;
  }
  // All of an expert's row tiles: as many as T rows have and no more, so that the band's tiles (tile_coord multiplies
  // them out) stay below the tiles of the launch, whose number the caller has checked.
  a.group = C::BAND_ROWS > 0 ? C::BAND_ROWS / C::TILE_M : (p.T + C::TILE_M - 1) / C::TILE_M;
  return a;
}

template <class C>
cudaError_t launch_group_cfg(const GroupProblem& p, const char** msg) {
  constexpr CUtensorMapDataType in =
      C::kKind == kKindBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  constexpr CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const uint64_t T = p.T, N = p.N, K = p.K, el = C::ELEM;
  GroupMaps m = {};
  auto* GU = static_cast<__nv_bfloat16*>(p.GU);
  CUresult e = CUDA_SUCCESS;
  auto rows = [&](CUtensorMap* map, const void* base, uint64_t cols, uint64_t pitch, uint32_t box_rows) {  // bf16, 64 columns
    if (e == CUDA_SUCCESS) e = encode_tmap_2d(map, bf, base, cols, T, pitch * 2, 64, box_rows);
  };
  if (C::WGRAD) {
    rows(&m.a, p.A, N, N, C::BK);
    rows(&m.b, p.W, K, K, C::BK);
    if (e == CUDA_SUCCESS) e = encode_tmap_3d(&m.d, bf, p.D, K, N, p.E, K * 2, N * K * 2, 64, C::BM);
  } else {
    e = encode_tmap_2d(&m.a, in, p.A, K, T, K * el, C::BK, C::A_BOX);
    if (e == CUDA_SUCCESS) e = encode_group_weights<C>(&m, in, p);
    if (C::TMA_OUT) rows(&m.d, p.D, N, N, C::BM);
    if (C::BWD) {
      rows(&m.g, GU, N, 2 * N, C::BM);
      rows(&m.u, GU + N, N, 2 * N, C::BM);
    }
  }
  if (e != CUDA_SUCCESS) {
    *msg = "cuTensorMapEncodeTiled rejected an operand (pointer, stride or extent)";
    return cudaErrorInvalidValue;
  }
  auto kernel = grouped_gemm_kernel<C>;
  int units = 0;
  cudaError_t ce = group_units<C, 1>(reinterpret_cast<const void*>(kernel), &units, msg);
  if (ce != cudaSuccess) return ce;
  const int64_t bound = group_tile_bound<C>(p);
  const int grid = static_cast<int>(bound < units ? bound : units);
  GroupArgs a = group_args<C>(p);
  // an expert with one row tile reads its weight once
  a.stream_w = !C::WGRAD && p.T <= static_cast<int64_t>(p.E) * C::TILE_M;
  void* kargs[] = {&m, &a};
  ce = launch_ex(reinterpret_cast<const void*>(kernel), dim3(grid), dim3(C::NUM_THREADS), C::SMEM_BYTES, p.stream,
                 p.pdl, kargs, 1, false);
  if (ce != cudaSuccess) *msg = "grouped GEMM kernel launch failed";
  return ce;
}

inline unsigned read_clear_index_impl() {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_index_status, sizeof(v)) != cudaSuccess) return ~0u;
  if (cudaMemcpyToSymbol(g_index_status, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace coda
