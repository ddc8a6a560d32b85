// Weight gradient of products grouped by expert, dW_e [N, K] = dY_e' X_e over
// the expert's rows, where the experts have many (grouped_gemm.cuh has the lone
// CTAs for the rest).
//
// A pair (tcgen05, cta_group::2) takes a tile of 256 x 512 of dW in two halves
// of 256 columns, each with an accumulator of its own, which fill the TMEM.
// All loads come from L2; a tile of 256 x 256, its accumulator double-buffered,
// moves 64 KB a k-block of 64 rows, this one 96 KB for twice the products (0 to
// 6% faster).  A half's accumulator is read in one go (two of its four boxes
// wait in registers), so the next tile's products do not wait for the stores.
//
// An expert's rows are copied in whole groups of 16, the MMA's k: its last
// k-block in a smaller box.  The rows behind the last whole group lie in a
// buffer of their own, which warp 10 fills while the tile's other rows are
// multiplied, and clears behind the expert's last row: both operands have to be
// zero there, not merely one (0 * inf).  Cleared in the ring, where its copies
// had to be waited for in turn, a last k-block cost 1 us a tile.
//
// Measured (64 experts of 2816 x 2048, 469 rows each on average, ragged): 277 us
// against 333 in tiles of 256 x 256 with the last k-block cleared in the ring,
// 1240 TFLOP/s, and 738 MB written at 2.6 TB/s.  8 experts of 28672 x 4096 and
// 512 rows: 700 us, 1370 TFLOP/s.  A tile of 512 rows takes 7.15 us: its MMAs
// alone 4.6, with the loads 5.6, with the epilogue but no stores 6.0; the stores
// share L2 with the loads.  Taking one half through up to 7 k-blocks before the
// other, so that each is handed over while the other works, left four k-blocks of
// loads in flight: 312 us.
#pragma once
#include "grouped_gemm.cuh"

namespace coda {

struct WgradCfg {
  static constexpr bool WGRAD = true;
  static constexpr bool EVEN = false;
  static constexpr int CG = 2;
  static constexpr int BM = 128;
  static constexpr int TILE_M = BM * CG;
  static constexpr int BAND_ROWS = CODA_RASTER_ROWS;
  static constexpr int HALF = 256;
  static constexpr int BN = 2 * HALF;
  static constexpr int STAGES = 3;
  static constexpr int BK = 64;
  static constexpr int UMMA_K = 16;
  static constexpr int STEPS = BK / UMMA_K;
  static constexpr int BOX = 64;  // columns of a copy
  static constexpr int BOX_BYTES = BOX * BK * 2;
  static constexpr int A_BYTES = BM / BOX * BOX_BYTES;
  static constexpr int HALF_BYTES = HALF / CG / BOX * BOX_BYTES;  // of X, in each CTA
  static constexpr int STAGE_BYTES = A_BYTES + 2 * HALF_BYTES;
  static constexpr int SLOT_BYTES = BM * BOX * 2;
  static constexpr int OFF_SLOTS = STAGES * STAGE_BYTES;
  static constexpr int OFF_TAIL = OFF_SLOTS + 4 * SLOT_BYTES;  // two slots a half
  static constexpr int TAIL_BOX_BYTES = UMMA_K * BOX * 2;
  static constexpr int TAIL_BYTES = STAGE_BYTES / BOX_BYTES * TAIL_BOX_BYTES;
  static constexpr int OFF_BARS = OFF_TAIL + TAIL_BYTES;
  static constexpr int NUM_BARS = 2 * STAGES + 3 + 4 + 1;
  static constexpr int SMEM_BYTES = OFF_BARS + NUM_BARS * 8 + 16 + 1024;
  static constexpr int NUM_EPI_THREADS = 128;  // of a half
  static constexpr int NUM_THREADS = 352;
  static constexpr uint32_t IDESC = make_idesc(1u, 1u, TILE_M, HALF, true, true);
  static_assert(SMEM_BYTES <= 232448, "exceeds 227 KB of shared memory");
};

struct WgradMaps {
  CUtensorMap a[4], b[4];  // dY and X in boxes of 16, 32, 48 and 64 rows
  CUtensorMap d;
};

// Roles: warps 0..3 epilogue of the tile's first half, 4..7 of its second, 8
// TMA producer, 9 TMEM owner and MMA issuer (of the pair's even CTA), 10 fixer
// of last k-blocks.
__global__ void __launch_bounds__(WgradCfg::NUM_THREADS, 1)
    grouped_wgrad_kernel(const __grid_constant__ WgradMaps maps, const __grid_constant__ GroupArgs args) {
  using C = WgradCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tail_full = empty + C::STAGES;  // the last rows' copies have landed in this CTA
  uint64_t* tail_ready = tail_full + 1;     // and the rows behind the expert's are zero, in both CTAs
  uint64_t* tail_empty = tail_ready + 1;
  uint64_t* acc_full = tail_empty + 1;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* mma_drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int cta_rank = static_cast<int>(cluster_ctarank());
  const int unit = blockIdx.x / C::CG;
  const int n_units = gridDim.x / C::CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tail_full, 1);
    mbar_init(tail_ready, C::CG);
    mbar_init(tail_empty, 1);
    for (int h = 0; h < 2; ++h) {
      mbar_init(&acc_full[h], 1);
      mbar_init(&acc_empty[h], C::CG * C::NUM_EPI_THREADS / 32);
    }
    mbar_init(mma_drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 8 && elect_one()) {
    tma_prefetch_desc(&maps.a[3]);
    tma_prefetch_desc(&maps.b[3]);
    tma_prefetch_desc(&maps.d);
  }
  if (warp == 9) {
    tmem_alloc<C::CG>(tmem_slot, C::BN);
    tmem_relinquish<C::CG>();
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;

  pdl_wait();
  pdl_launch_dependents();

  // halves of a tile with columns of dW in them; an expert's whole groups of 16 rows, and the rows behind them
  const auto halves_of = [&](const GroupTile& tl) { return args.K - tl.n * C::BN > C::HALF ? 2 : 1; };
  const auto groups_of = [](const GroupTile& tl) { return (tl.k1 - tl.k0) / C::UMMA_K; };
  const auto rest_of = [](const GroupTile& tl) { return (tl.k1 - tl.k0) % C::UMMA_K; };
  // a tile's columns of dY and X, in boxes of `box_bytes`, by load(destination, map, column)
  const auto copy_columns = [&](const GroupTile& tl, uint8_t* dst, int box_bytes, int map, auto&& load) {
    const int ax = tl.row0 + cta_rank * C::BM;
    const int bx = tl.n * C::BN + cta_rank * (C::HALF / C::CG);
#pragma unroll
    for (int i = 0; i < C::BM / C::BOX; ++i) load(dst + i * box_bytes, &maps.a[map], ax + i * C::BOX);
    dst += C::BM / C::BOX * box_bytes;
    for (int h = 0; h < halves_of(tl); ++h)
#pragma unroll
      for (int i = 0; i < C::HALF / C::CG / C::BOX; ++i, dst += box_bytes)
        load(dst, &maps.b[map], bx + h * C::HALF + i * C::BOX);
  };
  const auto boxes_of = [&](const GroupTile& tl) { return (C::BM + halves_of(tl) * (C::HALF / C::CG)) / C::BOX; };

  GroupWalk<C> walk(args);
  GroupTile tl;
  if (warp == 8) {
    // ------------------------------------------------------- TMA producer ----
    const uint64_t pol = l2_policy_evict_last();
    const uint32_t full0 = mapa_shared(smem_u32(full), 0);
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!walk.find(unit + k * n_units, tl)) break;
      if (elect_one()) {
        const int groups = groups_of(tl);
        for (int at = 0; at < groups; at += C::STEPS) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, &g_status)) {
            ok = false;
            break;
          }
          const int steps = min(C::STEPS, groups - at);
          const uint32_t bar = full0 + static_cast<uint32_t>(stage) * 8u;
          const int y = tl.k0 + at * C::UMMA_K;
          if (cta_rank == 0) mbar_arrive_expect_tx(&full[stage], C::CG * boxes_of(tl) * steps * C::TAIL_BOX_BYTES);
          copy_columns(tl, smem + stage * C::STAGE_BYTES, C::BOX_BYTES, steps - 1,
                       [&](uint8_t* dst, const CUtensorMap* m, int x) { tma_load_2d_pair(dst, m, bar, x, y, pol); });
          ++issued;
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (cta_rank == 0 && elect_one()) drain_ring(full, C::STAGES, issued, abort_flag);
  } else if (warp == 9) {
    // --------------------------------------------------------- MMA issuer ----
    if (cta_rank == 0) {
      constexpr uint16_t kPair = 3;
      int stage = 0;
      uint32_t phase = 0;
      uint32_t uses[2] = {0, 0}, tails = 0;  // of the accumulators, of the last rows' buffer
      bool ok = true;
      for (int it = 0; ok; ++it) {
        if (!walk.find(unit + it * n_units, tl)) break;
        if (elect_one()) {
          const int halves = halves_of(tl), groups = groups_of(tl), rest = rest_of(tl);
          // the products of `steps` groups of rows, of both halves; the accumulators are waited for and handed over
          auto products = [&](uint32_t a_s, int box_bytes, int steps, bool first, bool last) {
            const uint64_t adesc = sdesc_mnmajor_sw128(a_s, box_bytes);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (h >= halves) break;
              if (first && !mbar_wait(&acc_empty[h], (uses[h]++ & 1u) ^ 1u, abort_flag, &g_status)) return false;
              tc_fence_after_sync();
              const uint64_t bdesc = sdesc_mnmajor_sw128(a_s + (C::BM + h * (C::HALF / C::CG)) / C::BOX * box_bytes, box_bytes);
#pragma unroll
              for (int s = 0; s < C::STEPS; ++s)
                if (s < steps)
                  tc_mma<kKindBF16, C::CG>(tmem_base + static_cast<uint32_t>(h * C::HALF), adesc + C::UMMA_K * 8u * s,
                                           bdesc + C::UMMA_K * 8u * s, C::IDESC, !first || s != 0);
              if (last) tc_commit<C::CG>(&acc_full[h], kPair);
            }
            return true;
          };
          for (int at = 0; at < groups; at += C::STEPS) {
            ok = mbar_wait(&full[stage], phase, abort_flag, &g_status) &&
                 products(smem_u32(smem + stage * C::STAGE_BYTES), C::BOX_BYTES, min(C::STEPS, groups - at), at == 0,
                          rest == 0 && at + C::STEPS >= groups);
            if (!ok) break;
            tc_commit<C::CG>(&empty[stage], kPair);
            if (++stage == C::STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (ok && rest != 0) {
            ok = mbar_wait_cluster(tail_ready, tails++ & 1u, abort_flag, &g_status) &&
                 products(smem_u32(smem + C::OFF_TAIL), C::TAIL_BOX_BYTES, 1, groups == 0, true);
            if (ok) tc_commit<C::CG>(tail_empty, kPair);
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      if (elect_one()) {
        tc_commit<C::CG>(mma_drain, 1);
        (void)mbar_wait(mma_drain, 0, abort_flag, &g_status, false);
      }
    }
  } else if (warp == 10) {
    // ---------------- an expert's last rows, with zeros behind them ----
    const uint64_t pol = l2_policy_evict_last();
    const uint32_t ready0 = mapa_shared(smem_u32(tail_ready), 0);
    uint8_t* tail = smem + C::OFF_TAIL;
    uint32_t uses = 0;
    for (int k = 0;; ++k) {
      if (!walk.find(unit + k * n_units, tl)) break;
      const int rest = rest_of(tl), boxes = boxes_of(tl);
      if (rest == 0) continue;
      bool ok = true;
      if (elect_one()) {
        ok = mbar_wait(tail_empty, (uses & 1u) ^ 1u, abort_flag, &g_status);
        if (ok) {
          mbar_arrive_expect_tx(tail_full, boxes * C::TAIL_BOX_BYTES);
          copy_columns(tl, tail, C::TAIL_BOX_BYTES, 0, [&](uint8_t* dst, const CUtensorMap* m, int x) {
            tma_load_2d(dst, m, tail_full, x, tl.k1 - rest, pol);
          });
        }
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      // every lane waits, so every lane's writes follow the copies; an abort does not end this wait
      if (!__all_sync(0xffffffffu, mbar_wait(tail_full, uses & 1u, abort_flag, &g_status, false))) break;
      ++uses;
      const int chunks = (C::UMMA_K - rest) * 8;  // of 16 bytes; a box's rows lie side by side
      for (int b = 0; b < boxes; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (lane + 32 * i < chunks)
            *reinterpret_cast<uint4*>(tail + b * C::TAIL_BOX_BYTES + rest * 128 + (lane + 32 * i) * 16) =
                make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(ready0);
    }
  } else {
    // ----------------------------------------------------------- epilogue ----
    const int h = warp >> 2, q = warp & 3;
    const int row = q * 32 + lane;
    const bool store_warp = q == 0;  // the half's warp with the lane that stores
    const uint32_t bar_id = 1 + h;
    const uint32_t acc_empty0 = mapa_shared(smem_u32(&acc_empty[h]), 0);
    const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(h * C::HALF);
    uint8_t* slots = smem + C::OFF_SLOTS + 2 * h * C::SLOT_BYTES;
    uint32_t uses = 0;

    // 64 columns of the accumulator as bf16 (an expert without rows: zeros)
    auto take = [&](int b, bool some, uint32_t (&w)[32]) {
      if (!some) {
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = 0u;
        return;
      }
      uint32_t x[2][32];
      tmem_ld32(t_row + b * C::BOX, x[0]);
      tmem_ld32(t_row + b * C::BOX + 32, x[1]);
      tmem_wait_ld(x[0]);
      tmem_touch(x[1]);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        w[i] = pack_bf16x2(__uint_as_float(x[i >> 4][2 * i & 31]), __uint_as_float(x[i >> 4][(2 * i + 1) & 31]));
    };
    auto put = [&](int slot, const uint32_t (&w)[32]) {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4*>(slots + slot * C::SLOT_BYTES + swz(row, c)) =
            make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    };

    for (int it = 0;; ++it) {
      if (!walk.find(unit + it * n_units, tl)) break;
      const int col0 = tl.n * C::BN + h * C::HALF;
      if (col0 >= args.K) continue;
      const bool some = tl.k1 > tl.k0;
      const int row0 = tl.row0 + cta_rank * C::BM;
      const int boxes = row0 < args.N ? min(C::HALF, args.K - col0 + C::BOX - 1) / C::BOX : 0;
      // two of the four boxes go to the slots at once, which the last tile's stores have read, two wait in registers:
      // so the accumulator is free again before the first store
      if (store_warp && elect_one()) tma_store_wait_read_all();
      bool ok = true;
      if (some) ok = mbar_wait(&acc_full[h], uses++ & 1u, abort_flag, &g_status);
      if (!named_bar_and(bar_id, C::NUM_EPI_THREADS, ok)) break;
      tc_fence_after_sync();
      uint32_t w[32], w2[32], w3[32];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (b < boxes) {
          take(b, some, w);
          put(b, w);
        }
      }
      if (2 < boxes) take(2, some, w2);
      if (3 < boxes) take(3, some, w3);
      if (some) {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty0);
      }
      if (boxes == 0) continue;  // a pair's second CTA without rows
      auto store = [&](int first) {
        fence_proxy_async_smem();
        named_bar_sync(bar_id, C::NUM_EPI_THREADS);
        if (store_warp && elect_one()) {
          for (int b = first; b < min(boxes, first + 2); ++b)
            tma_store_3d(&maps.d, slots + (b - first) * C::SLOT_BYTES, col0 + b * C::BOX, row0, tl.e);
          tma_store_commit();
        }
      };
      store(0);
      if (boxes > 2) {
        if (store_warp && elect_one()) tma_store_wait_read_all();
        named_bar_sync(bar_id, C::NUM_EPI_THREADS);
        put(0, w2);
        if (boxes > 3) put(1, w3);
        store(2);
      }
    }
    if (store_warp && elect_one()) tma_store_wait_all();
  }

  // --------------------------------------------------------------- teardown ----
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();
  tc_fence_after_sync();
  if (warp == 9) tmem_dealloc<C::CG>(tmem_base, C::BN);
}

inline cudaError_t launch_wgrad_pairs(const GroupProblem& p, const char** msg) {
  using C = WgradCfg;
  constexpr CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const uint64_t T = p.T, N = p.N, K = p.K;
  WgradMaps m = {};
  CUresult e = encode_tmap_3d(&m.d, bf, p.D, K, N, p.E, K * 2, N * K * 2, C::BOX, C::BM);
  for (int i = 0; i < 4 && e == CUDA_SUCCESS; ++i) {
    e = encode_tmap_2d(&m.a[i], bf, p.A, N, T, N * 2, C::BOX, 16 * (i + 1));
    if (e == CUDA_SUCCESS) e = encode_tmap_2d(&m.b[i], bf, p.W, K, T, K * 2, C::BOX, 16 * (i + 1));
  }
  if (e != CUDA_SUCCESS) {
    *msg = "cuTensorMapEncodeTiled rejected an operand (pointer, stride or extent)";
    return cudaErrorInvalidValue;
  }
  const void* kernel = reinterpret_cast<const void*>(grouped_wgrad_kernel);
  int units = 0;
  cudaError_t ce = group_units<C, C::CG>(kernel, &units, msg);
  if (ce != cudaSuccess) return ce;
  const int64_t bound = group_tile_bound<C>(p);
  GroupArgs a = group_args<C>(p);
  void* kargs[] = {&m, &a};
  ce = launch_ex(kernel, dim3(static_cast<unsigned>(C::CG * (bound < units ? bound : units))), dim3(C::NUM_THREADS),
                 C::SMEM_BYTES, p.stream, p.pdl, kargs, C::CG, false);
  if (ce != cudaSuccess) *msg = "grouped GEMM kernel launch failed";
  return ce;
}

}  // namespace coda
