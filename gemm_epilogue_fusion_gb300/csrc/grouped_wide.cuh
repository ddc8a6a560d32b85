// Products of rows grouped by expert where the experts have many rows: CTA
// pairs (tcgen05, cta_group::2) with the weights as the MMA's M operand.
//
// The expert's rows are the MMA's N, which can be any multiple of 32 up to 256.
// An expert's rows are cut into as few tiles of at most 256 rows as hold them,
// of equal height: 530 rows are three tiles of 192, 192 and 146 (160), where
// tiles of 256 rows as the M operand, whose height is fixed, take three times
// 256.  Experts of some 500 rows waste 5% of the MMAs this way instead of 25%.
//
// A CTA's accumulator then holds its 128 weight rows (output columns; SwiGLU: 64
// gate and 64 up rows of the same columns) in the TMEM's lanes and the tile's
// rows in its columns.  The epilogue turns 32 rows at a time through shared
// memory in fp32 (written by output column, read by row), so a thread has eight
// neighbouring columns of one row, G beside U, and stores, or reads what the
// backward needs, in 16 bytes.  Rows behind the tile's end are not stored.
//
// A k-block of 64 takes 0.37 us at 256 rows (1740 TFLOP/s, near the power cap),
// 0.30 at 160 (52 KB a pair: L2's 13 TB/s; the MMAs alone 0.20), and with one tile
// an expert the weights' way from HBM.  64 experts of 2048 x 1408 with 30016 rows,
// ragged: SwiGLU 220 us (1570 TFLOP/s), down 130 (1330), their rows' gradient 233
// (1480), SwiGLU's gradient 159 (1090, 830 MB of traffic).
//
// Sums, scales and SwiGLU are fp32; an output is rounded once, to bf16: the
// products that follow take operands of 16 bits (or, requantised, 8), and the
// weighted sum over a row's experts reads them with half the traffic of fp32.
//
// Roles: warp 0 TMA producer, 1 TMEM owner and MMA issuer (of the pair's even
// CTA), 2..5 epilogue (SwiGLU's gradient: and 6..9).
#pragma once
#include "grouped_gemm.cuh"

namespace coda {

template <int KIND, int PROG>
struct WideCfg {
  static constexpr int kKind = KIND;
  static constexpr int kProg = PROG;
  static constexpr bool SWIGLU = PROG == kGroupSwiGLU || PROG == kGroupSwiGLUSave;
  static constexpr bool SAVE = PROG == kGroupSwiGLUSave;
  static constexpr bool BWD = PROG == kGroupSwiGLUBwd;
  static constexpr bool WGRAD = false;
  static constexpr bool EVEN = true;  // an expert's tiles have equal heights
  static constexpr bool W_MN = BWD || PROG == kGroupPlainMN;  // weights [E, K, N]
  static constexpr bool B_MN = W_MN;
  static constexpr int CG = 2;
  static constexpr int BM = 128;      // weight rows of a CTA
  static constexpr int TILE_M = 256;  // rows of the largest tile
  static constexpr int BAND_ROWS = SWIGLU ? CODA_RASTER_ROWS_SWIGLU : CODA_RASTER_ROWS;
  static constexpr int STAGES = 6;
  static constexpr int ELEM = KIND == kKindBF16 ? 2 : 1;
  static constexpr int BK = 128 / ELEM;
  static constexpr int UMMA_K = 32 / ELEM;
  static constexpr int K_STEPS = BK / UMMA_K;
  static constexpr int W_BYTES = BM * 128;
  static constexpr int X_BYTES = TILE_M / 2 * 128;
  static constexpr int CTA_COLS = SWIGLU ? BM / 2 : BM;  // output columns of a CTA
  static constexpr int OUT_COLS = CG * CTA_COLS;
  static constexpr int B_BOX = CTA_COLS;  // weight rows of a K-major box
  static constexpr int MN_BOX_BYTES = 64 * 128;
  static constexpr int CHUNK = 32;  // rows that the epilogue turns at a time
  static constexpr int PITCH = BM + 4;  // floats: eight threads' 16-byte reads lie in different banks
  static constexpr int TURN_BYTES = CHUNK * PITCH * 4;
  static constexpr int TMEM_COLS = 2 * TILE_M;
  static constexpr int NUM_EPI_THREADS = 128;  // of a group of epilogue warps
  // SwiGLU's gradient has twice the traffic of a plain product and a sigmoid: two groups of epilogue warps take its
  // chunks in turn (64 experts of 1408 x 2048 and 469 rows: 174 -> 167 us; the other programs did not gain.  Both were
  // measured before the issue by election, when the issuer's 0.32 us a k-block could hide an epilogue).
  static constexpr int EPI_GROUPS = BWD ? 2 : 1;
  static constexpr int NUM_THREADS = 64 + EPI_GROUPS * NUM_EPI_THREADS;
  static constexpr int OFF_X = STAGES * W_BYTES;
  static constexpr int OFF_TURN = OFF_X + STAGES * X_BYTES;
  static constexpr int OFF_BARS = OFF_TURN + 2 * TURN_BYTES;
  static constexpr int NUM_BARS = 2 * STAGES + 4 + 1;
  static constexpr int SMEM_BYTES = OFF_BARS + NUM_BARS * 8 + 16 + 1024;
  static constexpr uint32_t FMT = KIND == kKindBF16 ? 1u : 0u;
  static constexpr uint32_t IDESC = make_idesc(FMT, FMT, 2 * BM, 0, W_MN, false);  // and the tile's rows
  static_assert(KIND == kKindBF16 || !W_MN, "MN-major operands are bf16");
  static_assert(SMEM_BYTES <= 232448, "exceeds 227 KB of shared memory");
};

struct WideMaps {
  CUtensorMap a[8];  // A in boxes of 16, 32, ... 128 rows: one copy for any height (several, of 16 rows each, took
                     // twice the MMAs' time)
  CUtensorMap b, b2;
};

template <class C>
__global__ void __launch_bounds__(C::NUM_THREADS, 1)
    grouped_wide_kernel(const __grid_constant__ WideMaps maps, const __grid_constant__ GroupArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sW = smem;
  uint8_t* sX = smem + C::OFF_X;
  float* turn = reinterpret_cast<float*>(smem + C::OFF_TURN);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* mma_drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool mma_cta = rank == 0;
  const int unit = blockIdx.x / 2, n_units = gridDim.x / 2;
  const int k_blocks = (args.K + C::BK - 1) / C::BK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * C::EPI_GROUPS * C::NUM_EPI_THREADS / 32);
    }
    mbar_init(mma_drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && elect_one()) {
    for (int i = 0; i < 8; ++i) tma_prefetch_desc(&maps.a[i]);
    tma_prefetch_desc(&maps.b);
    if constexpr (C::SWIGLU) tma_prefetch_desc(&maps.b2);
  }
  if (warp == 1) {
    tmem_alloc<2>(tmem_slot, C::TMEM_COLS);
    tmem_relinquish<2>();
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();  // the peer's barriers exist before anyone signals them
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;

  pdl_wait();
  pdl_launch_dependents();

  GroupWalk<C> walk(args);
  GroupTile tl;
  // rows of the tile as the MMA counts them
  auto height = [](const GroupTile& t) { return (t.row_end - t.row0 + 31) & ~31; };
  if (warp == 0) {
    // ------------------------------------------------------- TMA producer ----
    const uint64_t pol = l2_policy_evict_last();
    const uint32_t full0 = mapa_shared(smem_u32(full), 0);
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!walk.find(unit + k * n_units, tl)) break;
      if (elect_one()) {
        const int half = height(tl) / 2;  // each CTA brings half of the rows
        const int row0 = tl.row0 + rank * half;
        const CUtensorMap* xmap = &maps.a[half / 16 - 1];
        const int col0 = tl.n * C::OUT_COLS + rank * C::CTA_COLS;
        for (int kb = 0; kb < k_blocks; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, &g_status)) {
            ok = false;
            break;
          }
          uint8_t* w = sW + stage * C::W_BYTES;
          uint8_t* x = sX + stage * C::X_BYTES;
          const uint32_t bar = full0 + static_cast<uint32_t>(stage) * 8u;
          const int kx = kb * C::BK;
          if (mma_cta) mbar_arrive_expect_tx(&full[stage], 2 * (C::W_BYTES + half * 128));
          if constexpr (C::W_MN) {
#pragma unroll
            for (int i = 0; i < C::BM / 64; ++i)
              tma_load_3d_pair(w + i * C::MN_BOX_BYTES, &maps.b, bar, col0 + i * 64, kx, tl.e, pol);
          } else {
            tma_load_3d_pair(w, &maps.b, bar, kx, col0, tl.e, pol);
            if constexpr (C::SWIGLU)  // gate rows, then the same columns' up rows
              tma_load_3d_pair(w + C::B_BOX * 128, &maps.b2, bar, kx, col0, tl.e, pol);
          }
          tma_load_2d_pair(x, xmap, bar, kx, row0, pol);
          ++issued;
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (mma_cta && elect_one()) drain_ring(full, C::STAGES, issued, abort_flag);
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer ----
    if (mma_cta) {
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
          const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * C::TILE_M);
          const uint32_t idesc = C::IDESC | (static_cast<uint32_t>(height(tl)) >> 3) << 17;
          for (int kb = 0; ok && kb < k_blocks; ++kb) {
            if (!mbar_wait(&full[stage], phase, abort_flag, &g_status)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            const uint32_t w_s = smem_u32(sW + stage * C::W_BYTES);
            const uint64_t wdesc = C::W_MN ? sdesc_mnmajor_sw128(w_s, C::MN_BOX_BYTES) : sdesc_kmajor_sw128(w_s);
            const uint64_t xdesc = sdesc_kmajor_sw128(smem_u32(sX + stage * C::X_BYTES));
            constexpr uint64_t w_step = C::W_MN ? C::UMMA_K * 8u : 2u;
#pragma unroll
            for (int s = 0; s < C::K_STEPS; ++s)
              tc_mma<C::kKind, 2>(d_tmem, wdesc + w_step * s, xdesc + 2u * s, idesc, (kb | s) != 0);
            tc_commit<2>(&empty[stage], 3);
            if (++stage == C::STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (ok) tc_commit<2>(&acc_full[buf], 3);
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      if (elect_one()) {
        tc_commit<2>(mma_drain, 1);
        (void)mbar_wait(mma_drain, 0, abort_flag, &g_status, false);
      }
    }
  } else {
    // ----------------------------------------------------------- epilogue ----
    const int q = warp & 3;
    const int group = (warp - 2) >> 2;
    const int tid = (static_cast<int>(threadIdx.x) - 64) & 127;
    const uint32_t bar_id = 1 + group;
    const uint32_t acc_empty0 = mapa_shared(smem_u32(acc_empty), 0);
    // this thread's row of a chunk, and its first eight columns (the next ones 32 further)
    const int my_row = tid >> 2, my_col = (tid & 3) * 8;
    constexpr int kVecs = C::CTA_COLS / 32;
    const int64_t N = args.N;
    int flip = 0;
    for (int it = 0;; ++it) {
      if (!walk.find(unit + it * n_units, tl)) break;
      const int buf = it & 1;
      const uint32_t use = static_cast<uint32_t>(it >> 1) & 1u;
      const int chunks = height(tl) / C::CHUNK;
      const int col0 = tl.n * C::OUT_COLS + rank * C::CTA_COLS + my_col;
      float ws = 1.0f;
      if constexpr (!C::BWD)
        if (args.w_scale != nullptr) ws = args.w_scale[tl.e];
      // what a chunk needs beside the accumulator, on its way before it
      float sc = ws;
      [[maybe_unused]] uint4 gin[C::BWD ? kVecs : 1], uin[C::BWD ? kVecs : 1];
      auto fetch = [&](int c) {
        const int64_t row = tl.row0 + c * C::CHUNK + my_row;
        if (row >= tl.row_end) return;
        if constexpr (C::BWD) {
          const __nv_bfloat16* gu = args.GU + row * 2 * N + col0;
#pragma unroll
          for (int v = 0; v < kVecs; ++v) {
            if (col0 + v * 32 >= args.N) continue;
            gin[v] = __ldcs(reinterpret_cast<const uint4*>(gu + v * 32));
            uin[v] = __ldcs(reinterpret_cast<const uint4*>(gu + N + v * 32));
          }
        } else if (args.row_scale != nullptr) {
          sc = args.row_scale[row] * ws;
        }
      };
      fetch(group);
      if (!named_bar_and(bar_id, C::NUM_EPI_THREADS, mbar_wait(&acc_full[buf], use, abort_flag, &g_status))) break;
      tc_fence_after_sync();
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(buf * C::TILE_M);
      auto release_acc = [&]() {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty0 + static_cast<uint32_t>(buf) * 8u);
      };
      if (group >= chunks) release_acc();  // a low tile's only chunk is the first group's
#pragma unroll 1
      for (int c = group; c < chunks; c += C::EPI_GROUPS, flip ^= 1) {
        uint32_t t[32];
        tmem_ld32(t_row + c * C::CHUNK, t);
        tmem_wait_ld(t);
        if (c + C::EPI_GROUPS >= chunks) release_acc();
        float* box = turn + (C::EPI_GROUPS == 2 ? group : flip) * (C::TURN_BYTES / 4);
        if (C::EPI_GROUPS == 2 && c != group) named_bar_sync(bar_id, C::NUM_EPI_THREADS);  // the group's only box is read
#pragma unroll
        for (int i = 0; i < 32; ++i) box[i * C::PITCH + q * 32 + lane] = __uint_as_float(t[i]);
        // the other box is written after the next chunk's barrier, when every thread has read it
        named_bar_sync(bar_id, C::NUM_EPI_THREADS);
        const int64_t row = tl.row0 + c * C::CHUNK + my_row;
        const bool mine = row < tl.row_end;
        const float* src = box + my_row * C::PITCH + my_col;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
          const int col = col0 + v * 32;
          if (!mine || col >= args.N) continue;
          float x[8], u[C::SWIGLU ? 8 : 1];
          auto read8 = [](const float* p, float* out) {
            const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
            out[0] = a.x, out[1] = a.y, out[2] = a.z, out[3] = a.w, out[4] = b.x, out[5] = b.y, out[6] = b.z, out[7] = b.w;
          };
          read8(src + v * 32, x);
          if constexpr (C::SWIGLU) read8(src + C::CTA_COLS + v * 32, u);
          uint32_t w[4];
          [[maybe_unused]] uint32_t wg[4], wu[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 p = make_float2(x[2 * e], x[2 * e + 1]);
            if constexpr (C::BWD) {
              const uint32_t g2 = e == 0 ? gin[v].x : e == 1 ? gin[v].y : e == 2 ? gin[v].z : gin[v].w;
              const uint32_t u2 = e == 0 ? uin[v].x : e == 1 ? uin[v].y : e == 2 ? uin[v].z : uin[v].w;
              group_swiglu_grad(p, g2, u2, wg[e], wu[e]);
            } else if constexpr (C::SWIGLU) {
              const float2 s2 = make_float2(sc, sc);
              const float2 G = fmul2(p, s2);
              const float2 U = fmul2(make_float2(u[2 * e], u[2 * e + 1]), s2);
              const float2 o = fmul2(silu2(G), U);
              w[e] = pack_bf16x2(o.x, o.y);
              if constexpr (C::SAVE) {
                wg[e] = pack_bf16x2(G.x, G.y);
                wu[e] = pack_bf16x2(U.x, U.y);
              }
            } else {
              w[e] = pack_bf16x2(p.x * sc, p.y * sc);
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
        if (c + C::EPI_GROUPS < chunks) fetch(c + C::EPI_GROUPS);
      }
    }
  }

  // --------------------------------------------------------------- teardown ----
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc<2>(tmem_base, C::TMEM_COLS);
}

template <class C>
cudaError_t launch_wide_cfg(const GroupProblem& p, const char** msg) {
  constexpr CUtensorMapDataType in =
      C::kKind == kKindBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const uint64_t T = p.T, K = p.K, el = C::ELEM;
  WideMaps m = {};
  CUresult e = CUDA_SUCCESS;
  for (uint32_t i = 0; i < 8 && e == CUDA_SUCCESS; ++i)
    e = encode_tmap_2d(&m.a[i], in, p.A, K, T, K * el, C::BK, 16 * (i + 1));
  if (e == CUDA_SUCCESS) e = encode_group_weights<C>(&m, in, p);
  if (e != CUDA_SUCCESS) {
    *msg = "cuTensorMapEncodeTiled rejected an operand (pointer, stride or extent)";
    return cudaErrorInvalidValue;
  }
  auto kernel = grouped_wide_kernel<C>;
  int units = 0;
  cudaError_t ce = group_units<C, C::CG>(reinterpret_cast<const void*>(kernel), &units, msg);
  if (ce != cudaSuccess) return ce;
  const int64_t bound = group_tile_bound<C>(p);
  GroupArgs a = group_args<C>(p);
  void* kargs[] = {&m, &a};
  ce = launch_ex(reinterpret_cast<const void*>(kernel), dim3(2 * static_cast<unsigned>(bound < units ? bound : units)),
                 dim3(C::NUM_THREADS), C::SMEM_BYTES, p.stream, p.pdl, kargs, C::CG, false);
  if (ce != cudaSuccess) *msg = "grouped GEMM kernel launch failed";
  return ce;
}

}  // namespace coda
