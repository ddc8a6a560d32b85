// Declarations of the mixture-of-experts operators: products of rows grouped
// by expert (grouped_gemm.cuh, coda_grouped_*.cu), the router and the rows'
// way into expert order and back (coda_experts.cu), and the norm with the
// residual's addition (coda_norm.cu).  Kept apart from coda_internal.h: the
// GEMM and auxiliary kernels do not see them, and figures recorded for those
// stay valid when these change.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "coda_decode.h"
#include "coda_internal.h"

namespace coda {

// Largest number of experts, of choices of a row, and width of a norm's row.
constexpr int kMaxExperts = 1024;
constexpr int kMaxChoices = 32;
constexpr int kMaxNormWidth = 32768;
// Rows that the router takes (fewer): a block's rows, and a warp's next one, are counted in 32 bits past the last.
constexpr int64_t kMaxRouteRows = (int64_t(1) << 31) - (1 << 24);

// ------------------------------------------------------- grouped products ----
// Programs of the grouped GEMM.  Rows [offsets[e], offsets[e + 1]) of the
// T-row operands belong to expert e.
//   kGroupPlain     D = s (A . W_e^T), W [E, N, K]
//   kGroupPlainMN   D = s (A . W_e), W [E, K, N] (the data gradient's product)
//   kGroupSwiGLU    D = silu(s A Wg_e^T) * (s A Wu_e^T), W [E, 2 N, K]: gate rows, then up rows
//   kGroupSwiGLUSave  the same, and G || U [T, 2 N] stored
//   kGroupSwiGLUBwd   dAct = A . W_e, W [E, K, N]; dG || dU [T, 2 N] from G || U
//   kGroupWgrad     D[e] [N, K] = sum over the rows of e of A[row, n] B[row, k]
// with s the row's scale times the expert's.
enum GroupProgram {
  kGroupPlain = 0,
  kGroupPlainMN = 1,
  kGroupSwiGLU = 2,
  kGroupSwiGLUSave = 3,
  kGroupSwiGLUBwd = 4,
  kGroupWgrad = 5
};

struct GroupProblem {
  int program;
  const void* A;           // [T, K]; kGroupWgrad: dY [T, N]
  const void* W;           // weights; kGroupWgrad: X [T, K]
  void* D;                 // [T, N]; kGroupSwiGLUBwd: dG || dU; kGroupWgrad: [E, N, K]
  void* GU;                // G || U [T, 2 N]: written by kGroupSwiGLUSave, read by kGroupSwiGLUBwd
  const int32_t* offsets;  // [E + 1]
  const float* row_scale;  // [T], nullable
  const float* w_scale;    // [E], nullable
  int T, E, N, K;          // N: output columns (SwiGLU: of act)
  cudaStream_t stream;
  bool pdl;
};
cudaError_t launch_grouped_bf16(const GroupProblem& p, const char** msg);
cudaError_t launch_grouped_grad(const GroupProblem& p, const char** msg);  // kGroupPlainMN, kGroupSwiGLUBwd, kGroupWgrad
cudaError_t launch_grouped_e4m3(const GroupProblem& p, const char** msg);
unsigned read_clear_status_grouped_bf16();  // kDevTimeout of the waits
unsigned read_clear_status_grouped_grad();
unsigned read_clear_status_grouped_e4m3();
unsigned read_clear_index_grouped_bf16();  // kDevBadIndex: offsets out of order or beyond T
unsigned read_clear_index_grouped_grad();
unsigned read_clear_index_grouped_e4m3();

// Tensor map of `rank` dimensions (innermost first; strides of all but the
// innermost, in bytes), 128-byte swizzle.
CUresult encode_tmap(CUtensorMap* m, CUtensorMapDataType dt, uint32_t rank, const void* base, const uint64_t* dims,
                     const uint64_t* strides, const uint32_t* box);
// 3-D tensor map [outer][middle][inner], 128-byte swizzle; a box is
// box_inner x box_middle elements of one outer index.
CUresult encode_tmap_3d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t middle,
                        uint64_t outer, uint64_t row_bytes, uint64_t outer_bytes, uint32_t box_inner,
                        uint32_t box_middle);

// ------------------------------------------------------------- router ----
struct RouteParams {
  const void* logits;  // rows ld elements apart
  int64_t ld;
  int32_t* ids;        // [M, k]
  float* weights;      // [M, k]
  int32_t* slots;      // [M, k]
  int32_t* offsets;    // [E + 1]
  int32_t* counts;     // workspace [blocks, E]
  int M, E, k;
  int renormalize;
  int rows_per_block;  // set by the launcher
};
struct RouteGradParams {
  const void* logits;
  int64_t ld;
  const int32_t* ids;
  const float* weights;
  const float* dweights;
  void* dlogits;
  int64_t ldd;
  int M, E, k;
  int renormalize;
};
int64_t route_workspace_bytes(int64_t M, int64_t E, int64_t k);
cudaError_t launch_route(const RouteParams& p, bool f32, cudaStream_t s, bool pdl);
cudaError_t launch_route_backward(const RouteGradParams& p, bool f32, cudaStream_t s, bool pdl);

// --------------------------------------------- rows to and from experts ----
struct DispatchParams {
  const void* X;         // [M, row_bytes]
  const float* scale;    // [M], nullable
  const int32_t* slots;  // [M, k]
  void* Xs;              // [T, row_bytes]
  float* scale_s;        // [T], with scale
  int64_t row_bytes;
  int M, k, T;
};
struct CombineParams {
  const void* Y;         // [T, N]
  const int32_t* slots;  // [M, k]
  const float* weights;  // [M, k], nullable (1)
  const void* R;         // [M, N], nullable
  void* H;               // [M, N]
  float* P;              // [M, ceil(N / 128)], nullable
  int M, N, k, T;
};
struct CombineGradParams {
  const void* dH;  // [M, N]
  const void* Y;   // [T, N]
  const int32_t* slots;
  const float* weights;
  void* dY;         // [T, N]
  float* dweights;  // [M, k]
  int M, N, k, T;
};
cudaError_t launch_dispatch(const DispatchParams& p, cudaStream_t s, bool pdl);
int combine_blocks(int64_t N, bool f32);  // of a row
cudaError_t launch_combine(const CombineParams& p, bool f32, cudaStream_t s, bool pdl);
cudaError_t launch_combine_backward(const CombineGradParams& p, bool f32, cudaStream_t s, bool pdl);
unsigned read_clear_status_experts();  // kDevBadIndex: a slot out of range

// --------------------------------------------------------------- norm ----
struct NormParams {
  const void* X;  // rows ldx elements apart
  int64_t ldx;
  const void* R;  // rows ldr elements apart, nullable
  int64_t ldr;
  const float* gamma;  // [N]; null: no norm, X itself is quantised
  float eps;
  void* H;       // [M, N], nullable
  void* Y;       // [M, N], nullable
  uint8_t* Yq;   // [M, N] e4m3, nullable
  float* scale;  // [M], with Yq
  float* r;      // [M], nullable
  int M, N;
};
struct NormGradParams {
  const void* dY;
  const void* H;
  const float* r;
  const float* gamma;
  const void* dH_in;  // nullable
  void* dH;
  float* dgamma;
  float* part;  // workspace [blocks, N]
  int M, N;
};
cudaError_t launch_norm(const NormParams& p, bool f32, cudaStream_t s, bool pdl);
int64_t norm_backward_workspace_bytes(int64_t M, int64_t N);
cudaError_t launch_norm_backward(const NormGradParams& p, bool f32, cudaStream_t s, bool pdl);

}  // namespace coda
