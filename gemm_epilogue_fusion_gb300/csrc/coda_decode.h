// Declarations of the decode and scoring kernels (coda_paged.cu,
// coda_logprobs.cu), kept apart from coda_internal.h: the GEMM and auxiliary
// kernels do not see them, and figures recorded for those stay valid when
// these change.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "coda_internal.h"

namespace coda {

// Device status bit beside kDevTimeout.
constexpr unsigned kDevBadIndex = 2u;  // a page, sequence or token index read on the device was out of range

// Largest head_dim of the paged cache calls and largest number of
// alternatives of coda_logprobs.
constexpr int kMaxHeadDim = 256;
constexpr int kMaxTop = 64;

// Paged key/value cache kernels (coda_paged.cu).  Caches are [num_pages,
// kv_heads, page_size, head_dim]; row_seq null = row i belongs to sequence i.
struct AppendParams {
  const void* Z;  // [M, (q_heads + 2 kv_heads) head_dim]
  const int32_t* positions;
  const int32_t* row_seq;
  const int32_t* page_table;  // [num_seqs, max_pages]
  void* Q;                    // [M, q_heads, head_dim], nullable
  void* Kc;
  void* Vc;
  const float* scale_k;  // e4m3 caches: dequantisation scales, else null
  const float* scale_v;
  int64_t M;
  int num_seqs, max_pages, q_heads, kv_heads, head_dim, num_pages, page_size;
  int page_shift;  // log2(page_size), or -1
  int lanes, rows;  // heads of a row, and rows, that a block has side by side
  int parts;        // blocks that share a row's heads
  int rotate;
  // Pair j turns by turn[j] / 2^64 of a whole turn per position: base^(-2j/head_dim) / 2 pi
  uint64_t turn[kMaxHeadDim / 2];
};
struct AttnParams {
  const void* Q;  // rows ldq elements apart, [q_heads, head_dim] each
  int64_t ldq;
  const void* Kc;
  const void* Vc;
  const int32_t* page_table;
  const int32_t* lengths;  // [M] keys of each row
  const int32_t* row_seq;
  void* O;     // [M, q_heads, head_dim]
  float* lse;  // [M, q_heads], nullable
  const float* scale_k;
  const float* scale_v;
  void* workspace;
  float scale;
  int M, num_seqs, max_pages, q_heads, kv_heads, head_dim, num_pages, page_size;
  int page_shift;  // log2(page_size), or -1
};
cudaError_t launch_paged_append(const AppendParams& p, bool f32, bool e4m3, cudaStream_t s, bool pdl);
cudaError_t launch_paged_attention(const AttnParams& p, bool f32, bool e4m3, cudaStream_t s, bool pdl);
int64_t paged_attention_workspace_bytes(int q_heads, int kv_heads, int head_dim);
unsigned read_clear_status_paged();

// Log probabilities (coda_logprobs.cu): logits rows ld elements apart.
struct LogprobsParams {
  const void* logits;
  int64_t ld;
  const int32_t* targets;
  float* logp;
  float* entropy;   // nullable
  float* lse;       // nullable
  float* top_logp;  // [M, top]
  int32_t* top_ids;
  int V, top;
  int ranks;  // blocks that share a row (set by the launcher)
};
struct LogprobsGradParams {
  const void* logits;
  int64_t ld;
  const int32_t* targets;
  const float* lse;
  const float* entropy;   // nullable without dentropy
  const float* dlogp;     // nullable (= 0)
  const float* dentropy;  // nullable (= 0)
  void* dlogits;
  int64_t ldd;
  int V;
  int blocks;  // blocks of a row (set by the launcher)
};
cudaError_t launch_logprobs(const LogprobsParams& p, int64_t M, bool f32, cudaStream_t s, bool pdl);
cudaError_t launch_logprobs_backward(const LogprobsGradParams& p, int64_t M, bool f32, cudaStream_t s, bool pdl);
int64_t logprobs_backward_blocks(int64_t V, bool f32);
unsigned read_clear_status_logprobs();

}  // namespace coda
