// C ABI of the fused GEMM-epilogue library: argument validation, dispatch to
// the kernel translation units, error reporting.  Nothing here allocates or
// synchronises (except coda_get_device_status, which says so).
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cinttypes>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <utility>

#include "coda.h"
#include "coda_decode.h"
#include "coda_experts.h"
#include "coda_internal.h"

namespace coda {
// The failure-path self-test kernel's launcher (coda_aux.cu).
cudaError_t launch_wait_probe(int64_t timeout_ns, cudaStream_t s);
}  // namespace coda

namespace {

thread_local char g_msg[512] = "";
// Largest M that coda_block_swiglu_noalloc accepts (its counters are built in).
constexpr int kNoAllocMaxRows = 131072;

coda_status fail(coda_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
coda_status fail(coda_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return s;
}

coda_status cuda_fail(cudaError_t e, const char* what) {
  return fail(CODA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

int elem_bytes(coda_dtype d) { return d == CODA_F32 ? 4 : d == CODA_BF16 ? 2 : 1; }
// residual / output element size for GEMMs with this operand type
int out_bytes(coda_dtype d) { return d == CODA_F32 ? 4 : 2; }
bool valid_dtype(int d) { return d == CODA_F32 || d == CODA_BF16 || d == CODA_E4M3; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range {
  const char* name;
  uintptr_t lo, hi;  // [lo, hi)
};
Range rng(const char* name, const void* p, int64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {name, a, a + static_cast<uintptr_t>(bytes)};
}
bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

// Every output range against every input range and every other output.
coda_status check_overlaps(const Range* outs, int n_out, const Range* ins, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlap(outs[i], ins[j]))
        return fail(CODA_ERR_INVALID_ARG, "output %s overlaps input %s", outs[i].name, ins[j].name);
    for (int j = i + 1; j < n_out; ++j)
      if (overlap(outs[i], outs[j]))
        return fail(CODA_ERR_INVALID_ARG, "outputs %s and %s overlap", outs[i].name, outs[j].name);
  }
  return CODA_OK;
}

#define REQUIRE(cond, ...)                                 \
  do {                                                     \
    if (!(cond)) return fail(CODA_ERR_INVALID_ARG, __VA_ARGS__); \
  } while (0)

coda_status check_ptr(const void* p, const char* name) {
  if (p == nullptr) return fail(CODA_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned16(p)) return fail(CODA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  return CODA_OK;
}

coda_status check_scalar_ptr(const void* p, const char* name) {
  if (p == nullptr) return fail(CODA_ERR_INVALID_ARG, "%s is NULL", name);
  if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0) return fail(CODA_ERR_INVALID_ARG, "%s is not 4-byte aligned", name);
  return CODA_OK;
}

#define TRY(expr)                        \
  do {                                   \
    coda_status s_ = (expr);             \
    if (s_ != CODA_OK) return s_;        \
  } while (0)

// Byte extents of every operand of an M x N x K product must fit int64, and
// the kernels' tile indices are 32-bit: bound both at the smallest tile,
// 128 x 128 outputs.  M, N, K are already within [0, 2^31).
coda_status check_extents(int64_t M, int64_t N, int64_t K, const char* nname) {
  REQUIRE(M * N < (int64_t(1) << 60) && M * K < (int64_t(1) << 60) && N * K < (int64_t(1) << 60),
          "M = %" PRId64 ", %s = %" PRId64 ", K = %" PRId64 ": a matrix of 2^60 elements or more", M, nname, N, K);
  REQUIRE(((M + 127) / 128) * ((N + 127) / 128) < INT32_MAX / 2,
          "M = %" PRId64 ", %s = %" PRId64 ": too many output tiles for the kernels' 32-bit tile indices", M, nname, N);
  return CODA_OK;
}

// Shape rules common to the GEMM calls.
coda_status check_gemm_dims(int64_t M, int64_t N, int64_t K, coda_dtype dt, const char* nname) {
  REQUIRE(valid_dtype(dt), "unknown dtype %d", static_cast<int>(dt));
  REQUIRE(M >= 0 && M < INT32_MAX, "M = %" PRId64 " out of range [0, 2^31)", M);
  REQUIRE(N > 0 && N < INT32_MAX, "%s = %" PRId64 " out of range [1, 2^31)", nname, N);
  REQUIRE(K > 0 && K < INT32_MAX, "K = %" PRId64 " out of range [1, 2^31)", K);
  REQUIRE((K * elem_bytes(dt)) % 16 == 0, "K = %" PRId64 " must be a multiple of %d for this dtype (16-byte rows)", K,
          16 / elem_bytes(dt));
  REQUIRE((N * out_bytes(dt)) % 16 == 0, "%s = %" PRId64 " must be a multiple of %d for this dtype (16-byte rows)",
          nname, N, 16 / out_bytes(dt));
  return check_extents(M, N, K, nname);
}

coda_status check_scales(coda_dtype dt, const float* a, const char* an, const float* b, const char* bn,
                         const float* c = nullptr, const char* cn = nullptr) {
  if (dt == CODA_E4M3) {
    TRY(check_scalar_ptr(a, an));
    TRY(check_scalar_ptr(b, bn));
    if (cn) TRY(check_scalar_ptr(c, cn));
  } else {
    REQUIRE(a == nullptr && b == nullptr && c == nullptr, "FP8 scales must be NULL unless dtype is CODA_E4M3");
  }
  return CODA_OK;
}

coda_status run_gemm(coda_dtype dt, const coda::GemmProblem& p) {
  const char* msg = "";
  cudaError_t e;
  switch (dt) {
    case CODA_BF16: e = coda::launch_gemm_bf16(p, &msg); break;
    case CODA_F32: e = coda::launch_gemm_tf32(p, &msg); break;
    default: e = coda::launch_gemm_e4m3(p, &msg); break;
  }
  if (e != cudaSuccess) return cuda_fail(e, msg);
  return CODA_OK;
}

// Programmatic dependent launch (kernel prologues overlap the previous
// kernel's tail) is on unless CODA_NO_PDL is set in the environment.
bool use_pdl() {
  static const bool on = getenv("CODA_NO_PDL") == nullptr;
  return on;
}

coda_status zero_scalar(float* p, cudaStream_t s) {
  if (p == nullptr) return CODA_OK;
  cudaError_t e = cudaMemsetAsync(p, 0, sizeof(float), s);
  return e == cudaSuccess ? CODA_OK : cuda_fail(e, "cudaMemsetAsync(amax)");
}

}  // namespace

// ------------------------------------------------------------ host helpers ----
namespace coda {

int device_sm_count() {
  // host threads may ask at once: each slot is written with the same value
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 1;
  if (dev < 64) {
    const int c = cached[dev].load(std::memory_order_relaxed);
    if (c > 0) return c;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 1;
  if (dev < 64) cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

CUresult encode_tmap_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t outer,
                        uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return CUDA_ERROR_NOT_FOUND;
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

CUresult encode_tmap(CUtensorMap* m, CUtensorMapDataType dt, uint32_t rank, const void* base, const uint64_t* dims,
                     const uint64_t* strides, const uint32_t* box) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return CUDA_ERROR_NOT_FOUND;
  cuuint64_t d[5], st[4];
  cuuint32_t b[5], one[5] = {1, 1, 1, 1, 1};
  for (uint32_t i = 0; i < rank; ++i) d[i] = dims[i], b[i] = box[i];
  for (uint32_t i = 0; i + 1 < rank; ++i) st[i] = strides[i];
  return fn(m, dt, rank, const_cast<void*>(base), d, st, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

CUresult encode_tmap_3d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t middle,
                        uint64_t outer, uint64_t row_bytes, uint64_t outer_bytes, uint32_t box_inner,
                        uint32_t box_middle) {
  const uint64_t dims[3] = {inner, middle, outer}, strides[2] = {row_bytes, outer_bytes};
  const uint32_t box[3] = {box_inner, box_middle, 1};
  return encode_tmap(m, dt, 3, base, dims, strides, box);
}

cudaError_t launch_ex(const void* kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t s, bool pdl,
                      void** args, int cluster, bool cooperative) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[3];
  int n = 0;
  if (cooperative) {
    attr[n].id = cudaLaunchAttributeCooperative;
    attr[n].val.cooperative = 1;
    ++n;
  }
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

}  // namespace coda

// ------------------------------------------------------------------- ABI ----
extern "C" {

int coda_version(void) { return 100; }

const char* coda_status_string(coda_status s) {
  switch (s) {
    case CODA_OK: return "CODA_OK";
    case CODA_ERR_INVALID_ARG: return "CODA_ERR_INVALID_ARG";
    case CODA_ERR_UNSUPPORTED: return "CODA_ERR_UNSUPPORTED";
    case CODA_ERR_CUDA: return "CODA_ERR_CUDA";
    case CODA_ERR_TIMEOUT: return "CODA_ERR_TIMEOUT";
  }
  return "unknown coda_status";
}

const char* coda_last_error(void) { return g_msg; }

int64_t coda_partial_cols(int64_t N) {
  if (N <= 0) return -1;
  return (N + coda::kPartialCols - 1) / coda::kPartialCols;
}

coda_status coda_fold_gamma(const void* Wt, const float* gamma, void* Wt_out, int64_t N_out, int64_t K,
                            coda_dtype dtype, cudaStream_t stream) {
  g_msg[0] = 0;
  REQUIRE(dtype == CODA_F32 || dtype == CODA_BF16, "coda_fold_gamma: dtype must be CODA_F32 or CODA_BF16");
  REQUIRE(N_out >= 0 && K > 0 && N_out < INT32_MAX && K < INT32_MAX && N_out * K < (int64_t(1) << 60),
          "coda_fold_gamma: bad shape");
  REQUIRE((K * elem_bytes(dtype)) % 16 == 0, "coda_fold_gamma: K must give 16-byte rows");
  if (N_out == 0) return CODA_OK;
  TRY(check_ptr(Wt, "Wt"));
  TRY(check_ptr(gamma, "gamma"));
  TRY(check_ptr(Wt_out, "Wt_out"));
  const int64_t wb = N_out * K * elem_bytes(dtype);
  const Range outs[] = {rng("Wt_out", Wt_out, wb)};
  const Range ins[] = {rng("Wt", Wt, wb), rng("gamma", gamma, K * 4)};
  TRY(check_overlaps(outs, 1, ins, 2));
  cudaError_t e = coda::launch_fold_gamma(Wt, gamma, Wt_out, N_out, K, dtype == CODA_F32, stream);
  return e == cudaSuccess ? CODA_OK : cuda_fail(e, "coda_fold_gamma launch");
}

coda_status coda_gemm_residual_partial_rms(const void* X, const void* W1t, const void* R, void* H, float* P,
                                           int64_t M, int64_t N, int64_t K, coda_dtype dtype,
                                           const float* scale_x, const float* scale_w, float* amax_h,
                                           cudaStream_t stream) {
  g_msg[0] = 0;
  TRY(check_gemm_dims(M, N, K, dtype, "N"));
  TRY(check_scales(dtype, scale_x, "scale_x", scale_w, "scale_w"));
  if (amax_h) TRY(check_scalar_ptr(amax_h, "amax_h"));
  if (M == 0) return zero_scalar(amax_h, stream);
  TRY(check_ptr(X, "X"));
  TRY(check_ptr(W1t, "W1t"));
  TRY(check_ptr(R, "R"));
  TRY(check_ptr(H, "H"));
  TRY(check_ptr(P, "P"));
  const int64_t T = coda_partial_cols(N);
  const int ob = out_bytes(dtype), ib = elem_bytes(dtype);
  const Range outs[] = {rng("H", H, M * N * ob), rng("P", P, M * T * 4), rng("amax_h", amax_h, amax_h ? 4 : 0)};
  const Range ins[] = {rng("X", X, M * K * ib), rng("W1t", W1t, N * K * ib), rng("R", R, M * N * ob),
                       rng("scale_x", scale_x, scale_x ? 4 : 0), rng("scale_w", scale_w, scale_w ? 4 : 0)};
  TRY(check_overlaps(outs, 3, ins, 5));
  TRY(zero_scalar(amax_h, stream));
  coda::GemmProblem p = {};
  p.epi = coda::kEpiResidualPartialRms;
  p.A = X;
  p.B = W1t;
  p.R = R;
  p.D = H;
  p.M = static_cast<int>(M);
  p.N_out = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.ep.P = P;
  p.ep.T = static_cast<int>(T);
  p.ep.scale_a = scale_x;
  p.ep.scale_b = scale_w;
  p.ep.amax_out = amax_h;
  p.stream = stream;
  p.pdl = use_pdl();
  return run_gemm(dtype, p);
}

coda_status coda_rms_reduce(const float* P, int64_t M, int64_t N, float eps, float* r, cudaStream_t stream) {
  g_msg[0] = 0;
  REQUIRE(M >= 0 && M < INT32_MAX, "coda_rms_reduce: M out of range");
  REQUIRE(N > 0 && N < INT32_MAX, "coda_rms_reduce: N out of range");
  REQUIRE(std::isfinite(eps) && eps >= 0.0f, "coda_rms_reduce: eps must be finite and >= 0");
  if (M == 0) return CODA_OK;
  TRY(check_ptr(P, "P"));
  TRY(check_ptr(r, "r"));
  const int64_t T = coda_partial_cols(N);
  const Range outs[] = {rng("r", r, M * 4)};
  const Range ins[] = {rng("P", P, M * T * 4)};
  TRY(check_overlaps(outs, 1, ins, 1));
  cudaError_t e = coda::launch_rms_reduce(P, M, static_cast<int>(T), N, eps, r, stream, use_pdl());
  return e == cudaSuccess ? CODA_OK : cuda_fail(e, "coda_rms_reduce launch");
}

}  // extern "C"

namespace {

// RoPE arguments of the row-scale program.
struct RopeArgs {
  int64_t head_dim, rope_cols;
  double base;
  int64_t seq_len;
  const int32_t* positions;
};

// Checks of the RoPE arguments of a row-scale program with N2 output columns.
coda_status check_rope(const RopeArgs* rope, int64_t M, int64_t N2, coda_dtype dtype) {
  const int64_t chunk = 16 / out_bytes(dtype);  // columns per 16-byte store chunk
  REQUIRE(rope->head_dim > 0 && rope->head_dim % chunk == 0,
          "head_dim must be a positive multiple of %" PRId64 " for this dtype", chunk);
  REQUIRE(rope->rope_cols >= 0 && rope->rope_cols <= N2 && rope->rope_cols % rope->head_dim == 0,
          "rope_cols must be a multiple of head_dim within [0, N2]");
  REQUIRE(std::isfinite(rope->base) && rope->base > 1.0, "base must be finite and > 1");
  REQUIRE(rope->positions != nullptr || (rope->seq_len > 0 && rope->seq_len < INT32_MAX),
          "seq_len must be in [1, 2^31) when positions is NULL");
  if (M > 0 && rope->positions) TRY(check_scalar_ptr(rope->positions, "positions"));
  return CODA_OK;
}

// The RoPE fields of a row-scale program's epilogue.
void set_rope(coda::EpiParams& ep, const RopeArgs* rope) {
  if (rope == nullptr || rope->rope_cols <= 0) return;
  ep.rope_pos = rope->positions;
  ep.rope_seq = static_cast<int>(rope->positions ? 1 : rope->seq_len);
  ep.rope_half = static_cast<int>(rope->head_dim / 2);
  ep.rope_cols = static_cast<int>(rope->rope_cols);
  ep.rope_log2b = static_cast<float>(std::log2(rope->base) / static_cast<double>(rope->head_dim / 2));
}

// Shared by the row-scale calls: r given, or reduced in the epilogue from P;
// optionally RoPE on the leading columns.
coda_status gemm_rowscale_impl(const void* H, const void* W2t, const float* r, const float* P, float eps,
                               float* r_out, void* Z, int64_t M, int64_t N2, int64_t K, coda_dtype dtype,
                               const float* scale_h, const float* scale_w, cudaStream_t stream,
                               const RopeArgs* rope = nullptr) {
  g_msg[0] = 0;
  if (rope) TRY(check_rope(rope, M, N2, dtype));
  TRY(check_gemm_dims(M, N2, K, dtype, "N2"));
  TRY(check_scales(dtype, scale_h, "scale_h", scale_w, "scale_w"));
  if (P) REQUIRE(std::isfinite(eps) && eps >= 0.0f, "eps must be finite and >= 0");
  if (M == 0) return CODA_OK;
  TRY(check_ptr(H, "H"));
  TRY(check_ptr(W2t, "W2t"));
  TRY(check_ptr(Z, "Z"));
  if (P) {
    TRY(check_ptr(P, "P"));
    if (r_out) TRY(check_scalar_ptr(r_out, "r_out"));
  } else {
    TRY(check_ptr(r, "r"));
  }
  const int ob = out_bytes(dtype), ib = elem_bytes(dtype);
  const int64_t T = coda_partial_cols(K);
  const Range outs[] = {rng("Z", Z, M * N2 * ob), rng("r_out", r_out, r_out ? M * 4 : 0)};
  const Range ins[] = {rng("H", H, M * K * ib), rng("W2t", W2t, N2 * K * ib), rng("r", r, r ? M * 4 : 0),
                       rng("P", P, P ? M * T * 4 : 0), rng("scale_h", scale_h, scale_h ? 4 : 0),
                       rng("scale_w", scale_w, scale_w ? 4 : 0),
                       rng("positions", rope ? rope->positions : nullptr, rope && rope->positions ? M * 4 : 0)};
  TRY(check_overlaps(outs, 2, ins, 7));
  coda::GemmProblem p = {};
  p.epi = coda::kEpiRowScale;
  p.A = H;
  p.B = W2t;
  p.D = Z;
  p.M = static_cast<int>(M);
  p.N_out = static_cast<int>(N2);
  p.K = static_cast<int>(K);
  p.ep.r = P ? nullptr : r;
  p.ep.P_in = P;
  p.ep.T_in = static_cast<int>(T);
  p.ep.n_norm = static_cast<float>(K);
  p.ep.eps = eps;
  p.ep.r_out = P ? r_out : nullptr;
  p.ep.scale_a = scale_h;
  p.ep.scale_b = scale_w;
  set_rope(p.ep, rope);
  p.stream = stream;
  p.pdl = use_pdl();
  return run_gemm(dtype, p);
}

// Shared by the SwiGLU calls.
coda_status gemm_swiglu_impl(const void* H, const void* Wgt, const void* Wut, const float* r, const float* P,
                             float eps, float* r_out, void* Act, int64_t M, int64_t I, int64_t K, coda_dtype dtype,
                             const float* scale_h, const float* scale_wg, const float* scale_wu, float* amax_act,
                             cudaStream_t stream) {
  g_msg[0] = 0;
  TRY(check_gemm_dims(M, I, K, dtype, "I"));
  TRY(check_scales(dtype, scale_h, "scale_h", scale_wg, "scale_wg", scale_wu, "scale_wu"));
  if (P) REQUIRE(std::isfinite(eps) && eps >= 0.0f, "eps must be finite and >= 0");
  if (amax_act) TRY(check_scalar_ptr(amax_act, "amax_act"));
  if (M == 0) return zero_scalar(amax_act, stream);
  TRY(check_ptr(H, "H"));
  TRY(check_ptr(Wgt, "Wgt"));
  TRY(check_ptr(Wut, "Wut"));
  if (P) {
    TRY(check_ptr(P, "P"));
    if (r_out) TRY(check_scalar_ptr(r_out, "r_out"));
  } else if (r) {
    TRY(check_scalar_ptr(r, "r"));
  }
  TRY(check_ptr(Act, "Act"));
  const int ob = out_bytes(dtype), ib = elem_bytes(dtype);
  const int64_t T = coda_partial_cols(K);
  const Range outs[] = {rng("Act", Act, M * I * ob), rng("amax_act", amax_act, amax_act ? 4 : 0),
                        rng("r_out", r_out, r_out ? M * 4 : 0)};
  const Range ins[] = {rng("H", H, M * K * ib),
                       rng("Wgt", Wgt, I * K * ib),
                       rng("Wut", Wut, I * K * ib),
                       rng("r", r, r ? M * 4 : 0),
                       rng("P", P, P ? M * T * 4 : 0),
                       rng("scale_h", scale_h, scale_h ? 4 : 0),
                       rng("scale_wg", scale_wg, scale_wg ? 4 : 0),
                       rng("scale_wu", scale_wu, scale_wu ? 4 : 0)};
  TRY(check_overlaps(outs, 3, ins, 8));
  TRY(zero_scalar(amax_act, stream));
  coda::GemmProblem p = {};
  p.epi = coda::kEpiSwiGLU;
  p.A = H;
  p.B = Wgt;
  p.B2 = Wut;
  p.D = Act;
  p.M = static_cast<int>(M);
  p.N_out = static_cast<int>(I);
  p.K = static_cast<int>(K);
  p.ep.r = P ? nullptr : r;
  p.ep.P_in = P;
  p.ep.T_in = static_cast<int>(T);
  p.ep.n_norm = static_cast<float>(K);
  p.ep.eps = eps;
  p.ep.r_out = P ? r_out : nullptr;
  p.ep.scale_a = scale_h;
  p.ep.scale_b = scale_wg;
  p.ep.scale_b2 = scale_wu;
  p.ep.amax_out = amax_act;
  p.stream = stream;
  p.pdl = use_pdl();
  return run_gemm(dtype, p);
}

}  // namespace

extern "C" {

coda_status coda_gemm_rowscale(const void* H, const void* W2t, const float* r, void* Z, int64_t M, int64_t N2,
                               int64_t K, coda_dtype dtype, const float* scale_h, const float* scale_w,
                               cudaStream_t stream) {
  if (r == nullptr && M > 0) {
    g_msg[0] = 0;
    return fail(CODA_ERR_INVALID_ARG, "r is NULL");
  }
  return gemm_rowscale_impl(H, W2t, r, nullptr, 0.0f, nullptr, Z, M, N2, K, dtype, scale_h, scale_w, stream);
}

coda_status coda_gemm_rowscale_fused_rms(const void* H, const void* W2t, const float* P, float eps, float* r_out,
                                         void* Z, int64_t M, int64_t N2, int64_t K, coda_dtype dtype,
                                         const float* scale_h, const float* scale_w, cudaStream_t stream) {
  if (P == nullptr && M > 0) {
    g_msg[0] = 0;
    return fail(CODA_ERR_INVALID_ARG, "P is NULL");
  }
  return gemm_rowscale_impl(H, W2t, nullptr, P, eps, r_out, Z, M, N2, K, dtype, scale_h, scale_w, stream);
}

coda_status coda_gemm_rowscale_rope(const void* H, const void* W2t, const float* r, const float* P, float eps,
                                    float* r_out, void* Z, int64_t M, int64_t N2, int64_t K, coda_dtype dtype,
                                    const float* scale_h, const float* scale_w, int64_t head_dim, int64_t rope_cols,
                                    double base, int64_t seq_len, const int32_t* positions, cudaStream_t stream) {
  if (M > 0 && (r == nullptr) == (P == nullptr)) {
    g_msg[0] = 0;
    return fail(CODA_ERR_INVALID_ARG, "exactly one of r and P must be given");
  }
  const RopeArgs rope = {head_dim, rope_cols, base, seq_len, positions};
  return gemm_rowscale_impl(H, W2t, P ? nullptr : r, P, eps, P ? r_out : nullptr, Z, M, N2, K, dtype, scale_h,
                            scale_w, stream, &rope);
}

coda_status coda_gemm_swiglu(const void* H, const void* Wgt, const void* Wut, const float* r, void* Act, int64_t M,
                             int64_t I, int64_t K, coda_dtype dtype, const float* scale_h, const float* scale_wg,
                             const float* scale_wu, float* amax_act, cudaStream_t stream) {
  return gemm_swiglu_impl(H, Wgt, Wut, r, nullptr, 0.0f, nullptr, Act, M, I, K, dtype, scale_h, scale_wg, scale_wu,
                          amax_act, stream);
}

coda_status coda_gemm_swiglu_fused_rms(const void* H, const void* Wgt, const void* Wut, const float* P, float eps,
                                       float* r_out, void* Act, int64_t M, int64_t I, int64_t K, coda_dtype dtype,
                                       const float* scale_h, const float* scale_wg, const float* scale_wu,
                                       float* amax_act, cudaStream_t stream) {
  if (P == nullptr && M > 0) {
    g_msg[0] = 0;
    return fail(CODA_ERR_INVALID_ARG, "P is NULL");
  }
  return gemm_swiglu_impl(H, Wgt, Wut, nullptr, P, eps, r_out, Act, M, I, K, dtype, scale_h, scale_wg, scale_wu,
                          amax_act, stream);
}

coda_status coda_gemm(const void* A, coda_layout a_layout, const void* B, coda_layout b_layout, void* D, int64_t M,
                      int64_t N, int64_t K, coda_dtype dtype, const float* row_scale, const float* col_scale,
                      cudaStream_t stream) {
  g_msg[0] = 0;
  REQUIRE(dtype == CODA_F32 || dtype == CODA_BF16, "coda_gemm: dtype must be CODA_F32 or CODA_BF16");
  REQUIRE((a_layout == CODA_K_MAJOR || a_layout == CODA_MN_MAJOR) && (b_layout == CODA_K_MAJOR || b_layout == CODA_MN_MAJOR),
          "unknown layout");
  const bool a_mn = a_layout == CODA_MN_MAJOR, b_mn = b_layout == CODA_MN_MAJOR;
  REQUIRE(!(a_mn || b_mn) || dtype == CODA_BF16, "MN-major operands are bf16 only");
  REQUIRE(!(a_mn && !b_mn), "an MN-major A needs an MN-major B");
  REQUIRE(M >= 0 && M < INT32_MAX && N > 0 && N < INT32_MAX && K > 0 && K < INT32_MAX, "bad shape");
  TRY(check_extents(M, N, K, "N"));
  const int eb = elem_bytes(dtype), ob = out_bytes(dtype);
  REQUIRE(((a_mn ? M : K) * eb) % 16 == 0, "A's rows must be a multiple of 16 bytes");
  REQUIRE(((b_mn ? N : K) * eb) % 16 == 0, "B's rows must be a multiple of 16 bytes");
  REQUIRE((N * ob) % 16 == 0, "D's rows must be a multiple of 16 bytes");
  if (M == 0) return CODA_OK;
  TRY(check_ptr(A, "A"));
  TRY(check_ptr(B, "B"));
  TRY(check_ptr(D, "D"));
  if (row_scale) TRY(check_scalar_ptr(row_scale, "row_scale"));
  if (col_scale) TRY(check_scalar_ptr(col_scale, "col_scale"));
  const Range outs[] = {rng("D", D, M * N * ob)};
  const Range ins[] = {rng("A", A, M * K * eb), rng("B", B, N * K * eb),
                       rng("row_scale", row_scale, row_scale ? M * 4 : 0),
                       rng("col_scale", col_scale, col_scale ? N * 4 : 0)};
  TRY(check_overlaps(outs, 1, ins, 4));
  coda::GemmProblem p = {};
  p.epi = coda::kEpiRowScale;
  p.A = A;
  p.B = B;
  p.D = D;
  p.M = static_cast<int>(M);
  p.N_out = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.ep.r = row_scale;
  p.ep.col_scale = col_scale;
  p.a_mn = a_mn;
  p.b_mn = b_mn;
  p.stream = stream;
  p.pdl = use_pdl();
  return run_gemm(dtype, p);
}

coda_status coda_gemm_grad_norm(const void* dOut, const void* Wt, const void* H, const float* gamma, void* dY,
                                float* S, int64_t M, int64_t N, int64_t K, coda_dtype dtype, cudaStream_t stream) {
  g_msg[0] = 0;
  REQUIRE(dtype == CODA_BF16, "coda_gemm_grad_norm: dtype must be CODA_BF16");
  TRY(check_gemm_dims(M, N, K, dtype, "N"));
  if (M == 0) return CODA_OK;
  TRY(check_ptr(dOut, "dOut"));
  TRY(check_ptr(Wt, "Wt"));
  TRY(check_ptr(H, "H"));
  TRY(check_ptr(gamma, "gamma"));
  TRY(check_ptr(dY, "dY"));
  TRY(check_ptr(S, "S"));
  const int64_t T = coda_partial_cols(N);
  const Range outs[] = {rng("dY", dY, M * N * 2), rng("S", S, M * T * 4)};
  const Range ins[] = {rng("dOut", dOut, M * K * 2), rng("Wt", Wt, K * N * 2), rng("H", H, M * N * 2),
                       rng("gamma", gamma, N * 4)};
  TRY(check_overlaps(outs, 2, ins, 4));
  coda::GemmProblem p = {};
  p.epi = coda::kEpiGradNorm;
  p.A = dOut;
  p.B = Wt;
  p.R = H;
  p.D = dY;
  p.M = static_cast<int>(M);
  p.N_out = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.ep.P = S;
  p.ep.T = static_cast<int>(T);
  p.ep.col_scale = gamma;
  p.b_mn = true;
  p.stream = stream;
  p.pdl = use_pdl();
  return run_gemm(dtype, p);
}

int64_t coda_rmsnorm_backward_workspace_bytes(int64_t M, int64_t N) {
  if (M < 0 || N <= 0) return -1;
  return coda::rmsnorm_bwd_chunks(M) * N * static_cast<int64_t>(sizeof(float));
}

coda_status coda_rmsnorm_backward(const void* dY, const void* H, const float* r, const float* gamma, const float* S,
                                  const void* dH_in, void* dH, void* Yt, float* dgamma, float* workspace, int64_t M,
                                  int64_t N, cudaStream_t stream) {
  g_msg[0] = 0;
  REQUIRE(M >= 0 && M < INT32_MAX && N > 0 && N < INT32_MAX && N % 8 == 0 && M * N < (int64_t(1) << 60),
          "coda_rmsnorm_backward: M in [0, 2^31), N a positive multiple of 8, M N below 2^60");
  if (M == 0) {
    TRY(check_scalar_ptr(dgamma, "dgamma"));
    cudaError_t e = cudaMemsetAsync(dgamma, 0, static_cast<size_t>(N) * sizeof(float), stream);
    return e == cudaSuccess ? CODA_OK : cuda_fail(e, "cudaMemsetAsync(dgamma)");
  }
  for (const auto& pr : {std::make_pair(dY, "dY"), std::make_pair(H, "H"), std::make_pair(static_cast<const void*>(dH), "dH"),
                         std::make_pair(static_cast<const void*>(Yt), "Yt"), std::make_pair(static_cast<const void*>(gamma), "gamma"),
                         std::make_pair(static_cast<const void*>(dgamma), "dgamma"),
                         std::make_pair(static_cast<const void*>(workspace), "workspace")})
    TRY(check_ptr(pr.first, pr.second));
  TRY(check_scalar_ptr(r, "r"));
  TRY(check_scalar_ptr(S, "S"));
  if (dH_in) TRY(check_ptr(dH_in, "dH_in"));
  const int64_t T = coda_partial_cols(N);
  const int64_t mn = M * N * 2;
  const Range outs[] = {rng("dH", dH, mn), rng("Yt", Yt, mn), rng("dgamma", dgamma, N * 4),
                        rng("workspace", workspace, coda_rmsnorm_backward_workspace_bytes(M, N))};
  const Range ins[] = {rng("dY", dY, mn), rng("H", H, mn), rng("r", r, M * 4), rng("gamma", gamma, N * 4),
                       rng("S", S, M * T * 4), rng("dH_in", dH_in, dH_in ? mn : 0)};
  TRY(check_overlaps(outs, 4, ins, 6));
  cudaError_t e = coda::launch_rmsnorm_backward(dY, H, r, gamma, S, static_cast<int>(T), dH_in, dH, Yt, dgamma,
                                                workspace, M, N, stream);
  return e == cudaSuccess ? CODA_OK : cuda_fail(e, "coda_rmsnorm_backward launch");
}

coda_status coda_gemm_swiglu_save(const void* H, const void* Wgt, const void* Wut, const float* r, const float* P,
                                  float eps, float* r_out, void* Act, void* GU, int64_t M, int64_t I, int64_t K,
                                  coda_dtype dtype, cudaStream_t stream) {
  g_msg[0] = 0;
  REQUIRE(dtype == CODA_BF16, "coda_gemm_swiglu_save: dtype must be CODA_BF16");
  // a 64-column box of the G half must not reach into the U half
  REQUIRE(I % 64 == 0, "coda_gemm_swiglu_save: I must be a multiple of 64");
  REQUIRE(M <= 0 || (r == nullptr) != (P == nullptr), "exactly one of r and P must be given");
  TRY(check_gemm_dims(M, I, K, dtype, "I"));
  if (P) REQUIRE(std::isfinite(eps) && eps >= 0.0f, "eps must be finite and >= 0");
  if (M == 0) return CODA_OK;
  TRY(check_ptr(H, "H"));
  TRY(check_ptr(Wgt, "Wgt"));
  TRY(check_ptr(Wut, "Wut"));
  TRY(check_ptr(Act, "Act"));
  TRY(check_ptr(GU, "GU"));
  if (P) TRY(check_ptr(P, "P"));
  else TRY(check_scalar_ptr(r, "r"));
  if (r_out) TRY(check_scalar_ptr(r_out, "r_out"));
  const int64_t T = coda_partial_cols(K);
  const Range outs[] = {rng("Act", Act, M * I * 2), rng("GU", GU, M * 2 * I * 2),
                        rng("r_out", r_out, (P && r_out) ? M * 4 : 0)};
  const Range ins[] = {rng("H", H, M * K * 2), rng("Wgt", Wgt, I * K * 2), rng("Wut", Wut, I * K * 2),
                       rng("r", r, r ? M * 4 : 0), rng("P", P, P ? M * T * 4 : 0)};
  TRY(check_overlaps(outs, 3, ins, 5));
  coda::GemmProblem p = {};
  p.epi = coda::kEpiSwiGLUSave;
  p.A = H;
  p.B = Wgt;
  p.B2 = Wut;
  p.D = Act;
  p.GU = GU;
  p.M = static_cast<int>(M);
  p.N_out = static_cast<int>(I);
  p.K = static_cast<int>(K);
  p.ep.r = P ? nullptr : r;
  p.ep.P_in = P;
  p.ep.T_in = static_cast<int>(T);
  p.ep.n_norm = static_cast<float>(K);
  p.ep.eps = eps;
  p.ep.r_out = P ? r_out : nullptr;
  p.ep.gu_off = static_cast<int>(I);
  p.stream = stream;
  p.pdl = use_pdl();
  return run_gemm(dtype, p);
}

coda_status coda_gemm_swiglu_backward(const void* dOut, const void* Wt, const void* GU, void* dGU, int64_t M,
                                      int64_t I, int64_t K, coda_dtype dtype, cudaStream_t stream) {
  g_msg[0] = 0;
  REQUIRE(dtype == CODA_BF16, "coda_gemm_swiglu_backward: dtype must be CODA_BF16");
  REQUIRE(I % 64 == 0, "coda_gemm_swiglu_backward: I must be a multiple of 64");
  TRY(check_gemm_dims(M, I, K, dtype, "I"));
  if (M == 0) return CODA_OK;
  TRY(check_ptr(dOut, "dOut"));
  TRY(check_ptr(Wt, "Wt"));
  TRY(check_ptr(GU, "GU"));
  TRY(check_ptr(dGU, "dGU"));
  const Range outs[] = {rng("dGU", dGU, M * 2 * I * 2)};
  const Range ins[] = {rng("dOut", dOut, M * K * 2), rng("Wt", Wt, K * I * 2), rng("GU", GU, M * 2 * I * 2)};
  TRY(check_overlaps(outs, 1, ins, 3));
  coda::GemmProblem p = {};
  p.epi = coda::kEpiSwiGLUBwd;
  p.A = dOut;
  p.B = Wt;
  p.R = GU;
  p.D = dGU;
  p.M = static_cast<int>(M);
  p.N_out = static_cast<int>(I);
  p.K = static_cast<int>(K);
  p.ep.gu_off = static_cast<int>(I);
  p.b_mn = true;
  p.stream = stream;
  p.pdl = use_pdl();
  return run_gemm(dtype, p);
}

int64_t coda_block_workspace_bytes(int64_t M) {
  if (M < 0) return -1;
  return ((M + 127) / 128 + 1) * static_cast<int64_t>(sizeof(unsigned));
}

}  // extern "C"

namespace {

// Shared by the one-launch blocks: residual GEMM (phase A) and its consumer
// (phase B) with the reduction folded into the consumer's epilogue.  Checks
// every argument and fills *p; enqueues nothing.  M == 0 leaves p->M at 0
// (nothing to launch).
coda_status block_prepare(int epi_b, const void* X, const void* W1t, const void* R, const void* Wb, const void* Wb2,
                          float eps, void* H, float* P, float* r_out, void* Out, int64_t M, int64_t N, int64_t K,
                          int64_t N_out, coda_dtype dtype, void* workspace, cudaStream_t stream,
                          coda::GemmProblem* pp) {
  g_msg[0] = 0;
  *pp = coda::GemmProblem{};
  if (dtype == CODA_E4M3)
    return fail(CODA_ERR_UNSUPPORTED,
                "one-launch blocks take CODA_F32 or CODA_BF16: FP8 needs the per-tensor amax of h before its consumer");
  TRY(check_gemm_dims(M, N, K, dtype, "N"));
  TRY(check_gemm_dims(M, N_out, N, dtype, epi_b == coda::kEpiSwiGLU ? "I" : "N2"));
  REQUIRE(std::isfinite(eps) && eps >= 0.0f, "eps must be finite and >= 0");
  if (M == 0) return CODA_OK;
  TRY(check_ptr(X, "X"));
  TRY(check_ptr(W1t, "W1t"));
  TRY(check_ptr(R, "R"));
  TRY(check_ptr(Wb, epi_b == coda::kEpiSwiGLU ? "Wgt" : "W2t"));
  if (epi_b == coda::kEpiSwiGLU) TRY(check_ptr(Wb2, "Wut"));
  TRY(check_ptr(H, "H"));
  TRY(check_ptr(P, "P"));
  if (r_out) TRY(check_scalar_ptr(r_out, "r_out"));
  TRY(check_ptr(Out, epi_b == coda::kEpiSwiGLU ? "Act" : "Z"));
  TRY(check_ptr(workspace, "workspace"));
  const int ob = out_bytes(dtype), ib = elem_bytes(dtype);
  const int64_t T = coda_partial_cols(N);
  const Range outs[] = {rng("H", H, M * N * ob), rng("P", P, M * T * 4), rng("r_out", r_out, r_out ? M * 4 : 0),
                        rng(epi_b == coda::kEpiSwiGLU ? "Act" : "Z", Out, M * N_out * ob),
                        rng("workspace", workspace, coda_block_workspace_bytes(M))};
  const Range ins[] = {rng("X", X, M * K * ib), rng("W1t", W1t, N * K * ib), rng("R", R, M * N * ob),
                       rng("W", Wb, N_out * N * ib), rng("Wut", Wb2, Wb2 ? N_out * N * ib : 0)};
  TRY(check_overlaps(outs, 5, ins, 5));
  coda::GemmProblem& p = *pp;
  p.epi = coda::kEpiResidualPartialRms;
  p.A = X;
  p.B = W1t;
  p.R = R;
  p.D = H;
  p.M = static_cast<int>(M);
  p.N_out = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.ep.P = P;
  p.ep.T = static_cast<int>(T);
  p.b.epi = epi_b;
  p.b.A = H;
  p.b.B = Wb;
  p.b.B2 = Wb2;
  p.b.D = Out;
  p.b.N_out = static_cast<int>(N_out);
  p.b.K = static_cast<int>(N);
  p.b.ep.P_in = P;
  p.b.ep.T_in = static_cast<int>(T);
  p.b.ep.n_norm = static_cast<float>(N);
  p.b.ep.eps = eps;
  p.b.ep.r_out = r_out;
  p.band_ready = static_cast<unsigned*>(workspace);
  p.stream = stream;
  p.pdl = use_pdl();
  return CODA_OK;
}

coda_status block_impl(int epi_b, const void* X, const void* W1t, const void* R, const void* Wb, const void* Wb2,
                       float eps, void* H, float* P, float* r_out, void* Out, int64_t M, int64_t N, int64_t K,
                       int64_t N_out, coda_dtype dtype, void* workspace, cudaStream_t stream) {
  coda::GemmProblem p;
  TRY(block_prepare(epi_b, X, W1t, R, Wb, Wb2, eps, H, P, r_out, Out, M, N, K, N_out, dtype, workspace, stream, &p));
  if (p.M == 0) return CODA_OK;
  return run_gemm(dtype, p);
}

}  // namespace

extern "C" {

coda_status coda_block_rowscale(const void* X, const void* W1t, const void* R, const void* W2t, float eps, void* H,
                                float* P, float* r_out, void* Z, int64_t M, int64_t N, int64_t K, int64_t N2,
                                coda_dtype dtype, void* workspace, cudaStream_t stream) {
  return block_impl(coda::kEpiRowScale, X, W1t, R, W2t, nullptr, eps, H, P, r_out, Z, M, N, K, N2, dtype, workspace,
                    stream);
}

coda_status coda_block_rowscale_rope(const void* X, const void* W1t, const void* R, const void* W2t, float eps,
                                     void* H, float* P, float* r_out, void* Z, int64_t M, int64_t N, int64_t K,
                                     int64_t N2, coda_dtype dtype, int64_t head_dim, int64_t rope_cols, double base,
                                     int64_t seq_len, const int32_t* positions, void* workspace,
                                     cudaStream_t stream) {
  coda::GemmProblem p;
  TRY(block_prepare(coda::kEpiRowScale, X, W1t, R, W2t, nullptr, eps, H, P, r_out, Z, M, N, K, N2, dtype, workspace,
                    stream, &p));
  const RopeArgs rope = {head_dim, rope_cols, base, seq_len, positions};
  TRY(check_rope(&rope, M, N2, dtype));
  if (p.M == 0) return CODA_OK;
  const int ob = out_bytes(dtype);
  const int64_t T = coda_partial_cols(N);
  const Range outs[] = {rng("H", H, M * N * ob), rng("P", P, M * T * 4), rng("r_out", r_out, r_out ? M * 4 : 0),
                        rng("Z", Z, M * N2 * ob), rng("workspace", workspace, coda_block_workspace_bytes(M))};
  const Range ins[] = {rng("positions", positions, positions ? M * 4 : 0)};
  TRY(check_overlaps(outs, 5, ins, 1));
  set_rope(p.b.ep, &rope);
  return run_gemm(dtype, p);
}

coda_status coda_block_swiglu(const void* X, const void* W1t, const void* R, const void* Wgt, const void* Wut,
                              float eps, void* H, float* P, float* r_out, void* Act, int64_t M, int64_t N, int64_t K,
                              int64_t I, coda_dtype dtype, void* workspace, cudaStream_t stream) {
  return block_impl(coda::kEpiSwiGLU, X, W1t, R, Wgt, Wut, eps, H, P, r_out, Act, M, N, K, I, dtype, workspace,
                    stream);
}

int64_t coda_block_fp8_workspace_bytes(int64_t M) {
  if (M < 0) return -1;
  return coda::block_counters((M + 127) / 128, true) * static_cast<int64_t>(sizeof(unsigned));
}

}  // extern "C"

namespace {

// Shared by the FP8 one-launch blocks.  Phase A: h = R + dequant(Aq . W1t^T)
// with P and amax_h; the quantiser warps then write Hq = e4m3(h / scale_h);
// phase B: the consumer on Hq with the reduction folded in.  With A_bf16
// given, the quantiser warps first write Aq = e4m3(A / (amax_a / 448)).
coda_status block_fp8_impl(int epi_b, const void* A_bf16, const float* amax_a, uint8_t* Aq, float* scale_a,
                           const uint8_t* W1t, const float* scale_w1, const void* R, const uint8_t* Wb,
                           const float* scale_wb, const uint8_t* Wb2, const float* scale_wb2, float eps, void* H,
                           float* P, float* r_out, float* amax_h, uint8_t* Hq, float* scale_h, void* Out,
                           float* amax_out, int64_t M, int64_t N, int64_t K, int64_t N_out, void* workspace,
                           cudaStream_t stream) {
  g_msg[0] = 0;
  const bool swiglu = epi_b == coda::kEpiSwiGLU;
  TRY(check_gemm_dims(M, N, K, CODA_E4M3, "N"));
  TRY(check_gemm_dims(M, N_out, N, CODA_E4M3, swiglu ? "I" : "N2"));
  REQUIRE(std::isfinite(eps) && eps >= 0.0f, "eps must be finite and >= 0");
  TRY(check_scalar_ptr(amax_h, "amax_h"));
  if (amax_out) TRY(check_scalar_ptr(amax_out, "amax_act"));
  if (M == 0) {
    TRY(zero_scalar(amax_h, stream));
    return zero_scalar(amax_out, stream);
  }
  const bool quant_a = A_bf16 != nullptr;
  if (quant_a) {
    TRY(check_ptr(A_bf16, "A"));
    TRY(check_scalar_ptr(amax_a, "amax_a"));
  }
  TRY(check_ptr(Aq, "Aq"));
  TRY(check_scalar_ptr(scale_a, "scale_a"));
  TRY(check_ptr(W1t, "W1t"));
  TRY(check_scalar_ptr(scale_w1, "scale_w1"));
  TRY(check_ptr(R, "R"));
  TRY(check_ptr(Wb, swiglu ? "Wgt" : "W2t"));
  TRY(check_scalar_ptr(scale_wb, swiglu ? "scale_wg" : "scale_w2"));
  if (swiglu) {
    TRY(check_ptr(Wb2, "Wut"));
    TRY(check_scalar_ptr(scale_wb2, "scale_wu"));
  }
  TRY(check_ptr(H, "H"));
  TRY(check_ptr(P, "P"));
  if (r_out) TRY(check_scalar_ptr(r_out, "r_out"));
  TRY(check_ptr(Hq, "Hq"));
  TRY(check_scalar_ptr(scale_h, "scale_h"));
  TRY(check_ptr(Out, swiglu ? "Act" : "Z"));
  TRY(check_ptr(workspace, "workspace"));
  const int64_t T = coda_partial_cols(N);
  const char* out_name = swiglu ? "Act" : "Z";
  // the launch writes Aq and scale_a when it quantises A; else it reads them
  const Range outs[] = {rng("H", H, M * N * 2), rng("P", P, M * T * 4), rng("r_out", r_out, r_out ? M * 4 : 0),
                        rng("amax_h", amax_h, 4), rng("Hq", Hq, M * N), rng("scale_h", scale_h, 4),
                        rng(out_name, Out, M * N_out * 2), rng("amax_act", amax_out, amax_out ? 4 : 0),
                        rng("workspace", workspace, coda_block_fp8_workspace_bytes(M)),
                        rng("Aq", quant_a ? Aq : nullptr, quant_a ? M * K : 0),
                        rng("scale_a", quant_a ? scale_a : nullptr, quant_a ? 4 : 0)};
  const Range ins[] = {rng("A", A_bf16, quant_a ? M * K * 2 : 0), rng("amax_a", amax_a, quant_a ? 4 : 0),
                       rng("Aq", quant_a ? nullptr : Aq, quant_a ? 0 : M * K),
                       rng("scale_a", quant_a ? nullptr : scale_a, quant_a ? 0 : 4), rng("W1t", W1t, N * K),
                       rng("scale_w1", scale_w1, 4), rng("R", R, M * N * 2), rng("W", Wb, N_out * N),
                       rng("scale_w", scale_wb, 4), rng("Wut", Wb2, Wb2 ? N_out * N : 0),
                       rng("scale_wu", scale_wb2, Wb2 ? 4 : 0)};
  TRY(check_overlaps(outs, 11, ins, 11));
  TRY(zero_scalar(amax_h, stream));
  TRY(zero_scalar(amax_out, stream));
  coda::GemmProblem p = {};
  p.epi = coda::kEpiResidualPartialRms;
  p.A = Aq;
  p.B = W1t;
  p.R = R;
  p.D = H;
  p.M = static_cast<int>(M);
  p.N_out = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.ep.P = P;
  p.ep.T = static_cast<int>(T);
  p.ep.scale_a = scale_a;
  p.ep.scale_b = scale_w1;
  p.ep.amax_out = amax_h;
  p.b.epi = epi_b;
  p.b.A = Hq;
  p.b.B = Wb;
  p.b.B2 = Wb2;
  p.b.D = Out;
  p.b.N_out = static_cast<int>(N_out);
  p.b.K = static_cast<int>(N);
  p.b.ep.P_in = P;
  p.b.ep.T_in = static_cast<int>(T);
  p.b.ep.n_norm = static_cast<float>(N);
  p.b.ep.eps = eps;
  p.b.ep.r_out = r_out;
  p.b.ep.scale_a = scale_h;
  p.b.ep.scale_b = scale_wb;
  p.b.ep.scale_b2 = scale_wb2;
  p.b.ep.amax_out = amax_out;
  p.band_ready = static_cast<unsigned*>(workspace);
  p.fp8_block = true;
  p.q.h = H;
  p.q.hq = Hq;
  p.q.amax_h = amax_h;
  p.q.scale_h = scale_h;
  p.q.a = A_bf16;
  p.q.aq = Aq;
  p.q.amax_a = amax_a;
  p.q.scale_a = scale_a;
  p.stream = stream;
  p.pdl = use_pdl();
  return run_gemm(CODA_E4M3, p);
}

}  // namespace

extern "C" {

coda_status coda_block_swiglu_fp8(const void* X, const float* amax_x, uint8_t* Xq, float* scale_x, const uint8_t* W1t,
                                  const float* scale_w1, const void* R, const uint8_t* Wgt, const float* scale_wg,
                                  const uint8_t* Wut, const float* scale_wu, float eps, void* H, float* P,
                                  float* r_out, float* amax_h, uint8_t* Hq, float* scale_h, void* Act,
                                  float* amax_act, int64_t M, int64_t N, int64_t K, int64_t I, void* workspace,
                                  cudaStream_t stream) {
  return block_fp8_impl(coda::kEpiSwiGLU, X, amax_x, Xq, scale_x, W1t, scale_w1, R, Wgt, scale_wg, Wut, scale_wu, eps,
                        H, P, r_out, amax_h, Hq, scale_h, Act, amax_act, M, N, K, I, workspace, stream);
}

coda_status coda_block_rowscale_fp8(const void* X, const float* amax_x, uint8_t* Xq, float* scale_x,
                                    const uint8_t* W1t, const float* scale_w1, const void* R, const uint8_t* W2t,
                                    const float* scale_w2, float eps, void* H, float* P, float* r_out,
                                    float* amax_h, uint8_t* Hq, float* scale_h, void* Z, int64_t M, int64_t N,
                                    int64_t K, int64_t N2, void* workspace, cudaStream_t stream) {
  return block_fp8_impl(coda::kEpiRowScale, X, amax_x, Xq, scale_x, W1t, scale_w1, R, W2t, scale_w2, nullptr, nullptr,
                        eps, H, P, r_out, amax_h, Hq, scale_h, Z, nullptr, M, N, K, N2, workspace, stream);
}

coda_status coda_amax(const void* x, int64_t n, coda_dtype dtype, float* amax, cudaStream_t stream) {
  g_msg[0] = 0;
  REQUIRE(dtype == CODA_F32 || dtype == CODA_BF16, "coda_amax: dtype must be CODA_F32 or CODA_BF16");
  REQUIRE(n >= 0 && n < (int64_t(1) << 60), "coda_amax: n out of range [0, 2^60)");
  TRY(check_scalar_ptr(amax, "amax"));
  TRY(zero_scalar(amax, stream));
  if (n == 0) return CODA_OK;
  TRY(check_ptr(x, "x"));
  const Range outs[] = {rng("amax", amax, 4)};
  const Range ins[] = {rng("x", x, n * elem_bytes(dtype))};
  TRY(check_overlaps(outs, 1, ins, 1));
  cudaError_t e = coda::launch_amax(x, n, dtype == CODA_F32, amax, stream);
  return e == cudaSuccess ? CODA_OK : cuda_fail(e, "coda_amax launch");
}

coda_status coda_quantize_e4m3(const void* x, int64_t n, coda_dtype dtype, const float* amax, uint8_t* q,
                               float* scale, cudaStream_t stream) {
  g_msg[0] = 0;
  REQUIRE(dtype == CODA_F32 || dtype == CODA_BF16, "coda_quantize_e4m3: dtype must be CODA_F32 or CODA_BF16");
  REQUIRE(n >= 0 && n < (int64_t(1) << 60), "coda_quantize_e4m3: n out of range [0, 2^60)");
  TRY(check_scalar_ptr(amax, "amax"));
  TRY(check_scalar_ptr(scale, "scale"));
  if (n > 0) {
    TRY(check_ptr(x, "x"));
    TRY(check_ptr(q, "q"));
  }
  const Range outs[] = {rng("q", q, n), rng("scale", scale, 4)};
  const Range ins[] = {rng("x", x, n * elem_bytes(dtype)), rng("amax", amax, 4)};
  TRY(check_overlaps(outs, 2, ins, 2));
  cudaError_t e = coda::launch_quantize_e4m3(x, n, dtype == CODA_F32, amax, q, scale, stream);
  return e == cudaSuccess ? CODA_OK : cuda_fail(e, "coda_quantize_e4m3 launch");
}

coda_status coda_selftest_wait_timeout(int64_t timeout_ns, cudaStream_t stream) {
  g_msg[0] = 0;
  REQUIRE(timeout_ns >= 1000 && timeout_ns <= 10000000000LL,
          "coda_selftest_wait_timeout: timeout_ns must lie in [1e3, 1e10]");
  cudaError_t e = coda::launch_wait_probe(timeout_ns, stream);
  return e == cudaSuccess ? CODA_OK : cuda_fail(e, "coda_selftest_wait_timeout launch");
}

coda_status coda_get_device_status(void) {
  g_msg[0] = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceSynchronize");
  const unsigned waits = coda::read_clear_status_bf16() | coda::read_clear_status_tf32() |
                         coda::read_clear_status_e4m3() | coda::read_clear_status_aux() |
                         coda::read_clear_status_grouped_bf16() | coda::read_clear_status_grouped_grad() |
                         coda::read_clear_status_grouped_e4m3();
  if (waits == ~0u) return fail(CODA_ERR_CUDA, "could not read the device status word");
  // the words of the other kernels, whose finding is another, are left for the next call
  if (waits & 1u) return fail(CODA_ERR_TIMEOUT, "a kernel gave up on a bounded wait (timeout)");
  const unsigned indices = coda::read_clear_status_paged() | coda::read_clear_status_logprobs() |
                           coda::read_clear_status_experts() | coda::read_clear_index_grouped_bf16() |
                           coda::read_clear_index_grouped_grad() | coda::read_clear_index_grouped_e4m3();
  if (indices == ~0u) return fail(CODA_ERR_CUDA, "could not read the device status word");
  if (indices & 2u)
    return fail(CODA_ERR_INVALID_ARG, "a page, sequence, length, token, expert, slot or offset on the device was out of range");
  return CODA_OK;
}

}  // extern "C"

// ------------------------------------------------- paged cache, attention ----
namespace {

// log2(n) of a power of two below 2^31, else -1.
int log2_or_none(int64_t n) {
  for (int b = 0; b < 31; ++b)
    if (n == int64_t(1) << b) return b;
  return -1;
}

// Shape rules common to the paged cache calls.
coda_status check_paged(int64_t M, int64_t num_seqs, int64_t max_pages, int64_t q_heads, int64_t kv_heads,
                        int64_t head_dim, int64_t num_pages, int64_t page_size, const int32_t* row_seq,
                        coda_dtype dtype, coda_dtype cache_dtype, const float* scale_k, const float* scale_v) {
  REQUIRE(dtype == CODA_F32 || dtype == CODA_BF16, "dtype must be CODA_F32 or CODA_BF16");
  REQUIRE(cache_dtype == dtype || (dtype == CODA_BF16 && cache_dtype == CODA_E4M3),
          "cache_dtype must equal dtype, or be CODA_E4M3 with CODA_BF16");
  REQUIRE(M >= 0 && M < INT32_MAX, "M = %" PRId64 " out of range [0, 2^31)", M);
  REQUIRE(num_seqs >= 0 && num_seqs < INT32_MAX, "num_seqs = %" PRId64 " out of range [0, 2^31)", num_seqs);
  REQUIRE(row_seq != nullptr || M <= num_seqs, "M = %" PRId64 " rows but %" PRId64 " sequences, and row_seq is NULL", M,
          num_seqs);
  REQUIRE(max_pages > 0 && max_pages < INT32_MAX, "max_pages = %" PRId64 " out of range [1, 2^31)", max_pages);
  REQUIRE(num_pages > 0 && num_pages < INT32_MAX, "num_pages = %" PRId64 " out of range [1, 2^31)", num_pages);
  REQUIRE(page_size > 0 && page_size < INT32_MAX, "page_size = %" PRId64 " out of range [1, 2^31)", page_size);
  REQUIRE(kv_heads > 0 && q_heads > 0 && q_heads < (1 << 20) && q_heads % kv_heads == 0,
          "q_heads = %" PRId64 " must be a positive multiple of kv_heads = %" PRId64 ", below 2^20", q_heads, kv_heads);
  const int64_t step = 16 / elem_bytes(cache_dtype);
  REQUIRE(head_dim > 0 && head_dim <= coda::kMaxHeadDim && head_dim % step == 0,
          "head_dim = %" PRId64 " must be a multiple of %" PRId64 " for this cache, at most %d", head_dim, step,
          coda::kMaxHeadDim);
  REQUIRE(num_pages < INT32_MAX / page_size / kv_heads,
          "num_pages * kv_heads * page_size: a cache of 2^31 rows or more");
  REQUIRE(M < (int64_t(1) << 60) / (q_heads + 2 * kv_heads) / head_dim, "rows of 2^60 elements or more");
  REQUIRE(num_seqs * max_pages < (int64_t(1) << 60), "a page table of 2^60 entries or more");
  if (cache_dtype == CODA_E4M3) {
    TRY(check_scalar_ptr(scale_k, "scale_k"));
    TRY(check_scalar_ptr(scale_v, "scale_v"));
  } else {
    REQUIRE(scale_k == nullptr && scale_v == nullptr, "scale_k and scale_v must be NULL unless the cache is CODA_E4M3");
  }
  return CODA_OK;
}

}  // namespace

extern "C" {

coda_status coda_paged_append(const void* Z, const int32_t* positions, const int32_t* row_seq,
                              const int32_t* page_table, void* Q, void* Kc, void* Vc, int64_t M, int64_t num_seqs,
                              int64_t max_pages, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                              int64_t num_pages, int64_t page_size, double base, coda_dtype dtype,
                              coda_dtype cache_dtype, const float* scale_k, const float* scale_v,
                              cudaStream_t stream) {
  g_msg[0] = 0;
  TRY(check_paged(M, num_seqs, max_pages, q_heads, kv_heads, head_dim, num_pages, page_size, row_seq, dtype,
                  cache_dtype, scale_k, scale_v));
  REQUIRE(base == 0.0 || (std::isfinite(base) && base > 1.0), "base must be 0 (no rotation), or finite and > 1");
  if (M == 0) return CODA_OK;
  TRY(check_ptr(Z, "Z"));
  TRY(check_scalar_ptr(positions, "positions"));
  if (row_seq) TRY(check_scalar_ptr(row_seq, "row_seq"));
  TRY(check_scalar_ptr(page_table, "page_table"));
  if (Q) TRY(check_ptr(Q, "Q"));
  TRY(check_ptr(Kc, "k_cache"));
  TRY(check_ptr(Vc, "v_cache"));
  const int64_t eb = elem_bytes(dtype), cache = num_pages * page_size * kv_heads * head_dim * elem_bytes(cache_dtype);
  const Range outs[] = {rng("Q", Q, Q ? M * q_heads * head_dim * eb : 0), rng("k_cache", Kc, cache),
                        rng("v_cache", Vc, cache)};
  const Range ins[] = {rng("Z", Z, M * (q_heads + 2 * kv_heads) * head_dim * eb),
                       rng("positions", positions, M * 4),
                       rng("row_seq", row_seq, row_seq ? M * 4 : 0),
                       rng("page_table", page_table, num_seqs * max_pages * 4),
                       rng("scale_k", scale_k, scale_k ? 4 : 0),
                       rng("scale_v", scale_v, scale_v ? 4 : 0)};
  TRY(check_overlaps(outs, 3, ins, 6));
  coda::AppendParams p = {};
  p.Z = Z;
  p.positions = positions;
  p.row_seq = row_seq;
  p.page_table = page_table;
  p.Q = Q;
  p.Kc = Kc;
  p.Vc = Vc;
  p.scale_k = scale_k;
  p.scale_v = scale_v;
  p.num_seqs = static_cast<int>(num_seqs);
  p.max_pages = static_cast<int>(max_pages);
  p.q_heads = static_cast<int>(q_heads);
  p.kv_heads = static_cast<int>(kv_heads);
  p.head_dim = static_cast<int>(head_dim);
  p.num_pages = static_cast<int>(num_pages);
  p.page_size = static_cast<int>(page_size);
  p.M = M;
  p.page_shift = log2_or_none(page_size);
  p.rotate = base != 0.0;
  if (p.rotate) {
    // base^(-2j / head_dim) / 2 pi < 1 as a 64-bit fraction of a turn, by repeated products in 64 bits: the
    // relative error of term j is j 2^-52 (the ratio's rounding and the products'), so the turn count at position 2^31
    // is off by j base^(-2j / head_dim) 2^-21 / 2 pi: less than 4e-7 of a turn from base 10000 on, and less than 1e-5
    // for any base (127 of 128 pairs in, at a base near 1)
    const double ratio = std::pow(base, -2.0 / static_cast<double>(head_dim));
    double f = 0.15915494309189535 * 0x1p64;
    for (int64_t j = 0; j < head_dim / 2; ++j, f *= ratio) p.turn[j] = static_cast<uint64_t>(f);
  }
  cudaError_t e =
      coda::launch_paged_append(p, dtype == CODA_F32, cache_dtype == CODA_E4M3, stream, use_pdl());
  return e == cudaSuccess ? CODA_OK : cuda_fail(e, "coda_paged_append launch");
}

int64_t coda_paged_attention_workspace_bytes(int64_t q_heads, int64_t kv_heads, int64_t head_dim) {
  if (kv_heads <= 0 || q_heads <= 0 || q_heads >= (1 << 20) || q_heads % kv_heads != 0 || head_dim <= 0 ||
      head_dim > coda::kMaxHeadDim)
    return -1;
  return coda::paged_attention_workspace_bytes(static_cast<int>(q_heads), static_cast<int>(kv_heads),
                                               static_cast<int>(head_dim));
}

coda_status coda_paged_attention(const void* Q, int64_t ldq, const void* Kc, const void* Vc,
                                 const int32_t* page_table, const int32_t* lengths, const int32_t* row_seq, void* O,
                                 float* lse, int64_t M, int64_t num_seqs, int64_t max_pages, int64_t q_heads,
                                 int64_t kv_heads, int64_t head_dim, int64_t num_pages, int64_t page_size,
                                 float scale, coda_dtype dtype, coda_dtype cache_dtype, const float* scale_k,
                                 const float* scale_v, void* workspace, cudaStream_t stream) {
  g_msg[0] = 0;
  TRY(check_paged(M, num_seqs, max_pages, q_heads, kv_heads, head_dim, num_pages, page_size, row_seq, dtype,
                  cache_dtype, scale_k, scale_v));
  const int64_t eb = elem_bytes(dtype), width = q_heads * head_dim;
  REQUIRE(ldq >= width && ldq < (int64_t(1) << 40) && (ldq * eb) % 16 == 0,
          "ldq = %" PRId64 " must hold a row of %" PRId64 " elements and be a multiple of %" PRId64, ldq, width, 16 / eb);
  REQUIRE(std::isfinite(scale) && scale > 0.0f, "scale must be finite and > 0");
  REQUIRE(M * q_heads < INT32_MAX, "M * q_heads = %" PRId64 " out of range [0, 2^31)", M * q_heads);
  REQUIRE(M == 0 || ldq < (int64_t(1) << 60) / M, "rows of 2^60 elements or more");
  if (M == 0) return CODA_OK;
  TRY(check_ptr(Q, "Q"));
  TRY(check_ptr(Kc, "k_cache"));
  TRY(check_ptr(Vc, "v_cache"));
  TRY(check_scalar_ptr(page_table, "page_table"));
  TRY(check_scalar_ptr(lengths, "lengths"));
  if (row_seq) TRY(check_scalar_ptr(row_seq, "row_seq"));
  TRY(check_ptr(O, "O"));
  if (lse) TRY(check_scalar_ptr(lse, "lse"));
  TRY(check_ptr(workspace, "workspace"));
  const int64_t cache = num_pages * page_size * kv_heads * head_dim * elem_bytes(cache_dtype);
  const Range outs[] = {rng("O", O, M * width * eb), rng("lse", lse, lse ? M * q_heads * 4 : 0),
                        rng("workspace", workspace, coda_paged_attention_workspace_bytes(q_heads, kv_heads, head_dim))};
  const Range ins[] = {rng("Q", Q, ((M - 1) * ldq + width) * eb),
                       rng("k_cache", Kc, cache),
                       rng("v_cache", Vc, cache),
                       rng("page_table", page_table, num_seqs * max_pages * 4),
                       rng("lengths", lengths, M * 4),
                       rng("row_seq", row_seq, row_seq ? M * 4 : 0),
                       rng("scale_k", scale_k, scale_k ? 4 : 0),
                       rng("scale_v", scale_v, scale_v ? 4 : 0)};
  TRY(check_overlaps(outs, 3, ins, 8));
  coda::AttnParams p = {};
  p.Q = Q;
  p.ldq = ldq;
  p.Kc = Kc;
  p.Vc = Vc;
  p.page_table = page_table;
  p.lengths = lengths;
  p.row_seq = row_seq;
  p.O = O;
  p.lse = lse;
  p.scale_k = scale_k;
  p.scale_v = scale_v;
  p.workspace = workspace;
  p.scale = scale;
  p.M = static_cast<int>(M);
  p.num_seqs = static_cast<int>(num_seqs);
  p.max_pages = static_cast<int>(max_pages);
  p.q_heads = static_cast<int>(q_heads);
  p.kv_heads = static_cast<int>(kv_heads);
  p.head_dim = static_cast<int>(head_dim);
  p.num_pages = static_cast<int>(num_pages);
  p.page_size = static_cast<int>(page_size);
  p.page_shift = log2_or_none(page_size);
  cudaError_t e = coda::launch_paged_attention(p, dtype == CODA_F32, cache_dtype == CODA_E4M3, stream, use_pdl());
  return e == cudaSuccess ? CODA_OK : cuda_fail(e, "coda_paged_attention launch");
}

}  // extern "C"

// ------------------------------------------------------- log probabilities ----
namespace {

// Shape rules common to the log-probability calls.
coda_status check_logits(int64_t M, int64_t V, int64_t ld, const char* ldname, coda_dtype dtype) {
  REQUIRE(dtype == CODA_F32 || dtype == CODA_BF16, "dtype must be CODA_F32 or CODA_BF16");
  REQUIRE(M >= 0 && M < INT32_MAX, "M = %" PRId64 " out of range [0, 2^31)", M);
  REQUIRE(V > 0 && V < INT32_MAX / 2, "V = %" PRId64 " out of range [1, 2^30)", V);
  REQUIRE(ld >= V && ld < (int64_t(1) << 40) && (ld * elem_bytes(dtype)) % 16 == 0,
          "%s = %" PRId64 " must be at least V = %" PRId64 " and a multiple of %d", ldname, ld, V,
          16 / elem_bytes(dtype));
  REQUIRE(M == 0 || ld < (int64_t(1) << 60) / M, "rows of 2^60 elements or more");
  return CODA_OK;
}

}  // namespace

extern "C" {

coda_status coda_logprobs(const void* logits, int64_t ld, const int32_t* targets, float* logp, float* entropy,
                          float* lse, float* top_logp, int32_t* top_ids, int64_t M, int64_t V, int64_t top,
                          coda_dtype dtype, cudaStream_t stream) {
  g_msg[0] = 0;
  TRY(check_logits(M, V, ld, "ld", dtype));
  REQUIRE(top >= 0 && top <= coda::kMaxTop && top <= V, "top = %" PRId64 " out of range [0, min(V, %d)]", top,
          coda::kMaxTop);
  if (M == 0) return CODA_OK;
  TRY(check_ptr(logits, "logits"));
  TRY(check_scalar_ptr(targets, "targets"));
  TRY(check_scalar_ptr(logp, "logp"));
  if (entropy) TRY(check_scalar_ptr(entropy, "entropy"));
  if (lse) TRY(check_scalar_ptr(lse, "lse"));
  if (top > 0) {
    TRY(check_scalar_ptr(top_logp, "top_logp"));
    TRY(check_scalar_ptr(top_ids, "top_ids"));
  }
  const Range outs[] = {rng("logp", logp, M * 4), rng("entropy", entropy, entropy ? M * 4 : 0),
                        rng("lse", lse, lse ? M * 4 : 0), rng("top_logp", top_logp, M * top * 4),
                        rng("top_ids", top_ids, M * top * 4)};
  const Range ins[] = {rng("logits", logits, ((M - 1) * ld + V) * elem_bytes(dtype)),
                       rng("targets", targets, M * 4)};
  TRY(check_overlaps(outs, 5, ins, 2));
  coda::LogprobsParams p = {};
  p.logits = logits;
  p.ld = ld;
  p.targets = targets;
  p.logp = logp;
  p.entropy = entropy;
  p.lse = lse;
  p.top_logp = top_logp;
  p.top_ids = top_ids;
  p.V = static_cast<int>(V);
  p.top = static_cast<int>(top);
  cudaError_t e = coda::launch_logprobs(p, M, dtype == CODA_F32, stream, use_pdl());
  return e == cudaSuccess ? CODA_OK : cuda_fail(e, "coda_logprobs launch");
}

coda_status coda_logprobs_backward(const void* logits, int64_t ld, const int32_t* targets, const float* lse,
                                   const float* entropy, const float* dlogp, const float* dentropy, void* dlogits,
                                   int64_t ldd, int64_t M, int64_t V, coda_dtype dtype, cudaStream_t stream) {
  g_msg[0] = 0;
  TRY(check_logits(M, V, ld, "ld", dtype));
  TRY(check_logits(M, V, ldd, "ldd", dtype));
  REQUIRE(M * coda::logprobs_backward_blocks(V, dtype == CODA_F32) < INT32_MAX,
          "M = %" PRId64 ", V = %" PRId64 ": too many blocks for one launch", M, V);
  if (M == 0) return CODA_OK;
  TRY(check_ptr(logits, "logits"));
  TRY(check_scalar_ptr(targets, "targets"));
  TRY(check_scalar_ptr(lse, "lse"));
  if (dlogp) TRY(check_scalar_ptr(dlogp, "dlogp"));
  if (dentropy) {
    TRY(check_scalar_ptr(dentropy, "dentropy"));
    TRY(check_scalar_ptr(entropy, "entropy"));
  }
  TRY(check_ptr(dlogits, "dlogits"));
  const int eb = elem_bytes(dtype);
  const Range outs[] = {rng("dlogits", dlogits, ((M - 1) * ldd + V) * eb)};
  const Range ins[] = {rng("logits", logits, ((M - 1) * ld + V) * eb),
                       rng("targets", targets, M * 4),
                       rng("lse", lse, M * 4),
                       rng("entropy", entropy, entropy ? M * 4 : 0),
                       rng("dlogp", dlogp, dlogp ? M * 4 : 0),
                       rng("dentropy", dentropy, dentropy ? M * 4 : 0)};
  TRY(check_overlaps(outs, 1, ins, 6));
  coda::LogprobsGradParams p = {};
  p.logits = logits;
  p.ld = ld;
  p.targets = targets;
  p.lse = lse;
  p.entropy = dentropy ? entropy : nullptr;
  p.dlogp = dlogp;
  p.dentropy = dentropy;
  p.dlogits = dlogits;
  p.ldd = ldd;
  p.V = static_cast<int>(V);
  cudaError_t e = coda::launch_logprobs_backward(p, M, dtype == CODA_F32, stream, use_pdl());
  return e == cudaSuccess ? CODA_OK : cuda_fail(e, "coda_logprobs_backward launch");
}

}  // extern "C"

// ------------------------------------------------------ mixture of experts ----
namespace {

// Rows of `width` elements `ld` apart, all within 2^60 elements.
coda_status check_rows(int64_t M, int64_t width, int64_t ld, const char* name, coda_dtype dtype) {
  REQUIRE(ld >= width && ld < (int64_t(1) << 40) && (ld * elem_bytes(dtype)) % 16 == 0,
          "%s = %" PRId64 " must hold a row of %" PRId64 " elements and be a multiple of %d", name, ld, width,
          16 / elem_bytes(dtype));
  REQUIRE(M == 0 || ld < (int64_t(1) << 60) / M, "rows of 2^60 elements or more");
  return CODA_OK;
}

// Shape rules common to the norm calls.
coda_status check_norm(int64_t M, int64_t N, coda_dtype dtype, bool codes) {
  REQUIRE(dtype == CODA_F32 || dtype == CODA_BF16, "dtype must be CODA_F32 or CODA_BF16");
  REQUIRE(M >= 0 && M < INT32_MAX, "M = %" PRId64 " out of range [0, 2^31)", M);
  const int step = codes ? 16 : 16 / elem_bytes(dtype);
  REQUIRE(N > 0 && N <= coda::kMaxNormWidth && N % step == 0,
          "N = %" PRId64 " must be a multiple of %d out of [1, %d]", N, step, coda::kMaxNormWidth);
  return CODA_OK;
}

coda_status norm_impl(const char* what, const void* X, int64_t ldx, const void* R, int64_t ldr, const float* gamma,
                      float eps, void* H, void* Y, uint8_t* Yq, float* scale, float* r, int64_t M, int64_t N,
                      coda_dtype dtype, cudaStream_t stream) {
  if (M == 0) return CODA_OK;
  TRY(check_ptr(X, "X"));
  if (R) TRY(check_ptr(R, "R"));
  if (gamma) TRY(check_ptr(gamma, "gamma"));
  if (H) TRY(check_ptr(H, "H"));
  if (Y) TRY(check_ptr(Y, "Y"));
  if (Yq) {
    TRY(check_ptr(Yq, "q"));
    TRY(check_scalar_ptr(scale, "scale"));
  }
  if (r) TRY(check_scalar_ptr(r, "r"));
  const int64_t eb = elem_bytes(dtype), mn = M * N * eb;
  const Range outs[] = {rng("H", H, H ? mn : 0), rng("Y", Y, Y ? mn : 0), rng("q", Yq, Yq ? M * N : 0),
                        rng("scale", scale, Yq ? M * 4 : 0), rng("r", r, r ? M * 4 : 0)};
  const Range ins[] = {rng("X", X, ((M - 1) * ldx + N) * eb), rng("R", R, R ? ((M - 1) * ldr + N) * eb : 0),
                       rng("gamma", gamma, gamma ? N * 4 : 0)};
  TRY(check_overlaps(outs, 5, ins, 3));
  coda::NormParams p = {};
  p.X = X;
  p.ldx = ldx;
  p.R = R;
  p.ldr = ldr;
  p.gamma = gamma;
  p.eps = eps;
  p.H = H;
  p.Y = Y;
  p.Yq = Yq;
  p.scale = scale;
  p.r = r;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  cudaError_t e = coda::launch_norm(p, dtype == CODA_F32, stream, use_pdl());
  return e == cudaSuccess ? CODA_OK : cuda_fail(e, what);
}

// Shape rules of the router calls.
coda_status check_route(int64_t M, int64_t E, int64_t k, coda_dtype dtype) {
  REQUIRE(dtype == CODA_F32 || dtype == CODA_BF16, "dtype must be CODA_F32 or CODA_BF16");
  REQUIRE(M >= 0 && M < coda::kMaxRouteRows, "M = %" PRId64 " out of range [0, 2^31 - 2^24)", M);
  REQUIRE(E > 0 && E <= coda::kMaxExperts, "E = %" PRId64 " out of range [1, %d]", E, coda::kMaxExperts);
  REQUIRE(k > 0 && k <= E && k <= coda::kMaxChoices, "top_k = %" PRId64 " out of range [1, min(E, %d)]", k,
          coda::kMaxChoices);
  REQUIRE(M * k < INT32_MAX, "M * top_k = %" PRId64 " out of range [0, 2^31)", M * k);
  return CODA_OK;
}

// Shape rules of the calls that move rows to and from expert order.
coda_status check_places(int64_t M, int64_t N, int64_t k, int64_t T, coda_dtype dtype) {
  REQUIRE(M >= 0 && M < INT32_MAX, "M = %" PRId64 " out of range [0, 2^31)", M);
  REQUIRE(T >= 0 && T < INT32_MAX, "T = %" PRId64 " out of range [0, 2^31)", T);
  REQUIRE(k > 0 && k <= coda::kMaxChoices, "top_k = %" PRId64 " out of range [1, %d]", k, coda::kMaxChoices);
  REQUIRE(N > 0 && N < INT32_MAX && (N * elem_bytes(dtype)) % 16 == 0,
          "N = %" PRId64 " must be a positive multiple of %d for this dtype (16-byte rows)", N, 16 / elem_bytes(dtype));
  REQUIRE(M * N < (int64_t(1) << 60) && T * N < (int64_t(1) << 60), "a matrix of 2^60 elements or more");
  return CODA_OK;
}

// Shape rules of the grouped products of A [T, K] with E weights of N x K.
coda_status check_grouped(int64_t T, int64_t E, int64_t N, int64_t K, coda_dtype dtype, const char* nname) {
  REQUIRE(T >= 0 && T <= INT32_MAX - 1024, "T = %" PRId64 " out of range [0, 2^31 - 1024)", T);
  REQUIRE(E > 0 && E <= coda::kMaxExperts, "E = %" PRId64 " out of range [1, %d]", E, coda::kMaxExperts);
  TRY(check_gemm_dims(T, N, K, dtype, nname));
  REQUIRE(N < (int64_t(1) << 30) && K < (int64_t(1) << 30) && N * K < (int64_t(1) << 37),
          "%s = %" PRId64 ", K = %" PRId64 ": an expert's weights of 2^37 elements or more", nname, N, K);
  REQUIRE((T / 32 + E) * ((N + 63) / 64) < (int64_t(1) << 30) &&
              E * ((N + 127) / 128) * ((K + 127) / 128) < (int64_t(1) << 30),
          "T = %" PRId64 ", %s = %" PRId64 ": too many output tiles for the kernels' 32-bit tile indices", T, nname, N);
  return CODA_OK;
}

coda_status check_group_scales(coda_dtype dtype, const float* row_scale, const float* w_scale) {
  if (dtype == CODA_E4M3) {
    TRY(check_scalar_ptr(row_scale, "row_scale"));
    TRY(check_scalar_ptr(w_scale, "w_scale"));
  } else {
    REQUIRE(w_scale == nullptr, "w_scale must be NULL unless dtype is CODA_E4M3");
    if (row_scale) TRY(check_scalar_ptr(row_scale, "row_scale"));
  }
  return CODA_OK;
}

coda_status run_grouped(const char* what, const coda::GroupProblem& p, coda_dtype dtype) {
  const char* msg = "";
  const bool grad =
      p.program == coda::kGroupPlainMN || p.program == coda::kGroupSwiGLUBwd || p.program == coda::kGroupWgrad;
  const cudaError_t e = dtype == CODA_E4M3 ? coda::launch_grouped_e4m3(p, &msg)
                        : grad             ? coda::launch_grouped_grad(p, &msg)
                                           : coda::launch_grouped_bf16(p, &msg);
  if (e == cudaSuccess) return CODA_OK;
  return fail(CODA_ERR_CUDA, "%s: %s: %s (%s)", what, msg, cudaGetErrorName(e), cudaGetErrorString(e));
}

coda::GroupProblem group_problem(int program, const void* A, const void* W, void* D, const int32_t* offsets, int64_t T,
                                 int64_t E, int64_t N, int64_t K, cudaStream_t stream) {
  coda::GroupProblem p = {};
  p.program = program;
  p.A = A;
  p.W = W;
  p.D = D;
  p.offsets = offsets;
  p.T = static_cast<int>(T);
  p.E = static_cast<int>(E);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.stream = stream;
  p.pdl = use_pdl();
  return p;
}

}  // namespace

extern "C" {

coda_status coda_add_rmsnorm(const void* X, int64_t ldx, const void* R, int64_t ldr, const float* gamma, float eps,
                             void* H, void* Y, uint8_t* Yq, float* scale, float* r, int64_t M, int64_t N,
                             coda_dtype dtype, cudaStream_t stream) {
  g_msg[0] = 0;
  TRY(check_norm(M, N, dtype, Yq != nullptr));
  TRY(check_rows(M, N, ldx, "ldx", dtype));
  if (R) TRY(check_rows(M, N, ldr, "ldr", dtype));
  REQUIRE(std::isfinite(eps) && eps >= 0.0f, "eps must be finite and >= 0");
  REQUIRE(M == 0 || Y != nullptr || Yq != nullptr, "one of Y and q must be given");
  if (M > 0) TRY(check_ptr(gamma, "gamma"));
  return norm_impl("coda_add_rmsnorm launch", X, ldx, R, ldr, gamma, eps, H, Y, Yq, scale, r, M, N, dtype, stream);
}

coda_status coda_quantize_rows_e4m3(const void* X, int64_t ldx, uint8_t* q, float* scale, int64_t M, int64_t N,
                                    coda_dtype dtype, cudaStream_t stream) {
  g_msg[0] = 0;
  TRY(check_norm(M, N, dtype, true));
  TRY(check_rows(M, N, ldx, "ldx", dtype));
  if (M > 0) TRY(check_ptr(q, "q"));
  return norm_impl("coda_quantize_rows_e4m3 launch", X, ldx, nullptr, 0, nullptr, 0.0f, nullptr, nullptr, q, scale,
                   nullptr, M, N, dtype, stream);
}

int64_t coda_add_rmsnorm_backward_workspace_bytes(int64_t M, int64_t N) {
  if (M < 0 || N <= 0 || N > coda::kMaxNormWidth) return -1;
  return coda::norm_backward_workspace_bytes(M, N);
}

coda_status coda_add_rmsnorm_backward(const void* dY, const void* H, const float* r, const float* gamma,
                                      const void* dH_in, void* dH, float* dgamma, float* workspace, int64_t M,
                                      int64_t N, coda_dtype dtype, cudaStream_t stream) {
  g_msg[0] = 0;
  TRY(check_norm(M, N, dtype, false));
  TRY(check_ptr(dgamma, "dgamma"));
  if (M == 0) {
    cudaError_t e = cudaMemsetAsync(dgamma, 0, static_cast<size_t>(N) * sizeof(float), stream);
    return e == cudaSuccess ? CODA_OK : cuda_fail(e, "cudaMemsetAsync(dgamma)");
  }
  TRY(check_ptr(dY, "dY"));
  TRY(check_ptr(H, "H"));
  TRY(check_scalar_ptr(r, "r"));
  TRY(check_ptr(gamma, "gamma"));
  if (dH_in) TRY(check_ptr(dH_in, "dH_in"));
  TRY(check_ptr(dH, "dH"));
  TRY(check_ptr(workspace, "workspace"));
  const int64_t mn = M * N * elem_bytes(dtype);
  const Range outs[] = {rng("dH", dH, mn), rng("dgamma", dgamma, N * 4),
                        rng("workspace", workspace, coda_add_rmsnorm_backward_workspace_bytes(M, N))};
  const Range ins[] = {rng("dY", dY, mn), rng("H", H, mn), rng("r", r, M * 4), rng("gamma", gamma, N * 4),
                       rng("dH_in", dH_in, dH_in ? mn : 0)};
  TRY(check_overlaps(outs, 3, ins, 5));
  coda::NormGradParams p = {};
  p.dY = dY;
  p.H = H;
  p.r = r;
  p.gamma = gamma;
  p.dH_in = dH_in;
  p.dH = dH;
  p.dgamma = dgamma;
  p.part = workspace;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  cudaError_t e = coda::launch_norm_backward(p, dtype == CODA_F32, stream, use_pdl());
  return e == cudaSuccess ? CODA_OK : cuda_fail(e, "coda_add_rmsnorm_backward launch");
}

int64_t coda_route_workspace_bytes(int64_t M, int64_t E, int64_t top_k) {
  if (M < 0 || E <= 0 || E > coda::kMaxExperts || top_k <= 0 || top_k > coda::kMaxChoices || top_k > E ||
      M >= coda::kMaxRouteRows || M * top_k >= INT32_MAX)
    return -1;
  return coda::route_workspace_bytes(M, E, top_k);
}

coda_status coda_route(const void* logits, int64_t ld, int64_t top_k, int renormalize, int32_t* ids, float* weights,
                       int32_t* slots, int32_t* offsets, void* workspace, int64_t M, int64_t E, coda_dtype dtype,
                       cudaStream_t stream) {
  g_msg[0] = 0;
  TRY(check_route(M, E, top_k, dtype));
  TRY(check_rows(M, E, ld, "ld", dtype));
  TRY(check_scalar_ptr(offsets, "offsets"));
  if (M == 0) {
    cudaError_t e = cudaMemsetAsync(offsets, 0, static_cast<size_t>(E + 1) * sizeof(int32_t), stream);
    return e == cudaSuccess ? CODA_OK : cuda_fail(e, "cudaMemsetAsync(offsets)");
  }
  const int64_t ws = coda::route_workspace_bytes(M, E, top_k);
  TRY(check_ptr(logits, "logits"));
  TRY(check_scalar_ptr(ids, "ids"));
  TRY(check_scalar_ptr(weights, "weights"));
  TRY(check_scalar_ptr(slots, "slots"));
  if (ws > 0) TRY(check_ptr(workspace, "workspace"));
  const int64_t pairs = M * top_k * 4;
  const Range outs[] = {rng("ids", ids, pairs), rng("weights", weights, pairs), rng("slots", slots, pairs),
                        rng("offsets", offsets, (E + 1) * 4), rng("workspace", workspace, ws)};
  const Range ins[] = {rng("logits", logits, ((M - 1) * ld + E) * elem_bytes(dtype))};
  TRY(check_overlaps(outs, 5, ins, 1));
  coda::RouteParams p = {};
  p.logits = logits;
  p.ld = ld;
  p.ids = ids;
  p.weights = weights;
  p.slots = slots;
  p.offsets = offsets;
  p.counts = static_cast<int32_t*>(workspace);
  p.M = static_cast<int>(M);
  p.E = static_cast<int>(E);
  p.k = static_cast<int>(top_k);
  p.renormalize = renormalize != 0;
  cudaError_t e = coda::launch_route(p, dtype == CODA_F32, stream, use_pdl());
  return e == cudaSuccess ? CODA_OK : cuda_fail(e, "coda_route launch");
}

coda_status coda_route_backward(const void* logits, int64_t ld, const int32_t* ids, const float* weights,
                                const float* dweights, int renormalize, void* dlogits, int64_t ldd, int64_t M,
                                int64_t E, int64_t top_k, coda_dtype dtype, cudaStream_t stream) {
  g_msg[0] = 0;
  TRY(check_route(M, E, top_k, dtype));
  if (!renormalize) TRY(check_rows(M, E, ld, "ld", dtype));
  TRY(check_rows(M, E, ldd, "ldd", dtype));
  if (M == 0) return CODA_OK;
  if (!renormalize) TRY(check_ptr(logits, "logits"));
  TRY(check_scalar_ptr(ids, "ids"));
  TRY(check_scalar_ptr(weights, "weights"));
  TRY(check_scalar_ptr(dweights, "dweights"));
  TRY(check_ptr(dlogits, "dlogits"));
  const int64_t pairs = M * top_k * 4, eb = elem_bytes(dtype);
  const Range outs[] = {rng("dlogits", dlogits, ((M - 1) * ldd + E) * eb)};
  const Range ins[] = {rng("logits", logits, renormalize ? 0 : ((M - 1) * ld + E) * eb), rng("ids", ids, pairs),
                       rng("weights", weights, pairs), rng("dweights", dweights, pairs)};
  TRY(check_overlaps(outs, 1, ins, 4));
  coda::RouteGradParams p = {};
  p.logits = logits;
  p.ld = ld;
  p.ids = ids;
  p.weights = weights;
  p.dweights = dweights;
  p.dlogits = dlogits;
  p.ldd = ldd;
  p.M = static_cast<int>(M);
  p.E = static_cast<int>(E);
  p.k = static_cast<int>(top_k);
  p.renormalize = renormalize != 0;
  cudaError_t e = coda::launch_route_backward(p, dtype == CODA_F32, stream, use_pdl());
  return e == cudaSuccess ? CODA_OK : cuda_fail(e, "coda_route_backward launch");
}

coda_status coda_expert_dispatch(const void* X, const float* scale, const int32_t* slots, void* Xs, float* scale_s,
                                 int64_t M, int64_t N, int64_t top_k, int64_t T, coda_dtype dtype,
                                 cudaStream_t stream) {
  g_msg[0] = 0;
  REQUIRE(valid_dtype(dtype), "unknown dtype %d", static_cast<int>(dtype));
  TRY(check_places(M, N, top_k, T, dtype));
  REQUIRE((scale == nullptr) == (scale_s == nullptr), "scale and scale_s must be given together");
  if (M == 0 || T == 0) return CODA_OK;
  TRY(check_ptr(X, "X"));
  TRY(check_scalar_ptr(slots, "slots"));
  TRY(check_ptr(Xs, "Xs"));
  if (scale) {
    TRY(check_scalar_ptr(scale, "scale"));
    TRY(check_scalar_ptr(scale_s, "scale_s"));
  }
  const int64_t eb = elem_bytes(dtype);
  const Range outs[] = {rng("Xs", Xs, T * N * eb), rng("scale_s", scale_s, scale_s ? T * 4 : 0)};
  const Range ins[] = {rng("X", X, M * N * eb), rng("slots", slots, M * top_k * 4),
                       rng("scale", scale, scale ? M * 4 : 0)};
  TRY(check_overlaps(outs, 2, ins, 3));
  coda::DispatchParams p = {};
  p.X = X;
  p.scale = scale;
  p.slots = slots;
  p.Xs = Xs;
  p.scale_s = scale_s;
  p.row_bytes = N * eb;
  p.M = static_cast<int>(M);
  p.k = static_cast<int>(top_k);
  p.T = static_cast<int>(T);
  cudaError_t e = coda::launch_dispatch(p, stream, use_pdl());
  return e == cudaSuccess ? CODA_OK : cuda_fail(e, "coda_expert_dispatch launch");
}

coda_status coda_expert_combine(const void* Y, const int32_t* slots, const float* weights, const void* R, void* H,
                                float* P, int64_t M, int64_t N, int64_t top_k, int64_t T, coda_dtype dtype,
                                cudaStream_t stream) {
  g_msg[0] = 0;
  REQUIRE(dtype == CODA_F32 || dtype == CODA_BF16, "dtype must be CODA_F32 or CODA_BF16");
  TRY(check_places(M, N, top_k, T, dtype));
  REQUIRE(M * coda::combine_blocks(N, dtype == CODA_F32) < INT32_MAX,
          "M = %" PRId64 ", N = %" PRId64 ": too many blocks for one launch", M, N);
  if (M == 0) return CODA_OK;
  if (T > 0) TRY(check_ptr(Y, "Y"));
  TRY(check_scalar_ptr(slots, "slots"));
  if (weights) TRY(check_scalar_ptr(weights, "weights"));
  if (R) TRY(check_ptr(R, "R"));
  TRY(check_ptr(H, "H"));
  if (P) TRY(check_ptr(P, "P"));
  const int64_t eb = elem_bytes(dtype), mn = M * N * eb;
  const Range outs[] = {rng("H", H, mn), rng("P", P, P ? M * coda_partial_cols(N) * 4 : 0)};
  const Range ins[] = {rng("Y", Y, T * N * eb), rng("slots", slots, M * top_k * 4),
                       rng("weights", weights, weights ? M * top_k * 4 : 0), rng("R", R, R ? mn : 0)};
  TRY(check_overlaps(outs, 2, ins, 4));
  coda::CombineParams p = {};
  p.Y = Y;
  p.slots = slots;
  p.weights = weights;
  p.R = R;
  p.H = H;
  p.P = P;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.k = static_cast<int>(top_k);
  p.T = static_cast<int>(T);
  cudaError_t e = coda::launch_combine(p, dtype == CODA_F32, stream, use_pdl());
  return e == cudaSuccess ? CODA_OK : cuda_fail(e, "coda_expert_combine launch");
}

coda_status coda_expert_combine_backward(const void* dH, const void* Y, const int32_t* slots, const float* weights,
                                         void* dY, float* dweights, int64_t M, int64_t N, int64_t top_k, int64_t T,
                                         coda_dtype dtype, cudaStream_t stream) {
  g_msg[0] = 0;
  REQUIRE(dtype == CODA_F32 || dtype == CODA_BF16, "dtype must be CODA_F32 or CODA_BF16");
  TRY(check_places(M, N, top_k, T, dtype));
  if (M == 0) return CODA_OK;
  TRY(check_ptr(dH, "dH"));
  if (T > 0) {
    TRY(check_ptr(Y, "Y"));
    TRY(check_ptr(dY, "dY"));
  }
  TRY(check_scalar_ptr(slots, "slots"));
  TRY(check_scalar_ptr(weights, "weights"));
  TRY(check_scalar_ptr(dweights, "dweights"));
  const int64_t eb = elem_bytes(dtype), pairs = M * top_k * 4;
  const Range outs[] = {rng("dY", dY, T * N * eb), rng("dweights", dweights, pairs)};
  const Range ins[] = {rng("dH", dH, M * N * eb), rng("Y", Y, T * N * eb), rng("slots", slots, pairs),
                       rng("weights", weights, pairs)};
  TRY(check_overlaps(outs, 2, ins, 4));
  coda::CombineGradParams p = {};
  p.dH = dH;
  p.Y = Y;
  p.slots = slots;
  p.weights = weights;
  p.dY = dY;
  p.dweights = dweights;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.k = static_cast<int>(top_k);
  p.T = static_cast<int>(T);
  cudaError_t e = coda::launch_combine_backward(p, dtype == CODA_F32, stream, use_pdl());
  return e == cudaSuccess ? CODA_OK : cuda_fail(e, "coda_expert_combine_backward launch");
}

coda_status coda_grouped_gemm(const void* X, const void* W, coda_layout w_layout, const int32_t* offsets,
                              const float* row_scale, const float* w_scale, void* Y, int64_t T, int64_t E, int64_t N,
                              int64_t K, coda_dtype dtype, cudaStream_t stream) {
  g_msg[0] = 0;
  REQUIRE(dtype == CODA_BF16 || dtype == CODA_E4M3, "coda_grouped_gemm: dtype must be CODA_BF16 or CODA_E4M3");
  REQUIRE(w_layout == CODA_K_MAJOR || w_layout == CODA_MN_MAJOR, "unknown layout");
  const bool mn = w_layout == CODA_MN_MAJOR;
  REQUIRE(!mn || dtype == CODA_BF16, "MN-major weights are bf16 only");
  TRY(check_grouped(T, E, N, K, dtype, "N"));
  if (T == 0) return CODA_OK;
  TRY(check_group_scales(dtype, row_scale, w_scale));
  TRY(check_ptr(X, "X"));
  TRY(check_ptr(W, "W"));
  TRY(check_scalar_ptr(offsets, "offsets"));
  TRY(check_ptr(Y, "Y"));
  const int64_t eb = elem_bytes(dtype);
  const Range outs[] = {rng("Y", Y, T * N * 2)};
  const Range ins[] = {rng("X", X, T * K * eb), rng("W", W, E * N * K * eb), rng("offsets", offsets, (E + 1) * 4),
                       rng("row_scale", row_scale, row_scale ? T * 4 : 0),
                       rng("w_scale", w_scale, w_scale ? E * 4 : 0)};
  TRY(check_overlaps(outs, 1, ins, 5));
  coda::GroupProblem p = group_problem(mn ? coda::kGroupPlainMN : coda::kGroupPlain, X, W, Y, offsets, T, E, N, K, stream);
  p.row_scale = row_scale;
  p.w_scale = w_scale;
  return run_grouped("coda_grouped_gemm", p, dtype);
}

coda_status coda_grouped_gemm_swiglu(const void* X, const void* Wgu, const int32_t* offsets, const float* row_scale,
                                     const float* w_scale, void* Act, void* GU, int64_t T, int64_t E, int64_t I,
                                     int64_t K, coda_dtype dtype, cudaStream_t stream) {
  g_msg[0] = 0;
  REQUIRE(dtype == CODA_BF16 || dtype == CODA_E4M3, "coda_grouped_gemm_swiglu: dtype must be CODA_BF16 or CODA_E4M3");
  REQUIRE(GU == nullptr || dtype == CODA_BF16, "saving the SwiGLU pre-activations is bf16 only");
  TRY(check_grouped(T, E, I, K, dtype, "I"));
  if (T == 0) return CODA_OK;
  TRY(check_group_scales(dtype, row_scale, w_scale));
  TRY(check_ptr(X, "X"));
  TRY(check_ptr(Wgu, "Wgu"));
  TRY(check_scalar_ptr(offsets, "offsets"));
  TRY(check_ptr(Act, "Act"));
  if (GU) TRY(check_ptr(GU, "GU"));
  const int64_t eb = elem_bytes(dtype);
  const Range outs[] = {rng("Act", Act, T * I * 2), rng("GU", GU, GU ? T * 2 * I * 2 : 0)};
  const Range ins[] = {rng("X", X, T * K * eb), rng("Wgu", Wgu, E * 2 * I * K * eb),
                       rng("offsets", offsets, (E + 1) * 4), rng("row_scale", row_scale, row_scale ? T * 4 : 0),
                       rng("w_scale", w_scale, w_scale ? E * 4 : 0)};
  TRY(check_overlaps(outs, 2, ins, 5));
  coda::GroupProblem p =
      group_problem(GU ? coda::kGroupSwiGLUSave : coda::kGroupSwiGLU, X, Wgu, Act, offsets, T, E, I, K, stream);
  p.GU = GU;
  p.row_scale = row_scale;
  p.w_scale = w_scale;
  return run_grouped("coda_grouped_gemm_swiglu", p, dtype);
}

coda_status coda_grouped_gemm_swiglu_backward(const void* dY, const void* Wd, const void* GU, const int32_t* offsets,
                                              void* dGU, int64_t T, int64_t E, int64_t I, int64_t K, coda_dtype dtype,
                                              cudaStream_t stream) {
  g_msg[0] = 0;
  REQUIRE(dtype == CODA_BF16, "coda_grouped_gemm_swiglu_backward: dtype must be CODA_BF16");
  TRY(check_grouped(T, E, I, K, dtype, "I"));
  if (T == 0) return CODA_OK;
  TRY(check_ptr(dY, "dY"));
  TRY(check_ptr(Wd, "Wd"));
  TRY(check_ptr(GU, "GU"));
  TRY(check_scalar_ptr(offsets, "offsets"));
  TRY(check_ptr(dGU, "dGU"));
  const Range outs[] = {rng("dGU", dGU, T * 2 * I * 2)};
  const Range ins[] = {rng("dY", dY, T * K * 2), rng("Wd", Wd, E * K * I * 2), rng("GU", GU, T * 2 * I * 2),
                       rng("offsets", offsets, (E + 1) * 4)};
  TRY(check_overlaps(outs, 1, ins, 4));
  coda::GroupProblem p = group_problem(coda::kGroupSwiGLUBwd, dY, Wd, dGU, offsets, T, E, I, K, stream);
  p.GU = const_cast<void*>(GU);
  return run_grouped("coda_grouped_gemm_swiglu_backward", p, dtype);
}

coda_status coda_grouped_gemm_wgrad(const void* dY, const void* X, const int32_t* offsets, void* dW, int64_t T,
                                    int64_t E, int64_t N, int64_t K, coda_dtype dtype, cudaStream_t stream) {
  g_msg[0] = 0;
  REQUIRE(dtype == CODA_BF16, "coda_grouped_gemm_wgrad: dtype must be CODA_BF16");
  TRY(check_grouped(T, E, N, K, dtype, "N"));
  TRY(check_ptr(dW, "dW"));
  if (T == 0) {
    cudaError_t e = cudaMemsetAsync(dW, 0, static_cast<size_t>(E * N * K) * 2, stream);
    return e == cudaSuccess ? CODA_OK : cuda_fail(e, "cudaMemsetAsync(dW)");
  }
  TRY(check_ptr(dY, "dY"));
  TRY(check_ptr(X, "X"));
  TRY(check_scalar_ptr(offsets, "offsets"));
  const Range outs[] = {rng("dW", dW, E * N * K * 2)};
  const Range ins[] = {rng("dY", dY, T * N * 2), rng("X", X, T * K * 2), rng("offsets", offsets, (E + 1) * 4)};
  TRY(check_overlaps(outs, 1, ins, 3));
  return run_grouped("coda_grouped_gemm_wgrad",
                     group_problem(coda::kGroupWgrad, dY, X, dW, offsets, T, E, N, K, stream), dtype);
}

}  // extern "C"

// --------------------------------------------------- allocation-free block ----
// Some callers cannot call cudaMalloc at all: runtimes that own every byte of
// device memory and hand a kernel library no workspace, and hot paths where
// an allocation (which may synchronise the device) is not acceptable.  For
// them coda_block_swiglu_noalloc keeps the one-launch block's band counters
// in this file-scope device array instead of a caller workspace.  Every GPU
// that loads the library holds it (4100 bytes) until the process exits.
static __device__ __align__(256) unsigned g_noalloc_band_counters[(kNoAllocMaxRows + 127) / 128 + 1];

namespace {

std::mutex g_noalloc_mu;
void* g_noalloc_addr[64] = {};

// The array's name is only a host-side stand-in: the kernel needs its device
// address, looked up once per device with that device current.
coda_status noalloc_counters(void** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= 64) return fail(CODA_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
  std::lock_guard<std::mutex> lock(g_noalloc_mu);
  if (g_noalloc_addr[dev] == nullptr) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_noalloc_band_counters);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(band counters)");
    g_noalloc_addr[dev] = p;
  }
  *out = g_noalloc_addr[dev];
  return CODA_OK;
}

}  // namespace

extern "C" coda_status coda_block_swiglu_noalloc(const void* X, const void* W1t, const void* R, const void* Wgt,
                                                 const void* Wut, float eps, void* H, float* P, float* r_out,
                                                 void* Act, int64_t M, int64_t N, int64_t K, int64_t I,
                                                 coda_dtype dtype, cudaStream_t stream) {
  g_msg[0] = 0;
  if (M > kNoAllocMaxRows)
    return fail(CODA_ERR_INVALID_ARG,
                "M = %" PRId64 " exceeds the %d rows of the library's built-in band counters; use coda_block_swiglu "
                "with a workspace",
                M, kNoAllocMaxRows);
  if (M <= 0) return coda_block_swiglu(X, W1t, R, Wgt, Wut, eps, H, P, r_out, Act, M, N, K, I, dtype, nullptr, stream);
  void* counters = nullptr;
  TRY(noalloc_counters(&counters));
  // every argument is checked before anything is enqueued, so a rejected
  // call leaves the shared array untouched
  coda::GemmProblem p;
  TRY(block_prepare(coda::kEpiSwiGLU, X, W1t, R, Wgt, Wut, eps, H, P, r_out, Act, M, N, K, I, dtype, counters, stream,
                    &p));
  // every call shares the array: start from zero whatever the last call left
  const int64_t bytes = coda_block_workspace_bytes(M);
  cudaError_t e = cudaMemsetAsync(counters, 0, static_cast<size_t>(bytes), stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync(band counters)");
  return run_gemm(dtype, p);
}
