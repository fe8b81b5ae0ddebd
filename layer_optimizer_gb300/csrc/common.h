// Internal helpers shared by the library's translation units: status and
// error-message plumbing, argument checks, small integer utilities.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>
#include <stdint.h>

#include <cstdarg>
#include <cstdio>
#include <string>

#include "sfopt.h"

namespace sf {

// NVTX range around one ABI call, so profiler timelines show library calls
// by name (header-only NVTX; a no-op unless a tool is attached).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

// Records a message for sf_last_error() (thread-local) and returns `st`.
sf_status fail(sf_status st, const char* fmt, ...);

// Clears the calling thread's last error message.
void clear_error();

// Maps a CUDA error to SF_ERR_CUDA with a message naming `what`.
sf_status cuda_fail(cudaError_t e, const char* what);

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

template <typename T>
constexpr T ceil_div(T a, T b) { return (a + b - 1) / b; }

// Number of SMs of the current device (cached per device).
int sm_count();

// Lets kernel `func` use up to `bytes` of dynamic shared memory on the
// current device (cudaFuncSetAttribute once per device, kernel and size;
// thread-safe).
sf_status allow_dynamic_smem(const void* func, size_t bytes);

// cuTensorMapEncodeTiled from the driver (looked up once), or null.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
  }();
  return fn;
}

// True when `p` points into device memory of the current device.  Every
// tensor map (TMA descriptor) this library encodes addresses such memory
// only; operands elsewhere (pinned host memory, a peer GPU's memory) take a
// path with plain loads or are rejected.
bool on_current_device(const void* p);

// Checks a matrix argument on the host: shape, leading dimension and type.
// want_rows / want_cols < 0 accept any size.  dtypes: a mask of 1 << sf_dtype.
sf_status check_matrix(const sf_matrix* m, const char* name, int64_t want_rows, int64_t want_cols, unsigned dtypes);

// Whether a byte belongs to elements of both matrices (null and empty ones have none): exact where their rows lie equally far
// apart or one of them has a single row, else judged by their first and last bytes.
bool overlap(const sf_matrix* a, const sf_matrix* b);

// Whether the two are one matrix: the same place, type and distance of rows (sizes are checked elsewhere).
bool same_matrix(const sf_matrix* a, const sf_matrix* b);

// Checks on the host that a vector (null passes) lies on a multiple of its element's size.
sf_status check_aligned(const void* p, size_t size, const char* name);

inline size_t dtype_bytes(int32_t t) { return t == SF_FP32 ? 4 : t == SF_BF16 ? 2 : 1; }

// Default bound for host waits, in milliseconds (SF_TIMEOUT_MS or 600 s).
int64_t default_timeout_ms();

// Polls `ev` (or a stream when ev is null) until it completes or the bound
// runs out.  Returns SF_OK, SF_ERR_TIMEOUT or SF_ERR_CUDA.
sf_status bounded_wait_event(cudaEvent_t ev, int64_t timeout_ms, const char* what);
sf_status bounded_wait_stream(cudaStream_t s, int64_t timeout_ms, const char* what);

// Checks for a pending launch error after enqueueing kernels.
inline sf_status check_launch(const char* what) {
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SF_OK : cuda_fail(e, what);
}

// Launch with programmatic stream serialisation: the kernel may be scheduled
// while the previous kernel in the stream drains; it must call
// griddepcontrol.wait before touching memory that kernel may write.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// fp32 constants of one AdamW step, derived in double and rounded once.
struct AdamConsts {
  float beta1, one_minus_beta1;
  float beta2, one_minus_beta2;
  float decay;          // 1 - lr * weight_decay
  float step_size;      // lr / (1 - beta1^t)
  float sqrt_bc2;       // sqrt(1 - beta2^t)
  float inv_sqrt_bc2;   // 1 / sqrt(1 - beta2^t), rounded once from double
  float eps;
};

// The device-side error words that bounded waits and index checks in the
// kernels set (0 = none; bit 1 = a wait ran out; bit 2 = an out-of-range index
// was skipped), one a translation unit, as symbols.
const void* device_error_lsp();
const void* device_error_adamw();
const void* device_error_gemm();
const void* device_error_lce();
const void* device_error_norm();
const void* device_error_wgrad();
const void* device_error_sandwich_fwd();
const void* device_error_sandwich_units();
const void* device_error_sandwich_strided();

// C = alpha A B^T (+ C) on the tensor cores (tc_gemm.cu): A bf16 [M][lda]
// row-major (K-major) or, with a_mn, [K][lda] (MN-major: A^T stored);
// B likewise [N][ldb] or, with b_mn, [K][ldb]; C fp32 [M][ldc].  With
// row_stats (float2 [M][ceil(N / 256)]) the epilogue also writes, per row and
// 256-column tile, the maximum of the row's values and the sum of
// exp(value - maximum).
constexpr int kTcTileN = 256;
constexpr int kTcStatCols = 128;     // columns of one entry of kTcStats' statistics
sf_status tc_gemm(const void* A, bool a_mn, const void* B, bool b_mn, float* C, int64_t M, int64_t N, int64_t K,
                  int64_t lda, int64_t ldb, int64_t ldc, float alpha, bool accumulate, cudaStream_t s,
                  float2* row_stats = nullptr);

// The same GEMM with the epilogues of the vocabulary-piece cross-entropy.
enum TcEpilogue : int {
  kTcF32 = 0,    // C fp32, as above
  kTcSplit = 1,  // C fp32 [splits][M][ldc]: partial products over parts of K
  kTcBf16 = 2,   // C bf16
  kTcStats = 3,  // row_stats, label_logit, and with `store` C = exp(A B^T - tile maximum) in bf16
  kTcRows = 5,   // C bf16 or fp32, product row i written to row row_map[i]
  kTcGrad = 4    // C = softmax - onehot(label) in bf16 from A B^T and lse, 0 in rows past M
};
struct TcJob {
  const void* A = nullptr;
  const void* B = nullptr;
  bool a_mn = false, b_mn = false;
  int64_t M = 0, N = 0, K = 0, lda = 0, ldb = 0;
  TcEpilogue epi = kTcF32;
  void* C = nullptr;               // fp32 or bf16 by the epilogue; null: not written (kTcStats without store)
  int64_t ldc = 0;
  float alpha = 1.0f;
  bool accumulate = false;         // fp32 epilogues
  int splits = 1;                  // kTcSplit
  float2* row_stats = nullptr;     // kTcF32: [M][tiles of kTcTileN]; kTcStats: [M][stats_ld], one entry per kTcStatCols
                                   // columns, at (col0 + column) / kTcStatCols
  int32_t stats_ld = 0;            // at least ceil((col0 + N) / kTcStatCols)
  int32_t col0 = 0;                // vocabulary id of column 0 (a multiple of 256)
  bool store = false;
  const int32_t* labels = nullptr; // [M] (kTcStats, kTcGrad); ids outside the product's columns match nothing
  float* label_logit = nullptr;    // [M]
  const float* lse = nullptr;      // [M]
  const float* scale = nullptr;    // device, one value: multiplies alpha (kTcSplit, kTcBf16, kTcRows)
  const int32_t* m_dev = nullptr;  // device-side M and K, at most the M and K above (not for kTcF32); an empty
  const int32_t* k_dev = nullptr;  // sum gives zeros
  const int32_t* row_map = nullptr;  // [M] (kTcRows)
  bool out_fp32 = false;           // kTcRows
  bool checked = false;            // the caller has checked that A, B and C are this device's memory
  bool chained = false;            // launched as a programmatic dependent of the previous kernel in the stream
};
sf_status tc_gemm(const TcJob& job, cudaStream_t s);

sf_status make_adam_consts(const sf_adamw_hparams* hp, int64_t step, bool with_decay,
                           AdamConsts* out);

// sf_checkpoint_load within the library (checkpoint.cu).
sf_status checkpoint_load(const sf_checkpoint* c, const float* row_factor, const void* gain, int32_t gain_dtype,
                          double gain_offset, const sf_matrix* y, cudaStream_t stream);

// The compressed AdamW step on the host cores for elements [b, e) of fp32
// S, m, v -> dS (host_adamw.cpp): bitwise the device kernel's results.
void host_adamw_compressed(const float* S, float* m, float* v, float* dS, int64_t b, int64_t e,
                           const AdamConsts& c);

// Cores this process may run on (its CPU affinity set), at least 1.
int usable_cores();

}  // namespace sf

#define SF_TRY(expr)                      \
  do {                                    \
    sf_status _st = (expr);               \
    if (_st != SF_OK) return _st;         \
  } while (0)

#define SF_CUDA_TRY(expr, what)                       \
  do {                                                \
    cudaError_t _e = (expr);                          \
    if (_e != cudaSuccess) return sf::cuda_fail(_e, what); \
  } while (0)
