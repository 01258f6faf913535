// C ABI of the library: argument validation, then the kernel launch (see include/jetfire.h).
#include <cstdint>
#include <cstdlib>
#include <mutex>
#include <cuda_runtime.h>

// NVTX ranges around the compute entry points, compiled in only with -DJF_NVTX (the separate
// instrumented build of build_lib.py --nvtx): header-only NVTX 3, no library to link.
#ifdef JF_NVTX
#include <nvtx3/nvToolsExt.h>
namespace {
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};
}  // namespace
#define JF_RANGE(name) const NvtxRange jf_nvtx_range_(name)
#else
#define JF_RANGE(name) ((void)0)
#endif

#include "jetfire.h"
#include "kernels.h"
#include "ptx.cuh"

namespace jf {
__device__ unsigned int g_status = 0u;
}

namespace {

struct DevInfo {
  int sm_count = 0;
  bool ok = false;
  unsigned int* status = nullptr;  // device address of jf::g_status on this device
};

// Per-device SM count and capability check (cached per device ordinal; the first call on a device
// fills its entry under a lock, so concurrent first calls from several threads are safe). The
// cached status-word address belongs to the device's primary context: resetting the device
// (cudaDeviceReset) while the library is loaded is not supported.
DevInfo device_info() {
  static std::mutex mu;
  static DevInfo cache[64];
  static bool probed[64] = {false};
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return DevInfo{};
  }
  std::lock_guard<std::mutex> lock(mu);
  if (!probed[dev]) {
    DevInfo d;
    int major = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) == cudaSuccess &&
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) {
      d.ok = (major == 10);
      d.sm_count = sms;
      void* addr = nullptr;
      if (cudaGetSymbolAddress(&addr, jf::g_status) == cudaSuccess) {
        d.status = static_cast<unsigned int*>(addr);
      } else {
        cudaGetLastError();
        d.ok = false;
      }
    } else {
      cudaGetLastError();
    }
    cache[dev] = d;
    probed[dev] = true;
  }
  return cache[dev];
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool dims_ok(int64_t r, int64_t c) {
  return r >= 0 && c >= 0 && (r % 32) == 0 && (c % 32) == 0 && r < (int64_t(1) << 31) && c < (int64_t(1) << 31);
}
inline bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  if (a == nullptr || b == nullptr || na <= 0 || nb <= 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + uintptr_t(nb) && b0 < a0 + uintptr_t(na);
}
inline int64_t elem_size(jf_dtype dt) { return dt == JF_F32 ? 4 : 2; }
inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? JF_OK : JF_ERR_CUDA; }

// JF_PLAIN_LOADS=1 in the environment when the library is loaded selects the quantizer's plain-load
// kernel, which otherwise serves only inputs the driver will not describe with a TMA tensor map. The
// variable is read once, at load time, so no call reads the environment.
const bool g_plain_loads = [] {
  const char* v = std::getenv("JF_PLAIN_LOADS");
  return v != nullptr && v[0] == '1';
}();
inline bool plain_loads_forced() { return g_plain_loads; }

int check_cq(const jf_cqtensor& t) {
  if (!dims_ok(t.rows, t.cols)) return JF_ERR_SHAPE;
  if (t.rows == 0 || t.cols == 0) return JF_OK;
  if (t.q == nullptr || t.s == nullptr) return JF_ERR_NULL;
  if (!aligned(t.q, 16) || !aligned(t.s, 4)) return JF_ERR_ALIGN;
  return JF_OK;
}

// Output quantized tensor; `need_q` false allows q == NULL (fp32-only output).
int check_q(const jf_qtensor& t, bool need_q) {
  if (!dims_ok(t.rows, t.cols)) return JF_ERR_SHAPE;
  if (t.rows == 0 || t.cols == 0) return JF_OK;
  if (t.q == nullptr) return need_q ? JF_ERR_NULL : JF_OK;
  if (t.s == nullptr) return JF_ERR_NULL;
  if (!aligned(t.q, 16) || !aligned(t.s, 4)) return JF_ERR_ALIGN;
  return JF_OK;
}

int64_t qbytes(const jf_cqtensor& t) { return t.rows * t.cols; }
int64_t sbytes(int64_t r, int64_t c) { return (r / 32) * (c / 32) * 4; }

// Shared validation + launch of the three GEMMs. A/B are the stored operands.
// `pre` (activation kActGelu only; q may be NULL) receives the re-quantized pre-activation.
int gemm_call(int mode, const jf_cqtensor& A, const jf_cqtensor& B, const jf_qtensor& Y, float* y_f32,
              int64_t rows, int64_t cols, int64_t depth, void* stream, int act = jf::kActNone,
              jf_qtensor pre = jf_qtensor{nullptr, nullptr, 0, 0}) {
  int st;
  if ((st = check_cq(A)) != JF_OK) return st;
  if ((st = check_cq(B)) != JF_OK) return st;
  if ((st = check_q(Y, false)) != JF_OK) return st;
  if (Y.rows != rows || Y.cols != cols) return JF_ERR_SHAPE;
  if (pre.q != nullptr) {
    if ((st = check_q(pre, true)) != JF_OK) return st;
    if (pre.rows != rows || pre.cols != cols) return JF_ERR_SHAPE;
  }
  if (rows == 0 || cols == 0) return JF_OK;
  if (Y.q == nullptr && y_f32 == nullptr) return JF_ERR_NULL;
  if (y_f32 != nullptr && !aligned(y_f32, 16)) return JF_ERR_ALIGN;
  // outputs must not overlap inputs (nor each other)
  const void* ins[4] = {A.q, A.s, B.q, B.s};
  const int64_t in_n[4] = {qbytes(A), sbytes(A.rows, A.cols), qbytes(B), sbytes(B.rows, B.cols)};
  const void* outs[5] = {Y.q, Y.q ? Y.s : nullptr, y_f32, pre.q, pre.q ? pre.s : nullptr};
  const int64_t out_n[5] = {rows * cols, sbytes(rows, cols), rows * cols * 4, rows * cols, sbytes(rows, cols)};
  for (int o = 0; o < 5; ++o) {
    for (int i = 0; i < 4; ++i)
      if (overlap(outs[o], out_n[o], ins[i], in_n[i])) return JF_ERR_ALIAS;
    for (int o2 = o + 1; o2 < 5; ++o2)
      if (overlap(outs[o], out_n[o], outs[o2], out_n[o2])) return JF_ERR_ALIAS;
  }
  const DevInfo d = device_info();
  if (!d.ok) return JF_ERR_DEVICE;
  jf::GemmArgs g = {};
  g.mode = mode;
  g.a_q = A.q;
  g.a_s = A.s;
  g.b_q = B.q;
  g.b_s = B.s;
  g.rows = rows;
  g.cols = cols;
  g.depth = depth;
  g.a_ld = A.cols;
  g.b_ld = B.cols;
  g.y_q = Y.q;
  g.y_s = Y.q ? Y.s : nullptr;
  g.y = y_f32;
  g.y_type = jf::kDenseF32;
  g.y_ld = cols;
  g.act = act;
  g.pre_q = pre.q;
  g.pre_s = pre.q ? pre.s : nullptr;
  g.status = d.status;
  if (depth == 0) {
    // empty contraction: the result is exactly zero (codes 0, scales 0)
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (Y.q) {
      e = cudaMemsetAsync(Y.q, 0, size_t(rows * cols), s);
      if (e == cudaSuccess) e = cudaMemsetAsync(Y.s, 0, size_t(sbytes(rows, cols)), s);
    }
    if (e == cudaSuccess && y_f32) e = cudaMemsetAsync(y_f32, 0, size_t(rows * cols * 4), s);
    // GELU(0) = 0: the fused output and the pre-activation are zero as well
    if (e == cudaSuccess && pre.q) {
      e = cudaMemsetAsync(pre.q, 0, size_t(rows * cols), s);
      if (e == cudaSuccess) e = cudaMemsetAsync(pre.s, 0, size_t(sbytes(rows, cols)), s);
    }
    return cuda_status(e);
  }
  return cuda_status(jf::launch_gemm(g, d.sm_count, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

// Bytes of the row statistics of a [rows, cols] tensor: int32 [rows][cols/32][2].
inline int64_t statbytes(int64_t rows, int64_t cols) { return rows * (cols / 32) * 2 * 4; }

static int quantize_impl(const void* x, jf_dtype dt, int64_t rows, int64_t cols, int8_t* q, float* s,
                         int32_t* stats, bool want_stats, void* stream) {
  if (dt != JF_F32 && dt != JF_BF16 && dt != JF_F16) return JF_ERR_DTYPE;
  if (!dims_ok(rows, cols)) return JF_ERR_SHAPE;
  if (rows == 0 || cols == 0) return JF_OK;
  if (x == nullptr || q == nullptr || s == nullptr || (want_stats && stats == nullptr)) return JF_ERR_NULL;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(s, 4) || (want_stats && !aligned(stats, 8))) return JF_ERR_ALIGN;
  const int64_t nx = rows * cols * elem_size(dt);
  if (overlap(q, rows * cols, x, nx) || overlap(s, sbytes(rows, cols), x, nx) ||
      overlap(q, rows * cols, s, sbytes(rows, cols)))
    return JF_ERR_ALIAS;
  if (want_stats) {
    const int64_t nst = statbytes(rows, cols);
    if (overlap(stats, nst, x, nx) || overlap(stats, nst, q, rows * cols) || overlap(stats, nst, s, sbytes(rows, cols)))
      return JF_ERR_ALIAS;
  }
  const DevInfo d = device_info();
  if (!d.ok) return JF_ERR_DEVICE;
  return cuda_status(jf::launch_quantize(x, int(dt), rows, cols, q, s, want_stats ? stats : nullptr,
                                          plain_loads_forced() ? nullptr : d.status, d.sm_count,
                                          static_cast<cudaStream_t>(stream)));
}

int jf_quantize_block(const void* x, jf_dtype dt, int64_t rows, int64_t cols, int8_t* q, float* s,
                      void* stream) {
  JF_RANGE(__func__);
  return quantize_impl(x, dt, rows, cols, q, s, nullptr, false, stream);
}

int jf_quantize_block_rowstats(const void* x, jf_dtype dt, int64_t rows, int64_t cols, int8_t* q, float* s,
                               int32_t* stats, void* stream) {
  JF_RANGE(__func__);
  return quantize_impl(x, dt, rows, cols, q, s, stats, true, stream);
}

int jf_dequantize_block(const int8_t* q, const float* s, int64_t rows, int64_t cols, void* y, jf_dtype dt,
                        void* stream) {
  JF_RANGE(__func__);
  if (dt != JF_F32 && dt != JF_BF16 && dt != JF_F16) return JF_ERR_DTYPE;
  if (!dims_ok(rows, cols)) return JF_ERR_SHAPE;
  if (rows == 0 || cols == 0) return JF_OK;
  if (q == nullptr || s == nullptr || y == nullptr) return JF_ERR_NULL;
  if (!aligned(q, 16) || !aligned(s, 4) || !aligned(y, 16)) return JF_ERR_ALIGN;
  const int64_t ny = rows * cols * elem_size(dt);
  if (overlap(y, ny, q, rows * cols) || overlap(y, ny, s, sbytes(rows, cols))) return JF_ERR_ALIAS;
  const DevInfo d = device_info();
  if (!d.ok) return JF_ERR_DEVICE;
  return cuda_status(jf::launch_dequantize(q, s, rows, cols, y, int(dt), d.sm_count, static_cast<cudaStream_t>(stream)));
}

int jf_linear_fwd(jf_cqtensor X, jf_cqtensor W, jf_qtensor Y, float* y_f32, void* stream) {
  JF_RANGE(__func__);
  if (!dims_ok(X.rows, X.cols) || !dims_ok(W.rows, W.cols)) return JF_ERR_SHAPE;
  if (X.cols != W.cols) return JF_ERR_SHAPE;
  return gemm_call(jf::kFwd, X, W, Y, y_f32, X.rows, W.rows, X.cols, stream);
}

int jf_linear_fwd_gelu(jf_cqtensor X, jf_cqtensor W, jf_qtensor Y, jf_qtensor Ypre, void* stream) {
  JF_RANGE(__func__);
  if (!dims_ok(X.rows, X.cols) || !dims_ok(W.rows, W.cols)) return JF_ERR_SHAPE;
  if (X.cols != W.cols) return JF_ERR_SHAPE;
  if (Y.q == nullptr && X.rows != 0 && W.rows != 0) return JF_ERR_NULL;
  return gemm_call(jf::kFwd, X, W, Y, nullptr, X.rows, W.rows, X.cols, stream, jf::kActGelu, Ypre);
}

int jf_linear_dgrad(jf_cqtensor dY, jf_cqtensor W, jf_qtensor dX, float* dx_f32, void* stream) {
  JF_RANGE(__func__);
  if (!dims_ok(dY.rows, dY.cols) || !dims_ok(W.rows, W.cols)) return JF_ERR_SHAPE;
  if (dY.cols != W.rows) return JF_ERR_SHAPE;
  return gemm_call(jf::kDgrad, dY, W, dX, dx_f32, dY.rows, W.cols, dY.cols, stream);
}

int jf_linear_wgrad(jf_cqtensor dY, jf_cqtensor X, jf_qtensor dW, float* dw_f32, void* stream) {
  JF_RANGE(__func__);
  if (!dims_ok(dY.rows, dY.cols) || !dims_ok(X.rows, X.cols)) return JF_ERR_SHAPE;
  if (dY.rows != X.rows) return JF_ERR_SHAPE;
  return gemm_call(jf::kWgrad, dY, X, dW, dw_f32, dY.cols, X.cols, dY.rows, stream);
}

int jf_gelu_i8(jf_cqtensor X, jf_qtensor Y, void* stream) {
  JF_RANGE(__func__);
  int st;
  if ((st = check_cq(X)) != JF_OK) return st;
  if ((st = check_q(Y, true)) != JF_OK) return st;
  if (X.rows != Y.rows || X.cols != Y.cols) return JF_ERR_SHAPE;
  if (X.rows == 0 || X.cols == 0) return JF_OK;
  const int64_t nq = qbytes(X), ns = sbytes(X.rows, X.cols);
  if (overlap(Y.q, nq, X.q, nq) || overlap(Y.q, nq, X.s, ns) || overlap(Y.s, ns, X.q, nq) ||
      overlap(Y.s, ns, X.s, ns) || overlap(Y.q, nq, Y.s, ns))
    return JF_ERR_ALIAS;
  const DevInfo d = device_info();
  if (!d.ok) return JF_ERR_DEVICE;
  return cuda_status(jf::launch_gelu_i8(X.q, X.s, X.rows, X.cols, Y.q, Y.s, d.sm_count, static_cast<cudaStream_t>(stream)));
}

static int layernorm_impl(jf_cqtensor X, const int32_t* stats, bool want_stats, const float* gamma,
                          const float* beta, float eps, jf_qtensor Y, void* stream) {
  int st;
  if ((st = check_cq(X)) != JF_OK) return st;
  if ((st = check_q(Y, true)) != JF_OK) return st;
  if (X.rows != Y.rows || X.cols != Y.cols) return JF_ERR_SHAPE;
  if (X.rows == 0 || X.cols == 0) return JF_OK;
  if (gamma == nullptr || beta == nullptr || (want_stats && stats == nullptr)) return JF_ERR_NULL;
  if (!aligned(gamma, 16) || !aligned(beta, 16) || (want_stats && !aligned(stats, 8))) return JF_ERR_ALIGN;
  const int64_t nq = qbytes(X), ns = sbytes(X.rows, X.cols);
  if (overlap(Y.q, nq, X.q, nq) || overlap(Y.q, nq, X.s, ns) || overlap(Y.s, ns, X.q, nq) ||
      overlap(Y.s, ns, X.s, ns) || overlap(Y.q, nq, Y.s, ns) || overlap(Y.q, nq, gamma, X.cols * 4) ||
      overlap(Y.q, nq, beta, X.cols * 4) || overlap(Y.s, ns, gamma, X.cols * 4) || overlap(Y.s, ns, beta, X.cols * 4))
    return JF_ERR_ALIAS;
  if (want_stats) {
    const int64_t nst = statbytes(X.rows, X.cols);
    if (overlap(Y.q, nq, stats, nst) || overlap(Y.s, ns, stats, nst)) return JF_ERR_ALIAS;
  }
  const DevInfo d = device_info();
  if (!d.ok) return JF_ERR_DEVICE;
  return cuda_status(jf::launch_layernorm_i8(X.q, X.s, X.rows, X.cols, gamma, beta, eps, Y.q, Y.s,
                                             want_stats ? stats : nullptr, static_cast<cudaStream_t>(stream)));
}

int jf_layernorm_i8(jf_cqtensor X, const float* gamma, const float* beta, float eps, jf_qtensor Y,
                    void* stream) {
  JF_RANGE(__func__);
  return layernorm_impl(X, nullptr, false, gamma, beta, eps, Y, stream);
}

int jf_layernorm_i8_rowstats(jf_cqtensor X, const int32_t* stats, const float* gamma, const float* beta, float eps,
                             jf_qtensor Y, void* stream) {
  JF_RANGE(__func__);
  return layernorm_impl(X, stats, true, gamma, beta, eps, Y, stream);
}

int jf_gelu_i8_bwd(jf_cqtensor X, jf_cqtensor dY, jf_qtensor dX, void* stream) {
  JF_RANGE(__func__);
  int st;
  if ((st = check_cq(X)) != JF_OK) return st;
  if ((st = check_cq(dY)) != JF_OK) return st;
  if ((st = check_q(dX, true)) != JF_OK) return st;
  if (X.rows != dY.rows || X.cols != dY.cols || X.rows != dX.rows || X.cols != dX.cols) return JF_ERR_SHAPE;
  if (X.rows == 0 || X.cols == 0) return JF_OK;
  const int64_t nq = qbytes(X), ns = sbytes(X.rows, X.cols);
  const void* ins[4] = {X.q, X.s, dY.q, dY.s};
  const int64_t in_n[4] = {nq, ns, nq, ns};
  for (int i = 0; i < 4; ++i)
    if (overlap(dX.q, nq, ins[i], in_n[i]) || overlap(dX.s, ns, ins[i], in_n[i])) return JF_ERR_ALIAS;
  if (overlap(dX.q, nq, dX.s, ns)) return JF_ERR_ALIAS;
  const DevInfo d = device_info();
  if (!d.ok) return JF_ERR_DEVICE;
  return cuda_status(jf::launch_gelu_i8_bwd(X.q, X.s, dY.q, dY.s, X.rows, X.cols, dX.q, dX.s, d.sm_count,
                                            static_cast<cudaStream_t>(stream)));
}

int64_t jf_layernorm_i8_bwd_workspace_bytes(int64_t rows, int64_t cols) {
  if (!dims_ok(rows, cols) || cols > jf::kLnBwdMaxCols) return -1;
  return jf::ln_bwd_ctas(rows) * 2 * cols * 4;
}

}  // extern "C"

namespace {
// Every check of the LayerNorm backward that does not involve the workspace, in the order both
// entry points apply them: tensors, shapes, NULL gamma, alignment, then overlaps among the
// inputs and outputs (the workspace is checked by the caller of this function).
int ln_bwd_validate(const jf_cqtensor& X, const jf_cqtensor& dY, const float* gamma, const jf_qtensor& dX,
                    const float* dgamma, const float* dbeta) {
  int st;
  if ((st = check_cq(X)) != JF_OK) return st;
  if ((st = check_cq(dY)) != JF_OK) return st;
  if ((st = check_q(dX, true)) != JF_OK) return st;
  if (X.rows != dY.rows || X.cols != dY.cols || X.rows != dX.rows || X.cols != dX.cols) return JF_ERR_SHAPE;
  if (X.cols > jf::kLnBwdMaxCols) return JF_ERR_SHAPE;
  if (X.rows == 0 || X.cols == 0) return JF_OK;
  if (gamma == nullptr) return JF_ERR_NULL;
  if (!aligned(gamma, 16) || !aligned(dgamma, 4) || !aligned(dbeta, 4)) return JF_ERR_ALIGN;
  const int64_t nq = qbytes(X), ns = sbytes(X.rows, X.cols), H = X.cols;
  const void* ins[5] = {X.q, X.s, dY.q, dY.s, gamma};
  const int64_t in_n[5] = {nq, ns, nq, ns, H * 4};
  const void* outs[4] = {dX.q, dX.s, dgamma, dbeta};
  const int64_t out_n[4] = {nq, ns, H * 4, H * 4};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 5; ++i)
      if (overlap(outs[o], out_n[o], ins[i], in_n[i])) return JF_ERR_ALIAS;
    for (int o2 = o + 1; o2 < 4; ++o2)
      if (overlap(outs[o], out_n[o], outs[o2], out_n[o2])) return JF_ERR_ALIAS;
  }
  return JF_OK;
}

// The launch shared by both entry points, after validation. `part` is the column-sum workspace
// (NULL when neither dgamma nor dbeta is wanted).
int ln_bwd_launch(const jf_cqtensor& X, const jf_cqtensor& dY, const float* gamma, float eps, const jf_qtensor& dX,
                  float* dgamma, float* dbeta, float* part, void* stream) {
  const DevInfo d = device_info();
  if (!d.ok) return JF_ERR_DEVICE;
  return cuda_status(jf::launch_layernorm_i8_bwd(X.q, X.s, dY.q, dY.s, X.rows, X.cols, gamma, eps, dX.q, dX.s, part,
                                                 dgamma, dbeta, static_cast<cudaStream_t>(stream)));
}
}  // namespace

extern "C" {

int jf_layernorm_i8_bwd(jf_cqtensor X, jf_cqtensor dY, const float* gamma, float eps, jf_qtensor dX, float* dgamma,
                        float* dbeta, void* workspace, int64_t workspace_bytes, void* stream) {
  JF_RANGE(__func__);
  int st;
  if ((st = ln_bwd_validate(X, dY, gamma, dX, dgamma, dbeta)) != JF_OK) return st;
  if (X.rows == 0 || X.cols == 0) return JF_OK;
  const bool want_param_grads = dgamma != nullptr || dbeta != nullptr;
  if (!want_param_grads) return ln_bwd_launch(X, dY, gamma, eps, dX, nullptr, nullptr, nullptr, stream);
  const int64_t nw = jf_layernorm_i8_bwd_workspace_bytes(X.rows, X.cols);
  if (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < nw) return JF_ERR_WORKSPACE;
  const int64_t nq = qbytes(X), ns = sbytes(X.rows, X.cols), H = X.cols;
  const void* others[7] = {X.q, X.s, dY.q, dY.s, gamma, dX.q, dX.s};
  const int64_t other_n[7] = {nq, ns, nq, ns, H * 4, nq, ns};
  for (int i = 0; i < 7; ++i)
    if (overlap(workspace, nw, others[i], other_n[i])) return JF_ERR_ALIAS;
  if (overlap(workspace, nw, dgamma, H * 4) || overlap(workspace, nw, dbeta, H * 4)) return JF_ERR_ALIAS;
  return ln_bwd_launch(X, dY, gamma, eps, dX, dgamma, dbeta, static_cast<float*>(workspace), stream);
}

int jf_layernorm_i8_bwd_noalloc(jf_cqtensor X, jf_cqtensor dY, const float* gamma, float eps, jf_qtensor dX,
                                float* dgamma, float* dbeta, void* stream) {
  JF_RANGE(__func__);
  // the same argument checks, in the same order, as jf_layernorm_i8_bwd; only then the scratch size
  int st;
  if ((st = ln_bwd_validate(X, dY, gamma, dX, dgamma, dbeta)) != JF_OK) return st;
  if (X.rows == 0 || X.cols == 0) return JF_OK;
  if (dgamma == nullptr && dbeta == nullptr) return ln_bwd_launch(X, dY, gamma, eps, dX, nullptr, nullptr, nullptr, stream);
  if (jf_layernorm_i8_bwd_workspace_bytes(X.rows, X.cols) > jf::kLnBwdScratchBytes) return JF_ERR_WORKSPACE;
  const DevInfo d = device_info();
  if (!d.ok) return JF_ERR_DEVICE;
  float* scratch = jf::ln_bwd_static_scratch();
  if (scratch == nullptr) return JF_ERR_CUDA;
  return ln_bwd_launch(X, dY, gamma, eps, dX, dgamma, dbeta, scratch, stream);
}

int64_t jf_granular_scale_count(int64_t rows, int64_t cols, jf_granularity g) {
  if (!dims_ok(rows, cols)) return -1;
  switch (g) {
    case JF_GRAN_BLOCK: return (rows / 32) * (cols / 32);
    case JF_GRAN_TOKEN: return rows;
    case JF_GRAN_CHANNEL: return cols;
    case JF_GRAN_TENSOR: return 1;
    default: return -1;
  }
}

namespace {
bool gran_ok(jf_granularity g) { return g == JF_GRAN_BLOCK || g == JF_GRAN_TOKEN || g == JF_GRAN_CHANNEL || g == JF_GRAN_TENSOR; }
}  // namespace

int jf_quantize_granular(const void* x, jf_dtype dt, int64_t rows, int64_t cols, jf_granularity g, int8_t* q,
                         float* s, void* stream) {
  JF_RANGE(__func__);
  if (dt != JF_F32 && dt != JF_BF16 && dt != JF_F16) return JF_ERR_DTYPE;
  if (!gran_ok(g)) return JF_ERR_ARG;
  if (!dims_ok(rows, cols)) return JF_ERR_SHAPE;
  if (rows == 0 || cols == 0) return JF_OK;
  if (x == nullptr || q == nullptr || s == nullptr) return JF_ERR_NULL;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(s, 4)) return JF_ERR_ALIGN;
  const int64_t nx = rows * cols * elem_size(dt), ns = jf_granular_scale_count(rows, cols, g) * 4;
  if (overlap(q, rows * cols, x, nx) || overlap(s, ns, x, nx) || overlap(q, rows * cols, s, ns)) return JF_ERR_ALIAS;
  const DevInfo d = device_info();
  if (!d.ok) return JF_ERR_DEVICE;
  return cuda_status(jf::launch_quantize_granular(x, int(dt), rows, cols, int(g), q, s,
                                                   plain_loads_forced() ? nullptr : d.status, d.sm_count,
                                                  static_cast<cudaStream_t>(stream)));
}

int jf_dequantize_granular(const int8_t* q, const float* s, int64_t rows, int64_t cols, jf_granularity g, void* y,
                           jf_dtype dt, void* stream) {
  JF_RANGE(__func__);
  if (dt != JF_F32 && dt != JF_BF16 && dt != JF_F16) return JF_ERR_DTYPE;
  if (!gran_ok(g)) return JF_ERR_ARG;
  if (!dims_ok(rows, cols)) return JF_ERR_SHAPE;
  if (rows == 0 || cols == 0) return JF_OK;
  if (q == nullptr || s == nullptr || y == nullptr) return JF_ERR_NULL;
  if (!aligned(q, 16) || !aligned(s, 4) || !aligned(y, 16)) return JF_ERR_ALIGN;
  const int64_t ny = rows * cols * elem_size(dt), ns = jf_granular_scale_count(rows, cols, g) * 4;
  if (overlap(y, ny, q, rows * cols) || overlap(y, ny, s, ns)) return JF_ERR_ALIAS;
  const DevInfo d = device_info();
  if (!d.ok) return JF_ERR_DEVICE;
  return cuda_status(jf::launch_dequantize_granular(q, s, rows, cols, int(g), y, int(dt), d.sm_count,
                                                    static_cast<cudaStream_t>(stream)));
}

int jf_quantization_error(const void* x, jf_dtype dt, const int8_t* q, const float* s, int64_t rows, int64_t cols,
                          jf_granularity g, double* sums, void* stream) {
  JF_RANGE(__func__);
  if (dt != JF_F32 && dt != JF_BF16 && dt != JF_F16) return JF_ERR_DTYPE;
  if (!gran_ok(g)) return JF_ERR_ARG;
  if (!dims_ok(rows, cols)) return JF_ERR_SHAPE;
  if (sums == nullptr) return JF_ERR_NULL;
  if (!aligned(sums, 8)) return JF_ERR_ALIGN;
  const int64_t nx = rows * cols * elem_size(dt), ns = jf_granular_scale_count(rows, cols, g) * 4;
  if (rows != 0 && cols != 0) {
    if (x == nullptr || q == nullptr || s == nullptr) return JF_ERR_NULL;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(s, 4)) return JF_ERR_ALIGN;
    if (overlap(sums, 24, x, nx) || overlap(sums, 24, q, rows * cols) || overlap(sums, 24, s, ns)) return JF_ERR_ALIAS;
  }
  const DevInfo d = device_info();
  if (!d.ok) return JF_ERR_DEVICE;
  if (rows == 0 || cols == 0)
    return cuda_status(cudaMemsetAsync(sums, 0, 3 * sizeof(double), static_cast<cudaStream_t>(stream)));
  return cuda_status(jf::launch_quant_error(x, int(dt), q, s, rows, cols, int(g), sums, d.sm_count,
                                            static_cast<cudaStream_t>(stream)));
}

int jf_mx_quantize(const void* x, jf_dtype dt, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                   void* stream) {
  JF_RANGE(__func__);
  if (dt != JF_F32 && dt != JF_BF16 && dt != JF_F16) return JF_ERR_DTYPE;
  if (!dims_ok(rows, cols)) return JF_ERR_SHAPE;
  if (rows == 0 || cols == 0) return JF_OK;
  if (x == nullptr || codes == nullptr || scales == nullptr) return JF_ERR_NULL;
  if (!aligned(x, 16) || !aligned(codes, 16)) return JF_ERR_ALIGN;
  const int64_t nx = rows * cols * elem_size(dt), nc = rows * cols, ns = rows * (cols / 32);
  if (overlap(codes, nc, x, nx) || overlap(scales, ns, x, nx) || overlap(codes, nc, scales, ns)) return JF_ERR_ALIAS;
  const DevInfo d = device_info();
  if (!d.ok) return JF_ERR_DEVICE;
  return cuda_status(jf::launch_mx_quantize(x, int(dt), rows, cols, codes, scales, d.sm_count,
                                            static_cast<cudaStream_t>(stream)));
}

int jf_mx_linear_fwd(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes, const uint8_t* b_scales,
                     int64_t M, int64_t N, int64_t K, float* y, void* stream) {
  JF_RANGE(__func__);
  if (!dims_ok(M, K) || !dims_ok(N, K) || K % 128 != 0) return JF_ERR_SHAPE;
  if (M == 0 || N == 0) return JF_OK;
  if (K == 0) return JF_ERR_SHAPE;
  if (a_codes == nullptr || a_scales == nullptr || b_codes == nullptr || b_scales == nullptr || y == nullptr)
    return JF_ERR_NULL;
  if (!aligned(a_codes, 16) || !aligned(b_codes, 16) || !aligned(a_scales, 4) || !aligned(b_scales, 4) ||
      !aligned(y, 16))
    return JF_ERR_ALIGN;
  const void* ins[4] = {a_codes, a_scales, b_codes, b_scales};
  const int64_t in_n[4] = {M * K, M * (K / 32), N * K, N * (K / 32)};
  for (int i = 0; i < 4; ++i)
    if (overlap(y, M * N * 4, ins[i], in_n[i])) return JF_ERR_ALIAS;
  const DevInfo d = device_info();
  if (!d.ok) return JF_ERR_DEVICE;
  return cuda_status(jf::launch_mx_gemm(a_codes, a_scales, b_codes, b_scales, M, N, K, y, d.status, d.sm_count,
                                        static_cast<cudaStream_t>(stream)));
}

namespace {

bool dtype_ok(jf_dtype dt) { return dt == JF_F32 || dt == JF_BF16 || dt == JF_F16; }

// More elements than an address space has bytes: extents below it do not overflow.
constexpr int64_t kMaxElements = int64_t(1) << 50;

// A dense [rows, cols] operand of the epilogue calls, and the bytes from its first to its last element.
int check_matrix(const void* p, jf_dtype dt, int64_t ld, int64_t rows, int64_t cols) {
  if (p == nullptr) return JF_OK;
  if (!dtype_ok(dt)) return JF_ERR_DTYPE;
  if (ld < cols || ld >= kMaxElements || (rows > 1 && ld > kMaxElements / (rows - 1))) return JF_ERR_SHAPE;
  if (!aligned(p, 16) || (ld * elem_size(dt)) % 16 != 0) return JF_ERR_ALIGN;
  return JF_OK;
}
int64_t extent(jf_dtype dt, int64_t ld, int64_t rows, int64_t cols) { return ((rows - 1) * ld + cols) * elem_size(dt); }

// The linear layer's forward (bias, pre-activation output) and input gradient (saved pre-activation input)
// with activation and residual. rows x cols: the output; depth: the contraction.
int epilogue_call(int mode, const jf_cqtensor& A, const jf_cqtensor& B, const float* bias, const jf_cqtensor& saved,
                  jf_activation act, const jf_cqtensor& Rq, const jf_cmatrix& R, const jf_qtensor& Y, const jf_matrix& y,
                  const jf_qtensor& pre, int64_t rows, int64_t cols, int64_t depth, void* stream) {
  int st;
  if (act < JF_ACT_NONE || act > JF_ACT_SILU) return JF_ERR_ARG;
  if ((st = check_cq(A)) != JF_OK) return st;
  if ((st = check_cq(B)) != JF_OK) return st;
  const bool want_saved = mode == jf::kDgrad && act != JF_ACT_NONE;
  if (want_saved && ((st = check_cq(saved)) != JF_OK)) return st;
  if (want_saved && (saved.rows != rows || saved.cols != cols)) return JF_ERR_SHAPE;
  if (Rq.q != nullptr && R.p != nullptr) return JF_ERR_ARG;
  if (Rq.q != nullptr) {
    if ((st = check_cq(Rq)) != JF_OK) return st;
    if (Rq.rows != rows || Rq.cols != cols) return JF_ERR_SHAPE;
  }
  if ((st = check_matrix(R.p, R.dt, R.ld, rows, cols)) != JF_OK) return st;
  if ((st = check_matrix(y.p, y.dt, y.ld, rows, cols)) != JF_OK) return st;
  const jf_qtensor* const outs_q[2] = {&Y, &pre};
  for (const jf_qtensor* o : outs_q) {
    if (o->q == nullptr) continue;
    if ((st = check_q(*o, true)) != JF_OK) return st;
    if (o->rows != rows || o->cols != cols) return JF_ERR_SHAPE;
  }
  if (rows == 0 || cols == 0) return JF_OK;
  if (Y.q == nullptr && y.p == nullptr) return JF_ERR_NULL;
  if (!aligned(bias, 16)) return JF_ERR_ALIGN;
  const int64_t nq = rows * cols, ns = sbytes(rows, cols);
  const int64_t ny = y.p ? extent(y.dt, y.ld, rows, cols) : 0, nr = R.p ? extent(R.dt, R.ld, rows, cols) : 0;
  const bool in_place = y.p != nullptr && y.p == R.p && y.dt == R.dt && y.ld == R.ld;
  const void* ins[10] = {A.q, A.s, B.q, B.s, bias, want_saved ? saved.q : nullptr, want_saved ? saved.s : nullptr, Rq.q,
                         Rq.q ? Rq.s : nullptr, R.p};
  const int64_t in_n[10] = {qbytes(A), sbytes(A.rows, A.cols), qbytes(B), sbytes(B.rows, B.cols), cols * 4, nq, ns, nq, ns, nr};
  const void* outs[5] = {Y.q, Y.q ? Y.s : nullptr, y.p, pre.q, pre.q ? pre.s : nullptr};
  const int64_t out_n[5] = {nq, ns, ny, nq, ns};
  for (int o = 0; o < 5; ++o) {
    for (int i = 0; i < 10; ++i)
      if (overlap(outs[o], out_n[o], ins[i], in_n[i]) && !(o == 2 && i == 9 && in_place)) return JF_ERR_ALIAS;
    for (int o2 = o + 1; o2 < 5; ++o2)
      if (overlap(outs[o], out_n[o], outs[o2], out_n[o2])) return JF_ERR_ALIAS;
  }
  const DevInfo d = device_info();
  if (!d.ok) return JF_ERR_DEVICE;
  jf::GemmArgs g = {};
  g.mode = mode;
  g.a_q = A.q;
  g.a_s = A.s;
  g.b_q = B.q;
  g.b_s = B.s;
  g.rows = rows;
  g.cols = cols;
  g.depth = depth;
  g.a_ld = A.cols;
  g.b_ld = B.cols;
  g.y_q = Y.q;
  g.y_s = Y.q ? Y.s : nullptr;
  g.y = y.p;
  g.y_type = y.p ? int(y.dt) : 0;
  g.y_ld = y.ld;
  g.bias = bias;
  g.act = int(act);
  g.split_ok = true;
  if (want_saved) {
    g.act_q = saved.q;
    g.act_s = saved.s;
  }
  g.pre_q = pre.q;
  g.pre_s = pre.q ? pre.s : nullptr;
  if (Rq.q != nullptr) {
    g.res = Rq.q;
    g.res_s = Rq.s;
    g.res_type = jf::kResI8;
  } else if (R.p != nullptr) {
    g.res = R.p;
    g.res_type = int(R.dt);
    g.res_ld = R.ld;
  }
  g.status = d.status;
  return cuda_status(jf::launch_gemm(g, d.sm_count, static_cast<cudaStream_t>(stream)));
}

// The description shared by the two QKV calls.
int check_qkv(int64_t rows, const jf_qkv_rope* a) {
  if (a == nullptr) return JF_ERR_NULL;
  const int64_t lim = int64_t(1) << 31;
  if (a->layout != JF_ROPE_HALF && a->layout != JF_ROPE_INTERLEAVED) return JF_ERR_ARG;
  if (!(a->eps > 0.0f)) return JF_ERR_ARG;
  if (a->batch < 0 || a->seq < 0 || a->batch >= lim || a->seq >= lim || a->q_heads < 0 || a->kv_heads < 0 ||
      a->q_heads > 65535 || a->kv_heads > 65535 || a->head_dim < 32 || a->head_dim > 256 || a->head_dim % 32 != 0 ||
      a->rot_dim < 0 || a->rot_dim > a->head_dim || a->rot_dim % 16 != 0 || a->table_len < 0 || a->table_len >= lim * lim / 512 ||
      a->batch * a->seq > rows)
    return JF_ERR_SHAPE;
  if (a->rot_dim > 0 && a->positions == nullptr && a->seq > a->table_len) return JF_ERR_SHAPE;
  return JF_OK;
}

// One dense tensor of heads; bytes: from the first to the last element.
int check_heads(const void* p, const int64_t (&stride)[3], const int64_t (&size)[3], int64_t d, int64_t es, bool output,
                int64_t& bytes) {
  bytes = 0;
  if (size[0] == 0 || size[1] == 0 || size[2] == 0) return JF_OK;
  if (p == nullptr) return JF_ERR_NULL;
  if (!aligned(p, 16)) return JF_ERR_ALIGN;
  int64_t last = d - 1;
  for (int k = 0; k < 3; ++k) {
    if (size[k] == 1) continue;
    if (stride[k] < 0 || stride[k] > kMaxElements / (size[k] - 1)) return JF_ERR_SHAPE;
    if ((stride[k] * es) % 16 != 0) return JF_ERR_ALIGN;
    last += stride[k] * (size[k] - 1);
  }
  if (output) {   // from the smallest stride up, each must step over all that lies below it
    int64_t below = d;
    bool done[3] = {size[0] == 1, size[1] == 1, size[2] == 1};
    for (int n = 0; n < 3; ++n) {
      int best = -1;
      for (int k = 0; k < 3; ++k)
        if (!done[k] && (best < 0 || stride[k] < stride[best])) best = k;
      if (best < 0) break;
      if (stride[best] < below) return JF_ERR_SHAPE;
      below = stride[best] * (size[best] - 1) + below;
      done[best] = true;
    }
  }
  bytes = (last + 1) * es;
  return JF_OK;
}

int qkv_call(bool backward, const jf_cqtensor& X, const jf_qkv_rope* a, const jf_cheads (&t)[3], jf_dtype dt,
             const jf_qtensor& dX, float* dgq, float* dgk, void* workspace, int64_t workspace_bytes, void* stream) {
  int st;
  if (!dtype_ok(dt)) return JF_ERR_DTYPE;
  if (!dims_ok(X.rows, X.cols)) return JF_ERR_SHAPE;
  if ((st = check_qkv(X.rows, a)) != JF_OK) return st;
  if (X.cols != (a->q_heads + 2 * a->kv_heads) * a->head_dim) return JF_ERR_SHAPE;
  if (backward && (dX.rows != X.rows || dX.cols != X.cols)) return JF_ERR_SHAPE;
  const int64_t tokens = a->batch * a->seq, d = a->head_dim;
  const bool norm = (a->gamma_q != nullptr && a->q_heads > 0) || (a->gamma_k != nullptr && a->kv_heads > 0);
  const bool rotates = a->rot_dim > 0 && tokens > 0 && X.cols > 0;
  if ((dgq != nullptr && a->gamma_q == nullptr) || (dgk != nullptr && a->gamma_k == nullptr)) return JF_ERR_NULL;
  const bool want_dg = dgq != nullptr || dgk != nullptr;
  const bool reads_x = (!backward || norm) && tokens > 0;
  if (reads_x && (st = check_cq(X)) != JF_OK) return st;
  if (backward && (st = check_q(dX, true)) != JF_OK) return st;
  if (rotates && (a->cos_table == nullptr || a->sin_table == nullptr)) return JF_ERR_NULL;
  if (!aligned(a->cos_table, 16) || !aligned(a->sin_table, 16) || !aligned(a->positions, 8) || !aligned(a->gamma_q, 16) ||
      !aligned(a->gamma_k, 16) || !aligned(dgq, 4) || !aligned(dgk, 4))
    return JF_ERR_ALIGN;
  int64_t tb[3];
  for (int k = 0; k < 3; ++k) {
    const int64_t stride[3] = {t[k].stride_b, t[k].stride_s, t[k].stride_h};
    const int64_t size[3] = {a->batch, a->seq, k == 0 ? a->q_heads : a->kv_heads};
    if ((st = check_heads(t[k].p, stride, size, d, elem_size(dt), !backward, tb[k])) != JF_OK) return st;
  }
  const int64_t nq = X.rows * X.cols, ns = sbytes(X.rows, X.cols);
  const int64_t ntab = rotates ? a->table_len * (a->rot_dim / 2) * 4 : 0;
  const void* ins[10] = {reads_x ? X.q : nullptr, reads_x ? X.s : nullptr, a->cos_table, a->sin_table, a->positions,
                         a->gamma_q, a->gamma_k, backward ? t[0].p : nullptr, backward ? t[1].p : nullptr,
                         backward ? t[2].p : nullptr};
  const int64_t in_n[10] = {nq, ns, ntab, ntab, rotates ? tokens * 8 : 0, d * 4, d * 4, tb[0], tb[1], tb[2]};
  const int64_t nw = want_dg ? jf::qkv_bwd_ctas(X.rows, a->q_heads, a->kv_heads) * 2 * d * 4 : 0;
  if (want_dg && (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < nw)) return JF_ERR_WORKSPACE;
  const void* fo[3] = {t[0].p, t[1].p, t[2].p};
  const void* bo[5] = {dX.q, dX.s, dgq, dgk, want_dg ? workspace : nullptr};
  const int64_t bo_n[5] = {nq, ns, d * 4, d * 4, nw};
  for (int i = 0; i < 10; ++i) {
    if (!backward)
      for (int o = 0; o < 3; ++o)
        if (overlap(fo[o], tb[o], ins[i], in_n[i])) return JF_ERR_ALIAS;
    if (backward)
      for (int o = 0; o < 5; ++o)
        if (overlap(bo[o], bo_n[o], ins[i], in_n[i])) return JF_ERR_ALIAS;
  }
  if (backward)
    for (int o = 0; o < 5; ++o)
      for (int o2 = o + 1; o2 < 5; ++o2)
        if (overlap(bo[o], bo_n[o], bo[o2], bo_n[o2])) return JF_ERR_ALIAS;
  if (!backward && (tokens == 0 || X.cols == 0)) return JF_OK;
  if (backward && nq == 0 && !want_dg) return JF_OK;
  const DevInfo dev = device_info();
  if (!dev.ok) return JF_ERR_DEVICE;
  jf::QkvRopeArgs g = {};
  g.x_q = X.q;
  g.x_s = X.s;
  g.rows = X.rows;
  g.cols = X.cols;
  g.tokens = tokens;
  g.seq = a->seq > 0 ? a->seq : 1;
  g.hq = int(a->q_heads);
  g.hkv = int(a->kv_heads);
  g.d = int(d);
  g.rot = int(a->rot_dim);
  g.interleaved = a->layout == JF_ROPE_INTERLEAVED;
  g.cos = a->cos_table;
  g.sin = a->sin_table;
  g.table_len = a->table_len;
  g.positions = a->positions;
  g.gamma_q = a->gamma_q;
  g.gamma_k = a->gamma_k;
  g.eps = a->eps;
  jf::DenseHeads* const h[3] = {&g.q, &g.k, &g.v};
  for (int k = 0; k < 3; ++k) *h[k] = jf::DenseHeads{const_cast<void*>(t[k].p), t[k].stride_b, t[k].stride_s, t[k].stride_h};
  g.dx_q = dX.q;
  g.dx_s = dX.s;
  g.part = want_dg ? static_cast<float*>(workspace) : nullptr;
  g.dgamma_q = dgq;
  g.dgamma_k = dgk;
  g.status = dev.status;
  return cuda_status(jf::launch_qkv_rope(g, backward, int(dt), dev.sm_count, static_cast<cudaStream_t>(stream)));
}

}  // namespace

int jf_linear_fwd_epilogue(jf_cqtensor X, jf_cqtensor W, const float* bias, jf_activation act, jf_cqtensor Rq,
                           jf_cmatrix R, jf_qtensor Y, jf_matrix y, jf_qtensor P, void* stream) {
  JF_RANGE(__func__);
  if (!dims_ok(X.rows, X.cols) || !dims_ok(W.rows, W.cols)) return JF_ERR_SHAPE;
  if (X.cols != W.cols) return JF_ERR_SHAPE;
  return epilogue_call(jf::kFwd, X, W, bias, jf_cqtensor{nullptr, nullptr, 0, 0}, act, Rq, R, Y, y, P, X.rows, W.rows,
                       X.cols, stream);
}

int jf_linear_dgrad_epilogue(jf_cqtensor dY, jf_cqtensor W, jf_cqtensor P, jf_activation act, jf_cqtensor Rq,
                             jf_cmatrix R, jf_qtensor Y, jf_matrix y, void* stream) {
  JF_RANGE(__func__);
  if (!dims_ok(dY.rows, dY.cols) || !dims_ok(W.rows, W.cols)) return JF_ERR_SHAPE;
  if (dY.cols != W.rows) return JF_ERR_SHAPE;
  return epilogue_call(jf::kDgrad, dY, W, nullptr, P, act, Rq, R, Y, y, jf_qtensor{nullptr, nullptr, 0, 0}, dY.rows, W.cols,
                       dY.cols, stream);
}

int jf_bias_grad(jf_cqtensor dY, float* db, void* stream) {
  JF_RANGE(__func__);
  int st;
  if ((st = check_cq(dY)) != JF_OK) return st;
  if (dY.cols == 0) return JF_OK;
  if (db == nullptr) return JF_ERR_NULL;
  if (!aligned(db, 4)) return JF_ERR_ALIGN;
  if (dY.rows != 0 && (overlap(db, dY.cols * 4, dY.q, qbytes(dY)) || overlap(db, dY.cols * 4, dY.s, sbytes(dY.rows, dY.cols))))
    return JF_ERR_ALIAS;
  const DevInfo d = device_info();
  if (!d.ok) return JF_ERR_DEVICE;
  return cuda_status(jf::launch_bias_grad(dY.q, dY.s, dY.rows, dY.cols, db, static_cast<cudaStream_t>(stream)));
}

int jf_rope_table(const double* inv_freq, int64_t half, double magnitude, int64_t length, float* cos_table, float* sin_table,
                  void* stream) {
  JF_RANGE(__func__);
  if (half < 1 || half > 128 || length < 0 || length >= (int64_t(1) << 40)) return JF_ERR_SHAPE;
  if (length == 0) return JF_OK;
  if (inv_freq == nullptr || cos_table == nullptr || sin_table == nullptr) return JF_ERR_NULL;
  if (!aligned(cos_table, 16) || !aligned(sin_table, 16)) return JF_ERR_ALIGN;
  if (overlap(cos_table, length * half * 4, sin_table, length * half * 4)) return JF_ERR_ALIAS;
  const DevInfo d = device_info();
  if (!d.ok) return JF_ERR_DEVICE;
  return cuda_status(jf::launch_rope_table(inv_freq, half, magnitude, length, cos_table, sin_table, d.sm_count,
                                           static_cast<cudaStream_t>(stream)));
}

int64_t jf_qkv_rope_bwd_workspace_bytes(int64_t rows, const jf_qkv_rope* a) {
  if (rows < 0 || rows % 32 != 0 || rows >= (int64_t(1) << 31) || check_qkv(rows, a) != JF_OK) return -1;
  return jf::qkv_bwd_ctas(rows, a->q_heads, a->kv_heads) * 2 * a->head_dim * 4;
}

int jf_qkv_rope_fwd(jf_cqtensor QKV, const jf_qkv_rope* a, jf_heads q, jf_heads k, jf_heads v, jf_dtype dt, void* stream) {
  JF_RANGE(__func__);
  const jf_cheads t[3] = {{q.p, q.stride_b, q.stride_s, q.stride_h}, {k.p, k.stride_b, k.stride_s, k.stride_h},
                          {v.p, v.stride_b, v.stride_s, v.stride_h}};
  return qkv_call(false, QKV, a, t, dt, jf_qtensor{nullptr, nullptr, 0, 0}, nullptr, nullptr, nullptr, 0, stream);
}

int jf_qkv_rope_bwd(jf_cqtensor QKV, const jf_qkv_rope* a, jf_cheads dq, jf_cheads dk, jf_cheads dv, jf_dtype dt,
                    jf_qtensor dQKV, float* dgamma_q, float* dgamma_k, void* workspace, int64_t workspace_bytes,
                    void* stream) {
  JF_RANGE(__func__);
  const jf_cheads t[3] = {dq, dk, dv};
  return qkv_call(true, QKV, a, t, dt, dQKV, dgamma_q, dgamma_k, workspace, workspace_bytes, stream);
}

int jf_gemm_i8_s32(const int8_t* A, const int8_t* B, int32_t* C, int64_t M, int64_t N, int64_t K, void* stream) {
  JF_RANGE(__func__);
  if (M < 0 || N < 0 || K < 0 || M % 128 != 0 || N % 256 != 0 || K % 128 != 0 || K > 65536 ||
      M >= (int64_t(1) << 31) || N >= (int64_t(1) << 31))
    return JF_ERR_SHAPE;
  if (M == 0 || N == 0) return JF_OK;
  if (C == nullptr) return JF_ERR_NULL;
  if (!aligned(C, 16)) return JF_ERR_ALIGN;
  if (K == 0) return cuda_status(cudaMemsetAsync(C, 0, size_t(M * N * 4), static_cast<cudaStream_t>(stream)));
  if (A == nullptr || B == nullptr) return JF_ERR_NULL;
  if (!aligned(A, 16) || !aligned(B, 16)) return JF_ERR_ALIGN;
  if (overlap(C, M * N * 4, A, M * K) || overlap(C, M * N * 4, B, N * K)) return JF_ERR_ALIAS;
  const DevInfo d = device_info();
  if (!d.ok) return JF_ERR_DEVICE;
  return cuda_status(jf::launch_gemm_s32(A, B, C, M, N, K, d.status, d.sm_count, static_cast<cudaStream_t>(stream)));
}

int jf_selftest_wait_timeout(int64_t limit_ns, void* stream) {
  JF_RANGE(__func__);
  if (limit_ns < 1000000 || limit_ns > 10000000000ll) return JF_ERR_ARG;
  const DevInfo d = device_info();
  if (!d.ok) return JF_ERR_DEVICE;
  return cuda_status(jf::launch_wait_selftest(d.status, static_cast<unsigned long long>(limit_ns),
                                              static_cast<cudaStream_t>(stream)));
}

const char* jf_strerror(int status) {
  switch (status) {
    case JF_OK: return "ok";
    case JF_ERR_NULL: return "a required pointer is NULL";
    case JF_ERR_SHAPE: return "bad shape: dimensions must be non-negative multiples of 32 and agree";
    case JF_ERR_ALIGN: return "misaligned pointer (codes and fp32/bf16/fp16 data: 16 bytes; scales: 4 bytes)";
    case JF_ERR_DTYPE: return "unknown dtype";
    case JF_ERR_ALIAS: return "an output overlaps an input or another output";
    case JF_ERR_CUDA: return "a CUDA runtime/driver call failed";
    case JF_ERR_TIMEOUT: return "a kernel's bounded wait timed out; outputs are undefined";
    case JF_ERR_DEVICE: return "no usable sm_100 (B200) device is current";
    case JF_ERR_WORKSPACE: return "workspace is NULL, not 16-byte aligned or smaller than the size asked for";
    case JF_ERR_ARG: return "an enumerated argument (granularity, activation, layout) is unknown, or a scalar one out of range";
    case JF_ERR_RANGE: return "a position lay outside the rotary table; its token's rotated part is undefined";
    default: return "unknown status";
  }
}

int jf_device_status(void* stream) {
  JF_RANGE(__func__);
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return JF_ERR_CUDA;
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, jf::g_status, sizeof(v)) != cudaSuccess) return JF_ERR_CUDA;
  if (v != 0 && cudaMemcpyToSymbol(jf::g_status, &zero, sizeof(zero)) != cudaSuccess) return JF_ERR_CUDA;
  if (v & jf::kStatusTimeout) return JF_ERR_TIMEOUT;
  if (v & jf::kStatusRange) return JF_ERR_RANGE;
  return v ? JF_ERR_CUDA : JF_OK;
}

int jf_sm_count(void) {
  const DevInfo d = device_info();
  return d.sm_count;
}

}  // extern "C"
