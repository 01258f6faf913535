// Internal launch functions (called by the C ABI in api.cu after argument validation).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

namespace jf {

// The driver's cuTensorMapEncodeTiled (null if the driver does not provide it).
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// `status`: the device status word, raised when a bounded wait in the kernel runs out; null selects
// the plain-load kernel (no TMA staging, no waits). `stats` (optional, int32 [R][C/32][2]): per row
// and block, the sums of q and q^2 (what LayerNorm_i8 needs of its input rows).
cudaError_t launch_quantize(const void* x, int dtype, int64_t R, int64_t C, int8_t* q, float* s, int32_t* stats,
                            unsigned int* status, int sm_count, cudaStream_t st);
cudaError_t launch_dequantize(const int8_t* q, const float* s, int64_t R, int64_t C, void* y, int dtype,
                              int sm_count, cudaStream_t st);
cudaError_t launch_gelu_i8(const int8_t* q, const float* s, int64_t R, int64_t C, int8_t* qo, float* so,
                           int sm_count, cudaStream_t st);
// Failure-path self-test (selftest.cu): a bounded wait that runs out after limit_ns and raises the
// timeout bit of *status.
cudaError_t launch_wait_selftest(unsigned int* status, unsigned long long limit_ns, cudaStream_t st);

// MXFP8 comparison path (mxfp8.cu): MX quantization (E4M3 codes, E8M0 scale bytes per 1x32 block of
// a row) and Y = A B^T with the tensor core's block scaling (K a multiple of 128).
cudaError_t launch_mx_quantize(const void* x, int dtype, int64_t R, int64_t K, uint8_t* codes, uint8_t* scales,
                               int sm_count, cudaStream_t st);
cudaError_t launch_mx_gemm(const uint8_t* a_q, const uint8_t* a_s, const uint8_t* b_q, const uint8_t* b_s, int64_t M,
                           int64_t N, int64_t K, float* y, unsigned int* status, int sm_count, cudaStream_t st);

// Granularity variants of the quantizer and the quantization-error sums (granular.cu). Scales:
// block [R/32, C/32], token [R], channel [C], tensor [1].
enum Granularity { kGranBlock = 0, kGranToken = 1, kGranChannel = 2, kGranTensor = 3 };
cudaError_t launch_quantize_granular(const void* x, int dtype, int64_t R, int64_t C, int g, int8_t* q, float* s,
                                     unsigned int* status, int sm_count, cudaStream_t st);
cudaError_t launch_dequantize_granular(const int8_t* q, const float* s, int64_t R, int64_t C, int g, void* y,
                                       int dtype, int sm_count, cudaStream_t st);
cudaError_t launch_quant_error(const void* x, int dtype, const int8_t* q, const float* s, int64_t R, int64_t C, int g,
                               double* sums, int sm_count, cudaStream_t st);

// INT8 backward of GELU_i8 and LayerNorm_i8 (backward.cu). `part` is the fp32 workspace of
// per-CTA column sums, [ln_bwd_ctas(R)][2][H]; null when neither dgamma nor dbeta is wanted.
constexpr int64_t kLnBwdMaxCtas = 296;   // two resident CTAs on each of 148 SMs
constexpr int64_t kLnBwdMaxCols = 24576; // the [2][H] fp32 accumulators fit in one SM's shared memory
int64_t ln_bwd_ctas(int64_t R);
// Size of the static scratch the allocation-free LayerNorm backward uses in place of a workspace,
// and its device address on the current device (looked up once per device; null on failure).
constexpr int64_t kLnBwdScratchBytes = int64_t(16) << 20;
float* ln_bwd_static_scratch();
cudaError_t launch_gelu_i8_bwd(const int8_t* xq, const float* xs, const int8_t* dq, const float* ds, int64_t R,
                               int64_t C, int8_t* qo, float* so, int sm_count, cudaStream_t st);
cudaError_t launch_layernorm_i8_bwd(const int8_t* xq, const float* xs, const int8_t* dq, const float* ds, int64_t R,
                                    int64_t H, const float* gamma, float eps, int8_t* qo, float* so, float* part,
                                    float* dgamma, float* dbeta, cudaStream_t st);
cudaError_t launch_layernorm_i8(const int8_t* q, const float* s, int64_t R, int64_t H, const float* gamma,
                                const float* beta, float eps, int8_t* qo, float* so, const int32_t* stats,
                                cudaStream_t st);

// Column sums of an INT8 tensor (bias_grad.cu).
cudaError_t launch_bias_grad(const int8_t* q, const float* s, int64_t R, int64_t C, float* db, cudaStream_t st);

// Per-head norm and rotary positions between the INT8 QKV tensor and dense heads (qkv_rope.cu).
struct DenseHeads {           // element (batch b, token t, head h, dimension 0) at p + b stride_b + t stride_t + h stride_h
  void* p;
  int64_t stride_b, stride_t, stride_h;
};
struct QkvRopeArgs {
  const int8_t* x_q;          // [rows, cols] codes and scales of the projection's output
  const float* x_s;
  int64_t rows, cols;
  int64_t tokens, seq;        // valid rows; tokens of a sequence (row = batch * seq + token)
  int hq, hkv, d, rot;
  bool interleaved;
  const float* cos;           // [table_len, rot / 2]
  const float* sin;
  int64_t table_len;
  const int64_t* positions;   // [tokens], null: the token's index in its sequence
  const float* gamma_q;       // [d] norm weights, null: no norm
  const float* gamma_k;
  float eps;
  DenseHeads q, k, v;         // forward: outputs; backward: the gradients dq, dk, dv
  int8_t* dx_q;               // backward outputs
  float* dx_s;
  float* part;                // backward workspace [ctas][2][d], null when no weight gradient is wanted
  float* dgamma_q;
  float* dgamma_k;
  unsigned int* status;
};
int64_t qkv_bwd_ctas(int64_t rows, int64_t hq, int64_t hkv);
cudaError_t launch_qkv_rope(const QkvRopeArgs& a, bool backward, int dtype, int sm_count, cudaStream_t st);
// Tables of cos and sin (position * inv_freq[j]) * magnitude, [length, half], half <= 128; inv_freq is host memory.
cudaError_t launch_rope_table(const double* inv_freq, int64_t half, double magnitude, int64_t length, float* cos_out,
                              float* sin_out, int sm_count, cudaStream_t st);

// Block-scaled INT8 GEMM: out[r, c] = sum over 32-blocks kb of the contraction axis of
// fp32(sA(r/32, kb) * sB(c/32, kb)) * sum_{k in kb} A(r, k) B(c, k), re-quantized per 32x32 block.
// The operand views differ per mode (see gemm.cu).
enum GemmMode { kFwd = 0, kDgrad = 1, kWgrad = 2 };
// kActGelu is the GELU of jf_linear_fwd_gelu (gelu_f32), kActGeluEpi that of the epilogue calls (jf_activation's
// JF_ACT_GELU, gelu_epilogue_x2): the same function and fit, evaluated with fewer instructions.
enum GemmAct { kActNone = 0, kActRelu = 1, kActGeluEpi = 2, kActGeluTanh = 3, kActSilu = 4, kActGelu = 5 };
// Element type of a dense matrix (jf_dtype's values) or an INT8 residual.
enum DenseType { kDenseF32 = 0, kDenseBf16 = 1, kDenseF16 = 2, kResI8 = 3 };

struct GemmArgs {
  int mode;
  const int8_t* a_q;  // A codes (X for fwd, dY for dgrad and wgrad)
  const float* a_s;
  const int8_t* b_q;  // B codes (W for fwd and dgrad, X for wgrad)
  const float* b_s;
  int64_t rows, cols, depth;  // output rows, output cols, contraction length
  int64_t a_ld, b_ld;         // row pitch (elements) of the stored A and B matrices
  int8_t* y_q;                // nullable: the re-quantized result
  float* y_s;                 // non-null when y_q is
  void* y;                    // nullable: the dense result, y_type a DenseType, y_ld elements per row
  int y_type;
  int64_t y_ld;
  // the linear layers' epilogues (epilogue.cuh); null pointers are absent parts
  const float* bias;          // forward: fp32 [cols]
  int act;                    // GemmAct: forward, applied to the result; dgrad, its derivative at act_q / act_s
  const int8_t* act_q;        // dgrad with an activation: the saved pre-activation
  const float* act_s;
  int8_t* pre_q;              // forward: the re-quantized pre-activation
  float* pre_s;
  bool split_ok;              // few tiles may split a long contraction (another order of the fp32 sum)
  const void* res;            // residual: dense of DenseType res_type, or kResI8 codes with scales res_s
  const float* res_s;
  int res_type;
  int64_t res_ld;             // elements
  unsigned int* status;       // device status word (bit flags of ptx.cuh)
};

cudaError_t launch_gemm(const GemmArgs& g, int sm_count, cudaStream_t st);

// Plain INT8 GEMM C = A B^T (int32), A [M, K] and B [N, K] row-major: the tensor core's INT8 rate with
// no per-block rescale. M % 128 == 0, N % 256 == 0, K % 128 == 0.
cudaError_t launch_gemm_s32(const int8_t* a, const int8_t* b, int32_t* c, int64_t M, int64_t N, int64_t K,
                            unsigned int* status, int sm_count, cudaStream_t st);

}  // namespace jf
