// Tile epilogues of the block-scaled GEMM for a linear layer with bias, activation and residual:
//   forward          P = X W^T + bias,  Z = act(P) + R        (P optionally re-quantized, for the backward)
//   input gradient   Z = (dY W) * act'(P) + R                  with P the saved INT8 pre-activation
// Z leaves re-quantized per 32x32 block or rounded once to a dense fp32 / bf16 / fp16 matrix.
//
// One warp holds two horizontally adjacent 32x32 blocks of the finished fp32 tile, lane = row, so a
// lane's own 32 or 64 bytes of a row are contiguous but the 32 lanes' rows are far apart: direct
// 16-byte accesses would touch 32 half-used sectors each. Every matrix access here goes through a
// 2 KB shared-memory staging area per warp instead, as 32 rows of 64 bytes: four neighbouring lanes
// move a row's 64 bytes, eight rows per instruction. Row r keeps its 16-byte chunk c at chunk position
// c ^ ((r >> 1) & 3), so both sides of the transposition are free of bank conflicts.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "act.cuh"
#include "kernels.h"
#include "quant.cuh"

namespace jf {

constexpr int kStageBytes = 2048;   // staging of one epilogue warp: 32 rows x 64 bytes

// What a tile epilogue reads and writes besides the accumulators (device pointers; null = absent).
struct EpilogueParams {
  const float* bias;        // forward: [cols]
  const int8_t* act_q;      // input gradient: codes and scales of the saved pre-activation
  const float* act_s;
  const uint8_t* res;       // residual: dense of type res_type, or INT8 codes with scales res_s
  const float* res_s;
  uint8_t* y;               // dense output
  int64_t res_ld, y_ld;     // row pitches in bytes
  int res_type, y_type;     // kDenseF32 / kDenseBf16 / kDenseF16; res_type may be kResI8
};

__device__ __forceinline__ uint8_t* stage_at(uint8_t* sm, int row, int chunk) {
  return sm + row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}

// Lane r's 64 bytes (w) to row r of a matrix with row pitch ld; only the first `chunks` of a row's four
// 16-byte chunks exist.
__device__ __forceinline__ void rows64_store(uint8_t* g, int64_t ld, int chunks, const uint32_t (&w)[16], uint8_t* sm,
                                             int lane) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4*>(stage_at(sm, lane, c)) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  __syncwarp();
  const int c = lane & 3;
#pragma unroll
  for (int r = lane >> 2; r < 32; r += 8)
    if (c < chunks) *reinterpret_cast<uint4*>(g + r * ld + c * 16) = *reinterpret_cast<const uint4*>(stage_at(sm, r, c));
  __syncwarp();
}

// The reverse: lane r receives row r's 64 bytes (zeros in chunks that do not exist). Plain loads, not
// the read-only path: the residual may be the output matrix itself.
__device__ __forceinline__ void rows64_load(const uint8_t* g, int64_t ld, int chunks, uint32_t (&w)[16], uint8_t* sm,
                                            int lane) {
  const int c = lane & 3;
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = c < chunks ? *reinterpret_cast<const uint4*>(g + ((lane >> 2) + 8 * i) * ld + c * 16) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(stage_at(sm, (lane >> 2) + 8 * i, c)) = v[i];
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint4 u = *reinterpret_cast<const uint4*>(stage_at(sm, lane, k));
    w[4 * k] = u.x; w[4 * k + 1] = u.y; w[4 * k + 2] = u.z; w[4 * k + 3] = u.w;
  }
  __syncwarp();
}

// Re-quantize one block (lane = row): its 32 codes in w[0..7]; lane 0 writes the scale.
__device__ __forceinline__ void block_codes(const float (&v)[32], uint32_t* w, float* s, int lane) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) m = fmaxf(m, fabsf(v[i]));
  const BlockQuant bq = block_quant(warp_max_nonneg(m));
  quant_pack<32>(v, bq, w);
  if (lane == 0) *s = bq.s;
}

// Both blocks' codes (`two` false: only the first exists) and scales.
__device__ __forceinline__ void store_codes(const float (&v)[2][32], int8_t* q, int64_t ld, float* s, bool two,
                                            uint8_t* sm, int lane) {
  uint32_t w[16];
  block_codes(v[0], w, s, lane);
  if (two) block_codes(v[1], w + 8, s + 1, lane);
  else
#pragma unroll
    for (int i = 8; i < 16; ++i) w[i] = 0u;
  rows64_store(reinterpret_cast<uint8_t*>(q), ld, two ? 4 : 2, w, sm, lane);
}

// One row's 32 values of a block, rounded to nearest even, as a 16-bit type.
template <bool BF16>
__device__ __forceinline__ void pack16(const float (&v)[32], uint32_t (&w)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (BF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
}

__device__ __forceinline__ void store_dense(const float (&v)[32], uint8_t* y, int64_t ld, int type, uint8_t* sm, int lane) {
  uint32_t w[16];
  if (type == kDenseF32) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[16 * half + i]);
      rows64_store(y + 64 * half, ld, 4, w, sm, lane);
    }
    return;
  }
  if (type == kDenseBf16) pack16<true>(v, w);
  else pack16<false>(v, w);
  rows64_store(y, ld, 4, w, sm, lane);
}

__device__ __forceinline__ void add_dense(float (&v)[32], const uint8_t* r, int64_t ld, int type, uint8_t* sm, int lane) {
  uint32_t w[16];
  if (type == kDenseF32) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      rows64_load(r + 64 * half, ld, 4, w, sm, lane);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[16 * half + i] += __uint_as_float(w[i]);
    }
    return;
  }
  rows64_load(r, ld, 4, w, sm, lane);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (type == kDenseBf16) {
      v[2 * i] += __uint_as_float(w[i] << 16);
      v[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] += f.x;
      v[2 * i + 1] += f.y;
    }
  }
}

// v += q s for one block's row of codes.
__device__ __forceinline__ void add_codes(float (&v)[32], const uint32_t* w, float s) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f[4];
    i8x4_to_f32(w[i], f);
#pragma unroll
    for (int j = 0; j < 4; j += 2)
      fma_x2(f[j], f[j + 1], s, s, v[4 * i + j], v[4 * i + j + 1], v[4 * i + j], v[4 * i + j + 1]);
  }
}

__device__ __forceinline__ void activate(float (&v)[32], int act) {
  if (act == kActGelu) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) gelu_f32_x2(v[i], v[i + 1]);
  } else if (act == kActGeluTanh) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = gelu_tanh_f32(v[i]);
  } else if (act == kActSilu) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = silu_f32(v[i]);
  } else if (act == kActRelu) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = fmaxf(v[i], 0.0f);
  }
}

// v *= act'(q s) for one block: a block's pre-activation has at most 256 distinct values, so the warp
// tabulates act' of all of them (8 evaluations a lane instead of 32) in its staging area, indexed by the
// code's raw byte.
__device__ __forceinline__ void times_act_grad(float (&v)[32], const uint32_t* w, float s, int act, float* tab, int lane) {
#pragma unroll 1
  for (int b = lane; b < 256; b += 32) tab[b] = act_grad_f32(float(int8_t(b)) * s, act);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] *= tab[(w[i >> 2] >> (8 * (i & 3))) & 0xFFu];
  __syncwarp();
}

// The finished fp32 tile part acc (blocks (rbk, cbk) and, when `two`, (rbk, cbk + 1) of an output of ncb
// block columns and ld_q columns) through bias / activation / residual to its outputs.
template <bool GRAD>
__device__ __forceinline__ void linear_epilogue(const EpilogueParams& e, int act, float (&acc)[2][32], int8_t* y_q,
                                                float* y_s, int8_t* pre_q, float* pre_s, int64_t ld_q, int rbk, int cbk,
                                                int ncb, bool two, uint8_t* sm, int lane) {
  const int64_t off = int64_t(rbk) * 32 * ld_q + int64_t(cbk) * 32, soff = int64_t(rbk) * ncb + cbk;
  if constexpr (!GRAD) {
    if (e.bias != nullptr) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && !two) break;
        const float4* b4 = reinterpret_cast<const float4*>(e.bias + (cbk + h) * 32);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 b = __ldg(b4 + i);
          add_x2(acc[h][4 * i], acc[h][4 * i + 1], b.x, b.y, acc[h][4 * i], acc[h][4 * i + 1]);
          add_x2(acc[h][4 * i + 2], acc[h][4 * i + 3], b.z, b.w, acc[h][4 * i + 2], acc[h][4 * i + 3]);
        }
      }
    }
    if (pre_q != nullptr) store_codes(acc, pre_q + off, ld_q, pre_s + soff, two, sm, lane);
    activate(acc[0], act);
    if (two) activate(acc[1], act);
  } else if (act != kActNone) {
    uint32_t w[16];
    rows64_load(reinterpret_cast<const uint8_t*>(e.act_q) + off, ld_q, two ? 4 : 2, w, sm, lane);
    times_act_grad(acc[0], w, __ldg(e.act_s + soff), act, reinterpret_cast<float*>(sm), lane);
    if (two) times_act_grad(acc[1], w + 8, __ldg(e.act_s + soff + 1), act, reinterpret_cast<float*>(sm), lane);
  }
  if (e.res != nullptr) {
    if (e.res_type == kResI8) {
      uint32_t w[16];
      rows64_load(e.res + off, ld_q, two ? 4 : 2, w, sm, lane);
      add_codes(acc[0], w, __ldg(e.res_s + soff));
      if (two) add_codes(acc[1], w + 8, __ldg(e.res_s + soff + 1));
    } else {
      const int64_t eb = e.res_type == kDenseF32 ? 128 : 64;   // bytes of 32 columns
      const uint8_t* r = e.res + int64_t(rbk) * 32 * e.res_ld + cbk * eb;
      add_dense(acc[0], r, e.res_ld, e.res_type, sm, lane);
      if (two) add_dense(acc[1], r + eb, e.res_ld, e.res_type, sm, lane);
    }
  }
  if (y_q != nullptr) store_codes(acc, y_q + off, ld_q, y_s + soff, two, sm, lane);
  if (e.y != nullptr) {
    const int64_t eb = e.y_type == kDenseF32 ? 128 : 64;
    uint8_t* y = e.y + int64_t(rbk) * 32 * e.y_ld + cbk * eb;
    store_dense(acc[0], y, e.y_ld, e.y_type, sm, lane);
    if (two) store_dense(acc[1], y + eb, e.y_ld, e.y_type, sm, lane);
  }
}

}  // namespace jf
