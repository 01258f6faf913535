// Tile epilogues of the block-scaled GEMM for a linear layer with bias, activation and residual:
//   forward          P = X W^T + bias,  Z = act(P) + R        (P optionally re-quantized, for the backward)
//   input gradient   Z = (dY W) * act'(P) + R                  with P the saved INT8 pre-activation
// Z leaves re-quantized per 32x32 block or rounded once to a dense fp32 / bf16 / fp16 matrix.
//
// An output warp takes one finished 32x32 fp32 block at a time, lane = row. A lane's own 32 to 128 bytes of a
// row are contiguous but the 32 lanes' rows are far apart: direct 16-byte accesses would touch 32 half-used
// sectors each. Every matrix access here goes through the block's own shared memory (free once the block is in
// registers) instead, as 32 rows of 32 or 64 bytes: two or four neighbouring lanes move a row's bytes. Row r
// keeps its 16-byte chunk c at chunk position c ^ swizzle(r), so both sides of the transposition are
// free of bank conflicts.
//
// What bounds it: the chain of one warp (shared memory -> absmax -> scale -> codes -> shared memory -> global
// memory) beside two sum warps of the same sub-partition, ~1900 cycles a block, ~2600 a pass with GELU; four output
// warps have a tile's 16 blocks to go through, which a plain re-quantization does in the time of 16 contraction blocks and
// GELU with two outputs in that of 35-43.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "act.cuh"
#include "kernels.h"
#include "quant.cuh"

namespace jf {

// Which epilogue a kernel carries: none of the extras (weight gradient), a forward, an input gradient.
enum Epilogue { kEpiPlain = 0, kEpiForward = 1, kEpiGrad = 2 };

// What a tile epilogue reads and writes besides the accumulators (device pointers; null = absent).
struct EpilogueParams {
  const float* bias;        // forward: [cols]
  const int8_t* act_q;      // input gradient: codes and scales of the saved pre-activation
  const float* act_s;
  const uint8_t* res;       // residual: dense of type res_type, or INT8 codes with scales res_s
  const float* res_s;
  int8_t* y_q;              // re-quantized output
  float* y_s;
  int8_t* pre_q;            // forward: re-quantized pre-activation
  float* pre_s;
  uint8_t* y;               // dense output
  int64_t ld_q;             // columns of the output: the pitch of every INT8 matrix here
  int64_t res_ld, y_ld;     // row pitches in bytes of the dense ones
  int act;                  // GemmAct
  int res_type, y_type;     // kDenseF32 / kDenseBf16 / kDenseF16; res_type may be kResI8
};

// Staging position of 16-byte chunk c of row r, NC (2 or 4) chunks a row.
template <int NC>
__device__ __forceinline__ uint8_t* stage_at(uint8_t* sm, int r, int c) {
  return sm + r * (16 * NC) + ((c ^ (NC == 4 ? (r >> 1) & 3 : (r >> 2) & 1)) << 4);
}

// Lane r's 16 NC bytes (w) to row r of a matrix with row pitch ld.
template <int NC>
__device__ __forceinline__ void rows_store(uint8_t* g, int64_t ld, const uint32_t (&w)[4 * NC], uint8_t* sm, int lane) {
#pragma unroll
  for (int c = 0; c < NC; ++c)
    *reinterpret_cast<uint4*>(stage_at<NC>(sm, lane, c)) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  __syncwarp();
  const int c = lane % NC;
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += 32 / NC) {
    const int r = r0 + lane / NC;
    *reinterpret_cast<uint4*>(g + r * ld + c * 16) = *reinterpret_cast<const uint4*>(stage_at<NC>(sm, r, c));
  }
  __syncwarp();
}

// The reverse: lane r receives row r's bytes. Plain loads, not the read-only path: the residual may be the
// output matrix itself.
template <int NC>
__device__ __forceinline__ void rows_load(const uint8_t* g, int64_t ld, uint32_t (&w)[4 * NC], uint8_t* sm, int lane) {
  const int c = lane % NC;
  uint4 v[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) v[i] = *reinterpret_cast<const uint4*>(g + (lane / NC + 32 / NC * i) * ld + c * 16);
#pragma unroll
  for (int i = 0; i < NC; ++i) *reinterpret_cast<uint4*>(stage_at<NC>(sm, lane / NC + 32 / NC * i, c)) = v[i];
  __syncwarp();
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const uint4 u = *reinterpret_cast<const uint4*>(stage_at<NC>(sm, lane, k));
    w[4 * k] = u.x; w[4 * k + 1] = u.y; w[4 * k + 2] = u.z; w[4 * k + 3] = u.w;
  }
  __syncwarp();
}

// Re-quantize one block (lane = row) and write its codes (q: its first code) and its scale.
__device__ __forceinline__ void store_codes(const float (&v)[32], int8_t* q, int64_t ld, float* s, uint8_t* sm, int lane) {
  const BlockQuant bq = block_quant_approx(warp_max_nonneg(absmax32(v)));
  uint32_t w[8];
  // halves: a test per 8 values or for all 32 at once is 1-2% slower for the whole kernel (4096 x 1024 x 4096, GELU)
#pragma unroll
  for (int k = 0; k < 32; k += 16) {
    float far = bq.mode != 2 ? 1.0f : 0.0f;
    codes_fast<16>(v + k, bq.inv, w + k / 4, far);
    if (!(far < kFarLimit)) codes_exact<16>(v + k, bq.s, w + k / 4);
  }
  if (lane == 0) *s = bq.s;
  rows_store<2>(reinterpret_cast<uint8_t*>(q), ld, w, sm, lane);
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
      rows_store<4>(y + 64 * half, ld, w, sm, lane);
    }
    return;
  }
  if (type == kDenseBf16) pack16<true>(v, w);
  else pack16<false>(v, w);
  rows_store<4>(y, ld, w, sm, lane);
}

__device__ __forceinline__ void add_dense(float (&v)[32], const uint8_t* r, int64_t ld, int type, uint8_t* sm, int lane) {
  uint32_t w[16];
  if (type == kDenseF32) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      rows_load<4>(r + 64 * half, ld, w, sm, lane);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[16 * half + i] += __uint_as_float(w[i]);
    }
    return;
  }
  rows_load<4>(r, ld, w, sm, lane);
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
__device__ __forceinline__ void add_codes(float (&v)[32], const uint32_t (&w)[8], float s) {
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
  if (act == kActGeluEpi) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) gelu_epilogue_x2(v[i], v[i + 1]);
  } else if (act == kActGelu) {
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
    for (int i = 0; i < 32; ++i) asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(v[i]));   // a NaN stays one
  }
}

// v *= act'(q s) for one block: a block's pre-activation has at most 256 distinct values, so the warp
// tabulates act' of all of them in its staging area, indexed by the code's raw byte: 4 evaluations a lane
// instead of 32, since each serves m and -m.
__device__ __forceinline__ void times_act_grad(float (&v)[32], const uint32_t (&w)[8], float s, int act, float* tab, int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int m = lane + 1 + 32 * j;   // |code| 1 .. 128
    float at_pos, at_neg;
    act_grad_pair_epilogue(float(m) * s, act, at_pos, at_neg);
    if (m < 128) tab[m] = at_pos;
    tab[256 - m] = at_neg;
  }
  if (lane == 0) tab[0] = act == kActRelu ? 0.0f : fmaf(0.0f, s, 0.5f);   // NaN for a scale that is not finite
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] *= tab[(w[i >> 2] >> (8 * (i & 3))) & 0xFFu];
  __syncwarp();
}

// One finished fp32 block v = block (rbk, cbk) of an output of ncb block columns through bias / activation /
// residual to its outputs.
template <int EPI>
__device__ __forceinline__ void block_epilogue(const EpilogueParams& e, float (&v)[32], int rbk, int cbk, int ncb, uint8_t* sm,
                                               int lane) {
  const int64_t ld_q = e.ld_q;
  const int64_t off = int64_t(rbk) * 32 * ld_q + int64_t(cbk) * 32, soff = int64_t(rbk) * ncb + cbk;
  if (EPI == kEpiForward && e.bias != nullptr) {
    const float4* b4 = reinterpret_cast<const float4*>(e.bias + cbk * 32);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 b = __ldg(b4 + i);
      add_x2(v[4 * i], v[4 * i + 1], b.x, b.y, v[4 * i], v[4 * i + 1]);
      add_x2(v[4 * i + 2], v[4 * i + 3], b.z, b.w, v[4 * i + 2], v[4 * i + 3]);
    }
  }
  // pass 0 re-quantizes the pre-activation, pass 1 what comes of it: one copy of the quantizer's code
#pragma unroll 1
  for (int pass = EPI == kEpiForward && e.pre_q != nullptr ? 0 : 1; pass < 2; ++pass) {
    if (pass == 1) {
      if (EPI == kEpiForward) activate(v, e.act);
      if (EPI == kEpiGrad && e.act != kActNone) {
        uint32_t w[8];
        rows_load<2>(reinterpret_cast<const uint8_t*>(e.act_q) + off, ld_q, w, sm, lane);
        times_act_grad(v, w, __ldg(e.act_s + soff), e.act, reinterpret_cast<float*>(sm), lane);
      }
      if (EPI != kEpiPlain && e.res != nullptr) {
        if (e.res_type == kResI8) {
          uint32_t w[8];
          rows_load<2>(e.res + off, ld_q, w, sm, lane);
          add_codes(v, w, __ldg(e.res_s + soff));
        } else {
          const int64_t eb = e.res_type == kDenseF32 ? 128 : 64;   // bytes of 32 columns
          add_dense(v, e.res + int64_t(rbk) * 32 * e.res_ld + cbk * eb, e.res_ld, e.res_type, sm, lane);
        }
      }
    }
    int8_t* q = pass == 0 ? e.pre_q : e.y_q;
    float* s = pass == 0 ? e.pre_s : e.y_s;
    if (q != nullptr) store_codes(v, q + off, ld_q, s + soff, sm, lane);
  }
  if (e.y != nullptr)
    store_dense(v, e.y + int64_t(rbk) * 32 * e.y_ld + cbk * int64_t(e.y_type == kDenseF32 ? 128 : 64), e.y_ld, e.y_type, sm,
                lane);
}

}  // namespace jf
