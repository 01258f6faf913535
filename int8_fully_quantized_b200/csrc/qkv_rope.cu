// From the INT8 output of a QKV projection to the dense queries, keys and values attention reads, and
// back: per-head RMS norm of queries and keys and their rotary positions in one pass, and its gradient.
//
// A row of the quantized tensor is one token's [q heads | k heads | v heads] of D columns each (D a multiple
// of 32, so every head is whole 32-column blocks). Per token and head, with x = q s:
//   norm      u = x r gamma, r = 1 / sqrt(mean(x^2) + eps)                (or u = x)
//   rotation  (y_a, y_b) = (u_a c - u_b s, u_b c + u_a s) for every pair (a, b) of the first `rot` dimensions:
//             (j, j + rot/2) in the half layout, (2j, 2j + 1) interleaved; c, s from the caller's tables.
// Backward, with dy the gradient of y: du = the rotation by the negative angle, and with g = du gamma and
// xhat = x r: dx = r (g - xhat mean(g xhat)), dgamma = sum over tokens and heads of du xhat. dx is
// re-quantized per 32x32 block.
//
// Work split: a lane holds 16 dimensions of one token's head, two 8-column chunks. Rotating lane i takes
// chunks i and i + rot/16: in the half layout these are the two members of 8 pairs, interleaved each
// chunk holds 4 whole pairs, so a rotation never leaves a lane; the lanes past rot/16 share the
// dimensions that do not rotate. A head's lanes (D/16 of them, padded to a power of two G) are neighbours, so
// the norm's sums are shuffles among G lanes. The cosines and sines depend on the token alone: a lane
// loads its 16 once and keeps them in registers while it goes through the heads.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "ptx.cuh"
#include "quant.cuh"
#include "vec.cuh"

namespace jf {

namespace {

// 8 consecutive elements of a dense tensor, to and from fp32.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    Vec<T>::unpack(ld_stream_v4(p), f);
  } else {
    const uint4 a = ld_stream_v4(p), b = ld_stream_v4(p + 4);
    f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y); f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
    f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y); f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) = Vec<T>::pack(f);
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

__device__ __forceinline__ void codes8(const uint2& w, float s, float (&x)[8]) {
  float f[4];
  i8x4_to_f32(w.x, f);
  mul_x2(f[0], f[1], s, s, x[0], x[1]);
  mul_x2(f[2], f[3], s, s, x[2], x[3]);
  i8x4_to_f32(w.y, f);
  mul_x2(f[0], f[1], s, s, x[4], x[5]);
  mul_x2(f[2], f[3], s, s, x[6], x[7]);
}

// What a lane keeps of its token: the rotation's cosines and sines (1 and 0 where it does not rotate).
struct Angles {
  float c[8], s[8];
};

// The two 8-dimension chunks of lane i of a head (in units of 8 columns).
__device__ __forceinline__ void lane_chunks(int i, int rot, int& c1, int& c2) {
  const int r = rot >> 4;
  c1 = i < r ? i : 2 * i;
  c2 = i < r ? i + r : 2 * i + 1;
}

// Loads the angles of token t for lane i. A position outside the table raises the range bit of *status and
// makes the angles NaN (fill), or zero in the backward, so that the token's rotated part is NaN (zero).
__device__ __forceinline__ void load_angles(const QkvRopeArgs& a, int64_t t, int i, float fill, Angles& g) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    g.c[j] = 1.0f;
    g.s[j] = 0.0f;
  }
  const int r = a.rot >> 4;
  if (i >= r) return;
  const int64_t pos = a.positions != nullptr ? __ldg(reinterpret_cast<const long long*>(a.positions) + t) : t % a.seq;
  if (pos < 0 || pos >= a.table_len) {
    if (i == 0) atomicOr(a.status, kStatusRange);
#pragma unroll
    for (int j = 0; j < 8; ++j) g.c[j] = g.s[j] = fill;
    return;
  }
  // half layout: pairs 8 i .. 8 i + 7; interleaved: chunk i holds pairs 4 i .. 4 i + 3, chunk i + r pairs 4 (i + r) ..
  const int64_t row = pos * (a.rot >> 1);
  const int j0 = a.interleaved ? 4 * i : 8 * i, j1 = a.interleaved ? 4 * (i + r) : 8 * i + 4;
  const float4 c0 = __ldg(reinterpret_cast<const float4*>(a.cos + row + j0)), c1 = __ldg(reinterpret_cast<const float4*>(a.cos + row + j1));
  const float4 s0 = __ldg(reinterpret_cast<const float4*>(a.sin + row + j0)), s1 = __ldg(reinterpret_cast<const float4*>(a.sin + row + j1));
  g.c[0] = c0.x; g.c[1] = c0.y; g.c[2] = c0.z; g.c[3] = c0.w; g.c[4] = c1.x; g.c[5] = c1.y; g.c[6] = c1.z; g.c[7] = c1.w;
  g.s[0] = s0.x; g.s[1] = s0.y; g.s[2] = s0.z; g.s[3] = s0.w; g.s[4] = s1.x; g.s[5] = s1.y; g.s[6] = s1.z; g.s[7] = s1.w;
}

// Rotates a lane's 16 values by its angles (sign +1) or back (sign -1).
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const Angles& g, bool interleaved, float sign) {
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float s0 = sign * g.s[j], s1 = sign * g.s[4 + j];
      const float x0 = a[2 * j], x1 = a[2 * j + 1], z0 = b[2 * j], z1 = b[2 * j + 1];
      a[2 * j] = fmaf(x0, g.c[j], -(x1 * s0));
      a[2 * j + 1] = fmaf(x1, g.c[j], x0 * s0);
      b[2 * j] = fmaf(z0, g.c[4 + j], -(z1 * s1));
      b[2 * j + 1] = fmaf(z1, g.c[4 + j], z0 * s1);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = sign * g.s[j], x = a[j], z = b[j];
      a[j] = fmaf(x, g.c[j], -(z * s));
      b[j] = fmaf(z, g.c[j], x * s);
    }
  }
}

// Sum over the G lanes of a head.
template <int G>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void load_gamma(const float* gamma, int c1, int c2, float (&g1)[8], float (&g2)[8]) {
  const float4* p = reinterpret_cast<const float4*>(gamma + 8 * c1);
  const float4* q = reinterpret_cast<const float4*>(gamma + 8 * c2);
  const float4 a = __ldg(p), b = __ldg(p + 1), c = __ldg(q), d = __ldg(q + 1);
  g1[0] = a.x; g1[1] = a.y; g1[2] = a.z; g1[3] = a.w; g1[4] = b.x; g1[5] = b.y; g1[6] = b.z; g1[7] = b.w;
  g2[0] = c.x; g2[1] = c.y; g2[2] = c.z; g2[3] = c.w; g2[4] = d.x; g2[5] = d.y; g2[6] = d.z; g2[7] = d.w;
}

// Element offset of (token t, head h) in a dense tensor.
__device__ __forceinline__ int64_t head_offset(const DenseHeads& d, int64_t t, int64_t seq, int64_t h) {
  const int64_t b = t / seq;
  return b * d.stride_b + (t - b * seq) * d.stride_t + h * d.stride_h;
}

// Sum of squares of 8 codes (exact).
__device__ __forceinline__ float sumsq8(const uint2& w) { return float(__dp4a(int(w.x), int(w.x), __dp4a(int(w.y), int(w.y), 0))); }

// ---------------------------------------------------------------------------------------------
// Forward: 1 byte read and sizeof(T) bytes written per element, bound by HBM. A warp takes 32 / G tokens
// and a range of the heads (blockIdx.y).
// ---------------------------------------------------------------------------------------------
constexpr int kFwdWarps = 4;

template <typename T, int G>
__global__ void __launch_bounds__(32 * kFwdWarps) qkv_rope_fwd_kernel(const QkvRopeArgs a, int heads_per_warp) {
  const int lane = threadIdx.x & 31, i = lane % G, n = a.d >> 4;
  const int64_t t = (int64_t(blockIdx.x) * kFwdWarps + (threadIdx.x >> 5)) * (32 / G) + lane / G;
  const bool live = i < n && t < a.tokens;
  const int heads = a.hq + 2 * a.hkv;
  const int h0 = blockIdx.y * heads_per_warp, h1 = min(h0 + heads_per_warp, heads);
  int c1, c2;
  lane_chunks(i, a.rot, c1, c2);
  Angles ang;
  if (live && h0 < a.hq + a.hkv) load_angles(a, t, i, __int_as_float(0x7FC00000), ang);
  const int64_t nbc = a.cols >> 5;
  const int8_t* row = a.x_q + t * a.cols;
  const float* srow = a.x_s + (t >> 5) * nbc;
  float g1[8], g2[8];
  const float* gamma = nullptr;
  for (int h = h0; h < h1; ++h) {
    const int kind = h < a.hq ? 0 : h < a.hq + a.hkv ? 1 : 2;
    const float* gm = kind == 0 ? a.gamma_q : kind == 1 ? a.gamma_k : nullptr;
    if (gm != gamma) {
      if (gm != nullptr && i < n) load_gamma(gm, c1, c2, g1, g2);
      gamma = gm;
    }
    uint2 w1 = make_uint2(0u, 0u), w2 = w1;
    float s1 = 0.0f, s2 = 0.0f;
    const int64_t col = int64_t(h) * a.d;
    if (live) {
      w1 = ld_stream_v2(row + col + 8 * c1);
      w2 = ld_stream_v2(row + col + 8 * c2);
      s1 = __ldg(srow + ((col + 8 * c1) >> 5));
      s2 = __ldg(srow + ((col + 8 * c2) >> 5));
    }
    float x1[8], x2[8];
    if (gm != nullptr) {
      const float ss = head_sum<G>(fmaf(s1 * s1, sumsq8(w1), s2 * s2 * sumsq8(w2)));
      const float r = 1.0f / sqrtf(ss / float(a.d) + a.eps);
      codes8(w1, s1 * r, x1);
      codes8(w2, s2 * r, x2);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x1[j] *= g1[j];
        x2[j] *= g2[j];
      }
    } else {
      codes8(w1, s1, x1);
      codes8(w2, s2, x2);
    }
    if (!live) continue;
    if (kind < 2) rotate(x1, x2, ang, a.interleaved, 1.0f);
    const DenseHeads& d = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const int hh = kind == 0 ? h : kind == 1 ? h - a.hq : h - a.hq - a.hkv;
    T* out = static_cast<T*>(d.p) + head_offset(d, t, a.seq, hh);
    store8(out + 8 * c1, x1);
    store8(out + 8 * c2, x2);
  }
}

// ---------------------------------------------------------------------------------------------
// Backward: reads dq, dk, dv, and with a norm the codes of the queries and keys; writes INT8. The G warps of a
// slot hold one head of a 32-token strip at a time, 16 values a lane; a block's absmax goes through
// shared memory (integer maxima of the bit patterns: their order does not matter). Persistent CTAs take
// work items (strip, run of heads of one kind) in turn; the weights' gradients stay in registers while the
// kind lasts and are then added into the CTA's row of the workspace; a second kernel adds the rows in a
// fixed order in fp64.
// ---------------------------------------------------------------------------------------------
constexpr int kBwdWarps = 8;

template <typename T, int G>
__global__ void __launch_bounds__(32 * (G > kBwdWarps ? G : kBwdWarps)) qkv_rope_bwd_kernel(const QkvRopeArgs a, int heads_per_item) {
  constexpr int W = G > kBwdWarps ? G : kBwdWarps;
  constexpr int SLOTS = W / G;          // heads in flight
  __shared__ uint32_t s_max[3][SLOTS][8];
  __shared__ float s_part[W][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slot = warp / G;
  const int i = lane % G, n = a.d >> 4;
  const int tl = (warp % G) * (32 / G) + lane / G;   // token in the strip
  int c1, c2;
  lane_chunks(i, a.rot, c1, c2);
  const int64_t nbc = a.cols >> 5, strips = a.rows >> 5;
  if (threadIdx.x < 3 * SLOTS * 8) (&s_max[0][0][0])[threadIdx.x] = 0u;
  __syncthreads();
  int it = 0;                            // this slot's blocks so far: s_max[it % 3] is in use
  for (int kind = 0; kind < 3; ++kind) {
    const int heads = kind == 0 ? a.hq : a.hkv;
    const int base = kind == 0 ? 0 : kind == 1 ? a.hq : a.hq + a.hkv;
    const DenseHeads& d = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const float* gamma = kind == 0 ? a.gamma_q : kind == 1 ? a.gamma_k : nullptr;
    float g1[8], g2[8], dg1[8], dg2[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dg1[j] = dg2[j] = 0.0f;
    if (gamma != nullptr && i < n) load_gamma(gamma, c1, c2, g1, g2);
    const int runs = (heads + heads_per_item - 1) / heads_per_item;
    for (int64_t item = blockIdx.x; item < strips * runs; item += gridDim.x) {
      const int64_t strip = item / runs;
      const int h0 = int(item - strip * runs) * heads_per_item, h1 = min(h0 + heads_per_item, heads);
      const int64_t t = strip * 32 + tl;
      const bool live = i < n && t < a.tokens;
      Angles ang;
      if (live && kind < 2) load_angles(a, t, i, 0.0f, ang);
      for (int h = h0 + slot; h < h1; h += SLOTS, ++it) {
        const int64_t col = int64_t(base + h) * a.d;
        const int64_t b1 = (col + 8 * c1) >> 5, b2 = (col + 8 * c2) >> 5;
        float y1[8], y2[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y1[j] = y2[j] = 0.0f;
        uint2 w1 = make_uint2(0u, 0u), w2 = w1;
        float s1 = 0.0f, s2 = 0.0f;
        if (live) {
          const T* src = static_cast<const T*>(d.p) + head_offset(d, t, a.seq, h);
          load8(src + 8 * c1, y1);
          load8(src + 8 * c2, y2);
          if (gamma != nullptr) {
            w1 = ld_stream_v2(a.x_q + t * a.cols + col + 8 * c1);
            w2 = ld_stream_v2(a.x_q + t * a.cols + col + 8 * c2);
            s1 = __ldg(a.x_s + strip * nbc + b1);
            s2 = __ldg(a.x_s + strip * nbc + b2);
          }
          if (kind < 2) rotate(y1, y2, ang, a.interleaved, -1.0f);
        }
        if (gamma != nullptr) {
          const float ss = head_sum<G>(fmaf(s1 * s1, sumsq8(w1), s2 * s2 * sumsq8(w2)));
          const float r = 1.0f / sqrtf(ss / float(a.d) + a.eps);
          float x1[8], x2[8], m = 0.0f;   // xhat, and the sum of g xhat
          codes8(w1, s1 * r, x1);
          codes8(w2, s2 * r, x2);
          if (live) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              dg1[j] = fmaf(y1[j], x1[j], dg1[j]);
              dg2[j] = fmaf(y2[j], x2[j], dg2[j]);
              y1[j] *= g1[j];
              y2[j] *= g2[j];
              m = fmaf(y1[j], x1[j], m);
              m = fmaf(y2[j], x2[j], m);
            }
          }
          m = head_sum<G>(m) / float(a.d);   // eps > 0 keeps r finite: a head that is not there stays 0
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            y1[j] = r * fmaf(-x1[j], m, y1[j]);
            y2[j] = r * fmaf(-x2[j], m, y2[j]);
          }
        }
        // absmax of the head's D / 32 blocks over the strip's 32 tokens
        float m1 = 0.0f, m2 = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          m1 = fmaxf(m1, fabsf(y1[j]));
          m2 = fmaxf(m2, fabsf(y2[j]));
        }
#pragma unroll
        for (int o = G; o < 32; o <<= 1) {
          m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
          m2 = fmaxf(m2, __shfl_xor_sync(0xffffffffu, m2, o));
        }
        uint32_t* mx = s_max[it % 3][slot];
        if (lane < G && i < n) {
          atomicMax(mx + (c1 >> 2), __float_as_uint(m1));
          atomicMax(mx + (c2 >> 2), __float_as_uint(m2));
        }
        named_bar_sync(1 + slot, 32 * G);
        // the buffer of the block before this one is free now: every warp has read it before this barrier
        if (warp % G == 0 && lane < 8) s_max[(it + 2) % 3][slot][lane] = 0u;
        if (i < n) {
          const BlockQuant q1 = block_quant(__uint_as_float(mx[c1 >> 2])), q2 = block_quant(__uint_as_float(mx[c2 >> 2]));
          uint32_t o1[2], o2[2];
          quant_pack<8>(y1, q1, o1);
          quant_pack<8>(y2, q2, o2);
          int8_t* dst = a.dx_q + t * a.cols + col;
          *reinterpret_cast<uint2*>(dst + 8 * c1) = make_uint2(o1[0], o1[1]);
          *reinterpret_cast<uint2*>(dst + 8 * c2) = make_uint2(o2[0], o2[1]);
          if (tl == 0) {
            if ((c1 & 3) == 0) a.dx_s[strip * nbc + b1] = q1.s;
            if ((c2 & 3) == 0) a.dx_s[strip * nbc + b2] = q2.s;
          }
        }
      }
    }
    if (gamma != nullptr && a.part != nullptr) {
      // this CTA's sums: over a warp's tokens by shuffles, then over the warps in order
#pragma unroll
      for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int o = G; o < 32; o <<= 1) {
          dg1[j] += __shfl_xor_sync(0xffffffffu, dg1[j], o);
          dg2[j] += __shfl_xor_sync(0xffffffffu, dg2[j], o);
        }
      }
      __syncthreads();                   // the previous kind's sums have been read
      if (lane < G && i < n) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s_part[warp][8 * c1 + j] = dg1[j];
          s_part[warp][8 * c2 + j] = dg2[j];
        }
      }
      __syncthreads();
      for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) sum += s_part[w][c];
        a.part[(int64_t(blockIdx.x) * 2 + kind) * a.d + c] = sum;
      }
    }
  }
}

// dgamma[kind][c] = the CTAs' partial sums added in fp64 in a fixed order; one CTA per kind and 32 columns.
__global__ void __launch_bounds__(256) qkv_dgamma_kernel(const float* __restrict__ part, int ctas, int d,
                                                         float* __restrict__ dgq, float* __restrict__ dgk) {
  __shared__ double sum[8][32];
  float* out = blockIdx.y == 0 ? dgq : dgk;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  double t = 0.0;
  for (int b = warp; b < ctas; b += 8) t += double(part[(int64_t(b) * 2 + blockIdx.y) * d + c]);
  sum[warp][lane] = t;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int w = 1; w < 8; ++w) t += sum[w][lane];
    out[c] = float(t);
  }
}

struct Frequencies {
  double f[128];
};

// cos and sin of position * frequency, times the magnitude, each formed in fp64 (the angle of a far
// position needs more bits than fp32 has) and rounded once.
__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ Frequencies fr, int half, double magnitude, int64_t length,
                                                         float* __restrict__ cos_out, float* __restrict__ sin_out) {
  const int64_t total = length * half;
  for (int64_t e = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; e < total; e += int64_t(gridDim.x) * blockDim.x) {
    const int64_t p = e / half;
    double s, c;
    sincos(double(p) * fr.f[e - p * half], &s, &c);
    cos_out[e] = float(c * magnitude);
    sin_out[e] = float(s * magnitude);
  }
}

int group_of(int64_t d) { return d <= 32 ? 2 : d <= 64 ? 4 : d <= 128 ? 8 : 16; }

template <typename T, int G>
cudaError_t fwd(const QkvRopeArgs& a, int sm_count, cudaStream_t st) {
  const int heads = a.hq + 2 * a.hkv;
  const int64_t gx = (a.tokens + kFwdWarps * (32 / G) - 1) / (kFwdWarps * (32 / G));
  // all heads of a token in one warp when the tokens alone fill the SMs (the angles are then loaded once),
  // otherwise as few heads per warp as it takes to fill them
  int64_t per = gx * heads / (int64_t(sm_count) * 16);
  per = per < 1 ? 1 : per > heads ? heads : per;
  const int64_t gy = (heads + per - 1) / per;
  if (gy > 65535 || gx > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  qkv_rope_fwd_kernel<T, G><<<dim3(unsigned(gx), unsigned(gy)), 32 * kFwdWarps, 0, st>>>(a, int(per));
  return cudaGetLastError();
}

template <typename T, int G>
cudaError_t bwd(const QkvRopeArgs& a, int sm_count, cudaStream_t st) {
  constexpr int W = G > kBwdWarps ? G : kBwdWarps, SLOTS = W / G;
  const int64_t strips = a.rows / 32, ctas = qkv_bwd_ctas(a.rows, a.hq, a.hkv);
  // runs of heads long enough to reuse a strip's angles, short enough for several items per CTA
  int64_t per = strips * a.hq / (ctas * 4);
  per = per < SLOTS ? SLOTS : per > 8 ? 8 : per;
  qkv_rope_bwd_kernel<T, G><<<unsigned(ctas), 32 * W, 0, st>>>(a, int(per));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.part == nullptr) return e;
  qkv_dgamma_kernel<<<dim3(unsigned(a.d / 32), 2), 256, 0, st>>>(a.part, int(ctas), a.d, a.dgamma_q, a.dgamma_k);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run(const QkvRopeArgs& a, bool backward, int sm_count, cudaStream_t st) {
  switch (group_of(a.d)) {
    case 2: return backward ? bwd<T, 2>(a, sm_count, st) : fwd<T, 2>(a, sm_count, st);
    case 4: return backward ? bwd<T, 4>(a, sm_count, st) : fwd<T, 4>(a, sm_count, st);
    case 8: return backward ? bwd<T, 8>(a, sm_count, st) : fwd<T, 8>(a, sm_count, st);
    default: return backward ? bwd<T, 16>(a, sm_count, st) : fwd<T, 16>(a, sm_count, st);
  }
}

}  // namespace

// CTAs of the backward: at most two for each of 148 SMs, at most one per strip and head.
int64_t qkv_bwd_ctas(int64_t rows, int64_t hq, int64_t hkv) {
  const int64_t work = rows / 32 * (hq + 2 * hkv);
  return work < 296 ? (work < 1 ? 1 : work) : 296;
}

cudaError_t launch_qkv_rope(const QkvRopeArgs& a, bool backward, int dtype, int sm_count, cudaStream_t st) {
  switch (dtype) {
    case kDenseF32: return run<float>(a, backward, sm_count, st);
    case kDenseBf16: return run<__nv_bfloat16>(a, backward, sm_count, st);
    default: return run<__half>(a, backward, sm_count, st);
  }
}

cudaError_t launch_rope_table(const double* inv_freq, int64_t half, double magnitude, int64_t length, float* cos_out,
                              float* sin_out, int sm_count, cudaStream_t st) {
  Frequencies fr = {};
  for (int64_t j = 0; j < half; ++j) fr.f[j] = inv_freq[j];
  const int64_t blocks = (length * half + 255) / 256, cap = int64_t(sm_count) * 8;
  rope_table_kernel<<<unsigned(blocks < cap ? blocks : cap), 256, 0, st>>>(fr, int(half), magnitude, length, cos_out, sin_out);
  return cudaGetLastError();
}

}  // namespace jf
