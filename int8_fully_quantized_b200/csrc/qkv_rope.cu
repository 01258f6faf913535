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

// 8 consecutive elements of a dense tensor, loaded and later converted to fp32.
template <typename T>
struct Raw {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int k = 0; k < int(sizeof(T) / 2); ++k) v[k] = ld_stream_v4(p + 4 * k);
  }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    if constexpr (sizeof(T) == 2) {
      Vec<T>::unpack(v[0], f);
    } else {
      f[0] = __uint_as_float(v[0].x); f[1] = __uint_as_float(v[0].y); f[2] = __uint_as_float(v[0].z); f[3] = __uint_as_float(v[0].w);
      f[4] = __uint_as_float(v[1].x); f[5] = __uint_as_float(v[1].y); f[6] = __uint_as_float(v[1].z); f[7] = __uint_as_float(v[1].w);
    }
  }
};
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

// The two 8-dimension chunks of lane i of a head (in units of 8 columns).
__device__ __forceinline__ void lane_chunks(int i, int rot, int& c1, int& c2) {
  const int r = rot >> 4;
  c1 = i < r ? i : 2 * i;
  c2 = i < r ? i + r : 2 * i + 1;
}

// A rotating lane's 8 cosines and 8 sines: in the half layout pair j of its two chunks turns by c[j], s[j];
// interleaved, the pairs of its first chunk by c[0..3], those of the second by c[4..7].
struct Angles {
  float c[8], s[8];
  __device__ __forceinline__ void none() {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j] = 1.0f;
      s[j] = 0.0f;
    }
  }
  // From the table row at `row` (elements), its two vectors of four at j0 and j1.
  __device__ __forceinline__ void load(const QkvRopeArgs& a, int64_t row, int j0, int j1) {
    const float4 c0 = __ldg(reinterpret_cast<const float4*>(a.cos + row + j0)), c1 = __ldg(reinterpret_cast<const float4*>(a.cos + row + j1));
    const float4 s0 = __ldg(reinterpret_cast<const float4*>(a.sin + row + j0)), s1 = __ldg(reinterpret_cast<const float4*>(a.sin + row + j1));
    c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w; c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
    s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w; s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
  }
};

// Where lane i finds its angles in a table row.
__device__ __forceinline__ void angle_vectors(const QkvRopeArgs& a, int i, int& j0, int& j1) {
  j0 = a.interleaved ? 4 * i : 8 * i;
  j1 = a.interleaved ? 4 * (i + (a.rot >> 4)) : 8 * i + 4;
}

// Table row (in elements) of token t, the in_seq-th of its sequence; -1 for a position outside the table,
// which raises the range bit of *status.
__device__ __forceinline__ int64_t table_row(const QkvRopeArgs& a, int64_t t, int64_t in_seq, bool report) {
  const int64_t pos = a.positions != nullptr ? __ldg(reinterpret_cast<const long long*>(a.positions) + t) : in_seq;
  if (pos < 0 || pos >= a.table_len) {
    if (report) atomicOr(a.status, kStatusRange);
    return -1;
  }
  return pos * (a.rot >> 1);
}

// Rotates a lane's 16 values by its angles (forward) or back: packed where the pairs' members are
// neighbours in registers (half layout), scalar with its free negations for interleaved pairs.
template <bool BACK, bool INTER>
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const Angles& g) {
  if constexpr (INTER) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float& x = j < 4 ? a[2 * j] : b[2 * j - 8];
      float& z = j < 4 ? a[2 * j + 1] : b[2 * j - 7];
      const float u = BACK ? fmaf(x, g.c[j], z * g.s[j]) : fmaf(x, g.c[j], -(z * g.s[j]));
      z = BACK ? fmaf(z, g.c[j], -(x * g.s[j])) : fmaf(z, g.c[j], x * g.s[j]);
      x = u;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      float p0, p1, q0, q1, r0, r1;
      mul_x2(b[j], b[j + 1], g.s[j], g.s[j + 1], p0, p1);
      mul_x2(a[j], a[j + 1], g.s[j], g.s[j + 1], q0, q1);
      // the difference as product plus -1 times the other product: a packed operand has no sign of its own
      if (BACK) {
        fma_x2(a[j], a[j + 1], g.c[j], g.c[j + 1], p0, p1, r0, r1);
        mul_x2(b[j], b[j + 1], g.c[j], g.c[j + 1], p0, p1);
        fma_x2(q0, q1, -1.0f, -1.0f, p0, p1, b[j], b[j + 1]);
      } else {
        mul_x2(a[j], a[j + 1], g.c[j], g.c[j + 1], r0, r1);
        fma_x2(p0, p1, -1.0f, -1.0f, r0, r1, r0, r1);
        fma_x2(b[j], b[j + 1], g.c[j], g.c[j + 1], q0, q1, b[j], b[j + 1]);
      }
      a[j] = r0;
      a[j + 1] = r1;
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

// a / b for non-negative a and positive b, in 32 bits where both fit (a fifth of the instructions).
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
}

// Sequence b and place s in it of token t.
__device__ __forceinline__ void token_place(const QkvRopeArgs& a, int64_t t, int64_t& b, int64_t& s) {
  b = divide(t, a.seq);
  s = t - b * a.seq;
}
// Element offset of that token in a dense tensor.
__device__ __forceinline__ int64_t token_offset(const DenseHeads& d, int64_t b, int64_t s) { return b * d.stride_b + s * d.stride_t; }

// Sum of squares of 8 codes (exact).
__device__ __forceinline__ float sumsq8(const uint2& w) { return float(__dp4a(int(w.x), int(w.x), __dp4a(int(w.y), int(w.y), 0))); }

// ---------------------------------------------------------------------------------------------
// Forward: 1 byte read and sizeof(T) bytes written per element. A warp takes 32 / G tokens and a range of the heads
// (blockIdx.y). 8192 tokens of 32 + 8 heads of 128 with norms to bf16 (151 MB): 34.8 us, 4.4 TB/s including the
// launch; 152 MB at the copy rate would take 23. Neither DRAM (34% under ncu) nor the issue slots (61%) are full:
// latency bounds it. The codes of 4 heads wait in registers (92, so 5 CTAs an SM), and none are on their way while those
// are worked on; 1 head ahead at 8 CTAs (45 us) and 4 CTAs (38.9) are slower. A ring in shared memory as in the backward
// would hold them without registers (not tried here).
// ---------------------------------------------------------------------------------------------
constexpr int kFwdWarps = 4;
constexpr int kAhead = 4;

template <typename T, int G, bool INTER>
__global__ void __launch_bounds__(32 * kFwdWarps, 5) qkv_rope_fwd_kernel(const QkvRopeArgs a, int heads_per_warp) {
  const int lane = threadIdx.x & 31, i = lane % G, n = a.d >> 4;
  const int64_t t = (int64_t(blockIdx.x) * kFwdWarps + (threadIdx.x >> 5)) * (32 / G) + lane / G;
  const bool live = i < n && t < a.tokens;
  const int heads = a.hq + 2 * a.hkv;
  const int h0 = blockIdx.y * heads_per_warp, h1 = min(h0 + heads_per_warp, heads);
  int c1, c2;
  lane_chunks(i, a.rot, c1, c2);
  Angles ang;
  int64_t bt = 0, st = 0;
  if (live) {
    token_place(a, t, bt, st);
    ang.none();
    if (h0 < a.hq + a.hkv && i < (a.rot >> 4)) {
      const int64_t row = table_row(a, t, st, i == 0);
      int j0, j1;
      angle_vectors(a, i, j0, j1);
      if (row >= 0) {
        ang.load(a, row, j0, j1);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) ang.c[j] = ang.s[j] = __int_as_float(0x7FC00000);   // NaN
      }
    }
  }
  const float inv_d = 1.0f / float(a.d);
  const int8_t* row = a.x_q + t * a.cols;
  const float* srow = a.x_s + (t >> 5) * (a.cols >> 5);
  // One kind of head at a time; the codes of kAhead heads are loaded together, before the first is used.
  for (int kind = 0; kind < 3; ++kind) {
    const int base = kind == 0 ? 0 : kind == 1 ? a.hq : a.hq + a.hkv, num = kind == 0 ? a.hq : a.hkv;
    const int lo = max(h0, base), hi = min(h1, base + num);
    if (lo >= hi) continue;
    const float* gamma = kind == 0 ? a.gamma_q : kind == 1 ? a.gamma_k : nullptr;
    float g1[8], g2[8];
    if (gamma != nullptr && i < n) load_gamma(gamma, c1, c2, g1, g2);
    const DenseHeads& d = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    T* out = static_cast<T*>(d.p) + token_offset(d, bt, st) - base * d.stride_h;
    for (int hb = lo; hb < hi; hb += kAhead) {
      uint2 w1[kAhead], w2[kAhead];
      float s1[kAhead], s2[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        w1[u] = w2[u] = make_uint2(0u, 0u);
        s1[u] = s2[u] = 0.0f;
        if (live && hb + u < hi) {
          const int64_t col = int64_t(hb + u) * a.d;
          w1[u] = ld_stream_v2(row + col + 8 * c1);
          w2[u] = ld_stream_v2(row + col + 8 * c2);
          s1[u] = __ldg(srow + ((col + 8 * c1) >> 5));
          s2[u] = __ldg(srow + ((col + 8 * c2) >> 5));
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (hb + u >= hi) break;
        float x1[8], x2[8];
        if (gamma != nullptr) {
          const float ss = head_sum<G>(fmaf(s1[u] * s1[u], sumsq8(w1[u]), s2[u] * s2[u] * sumsq8(w2[u])));
          const float r = rsqrtf(fmaf(ss, inv_d, a.eps));
          codes8(w1[u], s1[u] * r, x1);
          codes8(w2[u], s2[u] * r, x2);
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            mul_x2(x1[j], x1[j + 1], g1[j], g1[j + 1], x1[j], x1[j + 1]);
            mul_x2(x2[j], x2[j + 1], g2[j], g2[j + 1], x2[j], x2[j + 1]);
          }
        } else {
          codes8(w1[u], s1[u], x1);
          codes8(w2[u], s2[u], x2);
        }
        if (!live) continue;
        if (kind < 2) rotate<false, INTER>(x1, x2, ang);
        T* o = out + (hb + u) * d.stride_h;
        store8(o + 8 * c1, x1);
        store8(o + 8 * c2, x2);
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Backward: reads dq, dk, dv, and with a norm the codes of the queries and keys; writes INT8. The G warps of a
// slot hold one head of a 32-token strip at a time, 16 values a lane; a block's absmax goes through
// shared memory (integer maxima of the bit patterns: their order does not matter). A lane copies what it
// will need of the next heads into its own places of a shared-memory ring (cp.async), so that loads in
// flight take no registers. The slots of a persistent grid share the strips and heads of one kind evenly,
// each a contiguous range; the weights' gradients stay in registers while the kind lasts and are then added
// into the CTA's row of the workspace; a second kernel adds the rows in a fixed order in fp64.
// What bounds it: latency between 470 instructions per 16 values, at 57% of the issue slots with 16 warps an SM (128
// registers; the half-layout instances store up to 16 bytes a thread to the stack), not the 195 MB (DRAM 27%). The
// instance serves norm, no norm and values alike, so calls without a norm carry its registers. 8192 tokens of 32 + 8
// heads of 128 with norms in 83 us, where the copy rate allows 30 (without norms 60 of 23). Tried and slower: two tokens a lane (spills, 172 us), 3 CTAs an SM (135), angles and gamma re-read per
// head (139) or gamma from shared memory (96), a slot's heads dealt out in turn instead of in ranges (116), a branch
// to the quotient per 8 values (98).
// ---------------------------------------------------------------------------------------------
constexpr int kBwdWarps = 8;

constexpr int kRing = 3;   // heads of the ring: two on their way while one is at work

// A lane's places in the ring: 16-byte pieces of the gradient's two chunks, then 8 bytes of codes of each.
template <typename T, int THREADS>
struct Ring {
  static constexpr int kPieces = int(sizeof(T)) / 2;                     // 16-byte pieces of 8 elements
  static constexpr int kHead = THREADS * (2 * kPieces * 16 + 16);        // bytes of one head's data
  static constexpr int kBytes = kRing * kHead;
};

template <typename T, int G, bool INTER>
__global__ void __launch_bounds__(32 * (G > kBwdWarps ? G : kBwdWarps), G > kBwdWarps ? 1 : 2) qkv_rope_bwd_kernel(const QkvRopeArgs a) {
  constexpr int W = G > kBwdWarps ? G : kBwdWarps;
  constexpr int SLOTS = W / G;              // heads in flight
  using R = Ring<T, 32 * W>;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ uint32_t s_max[3][SLOTS][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slot = warp / G;
  const int i = lane % G, n = a.d >> 4, nblk = a.d >> 5;
  const int tl = (warp % G) * (32 / G) + lane / G;   // token in the strip
  int c1, c2, j0, j1;
  lane_chunks(i, a.rot, c1, c2);
  angle_vectors(a, i, j0, j1);
  // shared-memory addresses of the lane's pieces (at stride 16 x threads) and codes in ring place 0
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16;
  const uint32_t mine_w = smem_u32(ring) + 32 * W * 2 * R::kPieces * 16 + threadIdx.x * 8;
  const int64_t nbc = a.cols >> 5, strips = a.rows >> 5;
  if (threadIdx.x < 3 * SLOTS * 8) (&s_max[0][0][0])[threadIdx.x] = 0u;
  __syncthreads();
  const float inv_d = 1.0f / float(a.d);
  int it = 0;                            // this slot's blocks so far: s_max[it] (modulo 3) is in use
  for (int kind = 0; kind < 3; ++kind) {
    const int heads = kind == 0 ? a.hq : a.hkv;
    const int base = kind == 0 ? 0 : kind == 1 ? a.hq : a.hq + a.hkv;
    const DenseHeads& d = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const float* gamma = kind == 0 ? a.gamma_q : kind == 1 ? a.gamma_k : nullptr;
    float dg1[8], dg2[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dg1[j] = dg2[j] = 0.0f;
    float g1[8], g2[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) g1[j] = g2[j] = 0.0f;
    if (gamma != nullptr && i < n) load_gamma(gamma, c1, c2, g1, g2);
    // the slots share the strips x heads of this kind evenly, each a contiguous range (strip by strip)
    const int64_t units = strips * heads, slots = int64_t(gridDim.x) * SLOTS, me = int64_t(blockIdx.x) * SLOTS + slot;
    const int64_t share = divide(units, slots), more = units - share * slots;
    const int64_t u0 = me * share + min(me, more);
    int64_t left = heads > 0 ? share + (me < more ? 1 : 0) : 0;
    int64_t strip = heads > 0 ? divide(u0, heads) : 0;
    int h0 = int(u0 - strip * heads);
    for (; left > 0; ++strip, h0 = 0) {
      const int h1 = int(min(int64_t(heads), h0 + left));
      left -= h1 - h0;
      const int64_t t = strip * 32 + tl;
      const bool live = i < n && t < a.tokens;
      const bool turns = kind < 2 && live && i < (a.rot >> 4);
      int64_t bt = 0, st = 0;
      if (live) token_place(a, t, bt, st);
      Angles ang;
      ang.none();
      if (turns) {
        const int64_t row = table_row(a, t, st, i == 0);
        if (row >= 0) {
          ang.load(a, row, j0, j1);
        } else {   // a position outside the table: no gradient
#pragma unroll
          for (int j = 0; j < 8; ++j) ang.c[j] = ang.s[j] = 0.0f;
        }
      }
      // a lane without a token copies nothing (from an address that is valid all the same) and gets zeros,
      // from which everything below is zero
      const T* src = live ? static_cast<const T*>(d.p) + token_offset(d, bt, st) + h0 * d.stride_h + 8 * c1
                          : reinterpret_cast<const T*>(a.dx_q);
      const int8_t* xr = live ? a.x_q + t * a.cols + int64_t(base + h0) * a.d + 8 * c1 : a.dx_q;
      const int64_t step_s = live ? d.stride_h : 0, step_x = live ? a.d : 0;
      const int next_s = live ? 8 * (c2 - c1) : 0;
      int8_t* dst = a.dx_q + t * a.cols + int64_t(base + h0) * a.d + 8 * c1;
      int64_t blk = strip * nbc + ((int64_t(base + h0) * a.d) >> 5);   // the head's first block
      const uint32_t take16 = live ? 16u : 0u, take8 = live ? 8u : 0u;
      uint32_t put = 0;                  // byte offset of the ring place to fill next
      auto fetch = [&]() {               // the next head in turn
        const T* src2 = src + next_s;
#pragma unroll
        for (int k = 0; k < R::kPieces; ++k) {
          cp_async_16(mine + put + k * (32 * W * 16), reinterpret_cast<const uint4*>(src) + k, take16);
          cp_async_16(mine + put + (R::kPieces + k) * (32 * W * 16), reinterpret_cast<const uint4*>(src2) + k, take16);
        }
        if (gamma != nullptr) {
          cp_async_8(mine_w + put, xr, take8);
          cp_async_8(mine_w + put + 32 * W * 8, xr + next_s, take8);
        }
        src += step_s;
        xr += step_x;
        put = put == (kRing - 1) * R::kHead ? 0 : put + R::kHead;
      };
#pragma unroll
      for (int k = 0; k < kRing - 1; ++k) {
        if (h0 + k < h1) fetch();
        cp_async_commit();
      }
      uint32_t get = 0;                  // ring place of the head at work
      float s1n = 0.0f, s2n = 0.0f;      // the next head's scales
      auto scales = [&](int64_t b) {
        if (gamma != nullptr && live) {
          s1n = __ldg(a.x_s + b + (c1 >> 2));
          s2n = __ldg(a.x_s + b + (c2 >> 2));
        }
      };
      if (h0 < h1) scales(blk);
      for (int h = h0; h < h1; ++h) {
        cp_async_wait<kRing - 2>();      // this lane's own copies: no barrier
        float y1[8], y2[8];
        uint2 w1 = make_uint2(0u, 0u), w2 = w1;
        const float s1 = s1n, s2 = s2n;
        Raw<T> r1, r2;
#pragma unroll
        for (int k = 0; k < R::kPieces; ++k) {
          r1.v[k] = lds_v4(mine + get + k * (32 * W * 16));
          r2.v[k] = lds_v4(mine + get + (R::kPieces + k) * (32 * W * 16));
        }
        if (gamma != nullptr) {
          w1 = lds_v2(mine_w + get);
          w2 = lds_v2(mine_w + get + 32 * W * 8);
        }
        r1.unpack(y1);
        r2.unpack(y2);
        if (h + kRing - 1 < h1) fetch();
        cp_async_commit();
        get = get == (kRing - 1) * R::kHead ? 0 : get + R::kHead;
        if (h + 1 < h1) scales(blk + (a.d >> 5));
        if (kind < 2) rotate<true, INTER>(y1, y2, ang);
        if (gamma != nullptr) {
          const float ss = head_sum<G>(fmaf(s1 * s1, sumsq8(w1), s2 * s2 * sumsq8(w2)));
          const float r = rsqrtf(fmaf(ss, inv_d, a.eps));   // eps > 0: finite, and a head that is not there stays 0
          float x1[8], x2[8], m0 = 0.0f, m1 = 0.0f;         // xhat, and the sum of g xhat
          codes8(w1, s1 * r, x1);
          codes8(w2, s2 * r, x2);
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            fma_x2(y1[j], y1[j + 1], x1[j], x1[j + 1], dg1[j], dg1[j + 1], dg1[j], dg1[j + 1]);
            fma_x2(y2[j], y2[j + 1], x2[j], x2[j + 1], dg2[j], dg2[j + 1], dg2[j], dg2[j + 1]);
            mul_x2(y1[j], y1[j + 1], g1[j], g1[j + 1], y1[j], y1[j + 1]);
            mul_x2(y2[j], y2[j + 1], g2[j], g2[j + 1], y2[j], y2[j + 1]);
            fma_x2(y1[j], y1[j + 1], x1[j], x1[j + 1], m0, m1, m0, m1);
            fma_x2(y2[j], y2[j + 1], x2[j], x2[j + 1], m0, m1, m0, m1);
          }
          const float m = -(head_sum<G>(m0 + m1) * inv_d);
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            fma_x2(x1[j], x1[j + 1], m, m, y1[j], y1[j + 1], y1[j], y1[j + 1]);
            fma_x2(x2[j], x2[j + 1], m, m, y2[j], y2[j + 1], y2[j], y2[j + 1]);
            mul_x2(y1[j], y1[j + 1], r, r, y1[j], y1[j + 1]);
            mul_x2(y2[j], y2[j + 1], r, r, y2[j], y2[j + 1]);
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
        uint32_t* mx = s_max[it][slot];
        if (lane < G && i < n) {
          atomicMax(mx + (c1 >> 2), __float_as_uint(m1));
          atomicMax(mx + (c2 >> 2), __float_as_uint(m2));
        }
        named_bar_sync(1 + slot, 32 * G);
        // the buffer of the block before this one is free now: every warp has read it before this barrier
        if (warp % G == 0 && lane < 8) s_max[it == 0 ? 2 : it - 1][slot][lane] = 0u;
        it = it == 2 ? 0 : it + 1;
        // lane l computes block l % 8's scale; the others fetch their two blocks' reciprocals from there
        const BlockQuant bq = block_quant_approx(__uint_as_float(mx[lane & 7]));
        const float inv1 = __shfl_sync(0xffffffffu, bq.inv, c1 >> 2), inv2 = __shfl_sync(0xffffffffu, bq.inv, c2 >> 2);
        const bool plain = __all_sync(0xffffffffu, bq.mode == 2 || (lane & 7) >= nblk);   // normal scales only
        uint32_t o[4];
        float far = 0.0f;
        codes_fast<8>(y1, inv1, o, far);
        codes_fast<8>(y2, inv2, o + 2, far);
        if (i < n && (!(far < kFarLimit) || !plain)) {
          codes_exact<8>(y1, block_quant_approx(__uint_as_float(mx[c1 >> 2])).s, o);
          codes_exact<8>(y2, block_quant_approx(__uint_as_float(mx[c2 >> 2])).s, o + 2);
        }
        if (i < n) {
          *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
          *reinterpret_cast<uint2*>(dst + 8 * (c2 - c1)) = make_uint2(o[2], o[3]);
        }
        if (warp % G == 0 && lane < nblk) a.dx_s[blk + lane] = bq.s;
        dst += a.d;
        blk += a.d >> 5;
      }
      cp_async_wait<0>();                // the next strip starts with an empty ring
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
      float* s_part = reinterpret_cast<float*>(ring);   // [W][256]: the ring is empty between kinds
      __syncthreads();                   // the previous kind's sums have been read, every warp's copies are used
      if (lane < G && i < n) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s_part[warp * 256 + 8 * c1 + j] = dg1[j];
          s_part[warp * 256 + 8 * c2 + j] = dg2[j];
        }
      }
      __syncthreads();
      for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) sum += s_part[w * 256 + c];
        a.part[(int64_t(blockIdx.x) * 2 + kind) * a.d + c] = sum;
      }
      __syncthreads();                   // before the ring is filled again
    }
  }
  cudaTriggerProgrammaticLaunchCompletion();
}

// CTAs of the backward: at most two for each of 148 SMs, at most one per strip and head.
constexpr int kQkvBwdMaxCtas = 296;

// dgamma[kind][c] = the CTAs' partial sums added in fp64 in a fixed order; one CTA per kind and 32 columns. A lane
// has all its loads in flight at once: it waits for memory once (with 8 warps that waited for 37 loads in turn the
// backward of 8192 tokens took 6 us longer).
constexpr int kSumWarps = 32;
constexpr int kSumRows = (kQkvBwdMaxCtas + kSumWarps - 1) / kSumWarps;
__global__ void __launch_bounds__(32 * kSumWarps) qkv_dgamma_kernel(const float* part, int ctas, int d,
                                                                    float* __restrict__ dgq, float* __restrict__ dgk) {
  __shared__ double sum[kSumWarps][32];
  float* out = blockIdx.y == 0 ? dgq : dgk;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float v[kSumRows];
  cudaGridDependencySynchronize();
#pragma unroll
  for (int k = 0; k < kSumRows; ++k) {
    const int b = warp + k * kSumWarps;
    v[k] = b < ctas ? part[(int64_t(b) * 2 + blockIdx.y) * d + c] : 0.0f;
  }
  double t = 0.0;
#pragma unroll
  for (int k = 0; k < kSumRows; ++k) t += double(v[k]);
  sum[warp][lane] = t;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int w = 1; w < kSumWarps; ++w) t += sum[w][lane];
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

template <typename T, int G, bool INTER>
cudaError_t fwd(const QkvRopeArgs& a, int sm_count, cudaStream_t st) {
  const int heads = a.hq + 2 * a.hkv;
  const int64_t gx = (a.tokens + kFwdWarps * (32 / G) - 1) / (kFwdWarps * (32 / G));
  // One head a warp while all CTAs run at once (64 tokens of 32 + 8 heads of 128: 7.2 us, with 4 heads 9.2). Beyond
  // that whole groups of kAhead heads, whose loads a warp has in flight together (2048 tokens 15.4 us, with two
  // heads 19.4; 512 tokens 9.1 and 11.2), more of them the more tokens there are (8192 tokens: 4 heads a warp take 11%
  // longer than 12): the angles are loaded once a warp.
  int64_t per = 1;
  if (gx * heads > int64_t(sm_count) * 5) {
    per = (gx * heads / (int64_t(sm_count) * 16) + kAhead - 1) / kAhead * kAhead;
    per = per < kAhead ? kAhead : per;
    per = per > heads ? heads : per;
  }
  const int64_t gy = (heads + per - 1) / per;
  if (gy > 65535 || gx > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  qkv_rope_fwd_kernel<T, G, INTER><<<dim3(unsigned(gx), unsigned(gy)), 32 * kFwdWarps, 0, st>>>(a, int(per));
  return cudaGetLastError();
}

template <typename T, int G, bool INTER>
cudaError_t bwd(const QkvRopeArgs& a, int sm_count, cudaStream_t st) {
  constexpr int W = G > kBwdWarps ? G : kBwdWarps;
  constexpr int smem = Ring<T, 32 * W>::kBytes;
  static_assert(smem >= W * 256 * 4, "the warps' column sums fit in the ring");
  static unsigned long long attr_set = 0;   // one bit per device ordinal
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (smem > 48 * 1024 && !(attr_set >> (dev & 63) & 1)) {
    e = cudaFuncSetAttribute(qkv_rope_bwd_kernel<T, G, INTER>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    attr_set |= 1ull << (dev & 63);
  }
  const int64_t ctas = qkv_bwd_ctas(a.rows, a.hq, a.hkv);
  qkv_rope_bwd_kernel<T, G, INTER><<<unsigned(ctas), 32 * W, smem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.part == nullptr) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a.d / 32), 2, 1);
  cfg.blockDim = dim3(32 * kSumWarps, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qkv_dgamma_kernel, static_cast<const float*>(a.part), int(ctas), a.d, a.dgamma_q, a.dgamma_k);
}

template <typename T, bool INTER>
cudaError_t run(const QkvRopeArgs& a, bool backward, int sm_count, cudaStream_t st) {
  switch (group_of(a.d)) {
    case 2: return backward ? bwd<T, 2, INTER>(a, sm_count, st) : fwd<T, 2, INTER>(a, sm_count, st);
    case 4: return backward ? bwd<T, 4, INTER>(a, sm_count, st) : fwd<T, 4, INTER>(a, sm_count, st);
    case 8: return backward ? bwd<T, 8, INTER>(a, sm_count, st) : fwd<T, 8, INTER>(a, sm_count, st);
    default: return backward ? bwd<T, 16, INTER>(a, sm_count, st) : fwd<T, 16, INTER>(a, sm_count, st);
  }
}

template <typename T>
cudaError_t run(const QkvRopeArgs& a, bool backward, int sm_count, cudaStream_t st) {
  return a.interleaved ? run<T, true>(a, backward, sm_count, st) : run<T, false>(a, backward, sm_count, st);
}

}  // namespace

int64_t qkv_bwd_ctas(int64_t rows, int64_t hq, int64_t hkv) {
  const int64_t work = rows / 32 * (hq + 2 * hkv);
  return work < kQkvBwdMaxCtas ? (work < 1 ? 1 : work) : kQkvBwdMaxCtas;
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
