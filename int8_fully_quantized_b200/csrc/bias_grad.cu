// Bias gradient of an INT8 linear layer: db[n] = sum over the rows m of fp32(dY.q[m, n]) * dY.s[m/32, n/32].
//
// One pass over the codes (1 byte and 1/256 of a scale per element; the output is negligible): HBM sets the
// floor. A cluster of up to 8 CTAs owns a slab of 128 columns; its warps take the slab's 32-row
// blocks in turn. Of one block a lane reads 16 columns of 8 rows (8 independent 16-byte loads; 8 lanes
// cover a row's 128 bytes), adds its codes exactly in packed 16-bit integers, and multiplies the integer
// sums by the block's scale into 16 fp32 column sums. Lanes, warps and CTAs (through distributed shared
// memory) are then added in a fixed order: one launch, no workspace, no atomics, the same bits every time.
// 8192 x 16384 (135 MB): 29-33 us with the launch, where the copy rate would take 20.5. DRAM is at 52% under ncu and the
// warps wait for loads (long scoreboard 11.8): 1024 CTAs at 4 an SM are 1.73 waves, and a warp loads its next block only
// after it has summed the present one. 512 x 1056 8.4 us, a launch with its cluster and the loads' latency.
#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"
#include "ptx.cuh"

namespace jf {

namespace cg = cooperative_groups;

constexpr int kBgWarps = 8;
constexpr int kBgCols = 128;      // columns of a slab
constexpr int kBgMaxCluster = 8;

__global__ void __launch_bounds__(32 * kBgWarps) bias_grad_kernel(const int8_t* __restrict__ q, const float* __restrict__ s,
                                                                  int64_t R, int64_t C, float* __restrict__ db) {
  __shared__ float part[kBgWarps][kBgCols];
  __shared__ float total[kBgCols];
  const cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t nbc = C >> 5, nblk = R >> 5;
  const int64_t slab = blockIdx.x / cluster.num_blocks();
  const int64_t col = slab * kBgCols + (lane & 7) * 16;
  const bool in = col < C;
  float acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
  if (in) {
    for (int64_t b = int64_t(cluster.block_rank()) * kBgWarps + warp; b < nblk; b += int64_t(cluster.num_blocks()) * kBgWarps) {
      const int8_t* src = q + (b * 32 + (lane >> 3)) * C + col;
      const float sc = __ldg(s + b * nbc + (col >> 5));
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = ld_stream_v4(src + int64_t(4 * i) * C);
      // code + 128 as unsigned bytes, even and odd bytes of a word added as two packed 16-bit sums
      uint32_t ev[4] = {0u, 0u, 0u, 0u}, od[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t w[4] = {v[i].x ^ 0x80808080u, v[i].y ^ 0x80808080u, v[i].z ^ 0x80808080u, v[i].w ^ 0x80808080u};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          ev[k] += w[k] & 0x00FF00FFu;
          od[k] += (w[k] >> 8) & 0x00FF00FFu;
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {   // less the 8 x 128 that the eight rows' offsets add
        acc[4 * k] = fmaf(float(int(ev[k] & 0xFFFFu) - 1024), sc, acc[4 * k]);
        acc[4 * k + 1] = fmaf(float(int(od[k] & 0xFFFFu) - 1024), sc, acc[4 * k + 1]);
        acc[4 * k + 2] = fmaf(float(int(ev[k] >> 16) - 1024), sc, acc[4 * k + 2]);
        acc[4 * k + 3] = fmaf(float(int(od[k] >> 16) - 1024), sc, acc[4 * k + 3]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 8);
    acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 16);
  }
  if (lane < 8)
#pragma unroll
    for (int i = 0; i < 16; ++i) part[warp][lane * 16 + i] = acc[i];
  __syncthreads();
  if (threadIdx.x < kBgCols) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kBgWarps; ++w) t += part[w][threadIdx.x];
    total[threadIdx.x] = t;
  }
  cluster.sync();
  if (cluster.block_rank() == 0 && threadIdx.x < kBgCols) {
    float t = 0.0f;
    for (unsigned r = 0; r < cluster.num_blocks(); ++r) t += *cluster.map_shared_rank(&total[threadIdx.x], r);
    const int64_t c = slab * kBgCols + threadIdx.x;
    if (c < C) db[c] = t;
  }
  cluster.sync();   // no CTA leaves while its sums are being read
}

cudaError_t launch_bias_grad(const int8_t* q, const float* s, int64_t R, int64_t C, float* db, cudaStream_t st) {
  // as many CTAs per slab as there are eight-block turns, a power of two up to the portable cluster size
  int cl = 1;
  while (cl < kBgMaxCluster && int64_t(cl) * kBgWarps < R / 32) cl *= 2;
  const int64_t slabs = (C + kBgCols - 1) / kBgCols;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(slabs * cl), 1, 1);   // C < 2^31: at most 2^27 CTAs
  cfg.blockDim = dim3(32 * kBgWarps, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(cl);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, bias_grad_kernel, q, s, R, C, db);
}

}  // namespace jf
