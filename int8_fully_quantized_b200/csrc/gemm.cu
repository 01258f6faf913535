// Block-scaled INT8 GEMM on sm_100a tensor cores (tcgen05.mma kind::i8), used for the forward,
// input-gradient and weight-gradient products of a Jetfire linear layer, and a plain INT8 GEMM with
// an int32 result (the tensor-core ceiling the block-scaled one is measured against).
//
// Jetfire (atlas.scime.ai summary, "Approach"): linear operators read and write INT8 tensors with
// one scale per 32x32 block, quantization is applied on-chip, and the weight gradient is also an
// INT8 computation with per-block scales. For every 32-wide block kb of the contraction axis the
// exact int32 partial P = sum_k A(r,k) B(c,k) is multiplied by c = fp32(sA(r/32,kb) * sB(c/32,kb))
// and accumulated in fp32; after the last block the fp32 tile is re-quantized per 32x32 block.
//
// Design of the block-scaled kernel (one CTA per SM, persistent over 128 x 128 output tiles, in the
// order that keeps the smaller operand resident in L2: see TileWalk). The rescale needs, per output
// element and contraction block, a conversion and an FMA on the CUDA cores, several times the tensor core's
// time for the same block, so the kernel is built to keep the warps that sum busy. Each contraction
// block of a tile is one MMA into its own int32 TMEM accumulator of 128 columns; the four accumulators
// that fit in TMEM form two groups of two, filled and emptied in turn:
//   warp 0       producer: lane 0 loads 128-byte-deep stages of A and B (TMA, 128-byte swizzle,
//                no multicast) into a 4-stage shared-memory ring; a slot is refilled once the MMAs
//                that read it have completed (tcgen05.commit on the slot's `empty` barrier).
//   warp 1       MMA: lane 0 issues a group's MMAs (M=128, N=128, K=32: for each of its two contraction
//                blocks, one at a tile's odd end, one that sets the accumulator to a constant and one that
//                adds the block's product; see partial_x2) and commits them together to the group's
//                `tfull` barrier, once the sum warps have emptied the group (`tempty`).
//   warps 4-11   sum: warp w owns TMEM lanes 32 (w % 4) .. +31 and two 32-column blocks, i.e.
//                two 32x32 output blocks of the tile. It waits for the group, loads each block's 64
//                partials per thread (one tcgen05.ld), hands the group back after the last load, and
//                accumulates fp32(sA*sB) * P in registers. The block scales come from global memory
//                straight into registers, 32 contraction blocks per load (lane l holds block w0 + l), one
//                window ahead, and are broadcast by warp shuffles. After the last block it leaves its two
//                fp32 blocks in shared memory (`ofull` / `oempty`) and goes on with the next tile.
//   warps 12-..  output: four or eight warps (Roles) take the finished blocks through the tile's epilogue
//                (epilogue.cuh) while the next tile is summed. Where there is no next tile, or where it is summed in
//                less time than the epilogue takes, there are none and the sum warps do it themselves.
// What bounds it (B200, 1965 MHz). Per 128 x 128 tile and contraction block the sum warps of a
// sub-partition need 256 cycles of FMA pipe (two packed FMAs for 2 elements); measured 470 at a
// contraction of 16384 and 490 at 4096. The rest is latency the two warps of a sub-partition do
// not hide for each other (barrier wait, TMEM load 80 cycles) and the hand-off: an MMA's result is visible ~530
// cycles after its issue, two MMAs' ~620, and each commit holds the tensor pipe for ~57 cycles besides
// an MMA's 64, which is why two blocks share one commit (389 cycles per block in a reduced kernel with two
// groups of two, 473 with four of one) and why every thread of a sum warp polls the barrier itself (one
// polling lane and a warp synchronization: 492). The main loop is unrolled by four blocks: rolled, branches
// and instruction fetch cost 9% more.
// At a contraction of 1024 (4096 x 1024 x 4096, 7 tiles a CTA; clock64 of CTA 0) the sum warps need 485 cycles a block in
// the plain forward and 590-600 beside output warps with GELU and two INT8 outputs (or GELU'), which take 20500 cycles
// for a tile's 4 blocks a warp and so set the pace together with the sum warps (19300 a tile). A tile's end costs
// 850-1250 cycles, the start up to the first sum 3100-3500, the last tile's epilogue 6400 (plain) or 15000, of
// 128000 and 158000 in all.
// Operand orientation: A and B are read K-major (contraction contiguous) or MN-major (output
// index contiguous) straight from their row-major INT8 storage, so dgrad and wgrad re-block along
// the other axis with no transpose pass.
//
// Ordering of the hand-offs: tcgen05 operations of different threads are ordered by a barrier only between
// tcgen05.fence::before_thread_sync ahead of the arrival (tcgen05.commit implies it) and fence::after_thread_sync
// behind the wait, so every hand-off of a group carries both: a sum warp that has seen the commit fences before
// it loads; once its partials are in registers (tcgen05.wait::ld) it fences and its lanes meet before lane 0
// arrives; the MMA lane fences before it overwrites the group. The two MMAs of a block have one shape and one
// accumulator, so the tensor core runs them in order.
//
// Every mbarrier wait is bounded (ptx.cuh). On a timeout the warp that saw it sets the CTA's abort
// flag; every other wait then gives up too and the roles end; in-flight copies and MMAs are drained
// (bounded) before TMEM is freed.
#include <cooperative_groups.h>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "act.cuh"
#include "epilogue.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace jf {

namespace cg = cooperative_groups;

constexpr int BM = 128;             // tile rows = MMA M = TMEM lanes
constexpr int BN = 128;             // tile cols = MMA N = TMEM columns of one accumulator
constexpr int KB = 32;              // contraction block (one MMA, one rescale)
constexpr int KBS = 4;              // contraction blocks per pipeline stage (128 bytes)
constexpr int GROUP = 2;            // contraction blocks committed, waited for and handed back together
constexpr int NGROUPS = 2;          // groups in TMEM (2 x 2 x 128 = all 512 columns)
constexpr int STAGES = 4;
constexpr int MMA_WARP = 1;
constexpr int FIRST_SUM_WARP = 4;   // warps 2 and 3 have no role: the sum warps start a warpgroup
constexpr int NUM_SUM_WARPS = 8;    // each owns two 32x32 output blocks of the 128 x 128 tile
constexpr int FIRST_OUT_WARP = FIRST_SUM_WARP + NUM_SUM_WARPS;
// Output warps take the sum warps' blocks through the tile's epilogue: 4 (two sum warps each), or 8 where a
// tile's epilogue outlasts its main loop, or 0: each sum warp its own (launch_gemm). Registers: the threads start
// with an equal share; the warpgroup of the producer and the MMA warp gives most of its own up, the sum warps take SUM_REGS, enough for
// 64 accumulators and 64 partials each, the output warps the rest. The shares' sum must not exceed the launch's
// total, or setmaxnreg would wait for ever. What ptxas stores to the stack all the same: 180 bytes a thread with
// eight output warps (72 registers each), 4-28 in the forwards' other instances and in those without output warps.
template <int NOUT, int SUM_REGS>
struct Roles {
  static constexpr int kThreads = 32 * (FIRST_OUT_WARP + NOUT);
  static constexpr int kLaunch = 65536 / kThreads / 8 * 8;
  static constexpr int kSum = SUM_REGS, kCtl = NOUT == 8 ? 24 : NOUT == 4 && SUM_REGS > 168 ? 32 : 40;
  static constexpr int kOut = NOUT == 0 ? 0 : (kThreads * kLaunch / 128 - kCtl - 2 * kSum) / (NOUT == 0 ? 1 : NOUT / 4) / 8 * 8;
  static_assert(128 * (kCtl + 2 * kSum) + 32 * NOUT * kOut <= kThreads * kLaunch, "register split");
};
constexpr int A_STAGE = BM * KBS * KB;  // 16 KB
constexpr int B_STAGE = BN * KBS * KB;  // 16 KB
constexpr uint32_t TMEM_COLS = NGROUPS * GROUP * BN;
static_assert(KBS % GROUP == 0 && TMEM_COLS == 512, "groups do not cross pipeline stages and fill TMEM");

constexpr int SMEM_A = 0;
constexpr int SMEM_B = SMEM_A + STAGES * A_STAGE;
constexpr int SMEM_BAR = SMEM_B + STAGES * B_STAGE;
constexpr int NUM_BARS = 2 * STAGES + 2 * NGROUPS + 2 * NUM_SUM_WARPS + 1;
constexpr int SMEM_MISC = SMEM_BAR + NUM_BARS * 8;
constexpr int SMEM_BIAS = (SMEM_MISC + 16 + 1023) / 1024 * 1024;   // 4 KB of -128: the operand of the bias MMA
constexpr int SMEM_OUT = SMEM_BIAS + BM * KB;                      // the finished tile, 16 fp32 blocks of 4 KB
constexpr int SMEM_BYTES = SMEM_OUT + BM * BN * 4 + 1024;          // + slack to align the base to 1024
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory of one CTA");

struct __align__(64) GemmParams {
  CUtensorMap tma_a;
  CUtensorMap tma_b;
  const float* a_s;
  const float* b_s;
  int64_t a_s_blk, a_s_k;  // scale of A at (row block r, contraction block kb): a_s[r*a_s_blk + kb*a_s_k]
  int64_t b_s_blk, b_s_k;
  unsigned int* status;
  int rows, cols, kblocks;
  int tiles_m, tiles_n;
  int n_fast;   // tile order: 0 = row tiles vary fastest, 1 = column tiles vary fastest
  int share;    // split contraction: pipeline stages of each CTA of a cluster
  EpilogueParams ep;
};

// The CTA's tiles t = blockIdx.x, blockIdx.x + gridDim.x, ... in order, as row and column tiles. The 148
// tiles in flight at once share one operand's blocks: with row tiles varying fastest they cover nearly
// all row tiles (all of A) and a few column tiles, so A is re-read from L2 by every wave and B streams
// once; the host picks the order that keeps the smaller operand the re-read one, so that it stays in L2.
// Two divisions at the start and additions from tile to tile: divided anew for every tile, the
// coordinates took each sum warp ~1000 cycles between two tiles.
struct TileWalk {
  int a, b, da, db, na;   // tile t = b na + a, a varying fastest
  bool n_fast;
  // From tile `first` in steps of `step`.
  __device__ __forceinline__ TileWalk(const GemmParams& p, int first, int step)
      : na(p.n_fast ? p.tiles_n : p.tiles_m), n_fast(p.n_fast != 0) {
    a = first % na;
    b = first / na;
    da = step % na;
    db = step / na;
  }
  __device__ __forceinline__ void next() {
    a += da;
    b += db;
    if (a >= na) {
      a -= na;
      ++b;
    }
  }
  __device__ __forceinline__ int row() const { return n_fast ? b : a; }
  __device__ __forceinline__ int col() const { return n_fast ? a : b; }
};

// tcgen05 instruction descriptor: s32 accumulator, signed int8 A and B, A/B major-ness, N, M.
template <bool A_MN, bool B_MN, int N>
__device__ constexpr uint32_t instr_desc() {
  return (2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(A_MN) << 15) | (uint32_t(B_MN) << 16) |
         (uint32_t(N >> 3) << 17) | (uint32_t(BM >> 4) << 24);
}

// Shared-memory matrix descriptor, 128-byte swizzle, sm_100 descriptor version.
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t((lbo >> 4) & 0x3FFFu) << 16) |
         (uint64_t((sbo >> 4) & 0x3FFFu) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// The partial sums' encoding. An MMA of constant operands first sets every accumulator to
// 32 * 128 * 128 = 2^19, and the block's own MMA adds its exact partial P on top (|P| <= 2^19), so an
// accumulator holds n = P + 2^19 in [0, 2^20]. Read as an fp32 bit pattern that is the denormal number
// n 2^-149, and one FMA, n 2^-149 * 2^126 - 2^-4, is exactly P 2^-23: the conversion runs in the FMA pipe, two
// values per packed instruction, and not as one int -> float conversion per value. Those cost more than
// their own issue slots: while both sum warps of the MMA warp's sub-partition convert, its tcgen05
// instructions take 327 cycles each instead of 87.
constexpr float kSumScale = 8388608.0f;            // 2^23, multiplied into the block's scale
constexpr float kMaxScaled = 4.0564819207303340848e31f;   // 2^105: below it that multiplication is exact
__device__ __forceinline__ void partial_x2(uint32_t r0, uint32_t r1, float& f0, float& f1) {
  constexpr float k126 = 8.507059173023461587e37f;   // 2^126
  fma_x2(__uint_as_float(r0), __uint_as_float(r1), k126, k126, -0.0625f, -0.0625f, f0, f1);
}

// A finished block between a sum warp and an output warp: row = lane, 16-byte chunk c of a row at position
// c ^ (row % 8) (conflict-free both ways).
__device__ __forceinline__ void block_to_smem(const float (&v)[32], uint8_t* blk, int lane) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<float4*>(blk + lane * 128 + ((c ^ (lane & 7)) << 4)) =
        make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}
__device__ __forceinline__ void block_from_smem(float (&v)[32], const uint8_t* blk, int lane) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float4 f = *reinterpret_cast<const float4*>(blk + lane * 128 + ((c ^ (lane & 7)) << 4));
    v[4 * c] = f.x; v[4 * c + 1] = f.y; v[4 * c + 2] = f.z; v[4 * c + 3] = f.w;
  }
}

// The 32 scales of one operand's row (or column) block `blk` for contraction blocks w0 .. w0+31:
// lane l returns the scale of block w0 + l (0 past the end of the matrix or of the contraction).
__device__ __forceinline__ float scale_window(const float* __restrict__ base, int64_t s_blk, int64_t s_k, int blk,
                                              int nblk, int w0, int kblocks, int lane) {
  const int kb = w0 + lane;
  return (blk < nblk && kb < kblocks) ? __ldg(base + blk * s_blk + int64_t(kb) * s_k) : 0.0f;
}

// SPLIT: a cluster of CTAs takes one tile, each a part of its contraction (p.share pipeline stages, in rank
// order; a part may be empty). The sum warps write each 32 x 32 part into the shared memory of the CTA that
// owns its block (distributed shared memory: written, not read, as nobody waits for a write; reading the parts
// from there instead took 6 us more), and the owners' output warps add the parts in rank order.
template <bool A_MN, bool B_MN, int EPI, int NOUT, int SUM_REGS, bool SPLIT>
__global__ void __launch_bounds__(Roles<NOUT, SUM_REGS>::kThreads, 1) gemm_i8_kernel(const __grid_constant__ GemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem + SMEM_A;
  uint8_t* sB = smem + SMEM_B;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SMEM_BAR);  // per stage: A and B landed
  uint64_t* empty = full + STAGES;      // per stage: the MMAs that read it completed
  uint64_t* tfull = empty + STAGES;     // per group: its MMAs completed
  uint64_t* tempty = tfull + NGROUPS;   // per group: every epilogue warp has read it
  uint64_t* ofull = tempty + NGROUPS;         // per sum warp: its two finished blocks are in shared memory
  uint64_t* oempty = ofull + NUM_SUM_WARPS;   // per sum warp: they have been written out
  uint64_t* drain = oempty + NUM_SUM_WARPS;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + SMEM_MISC);
  volatile uint32_t* abort_flag = tmem_holder + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < NGROUPS; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], NUM_SUM_WARPS);
    }
    for (int w = 0; w < NUM_SUM_WARPS; ++w) {
      mbar_init(&ofull[w], 1);
      mbar_init(&oempty[w], 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 0) {
    if (lane == 0) {
      if (p.kblocks > 0) {   // an empty contraction has no operands and no maps
        prefetch_tensormap(&p.tma_a);
        prefetch_tensormap(&p.tma_b);
      }
    }
    __syncwarp();
    tmem_alloc(tmem_holder, TMEM_COLS);
    tmem_relinquish();
  }
  for (int i = threadIdx.x; i < BM * KB / 4; i += Roles<NOUT, SUM_REGS>::kThreads) reinterpret_cast<uint32_t*>(smem + SMEM_BIAS)[i] = 0x80808080u;
  fence_proxy_async_smem();   // the bias operand is read by the tensor core
  const cg::cluster_group cluster = cg::this_cluster();
  tc_fence_before();
  if constexpr (SPLIT) cluster.sync();   // every CTA has started: its shared memory may be written
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  // this CTA's part of the contraction: blocks kb0 .. kb0 + kblocks - 1
  const int rank = SPLIT ? int(cluster.block_rank()) : 0, parts = SPLIT ? int(cluster.num_blocks()) : 1;
  const int kb0 = SPLIT ? rank * p.share * KBS : 0;
  const int kblocks = SPLIT ? max(0, min(p.share * KBS, p.kblocks - kb0)) : p.kblocks;
  const int num_kstages = (kblocks + KBS - 1) / KBS;
  const int num_tiles = p.tiles_m * p.tiles_n;
  const int first_tile = int(blockIdx.x) / parts, tile_step = int(gridDim.x) / parts;
  const int my_tiles = SPLIT ? 1 : first_tile < num_tiles ? (num_tiles - 1 - first_tile) / tile_step + 1 : 0;
  const int total_stages = my_tiles * num_kstages;   // this CTA's stages, in order

  if (warp < FIRST_SUM_WARP) {
    setmaxnreg_dec<Roles<NOUT, SUM_REGS>::kCtl>();
    if (warp == 0) {
      // ------------------------------------------------------------------ producer warp
      if (lane == 0) {
        uint32_t pending = 0, pend_ph = 0;  // slots armed, and the parity armed
        TileWalk at(p, first_tile, tile_step);
        int ks = 0, st = 0;
        uint32_t ph = 0;
        for (int g = 0; g < total_stages; ++g) {
          const int row0 = at.row() * BM, col0 = at.col() * BN;
          // far ahead of the MMAs: it looks now and then instead of polling beside the warps at work
          for (int i = 0; i < 4096 && !mbar_try_wait<true>(&empty[st], ph ^ 1u); ++i) __nanosleep(300);
          if (!mbar_wait<true>(&empty[st], ph ^ 1u, abort_flag, p.status)) break;
          mbar_arrive_expect_tx(&full[st], A_STAGE + B_STAGE);
          pending |= 1u << st;
          pend_ph = (pend_ph & ~(1u << st)) | (ph << st);
          const int k0 = (kb0 + ks * KBS) * KB;
          if (!A_MN) tma_load_2d(sA + st * A_STAGE, &p.tma_a, &full[st], k0, row0);
          else tma_load_2d(sA + st * A_STAGE, &p.tma_a, &full[st], row0, k0);
          if (!B_MN) tma_load_2d(sB + st * B_STAGE, &p.tma_b, &full[st], k0, col0);
          else tma_load_2d(sB + st * B_STAGE, &p.tma_b, &full[st], col0, k0);
          if (++ks == num_kstages) {
            ks = 0;
            at.next();
          }
          if (++st == STAGES) {
            st = 0;
            ph ^= 1u;
          }
        }
        // Teardown: every copy issued has landed before the CTA exits.
        for (int s = 0; s < STAGES; ++s)
          if (pending & (1u << s)) mbar_wait_teardown<true>(&full[s], (pend_ph >> s) & 1u, p.status);
      }
      __syncwarp();
    } else if (warp == MMA_WARP) {
      // ------------------------------------------------------------------ MMA warp
      if (lane == 0) {
        constexpr uint32_t idesc = instr_desc<A_MN, B_MN, BN>();
        // K-major: the 32-byte K step moves inside the 128-byte swizzle row;
        // MN-major: it moves by 32 rows of 128 bytes (four 8-row swizzle atoms).
        // The descriptors differ in their address field alone (16-byte units, low word).
        const uint64_t ad0 = smem_desc(smem_u32(sA), A_MN ? 16384 : 16, 1024);
        const uint64_t bd0 = smem_desc(smem_u32(sB), B_MN ? 16384 : 16, 1024);
        const uint32_t a_lo = uint32_t(ad0), a_hi = uint32_t(ad0 >> 32), b_lo = uint32_t(bd0), b_hi = uint32_t(bd0 >> 32);
        constexpr uint32_t a_step = (A_MN ? 4096 : 32) / 16, b_step = (B_MN ? 4096 : 32) / 16;
        // every byte of the bias operand is -128, so any descriptor inside its 4 KB describes it (no swizzle)
        const uint64_t bias = uint64_t((smem_u32(smem + SMEM_BIAS) >> 4) & 0x3FFFu) | (uint64_t(128 >> 4) << 16) |
                              (uint64_t(256 >> 4) << 32) | (uint64_t(1) << 46);
        constexpr uint32_t bias_idesc = instr_desc<false, false, BN>();
        bool ok = true, issued = false;
        int gi = 0, slot = 0, left = kblocks;       // groups so far: group gi lives in TMEM half gi % 2
        uint32_t sph = 0;
        for (int s = 0; ok && s < total_stages; ++s) {
          if (!mbar_wait<true>(&full[slot], sph, abort_flag, p.status)) break;
          const int nk = min(KBS, left);
          uint32_t a = a_lo + slot * (A_STAGE / 16), bb = b_lo + slot * (B_STAGE / 16);
#pragma unroll
          for (int kk = 0; kk < KBS; kk += GROUP) {
            if (kk >= nk) break;
            const uint32_t b = uint32_t(gi) & 1u;
            if (!mbar_wait<true>(&tempty[b], (uint32_t(gi >> 1) & 1u) ^ 1u, abort_flag, p.status)) { ok = false; break; }
            tc_fence_after();
            const uint32_t d = tmem_base + b * (GROUP * BN);
            mma_i8(d, bias, bias, bias_idesc, 0u);
            if (kk + 1 < nk) mma_i8(d + BN, bias, bias, bias_idesc, 0u);
            mma_i8_add(d, a + kk * a_step, a_hi, bb + kk * b_step, b_hi, idesc);
            if (kk + 1 < nk) mma_i8_add(d + BN, a + (kk + 1) * a_step, a_hi, bb + (kk + 1) * b_step, b_hi, idesc);
            tc_commit(&tfull[b]);
            issued = true;
            ++gi;
          }
          if (ok) tc_commit(&empty[slot]);   // the slot may be refilled once these MMAs complete
          if (++slot == STAGES) { slot = 0; sph ^= 1u; }
          left -= KBS;
          if (left <= 0) left = kblocks;
        }
        // Teardown: no MMA may still be writing TMEM when it is freed.
        if (issued) {
          tc_commit(drain);
          mbar_wait_teardown<true>(drain, 0u, p.status);
        }
      }
      __syncwarp();
    }
  } else if (warp < FIRST_OUT_WARP) {
    // ------------------------------------------------------------------ sum warps
    setmaxnreg_inc<Roles<NOUT, SUM_REGS>::kSum>();
    const int w = warp - FIRST_SUM_WARP;
    const int sub = warp & 3;             // TMEM sub-partition this warp may access = row block in the tile
    const int cb0 = (w >> 2) * 2;         // first of the warp's two column blocks in the tile
    const uint32_t t_base = tmem_base + (uint32_t(sub * 32) << 16) + uint32_t(cb0 * 32);
    const int nrb = p.rows >> 5, ncb = p.cols >> 5;
    // Scales of the current window (lane l: contraction block w0 + l) of the warp's row block (sa)
    // and two column blocks (sb0, sb1); each window prefetches the next one.
    float sa_n, sb0_n, sb1_n;
    auto load_scales = [&](const TileWalk& at, int w0, bool valid) {
      const int rbk = at.row() * (BM / 32) + sub, cbk = at.col() * (BN / 32) + cb0;
      sa_n = scale_window(p.a_s, p.a_s_blk, p.a_s_k, rbk, valid ? nrb : 0, kb0 + w0, kb0 + kblocks, lane);
      sb0_n = scale_window(p.b_s, p.b_s_blk, p.b_s_k, cbk, valid ? ncb : 0, kb0 + w0, kb0 + kblocks, lane);
      sb1_n = scale_window(p.b_s, p.b_s_blk, p.b_s_k, cbk + 1, valid ? ncb : 0, kb0 + w0, kb0 + kblocks, lane);
    };
    TileWalk at(p, first_tile, tile_step);                       // the tile of the scales loaded last
    load_scales(at, 0, my_tiles > 0);
    int gi = 0;                           // groups consumed so far
    bool alive = true;
    for (int tile = 0; tile < my_tiles; ++tile) {
      const int rbk = at.row() * (BM / 32) + sub, cbk = at.col() * (BN / 32) + cb0;   // the tile's (`at` moves on below)
      float acc[2][32];
#pragma unroll
      for (int i = 0; i < 32; ++i) acc[0][i] = acc[1][i] = 0.0f;
      for (int w0 = 0; alive && w0 < kblocks; w0 += 32) {
        // lane l: fp32(sA * sB) of contraction block w0 + l for the warp's two output blocks. Times 2^23 that would
        // pass the largest fp32 from 2^105 on: a window with such a block takes a loop of its own, which multiplies the
        // partials by 2^23 instead (one test per 32 blocks; the same products and sums, bit for bit).
        float cw0 = sa_n * sb0_n, cw1 = sa_n * sb1_n;
        const bool large = !__all_sync(0xffffffffu, fabsf(cw0) < kMaxScaled && fabsf(cw1) < kMaxScaled);
        if (!large) {
          cw0 *= kSumScale;
          cw1 *= kSumScale;
        }
        const bool more = w0 + 32 < kblocks;   // the rest of this tile, or the start of the next one
        if (!more) at.next();
        load_scales(at, more ? w0 + 32 : 0, more || tile + 1 < my_tiles);
        const int nk = min(32, kblocks - w0);
        // one contraction block: TMEM -> registers, then acc += c P (packed fp32x2 FMAs, each lane rounded
        // as the scalar fmaf); `last`: the group is in registers and its accumulators may be overwritten
        auto block = [&](uint32_t b, int k, int j, bool last) {
          uint32_t r[64];
          tmem_ld_32x32b_x64(t_base + (b * GROUP + k) * BN, r);
          const float c0 = __shfl_sync(0xffffffffu, cw0, j), c1 = __shfl_sync(0xffffffffu, cw1, j);
          tc_wait_ld64(r);
          if (last) {
            tc_fence_before();
            __syncwarp();
            mbar_arrive_if(&tempty[b], lane == 0);
          }
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float f0, f1, f2, f3;
            partial_x2(r[i], r[i + 1], f0, f1);
            partial_x2(r[32 + i], r[33 + i], f2, f3);
            fma_x2(c0, c0, f0, f1, acc[0][i], acc[0][i + 1], acc[0][i], acc[0][i + 1]);
            fma_x2(c1, c1, f2, f3, acc[1][i], acc[1][i + 1], acc[1][i], acc[1][i + 1]);
          }
        };
        int j0 = 0;
        if (__builtin_expect(large, 0)) {
#pragma unroll 1
          for (; j0 < nk; j0 += GROUP, ++gi) {
            const uint32_t b = uint32_t(gi) & 1u;
            const bool good = mbar_wait_often(&tfull[b], uint32_t(gi >> 1) & 1u, abort_flag, p.status);
            if (!__all_sync(0xffffffffu, good)) {
              alive = false;
              j0 = nk;
              break;
            }
            tc_fence_after();
            const int n = min(GROUP, nk - j0);
#pragma unroll 1
            for (int k = 0; k < n; ++k) {
              const float c0 = __shfl_sync(0xffffffffu, cw0, j0 + k), c1 = __shfl_sync(0xffffffffu, cw1, j0 + k);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t r[32];
                tmem_ld_32x32b_x32(t_base + (b * GROUP + k) * BN + 32 * h, r);
                tc_wait_ld(r);
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                  float f0, f1;
                  partial_x2(r[i], r[i + 1], f0, f1);
                  mul_x2(f0, f1, kSumScale, kSumScale, f0, f1);
                  fma_x2(h ? c1 : c0, h ? c1 : c0, f0, f1, acc[h][i], acc[h][i + 1], acc[h][i], acc[h][i + 1]);
                }
              }
            }
            tc_fence_before();
            __syncwarp();
            mbar_arrive_if(&tempty[b], lane == 0);
          }
        }
#pragma unroll 2
        for (; j0 + GROUP <= nk; j0 += GROUP, ++gi) {
          const uint32_t b = uint32_t(gi) & 1u;
          const bool good = mbar_wait_often(&tfull[b], uint32_t(gi >> 1) & 1u, abort_flag, p.status);
          if (!__all_sync(0xffffffffu, good)) { alive = false; break; }
          tc_fence_after();
          block(b, 0, j0, false);
          block(b, 1, j0 + 1, true);
        }
        if (alive && j0 < nk) {           // the odd block at the end of a tile
          const uint32_t b = uint32_t(gi) & 1u;
          const bool good = mbar_wait_often(&tfull[b], uint32_t(gi >> 1) & 1u, abort_flag, p.status);
          alive = __all_sync(0xffffffffu, good);
          tc_fence_after();
          if (alive) block(b, 0, j0, true);
          ++gi;
        }
      }
      if (!alive) break;
      if constexpr (SPLIT) {
        // the parts of the valid blocks to the CTAs that add them: block b to rank b % parts
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int b = 2 * w + h, owner = b & (parts - 1);
          if (rbk < nrb && cbk + h < ncb)
            block_to_smem(acc[h], cluster.map_shared_rank(smem + SMEM_OUT + (b - owner + rank) * 4096, owner), lane);
        }
        break;
      }
      if constexpr (NOUT == 0) {
        if (kblocks == 0) at.next();      // no scales of the next tile were loaded
        const int nblk = rbk < nrb ? min(2, ncb - cbk) : 0;
#pragma unroll 1
        for (int h = 0; h < nblk; ++h) {
          block_epilogue<EPI>(p.ep, acc[0], rbk, cbk + h, ncb, smem + SMEM_OUT + (2 * w + h) * 4096, lane);
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[0][i] = acc[1][i];
        }
        continue;
      }
      // the finished blocks to the output warps, and on to the next tile
      const bool room = mbar_wait_often(&oempty[w], (uint32_t(tile) & 1u) ^ 1u, abort_flag, p.status);
      if (!__all_sync(0xffffffffu, room)) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) block_to_smem(acc[h], smem + SMEM_OUT + (2 * w + h) * 4096, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ofull[w]);
    }
  } else if constexpr (NOUT > 0) {
    // ------------------------------------------------------------------ output warps
    if constexpr (Roles<NOUT, SUM_REGS>::kOut > Roles<NOUT, SUM_REGS>::kLaunch) setmaxnreg_inc<Roles<NOUT, SUM_REGS>::kOut>();
    else setmaxnreg_dec<Roles<NOUT, SUM_REGS>::kOut>();
    const int nrb = p.rows >> 5, ncb = p.cols >> 5;
    TileWalk at(p, first_tile, tile_step);
    bool alive = true;
    for (int tile = 0; !SPLIT && alive && tile < my_tiles; ++tile, at.next()) {
      for (int w = warp - FIRST_OUT_WARP; w < NUM_SUM_WARPS; w += NOUT) {
        const bool good = mbar_wait_often(&ofull[w], uint32_t(tile) & 1u, abort_flag, p.status);
        alive = __all_sync(0xffffffffu, good);
        if (!alive) break;
        const int rbk = at.row() * (BM / 32) + (w & 3), cbk = at.col() * (BN / 32) + (w >> 2) * 2;
        const int nblk = rbk < nrb ? min(2, ncb - cbk) : 0;
#pragma unroll 1
        for (int h = 0; h < nblk; ++h) {
          uint8_t* blk = smem + SMEM_OUT + (2 * w + h) * 4096;
          float v[32];
          block_from_smem(v, blk, lane);
          __syncwarp();                   // the block's memory is the warp's staging area from here on
          block_epilogue<EPI>(p.ep, v, rbk, cbk + h, ncb, blk, lane);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&oempty[w]);
      }
    }
    if constexpr (SPLIT) {
      cluster.sync();                     // every part is where it is added
      const bool whole = *abort_flag == 0u;
      for (int b = rank + parts * (warp - FIRST_OUT_WARP); whole && b < 16; b += parts * NOUT) {
        const int w = b >> 1, rbk = at.row() * (BM / 32) + (w & 3), cbk = at.col() * (BN / 32) + (w >> 2) * 2 + (b & 1);
        if (rbk >= nrb || cbk >= ncb) continue;
        uint8_t* blk = smem + SMEM_OUT + (b - rank) * 4096;   // the parts in rank order
        float v[32], part[32];
        block_from_smem(v, blk, lane);
        for (int r = 1; r < parts; ++r) {
          block_from_smem(part, blk + r * 4096, lane);
#pragma unroll
          for (int i = 0; i < 32; i += 2) add_x2(v[i], v[i + 1], part[i], part[i + 1], v[i], v[i + 1]);
        }
        __syncwarp();                     // the block's memory is the warp's staging area from here on
        block_epilogue<EPI>(p.ep, v, rbk, cbk, ncb, blk, lane);
      }
    }
  }
  if constexpr (SPLIT) {
    if (warp < FIRST_OUT_WARP) cluster.sync();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem_base, TMEM_COLS);
}

// ---------------------------------------------------------------------------------------------
// Plain INT8 GEMM, C (int32) = A B^T, for measuring the tensor core's INT8 rate: the same TMA and
// tcgen05 machinery with the whole contraction accumulated in TMEM (no per-block rescale), tiles of
// 128 x 256 (MMA N = 256), two 256-column accumulators so the epilogue of one tile overlaps the
// MMAs of the next. Both operands K-major; M % 128 == 0, N % 256 == 0, K % 128 == 0.
//   warp 0 producer (as above), warp 1 MMA, warps 2-9 epilogue (TMEM -> int32 rows in global).
// ---------------------------------------------------------------------------------------------
constexpr int S32_BN = 256;
constexpr int S32_STAGES = 4;
constexpr int S32_EPI_WARPS = 8;
constexpr int S32_THREADS = 64 + 32 * S32_EPI_WARPS;
constexpr int S32_A_STAGE = BM * KBS * KB;       // 16 KB
constexpr int S32_B_STAGE = S32_BN * KBS * KB;   // 32 KB
constexpr int S32_SMEM_BAR = S32_STAGES * (S32_A_STAGE + S32_B_STAGE);
constexpr int S32_NUM_BARS = 2 * S32_STAGES + 4 + 1;
constexpr int S32_SMEM_BYTES = S32_SMEM_BAR + S32_NUM_BARS * 8 + 16 + 1024;

struct __align__(64) GemmS32Params {
  CUtensorMap tma_a;
  CUtensorMap tma_b;
  int32_t* c;
  int64_t ldc;
  unsigned int* status;
  int kblocks, tiles_m, tiles_n;
};

__global__ void __launch_bounds__(S32_THREADS, 1) gemm_i8_s32_kernel(const __grid_constant__ GemmS32Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + S32_STAGES * S32_A_STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S32_SMEM_BAR);
  uint64_t* empty = full + S32_STAGES;
  uint64_t* tfull = empty + S32_STAGES;   // per accumulator: the tile's MMAs completed
  uint64_t* tempty = tfull + 2;           // per accumulator: every epilogue warp has read it
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile uint32_t* abort_flag = tmem_holder + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S32_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], S32_EPI_WARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  const int num_kstages = p.kblocks / KBS;
  const int num_tiles = p.tiles_m * p.tiles_n;
  const int my_tiles = blockIdx.x < num_tiles ? (num_tiles - 1 - blockIdx.x) / gridDim.x + 1 : 0;
  const int total_stages = my_tiles * num_kstages;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t pending = 0, pend_ph = 0;
      for (int g = 0; g < total_stages; ++g) {
        const int t = blockIdx.x + (g / num_kstages) * gridDim.x;
        const int k0 = (g % num_kstages) * KBS * KB;
        const int row0 = (t % p.tiles_m) * BM, col0 = (t / p.tiles_m) * S32_BN;
        const int st = g % S32_STAGES;
        const uint32_t ph = uint32_t(g / S32_STAGES) & 1u;
        if (!mbar_wait(&empty[st], ph ^ 1u, abort_flag, p.status)) break;
        mbar_arrive_expect_tx(&full[st], S32_A_STAGE + S32_B_STAGE);
        pending |= 1u << st;
        pend_ph = (pend_ph & ~(1u << st)) | (ph << st);
        tma_load_2d(sA + st * S32_A_STAGE, &p.tma_a, &full[st], k0, row0);
        tma_load_2d(sB + st * S32_B_STAGE, &p.tma_b, &full[st], k0, col0);
      }
      for (int s = 0; s < S32_STAGES; ++s)
        if (pending & (1u << s)) mbar_wait_teardown(&full[s], (pend_ph >> s) & 1u, p.status);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = instr_desc<false, false, S32_BN>();
      bool issued = false, ok = true;
      int g = 0;
      for (int i = 0; ok && i < my_tiles; ++i) {
        const uint32_t buf = uint32_t(i) & 1u;
        if (!mbar_wait(&tempty[buf], (uint32_t(i >> 1) & 1u) ^ 1u, abort_flag, p.status)) break;
        tc_fence_after();
        for (int ks = 0; ks < num_kstages; ++ks, ++g) {
          const int st = g % S32_STAGES;
          if (!mbar_wait(&full[st], uint32_t(g / S32_STAGES) & 1u, abort_flag, p.status)) { ok = false; break; }
          const uint32_t a_addr = smem_u32(sA + st * S32_A_STAGE), b_addr = smem_u32(sB + st * S32_B_STAGE);
#pragma unroll
          for (int kk = 0; kk < KBS; ++kk)
            mma_i8(tmem_base + buf * S32_BN, smem_desc(a_addr + kk * 32, 16, 1024), smem_desc(b_addr + kk * 32, 16, 1024),
                   idesc, (ks | kk) != 0 ? 1u : 0u);
          tc_commit(&empty[st]);
          issued = true;
        }
        if (ok) tc_commit(&tfull[buf]);
      }
      if (issued) {
        tc_commit(drain);
        mbar_wait_teardown(drain, 0u, p.status);
      }
    }
    __syncwarp();
  } else {
    const int sub = warp & 3, half = (warp - 2) >> 2;
    const uint32_t t_base = tmem_base + (uint32_t(sub * 32) << 16) + uint32_t(half * 128);
    for (int i = 0; i < my_tiles; ++i) {
      const uint32_t buf = uint32_t(i) & 1u;
      const uint32_t ph = uint32_t(i >> 1) & 1u;
      const bool good = mbar_try_wait(&tfull[buf], ph) || mbar_wait(&tfull[buf], ph, abort_flag, p.status);
      if (!__all_sync(0xffffffffu, good)) break;
      tc_fence_after();
      const int t = blockIdx.x + i * gridDim.x;
      const int64_t row = int64_t(t % p.tiles_m) * BM + sub * 32 + lane;
      int32_t* dst = p.c + row * p.ldc + int64_t(t / p.tiles_m) * S32_BN + half * 128;
#pragma unroll 1
      for (int ch = 0; ch < 4; ++ch) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(t_base + buf * S32_BN + ch * 32, r);
        tc_wait_ld(r);
        int4* d4 = reinterpret_cast<int4*>(dst + ch * 32);
#pragma unroll
        for (int j = 0; j < 8; ++j) d4[j] = make_int4(int(r[4 * j]), int(r[4 * j + 1]), int(r[4 * j + 2]), int(r[4 * j + 3]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[buf]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem_base, 512);
}

// ---------------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (fn == nullptr) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }
  return fn;
}

// 2-D int8 tensor map over a row-major [outer, inner] matrix with row pitch `ld` bytes.
static bool make_map(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint64_t ld,
                     uint32_t box_inner, uint32_t box_outer) {
  auto fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {ld};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool A_MN, bool B_MN, int EPI, int NOUT, int SUM_REGS, bool SPLIT>
static cudaError_t run(const GemmParams& prm, int grid, int parts, cudaStream_t st) {
  static unsigned long long attr_set = 0;  // one bit per device ordinal
  auto kern = gemm_i8_kernel<A_MN, B_MN, EPI, NOUT, SUM_REGS, SPLIT>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(attr_set & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    attr_set |= bit;
  }
  if constexpr (SPLIT) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid * parts), 1, 1);
    cfg.blockDim = dim3(Roles<NOUT, SUM_REGS>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(parts);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, prm);
  }
  kern<<<grid, Roles<NOUT, SUM_REGS>::kThreads, SMEM_BYTES, st>>>(prm);
  return cudaGetLastError();
}

cudaError_t launch_gemm(const GemmArgs& g, int sm_count, cudaStream_t st) {
  GemmParams prm;
  memset(&prm, 0, sizeof(prm));
  const int64_t rb = g.rows / 32, cb = g.cols / 32, kbn = g.depth / 32;
  bool okA = true, okB = true;
  const bool operands = g.depth > 0;   // without a contraction (bias and residual alone) nothing is loaded
  switch (g.mode) {
    case kFwd:  // A = X [rows, depth], B = W [cols, depth]; both K-major
      okA = !operands || make_map(&prm.tma_a, g.a_q, g.depth, g.rows, g.a_ld, 128, BM);
      okB = !operands || make_map(&prm.tma_b, g.b_q, g.depth, g.cols, g.b_ld, 128, BN);
      prm.a_s_blk = kbn; prm.a_s_k = 1;
      prm.b_s_blk = kbn; prm.b_s_k = 1;
      break;
    case kDgrad:  // A = dY [rows, depth] K-major; B = W [depth, cols] MN-major
      okA = !operands || make_map(&prm.tma_a, g.a_q, g.depth, g.rows, g.a_ld, 128, BM);
      okB = !operands || make_map(&prm.tma_b, g.b_q, g.cols, g.depth, g.b_ld, 128, 128);
      prm.a_s_blk = kbn; prm.a_s_k = 1;
      prm.b_s_blk = 1; prm.b_s_k = cb;
      break;
    default:  // kWgrad: A = dY [depth, rows] MN-major; B = X [depth, cols] MN-major
      okA = !operands || make_map(&prm.tma_a, g.a_q, g.rows, g.depth, g.a_ld, 128, 128);
      okB = !operands || make_map(&prm.tma_b, g.b_q, g.cols, g.depth, g.b_ld, 128, 128);
      prm.a_s_blk = 1; prm.a_s_k = rb;
      prm.b_s_blk = 1; prm.b_s_k = cb;
      break;
  }
  if (!okA || !okB) return cudaErrorInvalidValue;
  prm.a_s = g.a_s;
  prm.b_s = g.b_s;
  prm.status = g.status;
  prm.rows = int(g.rows);
  prm.cols = int(g.cols);
  prm.kblocks = int(kbn);
  prm.tiles_m = int((g.rows + BM - 1) / BM);
  prm.n_fast = g.rows > g.cols ? 1 : 0;   // A (rows x depth) larger than B: keep B in L2
  prm.tiles_n = int((g.cols + BN - 1) / BN);
  const int tiles = prm.tiles_m * prm.tiles_n;
  const int grid = tiles < sm_count ? tiles : sm_count;
  const auto bytes = [](int type) { return int64_t(type == kDenseF32 ? 4 : 2); };
  prm.ep.bias = g.bias;
  prm.ep.act = g.act;
  prm.ep.act_q = g.act_q;
  prm.ep.act_s = g.act_s;
  prm.ep.res = static_cast<const uint8_t*>(g.res);
  prm.ep.res_s = g.res_s;
  prm.ep.res_type = g.res_type;
  prm.ep.res_ld = g.res_ld * bytes(g.res_type);
  prm.ep.y_q = g.y_q;
  prm.ep.y_s = g.y_s;
  prm.ep.pre_q = g.pre_q;
  prm.ep.pre_s = g.pre_s;
  prm.ep.ld_q = g.cols;
  prm.ep.y = static_cast<uint8_t*>(g.y);
  prm.ep.y_type = g.y_type;
  prm.ep.y_ld = g.y_ld * bytes(g.y_type);
  // The exact GELU (an erfc per element) takes 4 output warps longer than 64 contraction blocks take the sum warps:
  // up to there 8 of them are faster (4096 x 2048 x 4096 154 us against 160), beyond they only slow the sum warps down.
  // Every other epilogue keeps up with 4.
  const bool out8 = g.act == kActGelu && kbn <= 64;
  // Few tiles leave SMs idle: the contraction is then split over clusters of 2, 4 or 8 CTAs, each with at least
  // one pipeline stage (two in clusters of 8, where one costs 1 us more than clusters of 4), as long as all
  // clusters run at once: a GPC's last SMs do not make up a whole cluster (of 148 SMs, 33 clusters of 4 and 15
  // of 8 are resident), which the 5 clusters to spare allow for. Undivided and split, us (bias, SiLU, bf16):
  // 32 x 4096 x 4096 45 and 21, 32 x 16384 x 4096 135 and 45, 352 x 1056 x 544 20.5 and 16.4, 256^3 17.2 and
  // 15.5, 1024 x 4096 x 1024 45 and 31. The sum's order, and with it the last bits, differ from the undivided
  // sum's, so only the calls that were born with it take it (split_ok).
  const int stages = int((kbn + KBS - 1) / KBS);
  int parts = 1;
  for (int c = 2; g.split_ok && c <= 8; c *= 2)
    if ((tiles + 5) * c <= sm_count && stages >= (c < 8 ? c : 2 * c)) parts = c;
  prm.share = (stages + parts - 1) / parts;
  // The sum warps as output warps (`direct`): output warps pay for overlapping a tile's epilogue with the next tile, by
  // a copy through shared memory and cold code at a call's end, and 4 of them take twice as long as 8 for one epilogue.
  // With and without them, us in a graph of such calls, INT8 out: one tile a CTA, 128^3 8.5 and 5.8, 512^3 11.2 and
  // 8.7, 1024^3 with GELU (jf_linear_fwd_gelu) 21.0 and 17.6, 1024 x 4096 x 1024 38.1 and 36.3; more tiles,
  // 4096 x 32 x 4096 30.2 and 17.9, 4096 x 256 x 4096 36.2 and 28.7 (weight gradient 29.6 and 29.0, but 29.4 and 34.5 with
  // fp32 out, whose border is 128: 26.6 and 26.1), 4096 x 512 x 4096 as input gradient 42.0 and 42.0; the exact GELU
  // 4096 x 1024 x 4096 109 and 104, 4096 x 2048 x 4096 152 and 158.
  const bool direct = parts == 1 && (tiles <= sm_count || kbn <= (g.y == nullptr ? 8 : 4) || (g.act == kActGelu && kbn <= 32));
  // without bias, activation and residual the instance without their code (cold: 128^3 6.4 with it, 5.8 without)
  const bool plain = g.bias == nullptr && g.act == kActNone && g.res == nullptr && g.pre_q == nullptr;
  if (g.mode == kFwd) {
    if (parts > 1) return run<false, false, kEpiForward, 4, 168, true>(prm, tiles, parts, st);
    if (direct)
      return plain ? run<false, false, kEpiPlain, 0, 232, false>(prm, grid, 1, st)
                   : run<false, false, kEpiForward, 0, 232, false>(prm, grid, 1, st);
    if (out8) return run<false, false, kEpiForward, 8, 152, false>(prm, grid, 1, st);
    // The register split for the output warps (168) or for the sum warps (176): 4096 x 1024 x 4096 with GELU and both
    // outputs takes 6% longer with 176, 4096 x 2048 x 4096 with GELU 3% longer with 168 and 8192 x 16384 x 4096 3.5%.
    return kbn <= 32 ? run<false, false, kEpiForward, 4, 168, false>(prm, grid, 1, st)
                     : run<false, false, kEpiForward, 4, 176, false>(prm, grid, 1, st);
  }
  if (g.mode == kDgrad) {
    if (parts > 1) return run<false, true, kEpiGrad, 4, 176, true>(prm, tiles, parts, st);
    if (direct)
      return plain ? run<false, true, kEpiPlain, 0, 232, false>(prm, grid, 1, st)
                   : run<false, true, kEpiGrad, 0, 232, false>(prm, grid, 1, st);
    return run<false, true, kEpiGrad, 4, 176, false>(prm, grid, 1, st);
  }
  if (direct) return run<true, true, kEpiPlain, 0, 232, false>(prm, grid, 1, st);
  return run<true, true, kEpiPlain, 4, 176, false>(prm, grid, 1, st);
}

cudaError_t launch_gemm_s32(const int8_t* a, const int8_t* b, int32_t* c, int64_t M, int64_t N, int64_t K,
                            unsigned int* status, int sm_count, cudaStream_t st) {
  GemmS32Params prm;
  memset(&prm, 0, sizeof(prm));
  if (!make_map(&prm.tma_a, a, uint64_t(K), uint64_t(M), uint64_t(K), 128, BM) ||
      !make_map(&prm.tma_b, b, uint64_t(K), uint64_t(N), uint64_t(K), 128, S32_BN))
    return cudaErrorInvalidValue;
  prm.c = c;
  prm.ldc = N;
  prm.status = status;
  prm.kblocks = int(K / KB);
  prm.tiles_m = int(M / BM);
  prm.tiles_n = int(N / S32_BN);
  const int tiles = prm.tiles_m * prm.tiles_n;
  const int grid = tiles < sm_count ? tiles : sm_count;
  static unsigned long long attr_set = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(attr_set & bit)) {
    e = cudaFuncSetAttribute(gemm_i8_s32_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S32_SMEM_BYTES);
    if (e != cudaSuccess) return e;
    attr_set |= bit;
  }
  gemm_i8_s32_kernel<<<grid, S32_THREADS, S32_SMEM_BYTES, st>>>(prm);
  return cudaGetLastError();
}

}  // namespace jf
