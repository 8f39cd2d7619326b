// pair_gemm.cuh -- matrix products of 16-bit operands on pairs of
// multiprocessors (tcgen05, cta_group::2), as a frame that the kernels of the
// cross entropy fill with their own order of tiles and their own use of a
// finished tile.
//
// A cluster of two blocks works on one tile of 256 x 256 (or fewer columns, where
// that fills the GPU better): each block stages 128 rows of A and half of B's per
// 64 summed indexes (32 KB; six stages, more of narrower tiles), and gets the
// tile's upper or lower 128 rows.  The pair is what lets the tensor cores run: a
// block alone would have to load twice the bytes of B per product, 96 bytes per
// clock and SM at the full rate, which the L2 does not deliver to all SMs at once;
// so it is 64.  Measured: 2.2 * 10^12 operations of 8192 x 65536 x 2048 in 1.01 ms
// (2.18 PFLOP/s) alone; 1.61 in a training step under the power cap, where cuBLAS
// sustains 1.70.
//
// The tensor cores cut the sum off at every addition (toward zero): 4096 positive
// terms come out 1.1e-5 too small, 16384 7e-5.  So tensor memory only ever holds the
// sum over kSumBlocks blocks; what reads the tiles out adds these in registers,
// rounded to nearest, up to 128 columns of a row per lane.  Two such sums fit: one is
// made while the other is read.
//
// Warp 0 issues the loads (TMA, 128-byte swizzle), warp 1 of the even block
// the products, warps 4 to 11 read the sums out, half the columns to each four.
#pragma once

#include <cuda.h>

#include "cluster.cuh"
#include "seq.h"
#include "tcgen05.cuh"

namespace fftgb {

constexpr int kPairTile = 256, kPairK = 64, kPairStages = 10;  // stages at most
constexpr int kPairThreads = 384, kOutWarps = 8;
// Sums of 512 terms: 7e-7 too small at most, for 1 to 2% of the time (8192 tokens with
// gradients: 5.52 ms with 1024 terms, 5.57 with 512, 5.83 with 256).
constexpr int kSumBlocks = 8;
constexpr uint32_t kStageHalf = 128 * 128;  // bytes of A (of B) per stage and block
// the stages, and behind them 32 x 33 floats for each of the warps that read tiles out
constexpr uint32_t kPairStageBytes = 6 * 2 * kStageHalf;
constexpr size_t kPairSpare = kOutWarps * 32 * 33 * sizeof(float);
constexpr size_t kPairSmem = 1024 + kPairStageBytes + kPairSpare;
extern __shared__ char pair_smem[];
__device__ __forceinline__ float *pair_spare() {
  return reinterpret_cast<float *>(pair_smem + ((1024 - (smem_u32(pair_smem) & 1023)) & 1023) + kPairStageBytes);
}

// ---- instructions for a pair of blocks -------------------------------------------------

__device__ __forceinline__ void pair_tmem_alloc(uint32_t *slot) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                   smem_u32(slot))
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_free(uint32_t base) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(base) : "memory");
}
// A box of a tensor of three axes into this block's shared memory, counted by
// the barrier at the cluster address `bar`.
__device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x,
                                          int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// D (TMEM of both blocks) (+)= A (shared, half the rows each) B (shared, half the columns each).
__device__ __forceinline__ void pair_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                         bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)accumulate), "n"(kDescHigh)
      : "memory");
}
// One arrival at the barrier of both blocks when the products so far have completed.
__device__ __forceinline__ void pair_commit(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// What these barriers order lies in tensor memory and behind the asynchronous proxy, so
// arrivals and waits have block scope: with cluster scope each would wait for the
// stores to global memory under way.
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ bool wait_pair(uint64_t *bar, uint32_t parity, volatile int *failed,
                                          int *status, long long limit) {
  if (bar_poll(bar, parity)) return true;
  const long long t0 = clock64();
#pragma unroll 1
  for (uint32_t it = 0; it < (1u << 24); ++it) {
    if (bar_poll(bar, parity)) return true;
    if (*failed || clock64() - t0 > limit) break;
  }
  *failed = 1;
  atomicExch(status, 1);  // kDeviceErrorTimeout
  return false;
}
// Registers: 384 threads are launched with 168 each (64 512); the loads and products
// keep 56, the warps that add sums up have 224.  56 * 128 + 224 * 256 = 64 512.
constexpr int kPairRegs = 168;
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 56;" ::: "memory");
}
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 224;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void add32(float (&sums)[N], int j, const uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float2 v = add2(make_float2(sums[j + i], sums[j + i + 1]),
                          make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])));
    sums[j + i] = v.x;
    sums[j + i + 1] = v.y;
  }
}

// ---- a tile's work ---------------------------------------------------------------------

// One tile of A B^T summed over blocks k0 .. k1 - 1 of 64 indexes, for every
// pair of parts.  K-major operands have their rows along `row`; MN-major
// ones have the summed index along their rows, from row kbase on.
struct PairTile {
  int a_row, b_row;    // first row of the tile in A and B
  int k0, k1;          // blocks of summed indexes
  int a_base, b_base;  // row of summed index 0 in an MN-major operand
};
// A problem's operands.
struct PairOperands {
  CUtensorMap a, b;
  int a_mn, b_mn;
  int width;  // columns of a tile: a multiple of 64 up to 256
  uint32_t b_bytes;  // of B per block and stage, as the boxes of its map bring them
  uint32_t idesc;
  // Products of parts: an fp32 operand is the sum of three bf16 parts, of
  // which the six largest products are taken, the smallest first.
  int parts;
  Waits waits;  // of a launch: its first problem's
};
__device__ __forceinline__ int part_pairs(int parts) { return parts == 1 ? 1 : 6; }
__device__ __forceinline__ void part_pair(int parts, int q, int &pa, int &pb) {
  // (2,0) (0,2) (1,1) (1,0) (0,1) (0,0)
  pa = parts == 1 ? 0 : (0x001102 >> (4 * q)) & 15;
  pb = parts == 1 ? 0 : (0x010120 >> (4 * q)) & 15;
}

struct PairShared {
  uint64_t full[kPairStages], empty[kPairStages], ready[2], taken[2], done;
  uint32_t tmem;
  int failed;
};

// Runs the tiles pair, pair + pairs, ... < tiles.  of(t, which) gives a tile
// and which of the problems `ops` it belongs to; out(t, sums) uses one, in warps 4 ..
// 11: a lane of warp w has the tile's row 128 rank + 32 (w % 4) + lane and, in
// `sums`, the first (w < 8) or last half of its columns.
template <class Of, class Out>
__device__ __forceinline__ void pair_run(const PairOperands *ops, int tiles, int *status, Of of,
                                         Out out) {
  __shared__ PairShared sh;
  const uint32_t stage0 = (smem_u32(pair_smem) + 1023) & ~1023u;
  // all problems of a launch have one width
  const uint32_t stage_bytes = kStageHalf + ops[0].b_bytes;
  const uint32_t stages = min((uint32_t)kPairStages, kPairStageBytes / stage_bytes);
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t rank = block_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  volatile int *failed = &sh.failed;
  const long long limit = ops[0].waits.limit;
  if (tid == 0) {
    const int starved = blockIdx.x == 0 ? ops[0].waits.starved : 0;  // one arrival more than will come
    for (int s = 0; s < kPairStages; ++s) {
      bar_init(&sh.full[s], starved == 1 && s == 0 ? 2 : 1);
      bar_init(&sh.empty[s], starved == 2 && s == 0 ? 2 : 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&sh.ready[i], starved == 3 && i == 0 ? 2 : 1);
      bar_init(&sh.taken[i], 2 * kOutWarps + (starved == 4 && i == 0 ? 1 : 0));
    }
    bar_init(&sh.done, 1);
    sh.failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  let_next();
  if (warp == 2) pair_tmem_alloc(&sh.tmem);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  after_previous();
  const uint32_t tm = sh.tmem;

  if (warp < 4) {
    fewer_registers();
    if (warp == 0) {
      if (elect_one()) {
        uint32_t s = 0, round = 0;  // the stage, and how often the ring has gone round
        bool ok = true;
        for (int t = pair; ok && t < tiles; t += pairs) {
          int which = 0;
          const PairTile w = of(t, which);
          const PairOperands &p = ops[which];
          const int a_row = w.a_row + (int)rank * 128, b_row = w.b_row + (int)rank * (p.width / 2);
          const int nq = part_pairs(p.parts);
          for (int q = 0; ok && q < nq; ++q) {
            int pa, pb;
            part_pair(p.parts, q, pa, pb);
            for (int kb = w.k0; kb < w.k1; ++kb) {
              if (round > 0 && !wait_pair(&sh.empty[s], (round - 1) & 1, failed, status, limit)) {
                ok = false;
                break;
              }
              if (rank == 0) bar_arrive_tx(&sh.full[s], 2 * (kStageHalf + p.b_bytes));
              const uint32_t bar = peer(smem_u32(&sh.full[s]), 0);
              const uint32_t sa = stage0 + s * stage_bytes, sb = sa + kStageHalf;
              const int k = kb * kPairK;
              if (p.a_mn) {
                pair_load(sa, &p.a, bar, a_row, w.a_base + k, pa);
                pair_load(sa + kStageHalf / 2, &p.a, bar, a_row + 64, w.a_base + k, pa);
              } else {
                pair_load(sa, &p.a, bar, k, a_row, pa);
              }
              if (p.b_mn) {
                pair_load(sb, &p.b, bar, b_row, w.b_base + k, pb);
                if (p.width > 128)
                  pair_load(sb + kStageHalf / 2, &p.b, bar, b_row + 64, w.b_base + k, pb);
              } else {
                pair_load(sb, &p.b, bar, k, b_row, pb);
              }
              if (++s == stages) s = 0, ++round;
            }
          }
        }
        // no copy, and no arrival of a completed product, may land after a block has gone
        for (uint32_t i = 0; i < stages; ++i) {
          if (i >= s && round == 0) break;
          const uint32_t last = (i < s ? round : round - 1) & 1;
          if (ok) wait_pair(&sh.empty[i], last, failed, status, limit);
          else if (rank == 0) let_land(&sh.full[i], last);
        }
      }
    } else if (warp == 1 && rank == 0) {
      if (elect_one()) {
        uint32_t s = 0, round = 0, n = 0;
        bool ok = true;
        for (int t = pair; ok && t < tiles; t += pairs) {
          int which = 0;
          const PairTile w = of(t, which);
          const PairOperands &p = ops[which];
          const int blocks = (w.k1 - w.k0) * part_pairs(p.parts);
          // 16 summed indexes: 32 bytes of a K-major row, 16 rows of an MN-major tile
          const uint32_t step_a = p.a_mn ? 2048 : 32, step_b = p.b_mn ? 2048 : 32;
          for (int b0 = 0; ok && b0 < blocks; b0 += kSumBlocks, ++n) {
            const int acc = n & 1, count = min(kSumBlocks, blocks - b0);
            if (n > 1 && !wait_pair(&sh.taken[acc], ((n >> 1) - 1) & 1, failed, status, limit)) {
              ok = false;
              break;
            }
            tc_fence_after();
            for (int kb = 0; kb < count; ++kb) {
              if (!wait_pair(&sh.full[s], round & 1, failed, status, limit)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t sa = stage0 + s * stage_bytes, sb = sa + kStageHalf;
#pragma unroll
              for (uint32_t k = 0; k < kPairK / 16; ++k)
                pair_mma(tm + acc * kPairTile, tile_desc(sa + k * step_a, kStageHalf / 2),
                         tile_desc(sb + k * step_b, kStageHalf / 2), p.idesc, kb > 0 || k > 0);
              pair_commit(&sh.empty[s]);
              if (++s == stages) s = 0, ++round;
            }
            if (ok) pair_commit(&sh.ready[acc]);
          }
        }
        if (*failed) {  // no product may write tensor memory that has been given back
          pair_commit(&sh.done);
          let_land(&sh.done, 0);
        }
      }
    }
  } else {
    more_registers();
    uint32_t n = 0;
    const uint32_t base = tm + ((uint32_t)(warp & 3) << 21);
    bool ok = true;
    for (int t = pair; ok && t < tiles; t += pairs) {
      int which = 0;
      const PairTile w = of(t, which);
      const int wide = ops[which].width / 2;
      const int blocks = (w.k1 - w.k0) * part_pairs(ops[which].parts);
      float sums[kPairTile / 2];
#pragma unroll
      for (int i = 0; i < kPairTile / 2; ++i) sums[i] = 0.0f;
      for (int b0 = 0; b0 < blocks; b0 += kSumBlocks, ++n) {
        const int acc = n & 1;
        // a warp reads on or leaves as one: lanes may see the end of a wait differently
        ok = __all_sync(0xffffffffu, wait_pair(&sh.ready[acc], (n >> 1) & 1, failed, status, limit));
        if (!ok) break;
        __syncwarp();
        tc_fence_after();
        const uint32_t at = base + acc * kPairTile + (uint32_t)((warp - 4) >> 2) * wide;
        uint32_t r[2][32];
        tmem_ld(at, r[0]);
        if (wide > 32) tmem_ld(at + 32, r[1]);
        tmem_wait_ld();
        add32(sums, 0, r[0]);
        if (wide > 64) tmem_ld(at + 64, r[0]);
        if (wide > 32) add32(sums, 32, r[1]);
        if (wide > 96) tmem_ld(at + 96, r[1]);
        tmem_wait_ld();
        if (wide > 64) add32(sums, 64, r[0]);
        if (wide > 96) add32(sums, 96, r[1]);
        tc_fence_before();
        __syncwarp();
        if ((tid & 31) == 0) arrive_at(peer(smem_u32(&sh.taken[acc]), 0));
      }
      if (ok) out(t, sums);
    }
  }
  __syncwarp();
  __syncthreads();
  // Given up: what this block has on its way to the other (its loads count there, its products'
  // ends too), and what the other has on its way here, lands before either goes.
  if (*failed) linger();
  __syncwarp();
  cluster_sync();
  if (*failed) linger();
  __syncwarp();
  if (warp == 2) pair_tmem_free(tm);
}

}  // namespace fftgb
