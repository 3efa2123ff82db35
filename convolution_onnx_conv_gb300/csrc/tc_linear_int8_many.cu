// Linear layers on int8 operands for many rows per weight matrix: y^T = W x^T with integer sums, on tcgen05 (see
// linear_int8_dev.cuh), in tiles of 256 weight rows x 192 rows of x on CTA pairs.
//
// A unit, 64 values, takes the tensor cores 384 cycles; meanwhile each CTA of a pair has to convert 128 weight rows
// and 96 rows of x of it (a single CTA's 128 x 192 tile: 128 and 192), 84 integer instructions at half rate for each
// of four warps.  What a unit goes through is long (its bytes' arrival, the conversion, the pair's barrier, the MMAs,
// their end seen in both CTAs), and TMEM holds only four units of weights beside two accumulators of 192 columns:
// so weights are converted ahead, in registers, and wait for a place for their stores only; rows of x, with places
// for eight units in shared memory, have warps of their own.
//
//   warps 0, 1    TMA: weight and x tiles of 128 values; TMEM and MMA issue (of a pair: the leader's)
//   warp 2        the tile schedule
//   warps 4-11    int8 -> fp16 of the weights: two groups of four warps, each a unit of every stage
//   warps 12-15   int8 -> fp16 of x
//   warps 16-23   epilogue: warp w the weight rows 32 (w % 4) .. and half of the columns
#include "linear_int8_dev.cuh"

namespace convf {

namespace {

constexpr int TN = kInt8PairRows;   // columns: rows of x

struct Int8ManyCfg {
  static constexpr int kXRows = TN / 2;              // rows of x that a CTA loads and converts
  static constexpr int kCols = TN / 2;               // columns per epilogue thread
  static constexpr int kThreads = 768;
  static constexpr int kWBytes = 128 * kKBlockBytes, kXBytes = kXRows * kKBlockBytes;   // of a stage, int8
  static constexpr int kBBytes = kXRows * 2 * kUnit; // of a unit of x, fp16
  static constexpr int kStages = 4, kAUnits = 4, kBBlocks = 4;   // places: int8 stages, units of weights, pairs of units of x
  static constexpr int kDCol = kAUnits * kUnitCols;  // the accumulators' first column
  static constexpr int kBarBytes = 256;
  static constexpr int kSmem = kStages * (kWBytes + kXBytes) + 2 * kBBlocks * kBBytes + kBarBytes + kScheduleBytes;
  // registers: 80 per thread at launch; the epilogue's two warpgroups take what the others give up
  static constexpr int kRegs = 80, kRegsEpi = 136, kRegsW = 64, kRegsX = 40, kRegsOther = 40;
  static_assert(256 * kRegsEpi + 256 * kRegsW + 128 * (kRegsX + kRegsOther) <= kThreads * kRegs, "register split");
  static_assert((2 * kStages + 2 * kAUnits + 2 * kBBlocks + 4) * 8 + 8 <= kBarBytes && kSmem <= 232448, "shared memory");
  static_assert(kDCol + 2 * TN <= 512, "TMEM columns");
};

__global__ void __launch_bounds__(Int8ManyCfg::kThreads, 1)
    linear_int8_many_kernel(const LinearParams p, const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX) {
  using Cfg = Int8ManyCfg;
  constexpr int kStages = Cfg::kStages, kAUnits = Cfg::kAUnits, kBBlocks = Cfg::kBBlocks, kCols = Cfg::kCols;
  constexpr int kChunkBlocks = kInt8Chunk / kKBlockBytes;
  extern __shared__ __align__(1024) uint8_t sW[];   // (the swizzle goes by address bits 7 to 9)
  uint8_t* sX = sW + kStages * Cfg::kWBytes;
  uint8_t* sB = sX + kStages * Cfg::kXBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sB + 2 * kBBlocks * Cfg::kBBytes);   // int8 tiles are here
  uint64_t* empty = full + kStages;     // and have been read
  uint64_t* afull = empty + kStages;    // a unit of weights is in TMEM, of both CTAs (the leader's)
  uint64_t* aempty = afull + kAUnits;   // and its MMAs have read it
  uint64_t* bfull = aempty + kAUnits;   // two units of x are converted, of both CTAs (the leader's)
  uint64_t* bempty = bfull + kBBlocks;  // and their MMAs have read them
  uint64_t* tfull = bempty + kBBlocks;  // an accumulator holds a chunk's sums
  uint64_t* tempty = tfull + 2;         // and has been read, in both CTAs (the leader's)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* prefix = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(full) + Cfg::kBarBytes);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 12);
    }
    for (int u = 0; u < kAUnits; ++u) {
      mbar_init(&afull[u], 8);
      mbar_init(&aempty[u], 1);
    }
    for (int b = 0; b < kBBlocks; ++b) {
      mbar_init(&bfull[b], 8);
      mbar_init(&bempty[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 16);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_launch_dependents();   // after the TMEM allocation, which a dependent's CTA would otherwise take
  pdl_wait_prior();
  if (warp == 2) build_schedule(p, TN, prefix, blockIdx.x == 0);
  __syncthreads();

  const long long tiles = tile_count(p, prefix);
  const long long t0 = blockIdx.x >> 1, tstep = gridDim.x >> 1;
  const long long mine = tiles > t0 ? (tiles - t0 - 1) / tstep + 1 : 0;   // tiles of this pair
  const long long blocks = mine * p.num_kb;                               // and their stages

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsOther));
    if (warp == 0) {
      if (lane == 0) {
        int stage = 0;
        uint32_t phase = 0;
        for (long long t = t0; t < tiles; t += tstep) {
          const LinearTile q = tile_at<TN, kManyCols>(p, prefix, t);
          for (int kb = 0; kb < p.num_kb; ++kb) {
            if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, p.status)) goto teardown;
            mbar_arrive_expect_tx(&full[stage], Cfg::kWBytes + Cfg::kXBytes);
            tma_load_3d(sW + stage * Cfg::kWBytes, &tmW, &full[stage], kb * kKBlockBytes, q.n0 + rank * 128, q.e);
            tma_load_2d(sX + stage * Cfg::kXBytes, &tmX, &full[stage], kb * kKBlockBytes, q.row0 + rank * Cfg::kXRows);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
      }
    } else if (warp == 1 && rank == 0) {
      // the whole warp walks the loop and one lane issues: the loop's state then stays in uniform
      // registers, which is where the MMA takes its descriptors from
      const bool issue = elect_one();
      constexpr uint32_t idesc = idesc_f16_f32(256, TN);
      const uint64_t b0 = sdesc_kmajor_sw128(smem_u32(sB));
      int unit = 0, block = 0, buf = 0;
      uint32_t aphase = 0, bphase = 0, tphase = 0;
      for (long long j = 0; j < mine; ++j) {
        for (int kb = 0, in_chunk = 0; kb < p.num_kb; ++kb) {
          const bool first = in_chunk == 0, last = ++in_chunk == kChunkBlocks || kb == p.num_kb - 1;
          const uint32_t d = tmem_base + Cfg::kDCol + buf * TN;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // the barriers are asked at once, before any is waited for
            bool ready = mbar_test_wait_cluster(&afull[unit], aphase);
            if (h == 0) {
              ready = mbar_test_wait_cluster(&bfull[block], bphase) & ready;
              if (first) ready = mbar_test_wait(&tempty[buf], tphase ^ 1) & ready;
            }
            if (!ready) {
              if (!mbar_wait_cluster(&afull[unit], aphase, abort_flag, p.status)) goto teardown;
              if (h == 0 && !mbar_wait_cluster(&bfull[block], bphase, abort_flag, p.status)) goto teardown;
              if (h == 0 && first && !mbar_wait(&tempty[buf], tphase ^ 1, abort_flag, p.status)) goto teardown;
            }
            tc_fence_after();
            const uint32_t a = tmem_base + unit * kUnitCols;
            const uint64_t b = b0 + (2 * block + h) * (Cfg::kBBytes >> 4);
            if (issue) {
#pragma unroll
              for (int s = 0; s < kUnit / 16; ++s)   // 16 values: 8 columns of A, 32 bytes of B
                tc_mma_f16_ts_pair(d, a + 8 * s, b + 2 * s, idesc, !first || h > 0 || s > 0);
              tc_commit_pair(&aempty[unit], 3);
              if (h == 1) tc_commit_pair(&bempty[block], 3);
              if (h == 1 && last) tc_commit_pair(&tfull[buf], 3);
            }
            __syncwarp();
            if (++unit == kAUnits) {
              unit = 0;
              aphase ^= 1;
            }
          }
          if (++block == kBBlocks) {
            block = 0;
            bphase ^= 1;
          }
          if (last) {
            in_chunk = 0;
            buf ^= 1;
            if (buf == 0) tphase ^= 1;
          }
        }
      }
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsW));
    const int quad = warp & 3, id = threadIdx.x & 127, h = (warp - 4) >> 2;   // this thread's weight row; its unit of a stage
    const uint32_t to0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    int stage = 0, unit = h;
    uint32_t phase = 0, uphase = 0;
    for (long long k = 0; k < blocks; ++k) {
      if (!mbar_wait(&full[stage], phase, abort_flag, p.status)) goto teardown;
      const uint8_t* w = sW + stage * Cfg::kWBytes + id * kKBlockBytes;
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint4*>(w + (((id & 7) ^ j ^ (4 * h)) << 4));
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      const bool room = mbar_test_wait(&aempty[unit], uphase ^ 1);   // (asked before the arithmetic)
      uint32_t f[2][16];
#pragma unroll
      for (int j = 0; j < 4; ++j) f16_of_int8_16(v[j], &f[j >> 1][8 * (j & 1)]);
      if (!room && !mbar_wait(&aempty[unit], uphase ^ 1, abort_flag, p.status)) goto teardown;
      tc_fence_after();
      tmem_st_32x32b_x16(to0 + unit * kUnitCols, f[0]);
      tmem_st_32x32b_x16(to0 + unit * kUnitCols + 16, f[1]);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote_cta(map_to_rank(smem_u32(&afull[unit]), 0));
      if ((unit += 2) >= kAUnits) {
        unit = h;
        uphase ^= 1;
      }
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
  } else if (warp < 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsX));
    // 16 bytes at a time: thread id's are those of row (id + 128 i) % 96, and j = (id + 128 i) / 96 of a unit's four
    constexpr int kPer = Cfg::kXRows * 4 / 128;
    const int id = threadIdx.x & 127;
    int stage = 0, block = 0;
    uint32_t phase = 0, bphase = 0;
    for (long long k = 0; k < blocks; ++k) {
      if (!mbar_wait(&full[stage], phase, abort_flag, p.status)) goto teardown;
      const bool room = mbar_test_wait(&bempty[block], bphase ^ 1);
      const uint8_t* x = sX + stage * Cfg::kXBytes;
      uint8_t* b = sB + 2 * block * Cfg::kBBytes;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 v[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int row = (id + 128 * i) % Cfg::kXRows, j = (id + 128 * i) / Cfg::kXRows;
          v[i] = *reinterpret_cast<const uint4*>(x + row * kKBlockBytes + (((row & 7) ^ j ^ (4 * h)) << 4));
        }
        if (h == 0 && !room && !mbar_wait(&bempty[block], bphase ^ 1, abort_flag, p.status)) goto teardown;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int row = (id + 128 * i) % Cfg::kXRows, j = (id + 128 * i) / Cfg::kXRows;
          uint32_t o[8];
          f16_of_int8_16(v[i], o);
          uint8_t* to = b + h * Cfg::kBBytes + row * 128;
          *reinterpret_cast<uint4*>(to + (((2 * j) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(to + (((2 * j + 1) ^ (row & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
      fence_proxy_async_smem();   // what was stored to shared memory is the MMA's to read
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_remote_cta(map_to_rank(smem_u32(&bfull[block]), 0));
        mbar_arrive(&empty[stage]);
      }
      if (++block == kBBlocks) {
        block = 0;
        bphase ^= 1;
      }
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsEpi));
    const int quad = warp & 3;
    const int c0 = (warp - 16) / 4 * kCols;   // this thread's columns
    const uint32_t from0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + Cfg::kDCol + c0;
    int buf = 0;
    uint32_t tphase = 0;
    for (long long t = t0; t < tiles; t += tstep) {
      const LinearTile q = tile_at<TN, kManyCols>(p, prefix, t);
      const int n = q.n0 + rank * 128 + quad * 32 + lane;   // this thread's weight row
      int acc[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[c] = 0;
#pragma unroll 1
      for (int kb = 0; kb < p.num_kb; kb += kChunkBlocks) {
        if (!mbar_wait(&tfull[buf], tphase, abort_flag, p.status)) goto teardown;
        tc_fence_after();
        int8_add_columns(acc, from0 + buf * TN);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote_relaxed(map_to_rank(smem_u32(&tempty[buf]), 0));
        buf ^= 1;
        if (buf == 0) tphase ^= 1;
      }
      const long long en = static_cast<long long>(q.e) * p.N + n;
      const Int8Finish finish{n < p.N ? p.w_scale[en] : 0.f, p.bias && n < p.N ? p.bias[en] : 0.f, p.lo, p.hi};
      float held[kCols / 32];   // scales of the columns' rows, a lane's for its warp
#pragma unroll
      for (int i = 0; i < kCols / 32; ++i) {
        const int c = c0 + 32 * i + lane;
        held[i] = c < q.rows ? p.x_scale[(q.row0 + c) * p.xs_row] : 0.f;
      }
      int8_put_columns(p, finish, acc, held, q.row0 + c0, q.rows - c0, n);
    }
  }

teardown:
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {
    // a wait ran out: give copies and MMAs already in flight time to land before TMEM is freed
    for (int i = 0; i < 2000; ++i) __nanosleep(100000);
  }
  __syncthreads();
  cluster_sync();   // no CTA of the pair leaves while the other may still signal it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

}  // namespace

cudaError_t launch_linear_int8_many(const LinearParams& p, const LinearPlan& plan, const CUtensorMap& tmW, const CUtensorMap& tmX,
                                    cudaStream_t stream) {
  using Cfg = Int8ManyCfg;
  static OncePerDevice once;
  const cudaError_t e = once([] {
    // the register split waits for ever if the kernel was given fewer registers than it shares out
    cudaFuncAttributes at;
    const cudaError_t got = cudaFuncGetAttributes(&at, linear_int8_many_kernel);
    if (got != cudaSuccess) return got;
    if (at.numRegs < Cfg::kRegs) return cudaErrorInvalidKernelImage;
    return cudaFuncSetAttribute(linear_int8_many_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(linear_int8_many_kernel, dim3(plan.grid), dim3(Cfg::kThreads), Cfg::kSmem, stream, 2, p, tmW, tmX);
}

}  // namespace convf
