// Linear layers on int8 operands for many rows per weight matrix: y = x W^T with integer sums, on tcgen05 (see
// linear_int8_dev.cuh), in tiles of 256 rows of x x 192 weight rows on CTA pairs.
//
// Here the rows of x are the MMA's first operand, in TMEM, so that a thread of the epilogue holds one row of y and
// writes 16 bytes at a time (with the weights there it held a column, and its 2-byte stores took the load/store
// units, which the conversion needs, 4 us a tile).
//
// A unit, 64 values, takes the tensor cores 384 cycles; meanwhile each CTA of a pair has to convert 128 rows of x
// and 96 weight rows of it (a single CTA's 128 x 192 tile: 128 and 192), 84 integer instructions at half rate for
// each of four warps.  What a unit goes through is long (its bytes' arrival, the conversion, the pair's barrier, the
// MMAs, their end seen in both CTAs), and TMEM holds only four units of x beside two accumulators of 192 columns: so
// x is converted ahead, in registers, and waits for a place for its stores only, and weights have warps of their own.
// A unit's weights go to shared memory with as many places, and one barrier each way serves both operands.
//
// Bound by the MMAs: 8192 x 8192 x 8192 606 to 613 us, 1.81 PFLOP/s, 94% of the library's measured bf16 burst (fp16 operands of
// as many values, ready, would take 570; small values, which take less power, 584 us); 4096 x 4096 x 4096 86 us (tensor pipe
// 74% of the cycles, ALU pipe 53%).
//
// A pair's MMAs are issued by one of its CTAs, the leader, and read what both have converted.  The other CTA's converting
// warps hand over within their own CTA, and a thread of it passes that on to the leader at cluster scope, where it is
// ordered for a thread of another CTA, by a fence for what is in shared memory (8192 x 8192 x 8192 622 us; by an arrival that
// releases all memory, which also waits for the results on their way out, 905; by such fences of the converting warps
// themselves 634).
//
//   warps 0, 1    TMA: weight and x tiles of 128 values; TMEM and MMA issue (the leader's)
//   warp 2        works out the CTA's next tiles
//   warps 1, 3    of the other CTA: each passes on one unit of every stage
//   warps 4-11    int8 -> fp16 of x: two groups of four warps, each a unit of every stage
//   warps 12-19   int8 -> fp16 of the weights, in two groups as well
//   warps 20-27   epilogue: warp w the rows 32 (w % 4) .. and half of the columns
#include <type_traits>

#include "linear_int8_dev.cuh"

namespace convf {

namespace {

constexpr int TN = kInt8PairCols;   // an MMA's columns: weight rows
constexpr int kTileBatch = 16;      // tiles that the scheduler works out at a time

struct Int8ManyCfg {
  static constexpr int kWRows = TN / 2;              // weight rows that a CTA loads and converts
  static constexpr int kCols = TN / 2;               // columns per epilogue thread
  static constexpr int kThreads = 896;
  static constexpr int kXBytes = 128 * kKBlockBytes, kWBytes = kWRows * kKBlockBytes;   // of a stage, int8
  static constexpr int kBBytes = kWRows * 2 * kUnit; // of a unit of weights, fp16
  static constexpr int kStages = 4, kUnits = 4;   // places: int8 stages, units
  static constexpr int kDCol = kUnits * kUnitCols;  // the accumulators' first column
  // per epilogue warp: three chunks of 32 rows of 64 bytes on their way out, its columns' scales and biases
  static constexpr int kOutBytes = 3 * 2048, kTableBytes = 2 * kCols * 4;
  static constexpr int kBarBytes = 256;
  static constexpr int kSmem = kStages * (kXBytes + kWBytes) + kUnits * kBBytes + 8 * (kOutBytes + kTableBytes) + kBarBytes + 2 * kTileBatch * 16 + kScheduleBytes;
  // registers: 72 per thread at launch; the epilogue's two warpgroups take what the others give up
  static constexpr int kRegs = 72, kRegsEpi = 128, kRegsX = 56, kRegsW = 48, kRegsOther = 40;
  static_assert(256 * (kRegsEpi + kRegsX + kRegsW) + 128 * kRegsOther <= kThreads * kRegs, "register split");
  static_assert((2 * kStages + 3 * kUnits + 8) * 8 + 8 <= kBarBytes && kSmem <= 232448, "shared memory");
  static_assert(kDCol + 2 * TN <= 512, "TMEM columns");
  static_assert(kUnits % 2 == 0, "each unit of a stage has places of its own");
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__global__ void __launch_bounds__(Int8ManyCfg::kThreads, 1)
    linear_int8_many_kernel(const LinearParams p, const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                            const __grid_constant__ CUtensorMap tmY) {
  using Cfg = Int8ManyCfg;
  constexpr int kStages = Cfg::kStages, kUnits = Cfg::kUnits, kCols = Cfg::kCols;
  constexpr int kChunkBlocks = kInt8Chunk / kKBlockBytes;
  extern __shared__ __align__(1024) uint8_t sX[];   // (the swizzle goes by address bits 7 to 9)
  uint8_t* sW = sX + kStages * Cfg::kXBytes;
  uint8_t* sB = sW + kStages * Cfg::kWBytes;
  uint8_t* sOut = sB + kUnits * Cfg::kBBytes;
  float* sTable = reinterpret_cast<float*>(sOut + 8 * Cfg::kOutBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(sOut + 8 * (Cfg::kOutBytes + Cfg::kTableBytes));   // int8 tiles are here
  uint64_t* empty = full + kStages;     // and have been read
  uint64_t* cfull = empty + kStages;    // a unit of x is in TMEM and one of weights in sB, of both CTAs (the leader's)
  uint64_t* cpeer = cfull + kUnits;     // of the other CTA (its own)
  uint64_t* cempty = cpeer + kUnits;    // and its MMAs have read them
  uint64_t* tfull = cempty + kUnits;    // an accumulator holds a chunk's sums
  uint64_t* tempty = tfull + 2;         // and has been read, in both CTAs (the leader's)
  uint64_t* tqfull = tempty + 2;        // a batch of tiles is worked out
  uint64_t* tqempty = tqfull + 2;       // and read by the loads' warp and the epilogue's
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tqempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  LinearTile* tileq = reinterpret_cast<LinearTile*>(reinterpret_cast<uint8_t*>(full) + Cfg::kBarBytes);
  int* prefix = reinterpret_cast<int*>(tileq + 2 * kTileBatch);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 16);
    }
    for (int u = 0; u < kUnits; ++u) {
      mbar_init(&cfull[u], 9);   // the leader's converting warps, and the other CTA's
      mbar_init(&cpeer[u], 8);
      mbar_init(&cempty[u], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 16);
      mbar_init(&tqfull[b], 1);
      mbar_init(&tqempty[b], 9);
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
  if (warp == 2) build_schedule(p, kInt8PairRows, prefix, blockIdx.x == 0);
  __syncthreads();

  const long long tiles = tile_count(p, prefix);
  const long long t0 = blockIdx.x >> 1, tstep = gridDim.x >> 1;
  const long long mine = tiles > t0 ? (tiles - t0 - 1) / tstep + 1 : 0;   // tiles of this pair
  // and their stages (operands that fit the device's memory give less than 2^26; 64 bits cost the converting loops
  // registers that they have not: 88.6 instead of 84.6 us for 4096^3)
  const int blocks = static_cast<int>(mine * p.num_kb);
  uint64_t* const converted = rank == 0 ? cfull : cpeer;   // where this CTA's converting warps arrive
  // this CTA's j-th tile, read by one thread (the loads') or a warp in the order of j; false: give up
  auto next_tile = [&](long long j, LinearTile& q, bool whole) {
    const int slot = static_cast<int>(j / kTileBatch) & 1, at = static_cast<int>(j % kTileBatch);
    if (at == 0) {
      const bool there = mbar_wait(&tqfull[slot], static_cast<uint32_t>(j / (2 * kTileBatch)) & 1, abort_flag, p.status);
      if (whole ? !whole_warp(there) : !there) return false;
    }
    q = tileq[slot * kTileBatch + at];
    if (at == kTileBatch - 1) {
      if (whole) __syncwarp();
      if (!whole || lane == 0) mbar_arrive(&tqempty[slot]);
    }
    return true;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsOther));
    if (warp == 0) {
      if (lane == 0) {
        int stage = 0;
        uint32_t phase = 0;
        for (long long j = 0; j < mine; ++j) {
          LinearTile q;
          if (!next_tile(j, q, false)) goto teardown;
          for (int kb = 0; kb < p.num_kb; ++kb) {
            if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, p.status)) goto teardown;
            mbar_arrive_expect_tx(&full[stage], Cfg::kWBytes + Cfg::kXBytes);
            tma_load_3d(sW + stage * Cfg::kWBytes, &tmW, &full[stage], kb * kKBlockBytes, q.n0 + rank * Cfg::kWRows, q.e);
            tma_load_2d(sX + stage * Cfg::kXBytes, &tmX, &full[stage], kb * kKBlockBytes, q.row0 + rank * 128);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
      }
    } else if (warp == 2) {
      for (long long j = 0; j < mine; j += kTileBatch) {
        const int slot = static_cast<int>(j / kTileBatch) & 1;
        if (!whole_warp(mbar_wait(&tqempty[slot], (static_cast<uint32_t>(j / (2 * kTileBatch)) & 1) ^ 1, abort_flag, p.status))) goto teardown;
        if (lane < kTileBatch && j + lane < mine)
          tileq[slot * kTileBatch + lane] = tile_at<kInt8PairRows, TN>(p, prefix, t0 + (j + lane) * tstep);
        __syncwarp();
        if (lane == 0) mbar_arrive(&tqfull[slot]);
      }
    } else if (rank != 0) {
      if (lane == 0) {
        const uint32_t cfull0 = map_to_rank(smem_u32(cfull), 0);
        const int h = warp >> 1;   // its unit of a stage
        int unit = h;
        uint32_t phase = 0;
        for (int k = 0; k < blocks; ++k) {
          if (!mbar_wait(&cpeer[unit], phase, abort_flag, p.status)) goto teardown;
          tc_fence_after();   // (what was stored to TMEM is ordered by this thread's barriers too)
          tc_fence_before();
          mbar_arrive_remote_shared(cfull0 + 8 * unit);
          if ((unit += 2) >= kUnits) {
            unit = h;
            phase ^= 1;
          }
        }
      }
    } else if (warp == 1) {
      // the whole warp walks the loop and one lane issues: the loop's state then stays in uniform
      // registers, which is where the MMA takes its descriptors from
      const bool issue = elect_one();
      constexpr uint32_t idesc = idesc_f16_f32(kInt8PairRows, TN);
      const uint64_t b0 = sdesc_kmajor_sw128(smem_u32(sB));
      int unit = 0, buf = 0;
      uint32_t phase = 0, tphase = 0;
      for (long long j = 0; j < mine; ++j) {
        for (int kb = 0, in_chunk = 0; kb < p.num_kb; ++kb) {
          const bool first = in_chunk == 0, last = ++in_chunk == kChunkBlocks || kb == p.num_kb - 1;
          const uint32_t d = tmem_base + Cfg::kDCol + buf * TN;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // both barriers are asked at once, before either is waited for
            bool ready = mbar_test_wait_cluster(&cfull[unit], phase);
            if (h == 0 && first) ready = mbar_test_wait(&tempty[buf], tphase ^ 1) & ready;
            if (!ready) ready = mbar_wait_cluster(&cfull[unit], phase, abort_flag, p.status) &&
                                (h > 0 || !first || mbar_wait(&tempty[buf], tphase ^ 1, abort_flag, p.status));
            if (!whole_warp(ready)) goto teardown;
            tc_fence_after();
            const uint32_t a = tmem_base + unit * kUnitCols;
            const uint64_t b = b0 + unit * (Cfg::kBBytes >> 4);
            if (issue) {
#pragma unroll
              for (int s = 0; s < kUnit / 16; ++s)   // 16 values: 8 columns of A, 32 bytes of B
                tc_mma_f16_ts_pair(d, a + 8 * s, b + 2 * s, idesc, !first || h > 0 || s > 0);
              tc_commit_pair(&cempty[unit], 3);
              if (h == 1 && last) tc_commit_pair(&tfull[buf], 3);
            }
            __syncwarp();
            if (++unit == kUnits) {
              unit = 0;
              phase ^= 1;
            }
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
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsX));
    const int quad = warp & 3, id = threadIdx.x & 127, h = (warp - 4) >> 2;   // this thread's row; its unit of a stage
    const uint32_t to0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    const uint8_t* from[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) from[j] = sX + id * kKBlockBytes + (((id & 7) ^ j ^ (4 * h)) << 4);
    int stage = 0, unit = h;
    uint32_t phase = 0, uphase = 0;
    bool here = false;
#pragma unroll 1
    for (int k = 0; k < blocks; ++k) {
      const bool there = here || mbar_wait(&full[stage], phase, abort_flag, p.status);   // (one vote on both waits, below)
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint4*>(from[j] + stage * Cfg::kXBytes);
      const bool room = mbar_test_wait(&cempty[unit], uphase ^ 1);   // (asked before the arithmetic: an answer takes 100 cycles)
      uint32_t f[2][16];
#pragma unroll
      for (int j = 0; j < 4; ++j) f16_of_int8_16(v[j], &f[j >> 1][8 * (j & 1)]);
      if (!whole_warp(there && (room || mbar_wait(&cempty[unit], uphase ^ 1, abort_flag, p.status)))) goto teardown;
      tc_fence_after();
      tmem_st_32x32b_x16(to0 + unit * kUnitCols, f[0]);
      tmem_st_32x32b_x16(to0 + unit * kUnitCols + 16, f[1]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);   // (its bytes have been used by now, not only asked for)
      __syncwarp();
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
      here = mbar_test_wait(&full[stage], phase);   // of the next stage
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&converted[unit]);
      if ((unit += 2) >= kUnits) {
        unit = h;
        uphase ^= 1;
      }
    }
  } else if (warp < 20) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsW));
    // 16 bytes at a time: thread id's are those of row (id + 128 i) % 96, and j = (id + 128 i) / 96 of a unit's four
    constexpr int kPer = Cfg::kWRows * 4 / 128;
    const int id = threadIdx.x & 127, h = (warp - 12) >> 2;   // its unit of a stage
    const uint8_t* from[kPer];
    uint8_t* to[kPer];   // the first half of the 16; the other is at 16 bytes before or behind it
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int row = (id + 128 * i) % Cfg::kWRows, j = (id + 128 * i) / Cfg::kWRows;
      from[i] = sW + row * kKBlockBytes + (((row & 7) ^ j ^ (4 * h)) << 4);
      to[i] = sB + row * 128 + (((row & 7) ^ (2 * j)) << 4);
    }
    const int other = (id & 1) ? -16 : 16;   // (rows of a thread are all odd or all even)
    int stage = 0, unit = h;
    uint32_t phase = 0, uphase = 0;
    bool here = false;
#pragma unroll 2   // (593 -> 580 us for 8192^3; x's loop too, or either more often: slower, by the instruction caches)
    for (int k = 0; k < blocks; ++k) {
      const bool there = here || mbar_wait(&full[stage], phase, abort_flag, p.status);
      uint4 v[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = *reinterpret_cast<const uint4*>(from[i] + stage * Cfg::kWBytes);
      const bool room = mbar_test_wait(&cempty[unit], uphase ^ 1);
      // (no access of the whole warp follows: the vote is taken once the unit has been handed over; both waits' votes in
      // front of them 8 us more)
      const bool go = there && (room || mbar_wait(&cempty[unit], uphase ^ 1, abort_flag, p.status));
      const int at = unit * Cfg::kBBytes;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        uint32_t o[8];
        f16_of_int8_16(v[i], o);
        *reinterpret_cast<uint4*>(to[i] + at) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(to[i] + at + other) = make_uint4(o[4], o[5], o[6], o[7]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
      here = mbar_test_wait(&full[stage], phase);   // of the next stage
      fence_proxy_async_smem();   // what was stored to shared memory is the MMA's to read
      __syncwarp();
      if (lane == 0 && go) mbar_arrive(&converted[unit]);
      if (!whole_warp(go)) goto teardown;
      if ((unit += 2) >= kUnits) {
        unit = h;
        uphase ^= 1;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsEpi));
    const int quad = warp & 3, half = (warp - 20) >> 2;
    const int mrow = rank * 128 + quad * 32;   // this warp's first row of the tile
    const uint32_t from0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + Cfg::kDCol + half * kCols;
    uint8_t* out = sOut + (warp - 20) * Cfg::kOutBytes;
    float* table = sTable + (warp - 20) * (Cfg::kTableBytes / 4);   // scales, then biases
    int buf = 0;
    uint32_t tphase = 0;
    for (long long j = 0; j < mine; ++j) {
      LinearTile q;
      if (!next_tile(j, q, true)) goto teardown;
      const int n0 = q.n0 + half * kCols;   // this warp's first column
      const long long row0 = q.row0 + mrow;
      const float xs = p.x_scale[(q.row0 + min(mrow + lane, q.rows - 1)) * p.xs_row];
#pragma unroll
      for (int i = 0; i < kCols / 32; ++i) {
        const int n = n0 + 32 * i + lane;
        const long long en = static_cast<long long>(q.e) * p.N + n;
        table[32 * i + lane] = n < p.N ? p.w_scale[en] : 0.f;
        table[kCols + 32 * i + lane] = p.bias && n < p.N ? p.bias[en] : 0.f;
      }
      __syncwarp();
      int acc[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[c] = 0;
#pragma unroll 1
      for (int kb = 0; kb < p.num_kb; kb += kChunkBlocks) {
        if (!whole_warp(mbar_wait(&tfull[buf], tphase, abort_flag, p.status))) goto teardown;
        tc_fence_after();
        int8_add_columns(acc, from0 + buf * TN);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote_relaxed(map_to_rank(smem_u32(&tempty[buf]), 0));
        buf ^= 1;
        if (buf == 0) tphase ^= 1;
      }
      if (mrow < q.rows && n0 < p.N) {
        // Three chunks of 64 bytes of each row at a time (all bf16 columns, half of the fp32 ones) through shared memory,
        // 16-byte units swizzled by row: whole warps' rows leave by TMA, a group's last rows by such units, unaligned or
        // ragged ones by the elements, lanes side by side.  (A TMA store clips the columns past N by units of 16 bytes
        // and would write over what follows rows that end inside one.)
        auto send = [&](auto bf16) {
          constexpr bool BF16 = decltype(bf16)::value;
          constexpr int kEach = BF16 ? 32 : 16;   // columns of a chunk
          const bool whole = p.vec_y && mrow + 32 <= q.rows;
#pragma unroll
          for (int c0 = 0; c0 < kCols; c0 += 3 * kEach) {
            if (lane < 3) bulk_wait_read<0>();   // the stores from these places
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 12; ++i) {   // unit i % 4 of chunk i / 4
              constexpr int kOf = kEach / 4;
              float v[kOf];
#pragma unroll
              for (int k = 0; k < kOf; k += 4) {
                const int at = c0 + i * kOf + k;
                const float4 s = *reinterpret_cast<const float4*>(table + at);
                v[k] = __fmul_rn(__int2float_rn(acc[at]), __fmul_rn(xs, s.x));
                v[k + 1] = __fmul_rn(__int2float_rn(acc[at + 1]), __fmul_rn(xs, s.y));
                v[k + 2] = __fmul_rn(__int2float_rn(acc[at + 2]), __fmul_rn(xs, s.z));
                v[k + 3] = __fmul_rn(__int2float_rn(acc[at + 3]), __fmul_rn(xs, s.w));
                if (p.bias) {
                  const float4 b = *reinterpret_cast<const float4*>(table + kCols + at);
                  v[k] = __fadd_rn(v[k], b.x);
                  v[k + 1] = __fadd_rn(v[k + 1], b.y);
                  v[k + 2] = __fadd_rn(v[k + 2], b.z);
                  v[k + 3] = __fadd_rn(v[k + 3], b.w);
                }
              }
              if (p.clamp) {
#pragma unroll
                for (int k = 0; k < kOf; ++k) v[k] = act_clamp(v[k], p.lo, p.hi);
              }
              uint4 w;
              if constexpr (BF16)
                w = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
              else
                w = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
              *reinterpret_cast<uint4*>(out + (i >> 2) * 2048 + lane * 64 + (((i & 3) ^ ((lane >> 1) & 3)) << 4)) = w;
            }
            if (whole) fence_proxy_async_smem();
            __syncwarp();
            if (whole && lane < 3) {   // a chunk each
              const int n = n0 + c0 + lane * kEach;
              if (n < p.N && (p.whole_units || n + kEach <= p.N)) tma_store_2d(&tmY, out + lane * 2048, n, static_cast<int>(row0));
              bulk_commit();
            }
#pragma unroll 1
            for (int i = 0; i < 3; ++i) {
              const int n = n0 + c0 + i * kEach;
              const bool units = p.vec_y && (p.whole_units || n + kEach <= p.N);   // the rows' 16-byte units are whole
              if ((whole && units) || n >= p.N) continue;
              const uint8_t* chunk = out + i * 2048;
              const int rows = min(32, q.rows - mrow);
              if (units) {
                const int u = lane & 3;
                for (int r = lane >> 2; r < rows; r += 8)
                  if (n + u * (kEach / 4) < p.N && CONVF_IN_BOUNDS(row0 + r < p.rows, p.status))
                    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.y) + ((row0 + r) * p.ldy + n) * (64 / kEach) + u * 16) =
                        *reinterpret_cast<const uint4*>(chunk + r * 64 + ((u ^ ((r >> 1) & 3)) << 4));
              } else {
                constexpr int kRows = 32 / kEach;   // rows at a time
                const int col = lane % kEach;
                for (int r = lane / kEach; r < rows; r += kRows) {
                  if (n + col < p.N && CONVF_IN_BOUNDS(row0 + r < p.rows, p.status)) {
                    const long long at = (row0 + r) * p.ldy + n + col;
                    const uint8_t* from = chunk + r * 64 + (((col * 64 / kEach >> 4) ^ ((r >> 1) & 3)) << 4) + col * (64 / kEach) % 16;
                    if constexpr (BF16)
                      static_cast<uint16_t*>(p.y)[at] = *reinterpret_cast<const uint16_t*>(from);
                    else
                      static_cast<uint32_t*>(p.y)[at] = *reinterpret_cast<const uint32_t*>(from);
                  }
                }
              }
            }
          }
        };
        if (p.out_bf16)
          send(std::true_type{});
        else
          send(std::false_type{});
      }
      __syncwarp();   // the table has been read
    }
    if (lane < 3) bulk_wait_all();   // the stores have been written before the CTA ends
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
                                    const CUtensorMap& tmY, cudaStream_t stream) {
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
  return launch_pdl(linear_int8_many_kernel, dim3(plan.grid), dim3(Cfg::kThreads), Cfg::kSmem, stream, 2, p, tmW, tmX, tmY);
}

}  // namespace convf
