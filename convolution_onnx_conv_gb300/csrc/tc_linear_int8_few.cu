// Linear layers on int8 operands for few rows per weight matrix: y^T = W x^T with integer sums, on tcgen05 (see
// linear_int8_dev.cuh).  16 or 64 rows of x are a tile's columns, and the CTAs of a cluster share a tile's
// reduction where there are fewer tiles than SMs, as in tc_linear_few.cu; their partial sums are integers too.
//
// For tens of rows, and for experts with a few each (fewer: linear_int8_direct.cu).  A launch takes 3.5 us, a k-block 285 to
// 500 ns (its bytes' arrival, the conversion of 128 weight rows, the MMAs; of these the bytes take 100), a tile's start and
// end 0.2 to 1.3 us and, where the reduction is shared, with the exchange 3 to 7: these are what bounds small layers, not
// the k-blocks (64 x 4096 x 4096, shared by 4, has 8 of them a CTA, 2.3 us of 15.2).  64 x 8192 x 8192 26.4 us (tensor
// pipe 12%, logic pipe 33%); 96 x 8192 x 2048 12.0; 1001 x 1000 x 2048 11.7; 128 rows over 24 experts of 2048 x 2048 25
// (floor 14.9).  A group of converting warps takes every other stage whole: its barriers' answers and its stores' ways then
// come once for two units (a unit of every stage each: 27.8, 12.6 and 12.3 us).
//
//   warp 0        TMA: weight and x tiles of 128 values
//   warp 1        TMEM, MMA issue
//   warps 2, 3    int8 -> fp16 of x (64 columns: warps 4-11)
//   8 warps       int8 -> fp16 of the weights: two groups of four warps, each every other stage
//   the last      epilogue: 4 warps, or 8 that take half of the columns each
#include "linear_int8_dev.cuh"

namespace convf {

namespace {

template <int TN>
struct Int8Cfg {
  // 16 columns: two CTAs on an SM, so that one's start, exchange and end are behind the other's loads (and a
  // dependent launch's start behind this one's end)
  static constexpr int kPerSm = TN == 16 ? 2 : 1;
  static constexpr int kXWarps = TN == 16 ? 2 : 8, kXFirst = TN == 16 ? 2 : 4;   // that convert x, and the first of them
  static constexpr int kWFirst = TN == 16 ? 4 : 12, kEpiFirst = kWFirst + 8;
  static constexpr int kEpiWarps = TN == 16 ? 4 : 8;
  static constexpr int kCols = TN == 16 ? TN : TN / 2;          // columns per epilogue thread
  static constexpr int kThreads = 32 * (kEpiFirst + kEpiWarps);
  static constexpr int kTmemCols = kPerSm == 2 ? 256 : 512;
  static constexpr int kWBytes = 128 * kKBlockBytes, kXBytes = TN * kKBlockBytes;   // of a stage, int8
  static constexpr int kBBytes = TN * 2 * kUnit;                // of a unit of x, fp16
  static constexpr int kBlocks = kPerSm == 2 ? 3 : 5;   // places of converted stages
  static constexpr int kDCol = 2 * kBlocks * kUnitCols;            // the accumulators' first column
  static constexpr int kRedBytes = TN * 128 * 4;                // partial sums of this CTA's columns, by rank
  static constexpr int kBarBytes = 512;
  static constexpr int kFixed = 1024 + 2 * kBlocks * kBBytes + kRedBytes + kScheduleBytes + kBarBytes;
  static constexpr int kBudget = kPerSm == 2 ? 115712 : 232448;
  static constexpr int kStages = (kBudget - kFixed) / (kWBytes + kXBytes);
  static constexpr int kSmem = kFixed + kStages * (kWBytes + kXBytes);
  static_assert(kStages >= 3 && (2 * kStages + 2 * kBlocks + 6) * 8 + 8 <= kBarBytes && kSmem <= kBudget, "shared memory");
  // A group of converting warps sees every phase of its places' barriers, one after another: loads may land out of order,
  // and a wait by parity that skipped a phase would take the one before it for its own.  Places of converted stages may
  // change between the groups, since MMAs end in order: a group at stage k has seen the end of stage k - 2 - kBlocks (its last
  // one's place), and so of k - 2 kBlocks, the phase that its wait for the end of k - kBlocks could be taken in by.
  static_assert(kStages % 2 == 0, "a place for int8 tiles belongs to one group");
  static_assert(kBlocks >= 2, "the phase before the one waited for has ended");
  static_assert(kDCol + 2 * TN <= kTmemCols, "TMEM columns");
};

template <int TN>
__global__ void __launch_bounds__(Int8Cfg<TN>::kThreads, Int8Cfg<TN>::kPerSm)
    linear_int8_few_kernel(const LinearParams p, const int split, const __grid_constant__ CUtensorMap tmW,
                       const __grid_constant__ CUtensorMap tmX) {
  using Cfg = Int8Cfg<TN>;
  constexpr int kStages = Cfg::kStages, kBlocks = Cfg::kBlocks, kCols = Cfg::kCols;
  constexpr int kChunkBlocks = kInt8Chunk / kKBlockBytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sW = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sX = sW + kStages * Cfg::kWBytes;
  uint8_t* sB = sX + kStages * Cfg::kXBytes;
  int* red = reinterpret_cast<int*>(sB + 2 * kBlocks * Cfg::kBBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(red) + Cfg::kRedBytes);   // int8 tiles are here
  uint64_t* empty = full + kStages;     // and have been read
  uint64_t* cfull = empty + kStages;    // a stage is converted: weights in TMEM, x in sB
  uint64_t* cempty = cfull + kBlocks;   // and its MMAs have read it
  uint64_t* tfull = cempty + kBlocks;   // an accumulator holds a chunk's sums
  uint64_t* tempty = tfull + 2;         // and has been read
  uint64_t* rfull = tempty + 2;         // every rank's partial sums of this CTA's columns have arrived
  uint64_t* rfree = rfull + 1;          // every rank has read what this CTA sent it
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rfree + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* prefix = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(full) + Cfg::kBarBytes);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4 + Cfg::kXWarps / 2);
    }
    for (int b = 0; b < kBlocks; ++b) {
      mbar_init(&cfull[b], 4 + Cfg::kXWarps / 2);
      mbar_init(&cempty[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], Cfg::kEpiWarps);
    }
    mbar_init(rfull, Cfg::kEpiWarps * split);
    mbar_init(rfree, Cfg::kEpiWarps * split);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, Cfg::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  if (split > 1) cluster_sync();   // the peers' barriers exist before anything is sent to them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const long long t0 = blockIdx.x / split, tstep = gridDim.x / split;
  const int ka = static_cast<int>(static_cast<long long>(p.num_kb) * rank / split);
  const int kb_end = static_cast<int>(static_cast<long long>(p.num_kb) * (rank + 1) / split);
  const long long first_tiles = static_cast<long long>((p.rows + TN - 1) / TN) * p.n_tiles;
  constexpr int kPrefetch = 16;
  // after the TMEM allocation, which a dependent's CTA would otherwise take
  pdl_launch_dependents();
  // one layer: the first wave's weight tiles are known before the previous kernel has ended (see tc_linear_few.cu)
  if (!p.offsets && warp == 0 && lane == 0 && t0 < first_tiles) {
    const int n0 = static_cast<int>(t0 / ((p.rows + TN - 1) / TN)) * 128;
    for (int kb = ka; kb < min(kb_end, ka + kPrefetch); ++kb) tma_prefetch_l2_3d(&tmW, kb * kKBlockBytes, n0, 0);
  }
  pdl_wait_prior();
  if (warp == 2) build_schedule(p, TN, prefix, blockIdx.x == 0);
  __syncthreads();

  const long long tiles = tile_count(p, prefix);
  const long long mine = tiles > t0 ? (tiles - t0 - 1) / tstep + 1 : 0;

  const int blocks = static_cast<int>(mine * (kb_end - ka));   // stages of this CTA (see tc_linear_int8_many.cu)

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (long long t = t0; t < tiles; t += tstep) {
        const LinearTile q = tile_at<TN, 128>(p, prefix, t);
        for (int kb = ka; kb < kb_end; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, p.status)) goto teardown;
          mbar_arrive_expect_tx(&full[stage], Cfg::kWBytes + Cfg::kXBytes);
          tma_load_3d(sW + stage * Cfg::kWBytes, &tmW, &full[stage], kb * kKBlockBytes, q.n0, q.e);
          tma_load_2d(sX + stage * Cfg::kXBytes, &tmX, &full[stage], kb * kKBlockBytes, q.row0);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    }
  } else if (warp == 1) {
    // the whole warp walks the loop and one lane issues: the loop's state then stays in uniform
    // registers, which is where the MMA takes its descriptors from
    const bool issue = elect_one();
    constexpr uint32_t idesc = idesc_f16_f32(128, TN);
    const uint64_t b0 = sdesc_kmajor_sw128(smem_u32(sB));
    int block = 0, buf = 0;
    uint32_t phase = 0, tphase = 0;
    for (long long j = 0; j < mine; ++j) {
      for (int kb = ka, in_chunk = 0; kb < kb_end; ++kb) {
        const bool first = in_chunk == 0, last = ++in_chunk == kChunkBlocks || kb == kb_end - 1;
        // both barriers are asked at once, before either is waited for
        bool ready = mbar_test_wait(&cfull[block], phase);
        if (first) ready = mbar_test_wait(&tempty[buf], tphase ^ 1) & ready;
        if (!ready) ready = mbar_wait(&cfull[block], phase, abort_flag, p.status) &&
                            (!first || mbar_wait(&tempty[buf], tphase ^ 1, abort_flag, p.status));
        if (!whole_warp(ready)) goto teardown;
        tc_fence_after();
        const uint32_t a = tmem_base + 2 * block * kUnitCols, d = tmem_base + Cfg::kDCol + buf * TN;
        const uint64_t b = b0 + 2 * block * (Cfg::kBBytes >> 4);
        if (issue) {
#pragma unroll
          for (int s = 0; s < 2 * kUnit / 16; ++s)   // 16 values: 8 columns of A, 32 bytes of a unit of B
            tc_mma_f16_ts(d, a + 8 * s, b + (s / 4) * (Cfg::kBBytes >> 4) + 2 * (s % 4), idesc, !first || s > 0);
          tc_commit(&cempty[block]);
          if (last) tc_commit(&tfull[buf]);
        }
        __syncwarp();
        if (++block == kBlocks) {
          block = 0;
          phase ^= 1;
        }
        if (last) {
          in_chunk = 0;
          buf ^= 1;
          if (buf == 0) tphase ^= 1;
        }
      }
    }
  } else if (warp >= Cfg::kXFirst && warp < Cfg::kXFirst + Cfg::kXWarps) {
    // 16 bytes at a time: of a stage's TN rows of 8, thread id takes those of row (id + i kX) % TN, 16-byte place
    // (id + i kX) / TN
    constexpr int kX = 16 * Cfg::kXWarps, kPer = TN * 8 / kX, kAtOnce = kPer < 4 ? kPer : 4;
    const int id = (threadIdx.x - 32 * Cfg::kXFirst) % kX, g = (threadIdx.x - 32 * Cfg::kXFirst) / kX;   // group: its stages are g, g + 2, ..
    int stage = g, block = g;
    uint32_t phase = 0, bphase = 0;
    bool here = false;
#pragma unroll 1
    for (int k = g; k < blocks; k += 2) {
      if (!whole_warp(here || mbar_wait(&full[stage], phase, abort_flag, p.status))) goto teardown;
      const bool room = mbar_test_wait(&cempty[block], bphase ^ 1);
      const uint8_t* x = sX + stage * Cfg::kXBytes;
      uint8_t* b = sB + 2 * block * Cfg::kBBytes;
#pragma unroll
      for (int i0 = 0; i0 < kPer; i0 += kAtOnce) {
        uint4 v[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const int task = id + (i0 + i) * kX, row = task % TN, j = task / TN;
          v[i] = *reinterpret_cast<const uint4*>(x + row * kKBlockBytes + ((j ^ (row & 7)) << 4));
        }
        if (i0 == 0 && !whole_warp(room || mbar_wait(&cempty[block], bphase ^ 1, abort_flag, p.status))) goto teardown;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const int task = id + (i0 + i) * kX, row = task % TN, j = task / TN;
          uint32_t o[8];
          f16_of_int8_16(v[i], o);
          uint8_t* to = b + (j >> 2) * Cfg::kBBytes + row * 128;   // unit j / 4, and of its 8 places 2 (j % 4) and the next
          *reinterpret_cast<uint4*>(to + (((2 * (j & 3)) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(to + (((2 * (j & 3) + 1) ^ (row & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
      const int next = stage + 2 >= kStages ? stage + 2 - kStages : stage + 2;
      phase ^= next < stage;
      here = mbar_test_wait(&full[next], phase);
      fence_proxy_async_smem();   // what was stored to shared memory is the MMA's to read
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&cfull[block]);
        mbar_arrive(&empty[stage]);   // (its bytes have been used by now, not only asked for)
      }
      stage = next;
      if ((block += 2) >= kBlocks) {
        block -= kBlocks;
        bphase ^= 1;
      }
    }
  } else if (warp >= Cfg::kWFirst && warp < Cfg::kEpiFirst) {
    const int quad = warp & 3, id = threadIdx.x & 127, g = (warp - Cfg::kWFirst) >> 2;   // this thread's weight row; its group's stages: g, g + 2, ..
    const uint32_t to0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    const uint8_t* from[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) from[j] = sW + id * kKBlockBytes + (((id & 7) ^ j) << 4);
    int stage = g, block = g;
    uint32_t phase = 0, bphase = 0;
    bool here = false;
#pragma unroll 1
    for (int k = g; k < blocks; k += 2) {
      if (!whole_warp(here || mbar_wait(&full[stage], phase, abort_flag, p.status))) goto teardown;
      uint4 v[8];   // (a row's second unit: its places with bit 6 the other way)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = *reinterpret_cast<const uint4*>(sW + ((static_cast<uint32_t>(from[j & 3] - sW) + stage * Cfg::kWBytes) ^ (j & 4 ? 64u : 0u)));
      const bool room = mbar_test_wait(&cempty[block], bphase ^ 1);   // (asked before the arithmetic: an answer takes 100 cycles)
      if (!whole_warp(room || mbar_wait(&cempty[block], bphase ^ 1, abort_flag, p.status))) goto teardown;
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        uint32_t f[16];
        f16_of_int8_16(v[j], f);
        f16_of_int8_16(v[j + 1], f + 8);
        tmem_st_32x32b_x16(to0 + 2 * block * kUnitCols + 8 * j, f);
      }
      const int next = stage + 2 >= kStages ? stage + 2 - kStages : stage + 2;
      phase ^= next < stage;
      here = mbar_test_wait(&full[next], phase);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&cfull[block]);
        mbar_arrive(&empty[stage]);   // (its bytes have been used by now, not only asked for)
      }
      stage = next;
      if ((block += 2) >= kBlocks) {
        block -= kBlocks;
        bphase ^= 1;
      }
    }
  } else if (warp >= Cfg::kEpiFirst) {
    const int quad = warp & 3;
    const int c0 = (warp - Cfg::kEpiFirst) / 4 * kCols;   // this thread's columns
    const uint32_t from0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + Cfg::kDCol + c0;
    int buf = 0;
    uint32_t bphase = 0, rphase = 0;
    constexpr int kHeld = (kCols + 31) / 32;   // row scales that a lane holds for its warp
    for (long long t = t0; t < tiles; t += tstep) {
      const LinearTile q = tile_at<TN, 128>(p, prefix, t);
      const int nrow = quad * 32 + lane;   // this thread's weight row of the CTA's tile
      const int n = q.n0 + nrow;
      const long long en = static_cast<long long>(q.e) * p.N + n;
      const float ws = n < p.N ? p.w_scale[en] : 0.f, bias = p.bias && n < p.N ? p.bias[en] : kNoBias;
      float held[kHeld];
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const int c = (split > 1 ? rank * (TN / split) : c0) + 32 * i + lane;   // (shared tiles: of what this rank finishes)
        held[i] = c < q.rows ? p.x_scale[(q.row0 + c) * p.xs_row] : 0.f;
      }
      int acc[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[c] = 0;
#pragma unroll 1
      for (int kb = ka; kb < kb_end; kb += kChunkBlocks) {
        if (!whole_warp(mbar_wait(&tfull[buf], bphase, abort_flag, p.status))) goto teardown;
        tc_fence_after();
        int8_add_columns(acc, from0 + buf * TN);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&tempty[buf]);
        }
        buf ^= 1;
        if (buf == 0) bphase ^= 1;
      }
      const Int8Finish finish{ws, bias, p.lo, p.hi};
      if (split == 1) {
        int8_put_columns(p, finish, acc, held, q.row0 + c0, q.rows - c0, n);
      } else {
        // column c is finished by rank c / per: send it there, then finish this rank's own
        const int per = TN / split;
        if (!whole_warp(mbar_wait_cluster(rfree, rphase ^ 1, abort_flag, p.status))) goto teardown;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const int col = c0 + c, to = col / per;
          if (col < q.rows)
            st_cluster_f32(map_to_rank(smem_u32(red + (rank * per + col - to * per) * 128 + nrow), to), __int_as_float(acc[c]));
        }
        asm volatile("fence.acq_rel.cluster;" ::: "memory");
        __syncwarp();
        if (lane < split) mbar_arrive_remote(map_to_rank(smem_u32(rfull), lane));
        if (!whole_warp(mbar_wait_cluster(rfull, rphase, abort_flag, p.status))) goto teardown;
        const int own = min(per, q.rows - rank * per);
        for (int j = c0 / kCols; j < own; j += Cfg::kEpiWarps / 4) {
          int sum = 0;
          for (int s = 0; s < split; ++s) sum += red[(s * per + j) * 128 + nrow];
          const float v = finish(sum, __shfl_sync(0xFFFFFFFFu, held[0], j));
          if (n < p.N) int8_put(p, q.row0 + rank * per + j, n, v);
        }
        __syncwarp();
        if (lane < split) mbar_arrive_remote(map_to_rank(smem_u32(rfree), lane));
        rphase ^= 1;
      }
    }
  }

teardown:
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {
    // a wait ran out: give copies and MMAs already in flight time to land before TMEM is freed
    for (int i = 0; i < 2000; ++i) __nanosleep(100000);
  }
  __syncthreads();
  if (split > 1) cluster_sync();   // no CTA leaves while a peer may still write to it or signal it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, Cfg::kTmemCols);
  }
}

template <int TN>
cudaError_t configure() {
  static OncePerDevice once;
  return once([] {
    return cudaFuncSetAttribute(linear_int8_few_kernel<TN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Int8Cfg<TN>::kSmem);
  });
}

template <int TN>
cudaError_t launch_t(const LinearParams& p, const LinearPlan& plan, const CUtensorMap& tmW, const CUtensorMap& tmX,
                     cudaStream_t stream) {
  const cudaError_t e = configure<TN>();
  if (e != cudaSuccess) return e;
  return launch_pdl(linear_int8_few_kernel<TN>, dim3(plan.grid), dim3(Int8Cfg<TN>::kThreads), Int8Cfg<TN>::kSmem,
                    stream, plan.split, p, plan.split, tmW, tmX);
}

template <int TN>
int max_clusters_t(int split, int num_sms) {
  if (split == 1) return num_sms * Int8Cfg<TN>::kPerSm;
  if (configure<TN>() != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(split);
  cfg.blockDim = dim3(Int8Cfg<TN>::kThreads);
  cfg.dynamicSmemBytes = Int8Cfg<TN>::kSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  return cudaOccupancyMaxActiveClusters(&n, linear_int8_few_kernel<TN>, &cfg) == cudaSuccess ? n : 0;
}

}  // namespace

cudaError_t launch_linear_int8_few(const LinearParams& p, const LinearPlan& plan, const CUtensorMap& tmW, const CUtensorMap& tmX,
                               cudaStream_t stream) {
  switch (plan.tile) {
    case 16: return launch_t<16>(p, plan, tmW, tmX, stream);
    case 64: return launch_t<64>(p, plan, tmW, tmX, stream);
  }
  return cudaErrorInvalidValue;
}

int linear_int8_max_clusters(int tile, int split, int num_sms) {
  switch (tile) {
    case 16: return max_clusters_t<16>(split, num_sms);
    case 64: return max_clusters_t<64>(split, num_sms);
  }
  return 0;
}

}  // namespace convf
