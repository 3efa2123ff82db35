// Linear layers for few rows per weight matrix (one token up to some hundred rows, or the ragged
// row groups of experts): y^T = W x^T on tcgen05.
//
// The weights are the MMA's 128-row operand and the rows of x its N columns (16, 32 or 64), so a call
// with one row wastes 15 columns of a narrow MMA instead of 127 rows of a wide one, and a ragged
// group's last tile wastes little.  Such a call is bound by the weights' bytes: each is read once,
// by TMA, many stages ahead.  When there are fewer tiles than SMs, the CTAs of a cluster share one
// tile's reduction (k-blocks r*S/num_kb ..) and add their fp32 partial sums through distributed
// shared memory, each finishing a slice of the tile's columns, in the order of their ranks (so
// results repeat bit for bit).
//
// Measured: 32 rows over 24 of 64 experts of 2048 x 2048 e4m3 weights (101 MB) 21.4 us, 4.7 TB/s; one row
// through 4096 x 4096 e4m3 7.8 us (from a graph; 9 us a call behind another), of which 2.5 us are the bytes at
// 6.8 TB/s and the rest the launch, the first loads' latency, the exchange between 4 CTAs and the end (11.3 us
// without the split).  bf16, 4096 x 4096: one row 10.2 us, 16 rows 12.4, 128 rows 18.2 (the bytes: 4.9).
//
// e4m3: the MMAs of one 128-value k-block go to a TMEM buffer of their own, and the epilogue
// adds buffer * (x_scale * w_scale) to fp32 sums in registers (a lane holds one weight row: the
// weight scale is the same for the whole tile, the row scales differ by column and come from a
// table that a warp fills ahead).  bf16: a buffer sums LinearParams::chunk_kb k-blocks.
//
//   warp 0      TMA: weight and x tiles of each k-block
//   warp 1      TMEM, MMA issue
//   warp 2      e4m3: the scale table
//   warps 4-7   epilogue (4-11 for 64 columns, each half of them)
#include "linear_dev.cuh"

namespace convf {

namespace {

template <bool F8, int TN>
struct FewCfg {
  static constexpr int kEpiWarps = TN >= 64 ? 8 : 4;
  static constexpr int kCols = TN >= 64 ? TN / 2 : TN;    // columns per epilogue thread
  static constexpr int kThreads = 128 + 32 * kEpiWarps;
  static constexpr int kWBytes = 128 * kKBlockBytes, kXBytes = TN * kKBlockBytes;
  static constexpr int kBufs = F8 ? 8 : 2;   // TMEM accumulators (and table slots)
  static constexpr int kTmemCols = kBufs * TN;
  static constexpr int kTableBytes = F8 ? kBufs * TN * 4 : 0;
  static constexpr int kRedBytes = TN * 128 * 4;               // partial sums of this CTA's columns, by rank
  static constexpr int kBarBytes = 512;
  static constexpr int kFixed = 1024 + kTableBytes + kRedBytes + kScheduleBytes + kBarBytes;
  // 16 and 32 columns: two CTAs on an SM, so that one's start, exchange and end are behind the
  // other's loads (and a dependent launch's start behind this one's end)
  static constexpr int kPerSm = TN <= 32 ? 2 : 1;
  static constexpr int kBudget = kPerSm == 2 ? 115712 : 232448;
  static constexpr int kStages = (kBudget - kFixed) / (kWBytes + kXBytes);
  static constexpr int kSmem = kFixed + kStages * (kWBytes + kXBytes);
  static_assert(kStages >= 4 && (2 * kStages + 3 * kBufs + 2) * 8 + 16 <= kBarBytes && kSmem <= kBudget, "shared memory");
  static_assert(kTmemCols >= 32 && kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "TMEM columns");
};

template <bool F8, int TN>
__global__ void __launch_bounds__(FewCfg<F8, TN>::kThreads, FewCfg<F8, TN>::kPerSm)
    linear_few_kernel(const LinearParams p, const int split, const __grid_constant__ CUtensorMap tmW,
                      const __grid_constant__ CUtensorMap tmX) {
  using Cfg = FewCfg<F8, TN>;
  constexpr int kStages = Cfg::kStages, kBufs = Cfg::kBufs, kCols = Cfg::kCols;
  constexpr int kElems = F8 ? 128 : 64;   // k values of a k-block
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sW = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sX = sW + kStages * Cfg::kWBytes;
  float* red = reinterpret_cast<float*>(sX + kStages * Cfg::kXBytes);
  float* table = red + TN * 128;
  uint64_t* full = reinterpret_cast<uint64_t*>(table + Cfg::kTableBytes / 4);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + kBufs;
  uint64_t* sfull = tempty + kBufs;
  uint64_t* rfull = sfull + kBufs;    // every rank's partial sums of this CTA's columns have arrived
  uint64_t* rfree = rfull + 1;        // every rank has read what this CTA sent it
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rfree + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* prefix = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(full) + Cfg::kBarBytes);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], Cfg::kEpiWarps);
      mbar_init(&sfull[b], 1);
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
  // after the TMEM allocation: a dependent kernel's CTA that took this SM's TMEM first would wait for
  // this kernel, and this kernel for it
  pdl_launch_dependents();
  // one layer: the first wave's weight tiles are known before the previous kernel has ended, and their way
  // to L2 can begin (a prefetch reads nothing stale: what that kernel still writes lands in L2).  Up to
  // kRasterRows row tiles n0 is this CTA's own first weight tile; past them it is one that other CTAs of the
  // wave take, and another CTA fetches this one's (by tile_at's order, with its 64-bit division: 0.1 us more)
  if (!p.offsets && warp == 0 && lane == 0 && t0 < first_tiles) {
    const int n0 = static_cast<int>(t0 / ((p.rows + TN - 1) / TN)) * 128;
    for (int kb = ka; kb < min(kb_end, ka + kPrefetch); ++kb) tma_prefetch_l2_3d(&tmW, kb * kElems, n0, 0);
  }
  pdl_wait_prior();
  if (warp == 2) build_schedule(p, TN, prefix, blockIdx.x == 0);
  __syncthreads();

  const long long tiles = tile_count(p, prefix);

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (long long t = t0; t < tiles; t += tstep) {
        const LinearTile q = tile_at<TN, 128>(p, prefix, t);
        for (int kb = ka; kb < kb_end; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, p.status)) goto teardown;
          mbar_arrive_expect_tx(&full[stage], Cfg::kWBytes + Cfg::kXBytes);
          tma_load_3d(sW + stage * Cfg::kWBytes, &tmW, &full[stage], kb * kElems, q.n0, q.e);
          tma_load_2d(sX + stage * Cfg::kXBytes, &tmX, &full[stage], kb * kElems, q.row0);
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
    constexpr uint32_t idesc = F8 ? idesc_e4m3_f32(128, TN) : idesc_bf16_f32(128, TN);
    const uint64_t a0 = sdesc_kmajor_sw128(smem_u32(sW)), b0 = sdesc_kmajor_sw128(smem_u32(sX));
    int stage = 0, buf = 0;
    uint32_t phase = 0, bphase = 0;
    const long long mine = tiles > t0 ? (tiles - t0 - 1) / tstep + 1 : 0;
    for (long long j = 0; j < mine; ++j) {
      for (int kb = ka, in_chunk = 0; kb < kb_end; ++kb) {
        const bool first = F8 || in_chunk == 0;
        const bool last = F8 || ++in_chunk == p.chunk_kb || kb == kb_end - 1;
        // both barriers are asked at once, before either is waited for
        bool ready = mbar_test_wait(&full[stage], phase);
        if (first) ready = mbar_test_wait(&tempty[buf], bphase ^ 1) & ready;
        if (!ready) {
          if (first && !mbar_wait(&tempty[buf], bphase ^ 1, abort_flag, p.status)) goto teardown;
          if (!mbar_wait(&full[stage], phase, abort_flag, p.status)) goto teardown;
        }
        tc_fence_after();
        const uint64_t a = a0 + stage * (Cfg::kWBytes >> 4), b = b0 + stage * (Cfg::kXBytes >> 4);
        const uint32_t d = tmem_base + buf * TN;
        if (issue) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {   // 32 bytes of k each
            if (F8)
              tc_mma_f8(d, a + 2 * i, b + 2 * i, idesc, i > 0);
            else
              tc_mma_bf16(d, a + 2 * i, b + 2 * i, idesc, !first || i > 0);
          }
          tc_commit(&empty[stage]);
          if (last) tc_commit(&tfull[buf]);
        }
        __syncwarp();
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
        if (last) {
          in_chunk = 0;
          if (++buf == kBufs) {
            buf = 0;
            bphase ^= 1;
          }
        }
      }
    }
  } else if (warp == 2) {
    if (F8) {
      // slot b: x_scale[row][kb] * w_scale[n0 / 128][kb] for the tile's rows (zero past them)
      constexpr int kPer = (TN + 31) / 32;   // columns per lane
      constexpr int kAhead = 4;              // k-blocks whose scales are on the way
      int buf = 0;
      uint32_t bphase = 0;
      const int nblk = (p.N + kScaleBlock - 1) / kScaleBlock;
      for (long long t = t0; t < tiles; t += tstep) {
        const LinearTile q = tile_at<TN, 128>(p, prefix, t);
        const float* ws = p.w_scale + (static_cast<long long>(q.e) * nblk + q.n0 / kScaleBlock) * p.num_kb;
        float v[kAhead][kPer], w[kAhead];
        auto fetch = [&](int kb, float (&vs)[kPer], float& wv) {
          wv = kb < kb_end ? ws[kb] : 0.f;
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            const int c = lane + 32 * j;
            vs[j] = kb < kb_end && c < q.rows ? p.x_scale[(q.row0 + c) * p.xs_row + kb * p.xs_blk] : 0.f;
          }
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch(ka + i, v[i], w[i]);
        for (int kb0 = ka; kb0 < kb_end; kb0 += kAhead) {
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            if (kb0 + i < kb_end) {
              if (!mbar_wait(&tempty[buf], bphase ^ 1, abort_flag, p.status)) goto teardown;
#pragma unroll
              for (int j = 0; j < kPer; ++j)
                if (lane + 32 * j < TN) table[buf * TN + lane + 32 * j] = v[i][j] * w[i];
              __syncwarp();
              if (lane == 0) mbar_arrive(&sfull[buf]);
              if (++buf == kBufs) {
                buf = 0;
                bphase ^= 1;
              }
              fetch(kb0 + i + kAhead, v[i], w[i]);
            }
          }
        }
      }
    }
  } else if (warp >= 4) {
    const int quad = warp & 3;
    const int c0 = (warp - 4) / 4 * kCols;   // this thread's columns
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    int buf = 0;
    uint32_t bphase = 0, rphase = 0;
    for (long long t = t0; t < tiles; t += tstep) {
      const LinearTile q = tile_at<TN, 128>(p, prefix, t);
      float acc[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
      for (int kb = ka; kb < kb_end; kb += F8 ? 1 : p.chunk_kb) {
        if (!whole_warp(mbar_wait(&tfull[buf], bphase, abort_flag, p.status) &&
                        (!F8 || mbar_wait(&sfull[buf], bphase, abort_flag, p.status)))) goto teardown;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(tmem_base + lane_base + buf * TN + c0 + c, r);
          tmem_ld_wait();
          if (F8) {
            const float4* s = reinterpret_cast<const float4*>(table + buf * TN + c0 + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 f = s[i];
              acc[c + 4 * i] = fmaf(__uint_as_float(r[4 * i]), f.x, acc[c + 4 * i]);
              acc[c + 4 * i + 1] = fmaf(__uint_as_float(r[4 * i + 1]), f.y, acc[c + 4 * i + 1]);
              acc[c + 4 * i + 2] = fmaf(__uint_as_float(r[4 * i + 2]), f.z, acc[c + 4 * i + 2]);
              acc[c + 4 * i + 3] = fmaf(__uint_as_float(r[4 * i + 3]), f.w, acc[c + 4 * i + 3]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[c + i] += __uint_as_float(r[i]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[buf]);
        if (++buf == kBufs) {
          buf = 0;
          bphase ^= 1;
        }
      }
      const int nrow = quad * 32 + lane;   // this thread's weight row of the tile
      const int n = q.n0 + nrow;
      const float bias = p.bias && n < p.N ? p.bias[static_cast<long long>(q.e) * p.N + n] : 0.f;
      auto put = [&](int c, float v) {
        v = act_clamp(v + bias, p.lo, p.hi);
        if (!CONVF_IN_BOUNDS(q.row0 + c < p.rows && n < p.N, p.status)) return;
        const long long at = static_cast<long long>(q.row0 + c) * p.ldy + n;
        if (p.out_bf16)
          static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v);
        else
          static_cast<float*>(p.y)[at] = v;
      };
      if (split == 1) {
        if (n < p.N) {
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            if (c0 + c < q.rows) put(c0 + c, acc[c]);
        }
      } else {
        // column c is finished by rank c / per: send it there, then finish this rank's own
        const int per = TN / split;
        if (!mbar_wait_cluster(rfree, rphase ^ 1, abort_flag, p.status)) goto teardown;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const int col = c0 + c, to = col / per;
          if (col < q.rows)
            st_cluster_f32(map_to_rank(smem_u32(red + (rank * per + col - to * per) * 128 + nrow), to), acc[c]);
        }
        asm volatile("fence.acq_rel.cluster;" ::: "memory");
        __syncwarp();
        if (lane < split) mbar_arrive_remote(map_to_rank(smem_u32(rfull), lane));
        if (!mbar_wait_cluster(rfull, rphase, abort_flag, p.status)) goto teardown;
        const int mine = min(per, q.rows - rank * per);
        for (int j = (warp - 4) / 4; j < mine; j += Cfg::kEpiWarps / 4) {
          float v = 0.f;
          for (int s = 0; s < split; ++s) v += red[(s * per + j) * 128 + nrow];
          if (n < p.N) put(rank * per + j, v);
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
  if (split > 1) cluster_sync();   // no CTA leaves while a peer may still write to it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, Cfg::kTmemCols);
  }
}

template <bool F8, int TN>
cudaError_t configure() {
  static OncePerDevice once;
  return once([] {
    return cudaFuncSetAttribute(linear_few_kernel<F8, TN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                FewCfg<F8, TN>::kSmem);
  });
}

template <bool F8, int TN>
cudaError_t launch_t(const LinearParams& p, const LinearPlan& plan, const CUtensorMap& tmW, const CUtensorMap& tmX,
                     cudaStream_t stream) {
  const cudaError_t e = configure<F8, TN>();
  if (e != cudaSuccess) return e;
  return launch_pdl(linear_few_kernel<F8, TN>, dim3(plan.grid), dim3(FewCfg<F8, TN>::kThreads), FewCfg<F8, TN>::kSmem,
                    stream, plan.split, p, plan.split, tmW, tmX);
}

template <bool F8, int TN>
int max_clusters_t(int split, int num_sms) {
  if (split == 1) return num_sms * FewCfg<F8, TN>::kPerSm;
  if (configure<F8, TN>() != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(split);
  cfg.blockDim = dim3(FewCfg<F8, TN>::kThreads);
  cfg.dynamicSmemBytes = FewCfg<F8, TN>::kSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  return cudaOccupancyMaxActiveClusters(&n, linear_few_kernel<F8, TN>, &cfg) == cudaSuccess ? n : 0;
}

}  // namespace

cudaError_t launch_linear_few(const LinearParams& p, const LinearPlan& plan, bool e4m3, const CUtensorMap& tmW,
                              const CUtensorMap& tmX, cudaStream_t stream) {
  switch (plan.tile) {
    case 16: return e4m3 ? launch_t<true, 16>(p, plan, tmW, tmX, stream) : launch_t<false, 16>(p, plan, tmW, tmX, stream);
    case 32: return e4m3 ? launch_t<true, 32>(p, plan, tmW, tmX, stream) : launch_t<false, 32>(p, plan, tmW, tmX, stream);
    case 64: return e4m3 ? launch_t<true, 64>(p, plan, tmW, tmX, stream) : launch_t<false, 64>(p, plan, tmW, tmX, stream);
  }
  return cudaErrorInvalidValue;
}

int linear_few_max_clusters(bool e4m3, int tile, int split, int num_sms) {
  switch (tile) {
    case 16: return e4m3 ? max_clusters_t<true, 16>(split, num_sms) : max_clusters_t<false, 16>(split, num_sms);
    case 32: return e4m3 ? max_clusters_t<true, 32>(split, num_sms) : max_clusters_t<false, 32>(split, num_sms);
    case 64: return e4m3 ? max_clusters_t<true, 64>(split, num_sms) : max_clusters_t<false, 64>(split, num_sms);
  }
  return 0;
}

}  // namespace convf
