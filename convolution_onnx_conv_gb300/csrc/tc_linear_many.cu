// Linear layers for many rows per weight matrix: y = x W^T on tcgen05, 128 x 256 tiles, or 256 x 256
// on CTA pairs.
//
// Here the rows of x are the MMA's rows, so that a thread of the epilogue holds one row of y and the
// e4m3 scale of a k-block is one number for all its columns.  The tensor cores are the bound: a
// 128 x 256 tile per SM needs 96 bytes of operands per cycle from shared memory at the e4m3 rate, a
// pair's 256 x 256 tile 64 (each CTA holds half of the weights), and L2 has to deliver 2/3 as many
// bytes.
//
// e4m3: TMEM holds two accumulators of 256 columns.  The MMAs of a 128-value k-block fill one while the
// epilogue adds the other, times x_scale * w_scale, to fp32 sums in registers: 128 columns per thread,
// two warpgroups, as packed multiply-adds (64 per thread and k-block, half of the issue slots of the
// 512 cycles that the MMAs take).  bf16: an accumulator sums LinearParams::chunk_kb k-blocks.
//
//   warp 0      TMA: x and weight tiles of each k-block
//   warp 1      TMEM, MMA issue (of a pair: the leader's)
//   warps 4-11  epilogue
#include "linear_dev.cuh"

namespace convf {

namespace {

template <bool PAIR>
struct ManyCfg {
  static constexpr int kThreads = 384;
  static constexpr int kTileM = PAIR ? 256 : 128;
  static constexpr int kXBytes = 128 * kKBlockBytes;
  static constexpr int kWBytes = (PAIR ? 128 : 256) * kKBlockBytes;   // a pair's CTA holds half
  static constexpr int kStages = PAIR ? 6 : 4;
  static constexpr int kOutBytes = 2048;   // per epilogue warp: 32 rows of 64 bytes on the way out
  static constexpr int kSchedBytes = (kMaxExperts + 1) * 4 + 12;
  static constexpr int kBarBytes = 256;
  static constexpr int kSmem = 1024 + kStages * (kXBytes + kWBytes) + 8 * kOutBytes + kBarBytes + kSchedBytes;
  static_assert(kSmem <= 232448, "shared memory");
  // registers: 168 per thread at launch; the epilogue's two warpgroups take what the others give up
  static constexpr int kRegs = 168, kRegsEpi = 224, kRegsOther = 56;
  static_assert(256 * kRegsEpi + 128 * kRegsOther <= kThreads * kRegs, "register split");
};

// two fp32 columns in a register pair
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair_of(uint32_t lo, uint32_t hi) {
  f32x2 v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
  return v;
}
__device__ __forceinline__ float2 split_of(f32x2 v) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
  return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

template <bool F8, bool PAIR>
__global__ void __launch_bounds__(ManyCfg<PAIR>::kThreads, 1)
    linear_many_kernel(const LinearParams p, const __grid_constant__ CUtensorMap tmW,
                       const __grid_constant__ CUtensorMap tmX) {
  using Cfg = ManyCfg<PAIR>;
  constexpr int kStages = Cfg::kStages;
  constexpr int kElems = F8 ? 128 : 64;
  constexpr uint32_t kTmemCols = 512;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sX = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sW = sX + kStages * Cfg::kXBytes;
  uint8_t* sOut = sW + kStages * Cfg::kWBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sOut + 8 * Cfg::kOutBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* prefix = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(full) + Cfg::kBarBytes);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int crank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const bool leader = crank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], PAIR ? 16 : 8);   // every epilogue warp, of both CTAs
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(tmem_slot, kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_launch_dependents();   // after the TMEM allocation, which a dependent's CTA would otherwise take
  pdl_wait_prior();
  if (warp == 2) build_schedule(p, Cfg::kTileM, prefix, blockIdx.x == 0);
  __syncthreads();

  const long long tiles = static_cast<long long>(prefix[p.experts]) * p.n_tiles;
  const long long t0 = PAIR ? blockIdx.x >> 1 : blockIdx.x, tstep = PAIR ? gridDim.x >> 1 : gridDim.x;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsOther));
    if (warp == 0 && lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (long long t = t0; t < tiles; t += tstep) {
        const LinearTile q = tile_at<Cfg::kTileM, kManyCols>(p, prefix, t);
        for (int kb = 0; kb < p.num_kb; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, p.status)) goto teardown;
          // a pair's loads all complete on the leader's barrier, which expects both CTAs' bytes
          if (leader) mbar_arrive_expect_tx(&full[stage], (PAIR ? 2 : 1) * (Cfg::kXBytes + Cfg::kWBytes));
          if (PAIR) {
            const uint32_t bar = map_to_rank(smem_u32(&full[stage]), 0);
            tma_load_2d_pair(sX + stage * Cfg::kXBytes, &tmX, bar, kb * kElems, q.row0 + crank * 128);
            tma_load_3d_pair(sW + stage * Cfg::kWBytes, &tmW, bar, kb * kElems, q.n0 + crank * 128, q.e);
          } else {
            tma_load_2d(sX + stage * Cfg::kXBytes, &tmX, &full[stage], kb * kElems, q.row0);
            tma_load_3d(sW + stage * Cfg::kWBytes, &tmW, &full[stage], kb * kElems, q.n0, q.e);
          }
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    } else if (warp == 1 && lane == 0 && leader) {
      constexpr uint32_t idesc = F8 ? idesc_e4m3_f32(Cfg::kTileM, kManyCols) : idesc_bf16_f32(Cfg::kTileM, kManyCols);
      int stage = 0, buf = 0;
      uint32_t phase = 0, bphase = 0;
      for (long long t = t0; t < tiles; t += tstep) {
        for (int kb = 0, in_chunk = 0; kb < p.num_kb; ++kb) {
          const bool first = F8 || in_chunk == 0;
          if (first && !mbar_wait(&tempty[buf], bphase ^ 1, abort_flag, p.status)) goto teardown;
          if (!mbar_wait(&full[stage], phase, abort_flag, p.status)) goto teardown;
          tc_fence_after();
          const uint64_t a = sdesc_kmajor_sw128(smem_u32(sX + stage * Cfg::kXBytes));
          const uint64_t b = sdesc_kmajor_sw128(smem_u32(sW + stage * Cfg::kWBytes));
          const uint32_t d = tmem_base + buf * kManyCols;
#pragma unroll
          for (int i = 0; i < 4; ++i) {   // 32 bytes of k each
            const uint32_t acc = !first || i > 0;
            if (F8 && PAIR)
              tc_mma_f8_pair(d, a + 2 * i, b + 2 * i, idesc, acc);
            else if (F8)
              tc_mma_f8(d, a + 2 * i, b + 2 * i, idesc, acc);
            else if (PAIR)
              tc_mma_bf16_pair(d, a + 2 * i, b + 2 * i, idesc, acc);
            else
              tc_mma_bf16(d, a + 2 * i, b + 2 * i, idesc, acc);
          }
          if (PAIR)
            tc_commit_pair(&empty[stage], 3);
          else
            tc_commit(&empty[stage]);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
          if (F8 || ++in_chunk == p.chunk_kb || kb == p.num_kb - 1) {
            in_chunk = 0;
            if (PAIR)
              tc_commit_pair(&tfull[buf], 3);
            else
              tc_commit(&tfull[buf]);
            if (++buf == 2) {
              buf = 0;
              bphase ^= 1;
            }
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsEpi));
    const int quad = warp & 3, half = (warp - 4) >> 2;
    uint8_t* out = sOut + (warp - 4) * Cfg::kOutBytes;
    const uint32_t lane_base = (static_cast<uint32_t>(quad * 32) << 16) + half * 128;
    const int nblk = (p.N + kScaleBlock - 1) / kScaleBlock;
    int buf = 0;
    uint32_t bphase = 0;
    for (long long t = t0; t < tiles; t += tstep) {
      const LinearTile q = tile_at<Cfg::kTileM, kManyCols>(p, prefix, t);
      const int mrow = crank * 128 + quad * 32;   // this warp's first row of the tile
      const int n0 = q.n0 + half * 128;           // and its first column
      const float *xs = nullptr, *ws = nullptr;
      if (F8) {
        // rows and columns past the edge read the last scale there is; their sums are not stored
        xs = p.x_scale + (q.row0 + min(mrow + lane, q.rows - 1)) * p.xs_row;
        ws = p.w_scale + (static_cast<long long>(q.e) * nblk + min(n0 / kScaleBlock, nblk - 1)) * p.num_kb;
      }
      // the scales of the next kAhead k-blocks are on their way (multiplied when they are used: a
      // product here would wait for them)
      constexpr int kAhead = 4;
      float sx[kAhead], sw[kAhead];
      auto fetch = [&](int kb, float& a, float& b) {
        const bool in = F8 && kb < p.num_kb;
        a = in ? __ldg(xs + kb * p.xs_blk) : 1.f;
        b = in ? __ldg(ws + kb) : 1.f;
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) fetch(i, sx[i], sw[i]);
      f32x2 acc[64];
#pragma unroll
      for (int c = 0; c < 64; ++c) acc[c] = 0;
      for (int kb = 0; kb < p.num_kb; kb += F8 ? 1 : p.chunk_kb) {
        const float both = sx[0] * sw[0];
        const f32x2 s = pair_of(__float_as_uint(both), __float_as_uint(both));
        if (F8) {
#pragma unroll
          for (int i = 0; i + 1 < kAhead; ++i) {
            sx[i] = sx[i + 1];
            sw[i] = sw[i + 1];
          }
          fetch(kb + kAhead, sx[kAhead - 1], sw[kAhead - 1]);
        }
        if (!mbar_wait(&tfull[buf], bphase, abort_flag, p.status)) goto teardown;
        tc_fence_after();
        const uint32_t from = tmem_base + lane_base + buf * kManyCols;
        // the next 16 columns are on their way while these are added
        uint32_t r[2][16];
        tmem_ld_32x32b_x16(from, r[0]);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          tmem_ld_wait_for(r[c & 1]);
          if (c < 7) {
            tmem_ld_32x32b_x16(from + 16 * (c + 1), r[(c + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if (PAIR)
                mbar_arrive_remote_relaxed(map_to_rank(smem_u32(&tempty[buf]), 0));
              else
                mbar_arrive(&tempty[buf]);
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[8 * c + i] = fma2(pair_of(r[c & 1][2 * i], r[c & 1][2 * i + 1]), s, acc[8 * c + i]);
        }
        if (++buf == 2) {
          buf = 0;
          bphase ^= 1;
        }
      }
      // the sums leave through shared memory, 32 rows of 64 bytes at a time (16-byte units swizzled
      // by row), as 16-byte stores of 64 consecutive bytes per row
      const float* bias = p.bias ? p.bias + static_cast<long long>(q.e) * p.N : nullptr;
      auto value = [&](float v, int n) { return act_clamp(bias && n < p.N ? v + __ldg(bias + n) : v, p.lo, p.hi); };
      const int per_unit = p.out_bf16 ? 8 : 4;   // columns of a 16-byte unit
      auto leave = [&](int n) {                  // the staged columns begin at n
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 8 + (lane >> 2), u = lane & 3;
          const uint4 v = *reinterpret_cast<const uint4*>(out + r * 64 + ((u ^ ((r >> 1) & 3)) << 4));
          const int c = n + u * per_unit;
          if (mrow + r < q.rows && c < p.N) {
            const long long at = static_cast<long long>(q.row0 + mrow + r) * p.ldy + c;
            if (p.vec_y && c + per_unit <= p.N) {
              *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.y) + at * (p.out_bf16 ? 2 : 4)) = v;
            } else {
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
              for (int j = 0; j < per_unit; ++j)
                if (c + j < p.N) {
                  if (p.out_bf16)
                    static_cast<uint16_t*>(p.y)[at + j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
                  else
                    static_cast<uint32_t*>(p.y)[at + j] = w[j];
                }
            }
          }
        }
        __syncwarp();
      };
      auto unit = [&](int u) { return reinterpret_cast<uint4*>(out + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4)); };
      if (p.out_bf16) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {   // 32 columns
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int n = n0 + 32 * c + 8 * u + 2 * i;
              const float2 v = split_of(acc[16 * c + 4 * u + i]);
              const __nv_bfloat162 h = __floats2bfloat162_rn(value(v.x, n), value(v.y, n + 1));
              w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *unit(u) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          leave(n0 + 32 * c);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) {   // 16 columns
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int n = n0 + 16 * c + 4 * u;
            const float2 v0 = split_of(acc[8 * c + 2 * u]), v1 = split_of(acc[8 * c + 2 * u + 1]);
            *unit(u) = make_uint4(__float_as_uint(value(v0.x, n)), __float_as_uint(value(v0.y, n + 1)),
                                  __float_as_uint(value(v1.x, n + 2)), __float_as_uint(value(v1.y, n + 3)));
          }
          leave(n0 + 16 * c);
        }
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
  if (PAIR) cluster_sync();   // no CTA of the pair leaves while the other may still signal it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem_base, kTmemCols);
    else
      tmem_dealloc(tmem_base, kTmemCols);
  }
}

template <bool F8, bool PAIR>
cudaError_t launch_t(const LinearParams& p, const LinearPlan& plan, const CUtensorMap& tmW, const CUtensorMap& tmX,
                     cudaStream_t stream) {
  using Cfg = ManyCfg<PAIR>;
  static bool configured = false;
  if (!configured) {
    // the register split waits for ever if the kernel was given fewer registers than it shares out
    cudaFuncAttributes at;
    cudaError_t e = cudaFuncGetAttributes(&at, linear_many_kernel<F8, PAIR>);
    if (e == cudaSuccess && at.numRegs < Cfg::kRegs) e = cudaErrorInvalidKernelImage;
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(linear_many_kernel<F8, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e != cudaSuccess) return e;
    configured = true;
  }
  return launch_pdl(linear_many_kernel<F8, PAIR>, dim3(plan.grid), dim3(Cfg::kThreads), Cfg::kSmem, stream, PAIR ? 2 : 1, p,
                    tmW, tmX);
}

}  // namespace

cudaError_t launch_linear_many(const LinearParams& p, const LinearPlan& plan, bool e4m3, const CUtensorMap& tmW,
                               const CUtensorMap& tmX, cudaStream_t stream) {
  if (plan.tile == 256)
    return e4m3 ? launch_t<true, true>(p, plan, tmW, tmX, stream) : launch_t<false, true>(p, plan, tmW, tmX, stream);
  return e4m3 ? launch_t<true, false>(p, plan, tmW, tmX, stream) : launch_t<false, false>(p, plan, tmW, tmX, stream);
}

}  // namespace convf
