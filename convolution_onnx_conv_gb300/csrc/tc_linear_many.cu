// Linear layers for many rows per weight matrix: y = x W^T on tcgen05, 128 x 256 tiles, or 256 x 256
// on CTA pairs.
//
// Here the rows of x are the MMA's rows, so that a thread of the epilogue holds one row of y and the
// e4m3 scale of a k-block is one number for all its columns.  The tensor cores are the bound: a
// 128 x 256 tile per SM needs 96 bytes of operands per cycle from shared memory at the e4m3 rate, a
// pair's 256 x 256 tile 64 (each CTA holds half of the weights), and L2 has to deliver 2/3 as many
// bytes.
//
// e4m3: a k-block's sums have to leave TMEM to be scaled, so the epilogue works all the time.  TMEM
// holds a ring of four accumulators of 128 columns; the MMAs of a 128-value k-block fill one for each
// half of the tile's columns, and a warpgroup adds its half's, times x_scale * w_scale, to fp32 sums in
// registers: 128 columns per thread, as packed multiply-adds.  While it does the MMAs fill the other
// three: 768 cycles for the way from the last MMA over the reads back to the next one (two accumulators
// of 256 columns leave 512, and ran at half the rate).  bf16: an accumulator of 256 columns sums
// LinearParams::chunk_kb k-blocks.
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
  static constexpr int kStages = PAIR ? 5 : 4;
  static constexpr int kOutBytes = 4096;   // per epilogue warp: 32 rows of 128 bytes on the way out
  static constexpr int kBarBytes = 256;
  static constexpr int kFixed = kStages * (kXBytes + kWBytes) + 8 * kOutBytes + kBarBytes;   // and the schedule
  static_assert((2 * kStages + 8) * 8 + 8 <= kBarBytes, "barriers");
  static_assert(kFixed + ((PAIR ? kMaxExperts : kManyExperts) + 4) * 4 <= 232448, "shared memory");
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
                       const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmY) {
  using Cfg = ManyCfg<PAIR>;
  constexpr int kStages = Cfg::kStages;
  constexpr int kElems = F8 ? 128 : 64;
  constexpr uint32_t kTmemCols = 512;
  extern __shared__ __align__(1024) uint8_t sX[];   // (the swizzle goes by address bits 7 to 9)
  uint8_t* sW = sX + kStages * Cfg::kXBytes;
  uint8_t* sOut = sW + kStages * Cfg::kWBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sOut + 8 * Cfg::kOutBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 4);
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
    for (int b = 0; b < 4; ++b) {   // accumulator b: 128 columns, of half b & 1 of a tile
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], PAIR ? 8 : 4);   // the warps of a half's warpgroup, of both CTAs
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

  // every earlier MMA of this thread has completed -> an arrival on `bar`, of a pair in both CTAs
  auto commit_to = [&](uint64_t* bar) {
    if (PAIR)
      tc_commit_pair(bar, 3);
    else
      tc_commit(bar);
  };
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
            if (F8) {   // this CTA's half of each half of the columns
              tma_load_3d_pair(sW + stage * Cfg::kWBytes, &tmW, bar, kb * kElems, q.n0 + crank * 64, q.e);
              tma_load_3d_pair(sW + stage * Cfg::kWBytes + 64 * kKBlockBytes, &tmW, bar, kb * kElems,
                               q.n0 + 128 + crank * 64, q.e);
            } else {
              tma_load_3d_pair(sW + stage * Cfg::kWBytes, &tmW, bar, kb * kElems, q.n0 + crank * 128, q.e);
            }
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
    } else if (warp == 1 && leader) {
      // The whole warp walks the loop and one lane issues: the loop's state then stays in uniform
      // registers, which is where the MMA takes its descriptors from.
      const bool issue = elect_one();
      constexpr int kCols = F8 ? 128 : 256;   // of an MMA
      constexpr uint32_t idesc = F8 ? idesc_e4m3_f32(Cfg::kTileM, kCols) : idesc_bf16_f32(Cfg::kTileM, kCols);
      // weight rows of the second half of the columns (a pair's CTA holds half of each half)
      constexpr uint32_t kHalf = (PAIR ? 64 : 128) * kKBlockBytes >> 4;
      const uint64_t a0 = sdesc_kmajor_sw128(smem_u32(sX)), b0 = sdesc_kmajor_sw128(smem_u32(sW));
      int stage = 0, buf = 0;   // buf: 0 or 2, the first accumulator of the k-block
      uint32_t phase = 0, bphase = 0;
      const long long mine = tiles > t0 ? (tiles - t0 - 1) / tstep + 1 : 0;
      for (long long j = 0; j < mine; ++j) {
        for (int kb = 0, in_chunk = 0; kb < p.num_kb; ++kb) {
          const bool first = F8 || in_chunk == 0;
          const bool last = F8 || ++in_chunk == p.chunk_kb || kb == p.num_kb - 1;
          // the three barriers are asked at once: their answers, one after the other, took longer
          // than the MMAs
          bool ready = mbar_test_wait(&full[stage], phase);
          if (first) {
            const bool r0 = mbar_test_wait(&tempty[buf], bphase ^ 1), r1 = mbar_test_wait(&tempty[buf + 1], bphase ^ 1);
            ready = ready & r0 & r1;
          }
          if (!ready) {
            if (!mbar_wait(&full[stage], phase, abort_flag, p.status)) goto teardown;
            if (first && !mbar_wait(&tempty[buf], bphase ^ 1, abort_flag, p.status)) goto teardown;
            if (first && !mbar_wait(&tempty[buf + 1], bphase ^ 1, abort_flag, p.status)) goto teardown;
          }
          tc_fence_after();
          const uint64_t a = a0 + stage * (Cfg::kXBytes >> 4), b = b0 + stage * (Cfg::kWBytes >> 4);
          const uint32_t d = tmem_base + buf * 128;
          if (issue) {
#pragma unroll
            for (int h = 0; h < (F8 ? 2 : 1); ++h) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {   // 32 bytes of k each
                if (F8 && PAIR)
                  tc_mma_f8_pair(d + h * 128, a + 2 * i, b + h * kHalf + 2 * i, idesc, i > 0);
                else if (F8)
                  tc_mma_f8(d + h * 128, a + 2 * i, b + h * kHalf + 2 * i, idesc, i > 0);
                else if (PAIR)
                  tc_mma_bf16_pair(d, a + 2 * i, b + 2 * i, idesc, !first || i > 0);
                else
                  tc_mma_bf16(d, a + 2 * i, b + 2 * i, idesc, !first || i > 0);
              }
              if (F8 && h == 0) commit_to(&tfull[buf]);
            }
            commit_to(&empty[stage]);
            if (!F8 && last) commit_to(&tfull[buf]);
            if (last) commit_to(&tfull[buf + 1]);
          }
          __syncwarp();
          if (last) {
            in_chunk = 0;
            if ((buf ^= 2) == 0) bphase ^= 1;
          }
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsEpi));
    const int quad = warp & 3, half = (warp - 4) >> 2;
    uint8_t* out = sOut + (warp - 4) * Cfg::kOutBytes;
    const uint32_t from0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + half * 128;
    const int nblk = (p.N + kScaleBlock - 1) / kScaleBlock;
    int buf = half;
    uint32_t bphase = 0;
    for (long long t = t0; t < tiles; t += tstep) {
      const LinearTile q = tile_at<Cfg::kTileM, kManyCols>(p, prefix, t);
      const int mrow = crank * 128 + quad * 32;   // this warp's first row of the tile
      const int n0 = q.n0 + half * 128;           // and its first column
      // the scales are loaded two k-blocks ahead (and multiplied when they are used: a product at the
      // load would wait for it); rows and columns past the edge read the last scale there is, and
      // their sums are not stored
      const float *xs = nullptr, *ws = nullptr;
      float x0 = 1.f, w0 = 1.f, x1 = 1.f, w1 = 1.f;
      if (F8) {
        xs = p.x_scale + (q.row0 + min(mrow + lane, q.rows - 1)) * p.xs_row;
        ws = p.w_scale + (static_cast<long long>(q.e) * nblk + min(n0 / kScaleBlock, nblk - 1)) * p.num_kb;
        x0 = __ldg(xs);
        w0 = __ldg(ws);
        if (p.num_kb > 1) {
          xs += p.xs_blk;
          ++ws;
        }
        x1 = __ldg(xs);
        w1 = __ldg(ws);
      }
      f32x2 acc[64];
#pragma unroll
      for (int c = 0; c < 64; ++c) acc[c] = 0;
#pragma unroll 1
      for (int kb = 0; kb < p.num_kb; kb += F8 ? 1 : p.chunk_kb) {
        const float both = x0 * w0;
        const f32x2 s = pair_of(__float_as_uint(both), __float_as_uint(both));
        if (F8) {
          x0 = x1;
          w0 = w1;
          if (kb + 2 < p.num_kb) {
            xs += p.xs_blk;
            ++ws;
          }
          x1 = __ldg(xs);
          w1 = __ldg(ws);
        }
        if (!mbar_wait(&tfull[buf], bphase, abort_flag, p.status)) goto teardown;
        tc_fence_after();
        const uint32_t from = from0 + (buf & 2) * 128;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t r[64];
          tmem_ld_32x32b_x64(from + 64 * c, r);   // waits for the values
          if (c == 1) {
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
          for (int i = 0; i < 32; ++i) acc[32 * c + i] = fma2(pair_of(r[2 * i], r[2 * i + 1]), s, acc[32 * c + i]);
        }
        buf ^= 2;
        if (buf == half) bphase ^= 1;
      }
      // out through shared memory, 32 rows of 128 bytes at a time (in the 128-byte swizzle): one TMA
      // store where all 32 rows are the tile's (it clips the columns past N), else row by row
      const bool whole = p.vec_y && mrow + 32 <= q.rows;
      const float* bias = p.bias ? p.bias + static_cast<long long>(q.e) * p.N : nullptr;
      auto finish = [&](float2 v, int n) {
        if (bias) {
          v.x += n < p.N ? __ldg(bias + n) : 0.f;
          v.y += n + 1 < p.N ? __ldg(bias + n + 1) : 0.f;
        }
        if (p.clamp) {
          v.x = act_clamp(v.x, p.lo, p.hi);
          v.y = act_clamp(v.y, p.lo, p.hi);
        }
        return v;
      };
      auto room = [&] {   // the staged rows of the last store have been read
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
      };
      auto unit = [&](int u) { return reinterpret_cast<uint4*>(out + lane * 128 + ((u ^ (lane & 7)) << 4)); };
      auto leave = [&](int n) {
        if (whole) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && n < p.N) {
            tma_store_2d(&tmY, out, n, q.row0 + mrow);
            bulk_commit();
          }
          return;
        }
        __syncwarp();
        const int osz = p.out_bf16 ? 2 : 4, per_unit = 16 / osz;
        for (int i = 0; i < 8; ++i) {
          const int r = i * 4 + (lane >> 3), u = lane & 7, c = n + u * per_unit;
          if (mrow + r >= q.rows || c >= p.N) continue;
          const uint8_t* v = out + r * 128 + ((u ^ (r & 7)) << 4);
          uint8_t* to = static_cast<uint8_t*>(p.y) + (static_cast<long long>(q.row0 + mrow + r) * p.ldy + c) * osz;
          if (p.vec_y && c + per_unit <= p.N) {
            *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(v);
          } else {
            for (int j = 0; j < per_unit && c + j < p.N; ++j) {
              if (osz == 2)
                reinterpret_cast<uint16_t*>(to)[j] = reinterpret_cast<const uint16_t*>(v)[j];
              else
                reinterpret_cast<uint32_t*>(to)[j] = reinterpret_cast<const uint32_t*>(v)[j];
            }
          }
        }
        __syncwarp();
      };
      if (mrow < q.rows) {
        if (p.out_bf16) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            room();
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 v = finish(split_of(acc[32 * c + 4 * u + i]), n0 + 64 * c + 8 * u + 2 * i);
                const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
              }
              *unit(u) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            leave(n0 + 64 * c);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            room();
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const int n = n0 + 32 * c + 4 * u;
              const float2 v0 = finish(split_of(acc[16 * c + 2 * u]), n);
              const float2 v1 = finish(split_of(acc[16 * c + 2 * u + 1]), n + 2);
              *unit(u) = make_uint4(__float_as_uint(v0.x), __float_as_uint(v0.y), __float_as_uint(v1.x),
                                    __float_as_uint(v1.y));
            }
            leave(n0 + 32 * c);
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();   // the stores have been written before the CTA ends
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
                     const CUtensorMap& tmY, cudaStream_t stream) {
  using Cfg = ManyCfg<PAIR>;
  static bool configured = false;
  if (!configured) {
    // the register split waits for ever if the kernel was given fewer registers than it shares out
    cudaFuncAttributes at;
    cudaError_t e = cudaFuncGetAttributes(&at, linear_many_kernel<F8, PAIR>);
    if (e == cudaSuccess && at.numRegs < Cfg::kRegs) e = cudaErrorInvalidKernelImage;
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(linear_many_kernel<F8, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    if (e != cudaSuccess) return e;
    configured = true;
  }
  const int smem = Cfg::kFixed + (p.experts + 4) / 4 * 16;   // experts + 1 ints
  if (smem > 232448) return cudaErrorInvalidValue;
  return launch_pdl(linear_many_kernel<F8, PAIR>, dim3(plan.grid), dim3(Cfg::kThreads), smem, stream, PAIR ? 2 : 1, p,
                    tmW, tmX, tmY);
}

}  // namespace

cudaError_t launch_linear_many(const LinearParams& p, const LinearPlan& plan, bool e4m3, const CUtensorMap& tmW,
                               const CUtensorMap& tmX, const CUtensorMap& tmY, cudaStream_t stream) {
  if (plan.tile == 256)
    return e4m3 ? launch_t<true, true>(p, plan, tmW, tmX, tmY, stream) : launch_t<false, true>(p, plan, tmW, tmX, tmY, stream);
  return e4m3 ? launch_t<true, false>(p, plan, tmW, tmX, tmY, stream) : launch_t<false, false>(p, plan, tmW, tmX, tmY, stream);
}

}  // namespace convf
