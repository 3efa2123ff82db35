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
// half of the tile's columns, and the epilogue adds it, times x_scale * w_scale, to fp32 sums in
// registers, as packed multiply-adds: 128 columns per thread.  An accumulator has 768 cycles for the way
// from its last MMA over the reads back to its next MMA before the tensor cores wait.  The MMAs take 512
// cycles per k-block, this takes 600 to 650 (tensor pipe 62% busy at 4096 x 4096 x 4096, tile ends
// included); two accumulators of 256 columns took 1080, sixteen epilogue warps of 64 columns 900.  What
// bounds it now is that way's latency, and, for long, the power limit: 8192 x 8192 x 8192 takes 357 us
// (3.1 PFLOP/s) in a short run and 420 us (2.6) in a long one.  bf16: an accumulator of 256 columns sums
// LinearParams::chunk_kb k-blocks, 512 cycles each for 64 values.
//
//   warps 0-7   epilogue: warp w the rows 32 (w % 4) .. and the columns 128 (w / 4) .. of the CTA's tile
//   warp 8      TMA: x and weight tiles of each k-block
//   warp 9      TMEM, MMA issue (of a pair: the leader's)
//   warp 10     works out the CTA's next tiles (the divisions and lookups cost the epilogue 1000 cycles a tile)
//   (warp 11: none; registers are handed over by warpgroups)
#include <type_traits>

#include "linear_dev.cuh"

namespace convf {

namespace {

constexpr int kTileBatch = 16;   // tiles that the scheduler works out at a time

template <bool PAIR>
struct ManyCfg {
  static constexpr int kThreads = 384;
  // registers: 168 per thread at launch; the epilogue's two warpgroups take what the third gives up.  (The
  // PLAIN kernels spill 8 to 16 bytes of the tile ends' state: 12 thousand local loads for the 256 tiles of
  // 4096 x 4096 in e4m3, whether K is 1024 or 4096, so none of them in the loop over k.)
  static constexpr int kRegs = 168, kRegsEpi = 224, kRegsOther = 56;
  static_assert(256 * kRegsEpi + 128 * kRegsOther <= kThreads * kRegs, "register split");
  static constexpr int kTileM = PAIR ? 256 : 128;
  static constexpr int kXBytes = 128 * kKBlockBytes;
  static constexpr int kWBytes = (PAIR ? 128 : 256) * kKBlockBytes;   // a pair's CTA holds half
  static constexpr int kStages = PAIR ? 5 : 4;
  // per epilogue warp on the way out: chunks of 32 rows of 128 bytes (64 bf16 columns, or 32 fp32)
  static constexpr int kOutChunks = PAIR ? 2 : 1, kOutBytes = 4096 * kOutChunks;
  static constexpr int kBarBytes = 256;
  static constexpr int kSmem = kStages * (kXBytes + kWBytes) + 8 * kOutBytes + kBarBytes + 2 * kTileBatch * 16 + kScheduleBytes;
  static_assert((2 * kStages + 12) * 8 + 8 <= kBarBytes, "barriers");
  static_assert(kSmem <= 232448, "shared memory");
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
__device__ __forceinline__ void fma2(f32x2& c, f32x2 a, f32x2 b) {
  asm volatile("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t bf16_pair(f32x2 v) {
  const float2 f = split_of(v);
  return bf16_pair(f.x, f.y);
}
__device__ __forceinline__ void load_pairs(const float* p, f32x2& a, f32x2& b) {
  asm volatile("ld.global.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "l"(p));
}
// the first `left` of a 16-byte unit's PER elements
template <int PER, typename E>
__device__ __forceinline__ void store_unit(E* to, uint4 v, int left) {
  if (left >= PER) {
    *reinterpret_cast<uint4*>(to) = v;
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (j < left) to[j] = PER == 8 ? static_cast<E>(w[j >> 1] >> (16 * (j & 1))) : static_cast<E>(w[j & 3]);
  }
}
__device__ __forceinline__ uint4 unit_of(f32x2 a, f32x2 b) {
  const float2 u = split_of(a), v = split_of(b);
  return make_uint4(__float_as_uint(u.x), __float_as_uint(u.y), __float_as_uint(v.x), __float_as_uint(v.y));
}
// four columns from n of a row of y (element `at`): the bias, the clamp, the one rounding
__device__ __forceinline__ void finish4(const LinearParams& p, long long at, int n, float4 v, const float (&b)[4]) {
  float f[4] = {v.x + b[0], v.y + b[1], v.z + b[2], v.w + b[3]};
  if (p.clamp) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = act_clamp(f[j], p.lo, p.hi);
  }
  if (p.vec_y && n + 4 <= p.N) {
    if (p.out_bf16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + at) = make_uint2(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) = make_float4(f[0], f[1], f[2], f[3]);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (n + j < p.N) {
      if (p.out_bf16)
        static_cast<__nv_bfloat16*>(p.y)[at + j] = __float2bfloat16_rn(f[j]);
      else
        static_cast<float*>(p.y)[at + j] = f[j];
    }
}
// PLAIN: rows of y begin on 16 bytes, and nothing is done to the sums but a bias that can be read as 16
// bytes and the clamp of bf16 results.  The other cases have a kernel of their own:
// their code's registers had the compiler keep the halves of the sums' pairs apart, and every multiply-
// add of the loop then cost two (800 instead of 600 cycles per k-block).
template <bool F8, bool PAIR, bool PLAIN>
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
  uint64_t* tqfull = tempty + 4;    // a batch of tiles is worked out
  uint64_t* tqempty = tqfull + 2;   // and read by the loads' warp and the epilogue's
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tqempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  LinearTile* tileq = reinterpret_cast<LinearTile*>(reinterpret_cast<uint8_t*>(full) + Cfg::kBarBytes);
  int* prefix = reinterpret_cast<int*>(tileq + 2 * kTileBatch);

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
      mbar_init(&tempty[b], PAIR ? 8 : 4);   // the epilogue warps of a half, of both CTAs
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tqfull[b], 1);
      mbar_init(&tqempty[b], 9);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 9) {
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
  if (warp == 8) build_schedule(p, Cfg::kTileM, prefix, blockIdx.x == 0);
  __syncthreads();

  const long long tiles = tile_count(p, prefix);
  const long long t0 = PAIR ? blockIdx.x >> 1 : blockIdx.x, tstep = PAIR ? gridDim.x >> 1 : gridDim.x;
  const long long mine = tiles > t0 ? (tiles - t0 - 1) / tstep + 1 : 0;   // tiles of this CTA
  // this CTA's j-th tile, read by one thread (the loads') or a warp in the order of j; false: give up
  auto next_tile = [&](long long j, LinearTile& q, bool whole_warp) {
    const int slot = static_cast<int>(j / kTileBatch) & 1, at = static_cast<int>(j % kTileBatch);
    if (at == 0 && !mbar_wait(&tqfull[slot], static_cast<uint32_t>(j / (2 * kTileBatch)) & 1, abort_flag, p.status)) return false;
    q = tileq[slot * kTileBatch + at];
    if (at == kTileBatch - 1) {
      if (whole_warp) __syncwarp();
      if (!whole_warp || lane == 0) mbar_arrive(&tqempty[slot]);
    }
    return true;
  };

  // every earlier MMA of this thread has completed -> an arrival on `bar`, of a pair in both CTAs
  auto commit_to = [&](uint64_t* bar) {
    if (PAIR)
      tc_commit_pair(bar, 3);
    else
      tc_commit(bar);
  };
  if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsOther));
  if (warp == 8) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (long long j = 0; j < mine; ++j) {
        LinearTile q;
        if (!next_tile(j, q, false)) goto teardown;
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
    }
  } else if (warp == 9) {
    if (leader) {
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
  } else if (warp == 10) {
    for (long long j = 0; j < mine; j += kTileBatch) {
      const int slot = static_cast<int>(j / kTileBatch) & 1;
      if (!mbar_wait(&tqempty[slot], (static_cast<uint32_t>(j / (2 * kTileBatch)) & 1) ^ 1, abort_flag, p.status)) goto teardown;
      if (lane < kTileBatch && j + lane < mine)
        tileq[slot * kTileBatch + lane] = tile_at<Cfg::kTileM, kManyCols>(p, prefix, t0 + (j + lane) * tstep);
      __syncwarp();
      if (lane == 0) mbar_arrive(&tqfull[slot]);
    }
  } else if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsEpi));
    const int quad = warp & 3, half = warp >> 2;
    const int mrow = crank * 128 + quad * 32;   // this warp's first row of the tile
    const uint32_t from0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + half * 128;
    int buf = half;
    uint32_t bphase = 0;
    bool ready = false;
    // the scales are loaded a k-block ahead (and multiplied when they are used: a product at the load would
    // wait for it); rows and columns past the edge read the last scale there is, and their sums are not
    // stored
    const float *xs = nullptr, *ws = nullptr;
    float x1 = 1.f, w1 = 1.f;
    const int nblk = (p.N + kScaleBlock - 1) / kScaleBlock;
    auto first_scales = [&](const LinearTile& q) {
      if (!F8) return;
      xs = p.x_scale + (q.row0 + min(mrow + lane, q.rows - 1)) * p.xs_row;
      ws = p.w_scale + (static_cast<long long>(q.e) * nblk + min(q.n0 / kScaleBlock + half, nblk - 1)) * p.num_kb;
      x1 = *xs;
      w1 = *ws;
    };
    LinearTile q, qn;
    if (mine > 0) {
      if (!next_tile(0, qn, true)) goto teardown;
      first_scales(qn);
    }
    for (long long j = 0; j < mine; ++j) {
      q = qn;
      const int n0 = q.n0 + half * 128;   // this warp's first column
      const float* bias = p.bias ? p.bias + static_cast<long long>(q.e) * p.N : nullptr;
      f32x2 acc[64];
#pragma unroll
      for (int c = 0; c < 64; ++c) acc[c] = 0;
      if (PLAIN && bias) {   // the sums begin with it
#pragma unroll
        for (int c = 0; c < 64; c += 2)
          if (n0 + 2 * c < p.N) load_pairs(bias + n0 + 2 * c, acc[c], acc[c + 1]);
      }
#pragma unroll 1
      for (int kb = 0; kb < p.num_kb; kb += F8 ? 1 : p.chunk_kb) {
        if (!ready && !mbar_wait(&tfull[buf], bphase, abort_flag, p.status)) goto teardown;
        tc_fence_after();
        const uint32_t from = from0 + (buf & 2) * 128;
        f32x2 r[32];
        tmem_ld_64_wait(from, r);
        const float both = x1 * w1;
        const f32x2 s = pair_of(__float_as_uint(both), __float_as_uint(both));
#pragma unroll
        for (int i = 0; i < 32; ++i) fma2(acc[i], r[i], s);
        tmem_ld_64_wait(from + 64, r);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR)
            mbar_arrive_remote_relaxed(map_to_rank(smem_u32(&tempty[buf]), 0));
          else
            mbar_arrive(&tempty[buf]);
        }
        buf ^= 2;
        if (buf == half) bphase ^= 1;
        // (here and not before the sums: there the kernel of pairs without PLAIN spilled, 101 us instead of 93
        // for 4096 x 4097 x 4096)
        if (F8 && kb + 1 < p.num_kb) {
          xs += p.xs_blk;
          ++ws;
          x1 = *xs;
          w1 = *ws;
        }
        // asked before the last sums, so that the answer is not waited for
        ready = mbar_test_wait(&tfull[buf], bphase);
#pragma unroll
        for (int i = 0; i < 32; ++i) fma2(acc[32 + i], r[i], s);
      }
      if (j + 1 < mine) {
        if (!next_tile(j + 1, qn, true)) goto teardown;
        first_scales(qn);
      }
      if (mrow >= q.rows || n0 >= p.N) continue;
      uint8_t* out = sOut + warp * Cfg::kOutBytes;
      // Whole warps' rows leave by TMA while the next tile's sums begin: the stores of all SMs at once, waited
      // for, cost 4700 cycles a tile.  (A TMA store clips the columns past N by units of 16 bytes and would
      // write over what follows rows that end inside one.)  bf16 results are clamped after
      // the rounding, which is monotonic: the bounds, rounded, give the same values, and the sums' pairs
      // stay whole.
      const uint32_t lo = bf16_pair(p.lo, p.lo), hi = bf16_pair(p.hi, p.hi);
      auto bf16_unit = [&](int u) {   // 8 columns
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] = bf16_pair(acc[4 * u + i]);
          if (p.clamp) asm("max.NaN.bf16x2 %0, %0, %1;\n\tmin.NaN.bf16x2 %0, %0, %2;" : "+r"(w[i]) : "r"(lo), "r"(hi));
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
      };
      if (PLAIN && mrow + 32 <= q.rows && (p.whole_units || n0 + 128 <= p.N)) {
        auto chunk_unit = [&](int c, int u) {
          return reinterpret_cast<uint4*>(out + (c % Cfg::kOutChunks) * 4096 + lane * 128 + ((u ^ (lane & 7)) << 4));
        };
        auto room = [&] {   // the chunk's place has been read by the store before
          if (lane == 0) bulk_wait_read<Cfg::kOutChunks - 1>();
          __syncwarp();
        };
        auto send = [&](int c, int n) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (n < p.N) tma_store_2d(&tmY, out + (c % Cfg::kOutChunks) * 4096, n, q.row0 + mrow);
            bulk_commit();
          }
        };
        if (p.out_bf16) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            room();
#pragma unroll
            for (int u = 0; u < 8; ++u) *chunk_unit(c, u) = bf16_unit(8 * c + u);
            send(c, n0 + 64 * c);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            room();
#pragma unroll
            for (int u = 0; u < 8; ++u) *chunk_unit(c, u) = unit_of(acc[16 * c + 2 * u], acc[16 * c + 2 * u + 1]);
            send(c, n0 + 32 * c);
          }
        }
      } else if (PLAIN) {
        // a group's last rows, or rows that end inside 16 bytes: each lane its own row
        if (mrow + lane < q.rows && CONVF_IN_BOUNDS(q.row0 + mrow + lane < p.rows, p.status)) {
          const long long at = static_cast<long long>(q.row0 + mrow + lane) * p.ldy + n0;
          if (p.out_bf16) {
            uint16_t* row = static_cast<uint16_t*>(p.y) + at;
#pragma unroll
            for (int u = 0; u < 16; ++u) store_unit<8>(row + 8 * u, bf16_unit(u), p.N - n0 - 8 * u);
          } else {
            uint32_t* row = static_cast<uint32_t*>(p.y) + at;
#pragma unroll
            for (int u = 0; u < 32; ++u) store_unit<4>(row + 4 * u, unit_of(acc[2 * u], acc[2 * u + 1]), p.N - n0 - 4 * u);
          }
        }
      } else {
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
        // Unaligned rows or bias, the ragged edge of N, clamped fp32: 64 columns at a time through shared
        // memory (16-byte units swizzled by row).  A part of a sector that is written costs L2 more than a
        // whole one, so a store's lanes are adjacent columns of one row: aligned rows 4 a lane; other bf16
        // rows 2 a lane from the row's first even address; other fp32 rows one.
        constexpr int kRound = Cfg::kOutBytes / 256;   // rows staged at a time
        const int rows = min(32, q.rows - mrow);
        const long long row0 = static_cast<long long>(q.row0 + mrow) * p.ldy;
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
          const int n = n0 + 64 * pass;
          float b[4];   // of the lane's columns: 4 from 4 (lane % 16), or 3 from 2 lane, or lane and lane + 32
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = p.vec_y ? 4 * (lane & 15) + i : p.out_bf16 ? 2 * lane + i : lane + 32 * i;
            b[i] = bias ? bias[min(n + c, p.N - 1)] : 0.f;
          }
          for (int r0 = 0; r0 < rows; r0 += kRound) {
            if ((lane & ~(kRound - 1)) == r0) {
#pragma unroll
              for (int u = 0; u < 16; ++u)
                *reinterpret_cast<uint4*>(out + (lane & (kRound - 1)) * 256 + ((u ^ (lane & 7)) << 4)) =
                    unit_of(acc[32 * pass + 2 * u], acc[32 * pass + 2 * u + 1]);
            }
            __syncwarp();
            const int some = min(kRound, rows - r0);
            auto staged = [&](int r, int c) {
              return *reinterpret_cast<const float*>(out + r * 256 + (((c >> 2) ^ (r & 7)) << 4) + (c & 3) * 4);
            };
            // AS_IS: all 64 columns, nothing to add or clamp
            auto send_rows = [&](auto as_is) {
              constexpr bool AS_IS = decltype(as_is)::value;
              auto done = [&](float v, float bias_c) {
                if (AS_IS) return v;
                v += bias_c;
                return p.clamp ? act_clamp(v, p.lo, p.hi) : v;
              };
              const int left = AS_IS ? 64 : p.N - n;   // columns of the row from n
              const long long at = row0 + r0 * p.ldy + n;
              if (p.out_bf16) {
                __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.y) + at;
#pragma unroll 4
                for (int r = 0; r < some; ++r, to += p.ldy) {
                  if (!CONVF_IN_BOUNDS(q.row0 + mrow + r0 + r < p.rows, p.status)) continue;
                  if ((reinterpret_cast<uintptr_t>(to) & 2) == 0) {
                    const float2 v = *reinterpret_cast<const float2*>(out + r * 256 + (((lane >> 1) ^ (r & 7)) << 4) + (lane & 1) * 8);
                    if (2 * lane + 1 < left)
                      *reinterpret_cast<uint32_t*>(to + 2 * lane) = bf16_pair(done(v.x, b[0]), done(v.y, b[1]));
                    else if (2 * lane < left)
                      to[2 * lane] = __float2bfloat16_rn(done(v.x, b[0]));
                  } else {
                    // an even address is at column 1: pairs from there, and the first and last column alone
                    const int c = 2 * lane + 1;
                    const float v0 = done(staged(r, c), b[1]), v1 = done(staged(r, min(c + 1, 63)), b[2]);
                    if (c + 1 < min(left, 64))
                      *reinterpret_cast<uint32_t*>(to + c) = bf16_pair(v0, v1);
                    else if (c < left)
                      to[c] = __float2bfloat16_rn(v0);
                    if (lane == 0 && left > 0) to[0] = __float2bfloat16_rn(done(staged(r, 0), b[0]));
                  }
                }
              } else {
                float* to = static_cast<float*>(p.y) + at;
#pragma unroll 4
                for (int r = 0; r < some; ++r, to += p.ldy) {
                  if (!CONVF_IN_BOUNDS(q.row0 + mrow + r0 + r < p.rows, p.status)) continue;
                  if (lane < left) to[lane] = done(staged(r, lane), b[0]);
                  if (lane + 32 < left) to[lane + 32] = done(staged(r, lane + 32), b[1]);
                }
              }
            };
            if (p.vec_y) {
              const int n4 = n + 4 * (lane & 15);
#pragma unroll 4
              for (int r = lane >> 4; r < some; r += 2) {
                const float4 v = *reinterpret_cast<const float4*>(out + r * 256 + (((lane & 15) ^ (r & 7)) << 4));
                if (n4 < p.N && CONVF_IN_BOUNDS(q.row0 + mrow + r0 + r < p.rows, p.status))
                  finish4(p, row0 + (r0 + r) * p.ldy + n4, n4, v, b);
              }
            } else if (!bias && !p.clamp && n + 64 <= p.N) {
              send_rows(std::true_type{});
            } else {
              send_rows(std::false_type{});
            }
            __syncwarp();
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
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem_base, kTmemCols);
    else
      tmem_dealloc(tmem_base, kTmemCols);
  }
}

template <bool F8, bool PAIR, bool PLAIN>
cudaError_t launch_t(const LinearParams& p, const LinearPlan& plan, const CUtensorMap& tmW, const CUtensorMap& tmX,
                     const CUtensorMap& tmY, cudaStream_t stream) {
  using Cfg = ManyCfg<PAIR>;
  static OncePerDevice once;
  const cudaError_t e = once([] {
    // the register split waits for ever if the kernel was given fewer registers than it shares out
    cudaFuncAttributes at;
    const cudaError_t got = cudaFuncGetAttributes(&at, linear_many_kernel<F8, PAIR, PLAIN>);
    if (got != cudaSuccess) return got;
    if (at.numRegs < Cfg::kRegs) return cudaErrorInvalidKernelImage;
    return cudaFuncSetAttribute(linear_many_kernel<F8, PAIR, PLAIN>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(linear_many_kernel<F8, PAIR, PLAIN>, dim3(plan.grid), dim3(Cfg::kThreads), Cfg::kSmem, stream, PAIR ? 2 : 1, p,
                    tmW, tmX, tmY);
}

}  // namespace

cudaError_t launch_linear_many(const LinearParams& p, const LinearPlan& plan, bool e4m3, const CUtensorMap& tmW,
                               const CUtensorMap& tmX, const CUtensorMap& tmY, cudaStream_t stream) {
  // (16-byte bias loads: every expert's bias begins on 16 bytes)
  const bool bias_ok = !p.bias || ((reinterpret_cast<uintptr_t>(p.bias) & 15) == 0 && p.N % 4 == 0);
  const bool plain = p.vec_y && bias_ok && (p.out_bf16 || !p.clamp);
  auto go = [&](auto f8, auto pair) {
    constexpr bool F8 = decltype(f8)::value, PAIR = decltype(pair)::value;
    return plain ? launch_t<F8, PAIR, true>(p, plan, tmW, tmX, tmY, stream) : launch_t<F8, PAIR, false>(p, plan, tmW, tmX, tmY, stream);
  };
  const std::true_type yes;
  const std::false_type no;
  if (plan.tile == 256) return e4m3 ? go(yes, yes) : go(no, yes);
  return e4m3 ? go(yes, no) : go(no, no);
}

}  // namespace convf
