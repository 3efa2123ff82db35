// Linear layers on int8 operands, exact: y^T = W x^T with integer sums, on tcgen05.
//
// sm_103a's tcgen05.mma has no integer kind, and its warp-level int8 MMA reaches a twelfth of the fp16 rate.  An
// int8 value is an fp16 number, the product of two is below 2^14 and fp32 holds every integer up to 2^24: fp16
// MMAs add kChunk products exactly, and the chunks' sums are added as int32 in registers.  So every sum is the
// integer, whatever the order, and all forms give the same bits.
//
// The bytes stay int8 up to shared memory (TMA); four warps make fp16 of them: a byte in the low bits of an fp16
// number 1024 + .. and a subtraction, 5 instructions for 4 values.  The weights are the MMA's 128 rows and go to
// TMEM, from where the MMA reads its first operand, and not back to shared memory, whose bandwidth is the scarce
// thing (reading 1 byte, writing 2 and the MMA reading those is 5 bytes a value); the rows of x are its columns and
// go back to shared memory.  Values keep no order within four of them: both operands are permuted alike.
//
// Few rows: 16, 32 or 64 columns a tile, and clusters that share a tile's reduction, as in tc_linear_few.cu; the
// partial sums are integers too.  Many rows: 256 weight rows x 192 columns on CTA pairs: each CTA converts 128
// weight rows and 96 rows of x for 384 cycles of MMAs per 64 values; two accumulators of 192 columns and four
// units of weights fill TMEM.
//
//   warp 0      TMA: weight and x tiles of 128 values
//   warp 1      TMEM, MMA issue (of a pair: the leader's)
//   warp 2      the tile schedule
//   warps 4-7   int8 -> fp16, units of 64 values
//   warps 8-..  epilogue: 4 warps, 8 where each takes half of the columns
#include <cuda_fp16.h>

#include "linear_dev.cuh"

namespace convf {

namespace {

constexpr int kUnit = 64;        // values of a unit: an fp16 row of 128 bytes
constexpr int kChunk = 512;      // values that an accumulator sums: 2^23 at most
constexpr int kConvertWarps = 4;

template <int TN, bool PAIR>
struct Int8Cfg {
  static constexpr int kXRows = PAIR ? TN / 2 : TN;             // rows of x that a CTA loads and converts
  static constexpr int kEpiWarps = TN > 64 ? 8 : 4;
  static constexpr int kCols = TN > 64 ? TN / 2 : TN;           // columns per epilogue thread
  static constexpr int kThreads = 256 + 32 * kEpiWarps;
  static constexpr int kPerSm = TN <= 32 ? 2 : 1;
  static constexpr int kTmemCols = kPerSm == 2 ? 256 : 512;
  static constexpr int kWBytes = 128 * kKBlockBytes, kXBytes = kXRows * kKBlockBytes;   // of a stage, int8
  static constexpr int kBBytes = kXRows * 2 * kUnit;            // of a unit of x, fp16
  static constexpr int kUnitCols = kUnit / 2;                   // TMEM columns of a unit of weights
  static constexpr int kUnits = PAIR ? 4 : 6;
  static constexpr int kDCol = kUnits * kUnitCols;              // the accumulators' first column
  static constexpr int kRedBytes = TN <= 64 ? TN * 128 * 4 : 0;
  static constexpr int kBarBytes = 512;
  static constexpr int kFixed = 1024 + kUnits * kBBytes + kRedBytes + kScheduleBytes + kBarBytes;
  static constexpr int kBudget = kPerSm == 2 ? 115712 : 232448;
  static constexpr int kStages = (kBudget - kFixed) / (kWBytes + kXBytes);
  static constexpr int kSmem = kFixed + kStages * (kWBytes + kXBytes);
  // registers of a pair's kernel: the epilogue's two warpgroups take what the other two give up
  static constexpr int kRegs = 128, kRegsEpi = 168, kRegsConvert = 96, kRegsOther = 72;
  static_assert(256 * kRegsEpi + 128 * (kRegsConvert + kRegsOther) <= 512 * kRegs, "register split");
  static_assert(kStages >= 3 && (2 * kStages + 2 * kUnits + 6) * 8 + 8 <= kBarBytes && kSmem <= kBudget, "shared memory");
  static_assert(kDCol + 2 * TN <= kTmemCols, "TMEM columns");
};

// Instruction descriptor, kind::f16 with fp16 A/B (formats 0), fp32 D, both K-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// D[tmem] (+)= A[tmem] * B[smem]^T: 16 values of k per call
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tc_mma_f16_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                   uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// mbar_test_wait for a phase that arrivals from another CTA complete
__device__ __forceinline__ bool mbar_test_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// store 32 consecutive 32-bit columns of lanes (base + i) from thread i of the warp
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// Four int8 values as fp16: {0, 2} and {1, 3}.  0x6400 | (b ^ 0x80) is 1024 + 128 + b.
__device__ __forceinline__ void f16_of_int8(uint32_t w, uint32_t& even, uint32_t& odd) {
  const __half2 bias = __half2half2(__ushort_as_half(0xE480));   // -1152
  const uint32_t e = (w & 0x00FF00FFu) ^ 0x64806480u, o = ((w >> 8) & 0x00FF00FFu) ^ 0x64806480u;
  const __half2 he = __hadd2(*reinterpret_cast<const __half2*>(&e), bias), ho = __hadd2(*reinterpret_cast<const __half2*>(&o), bias);
  even = *reinterpret_cast<const uint32_t*>(&he);
  odd = *reinterpret_cast<const uint32_t*>(&ho);
}

template <int TN, bool PAIR>
__global__ void __launch_bounds__(Int8Cfg<TN, PAIR>::kThreads, Int8Cfg<TN, PAIR>::kPerSm)
    linear_int8_kernel(const LinearParams p, const int split, const __grid_constant__ CUtensorMap tmW,
                       const __grid_constant__ CUtensorMap tmX) {
  using Cfg = Int8Cfg<TN, PAIR>;
  constexpr int kStages = Cfg::kStages, kUnits = Cfg::kUnits, kCols = Cfg::kCols;
  constexpr int kNTile = PAIR ? 256 : 128;   // weight rows of a tile
  constexpr int kChunkUnits = kChunk / kUnit;
  extern __shared__ uint8_t smem_raw[];
  // (the swizzle goes by address bits 7 to 9, and a pair's CTAs have their operands at the same offset: the
  // dynamic shared memory begins at the same address in both)
  uint8_t* sW = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sX = sW + kStages * Cfg::kWBytes;
  uint8_t* sB = sX + kStages * Cfg::kXBytes;
  int* red = reinterpret_cast<int*>(sB + kUnits * Cfg::kBBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(red) + Cfg::kRedBytes);   // int8 tiles are here
  uint64_t* empty = full + kStages;     // and have been read
  uint64_t* cfull = empty + kStages;    // a unit is converted (of a pair: the leader's, for both CTAs)
  uint64_t* cempty = cfull + kUnits;    // and its MMAs have read it
  uint64_t* tfull = cempty + kUnits;    // an accumulator holds a chunk's sums
  uint64_t* tempty = tfull + 2;         // and has been read (of a pair: the leader's)
  uint64_t* rfull = tempty + 2;         // every rank's partial sums of this CTA's columns have arrived
  uint64_t* rfree = rfull + 1;          // every rank has read what this CTA sent it
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rfree + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* prefix = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(full) + Cfg::kBarBytes);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = PAIR || split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const bool leader = !PAIR || rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kConvertWarps);
    }
    for (int u = 0; u < kUnits; ++u) {
      mbar_init(&cfull[u], kConvertWarps * (PAIR ? 2 : 1));
      mbar_init(&cempty[u], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], Cfg::kEpiWarps * (PAIR ? 2 : 1));
    }
    mbar_init(rfull, Cfg::kEpiWarps * split);
    mbar_init(rfree, Cfg::kEpiWarps * split);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(tmem_slot, Cfg::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, Cfg::kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR || split > 1) cluster_sync();   // the peers' barriers exist before anything is sent to them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int ctas = PAIR ? 2 : split;   // that share a tile
  const long long t0 = blockIdx.x / ctas, tstep = gridDim.x / ctas;
  const int ka = PAIR ? 0 : static_cast<int>(static_cast<long long>(p.num_kb) * rank / split);
  const int kb_end = PAIR ? p.num_kb : static_cast<int>(static_cast<long long>(p.num_kb) * (rank + 1) / split);
  const long long first_tiles = static_cast<long long>((p.rows + TN - 1) / TN) * p.n_tiles;
  constexpr int kPrefetch = 16;
  // after the TMEM allocation, which a dependent's CTA would otherwise take
  pdl_launch_dependents();
  // one layer: the first wave's weight tiles are known before the previous kernel has ended (see tc_linear_few.cu)
  if (!p.offsets && warp == 0 && lane == 0 && t0 < first_tiles) {
    const int n0 = static_cast<int>(t0 / ((p.rows + TN - 1) / TN)) * kNTile + (PAIR ? rank * 128 : 0);
    for (int kb = ka; kb < min(kb_end, ka + kPrefetch); ++kb) tma_prefetch_l2_3d(&tmW, kb * kKBlockBytes, n0, 0);
  }
  pdl_wait_prior();
  if (warp == 2) build_schedule(p, TN, prefix, blockIdx.x == 0);
  __syncthreads();

  const long long tiles = tile_count(p, prefix);
  const long long mine = tiles > t0 ? (tiles - t0 - 1) / tstep + 1 : 0;
  auto commit_to = [&](uint64_t* bar) {
    if (PAIR)
      tc_commit_pair(bar, 3);
    else
      tc_commit(bar);
  };

  if (warp < 4) {
    if (PAIR) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsOther));
    if (warp == 0) {
      if (lane == 0) {
        int stage = 0;
        uint32_t phase = 0;
        for (long long t = t0; t < tiles; t += tstep) {
          const LinearTile q = tile_at<TN, kNTile>(p, prefix, t);
          const int n0 = q.n0 + (PAIR ? rank * 128 : 0), row0 = q.row0 + (PAIR ? rank * Cfg::kXRows : 0);
          for (int kb = ka; kb < kb_end; ++kb) {
            if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, p.status)) goto teardown;
            mbar_arrive_expect_tx(&full[stage], Cfg::kWBytes + Cfg::kXBytes);
            tma_load_3d(sW + stage * Cfg::kWBytes, &tmW, &full[stage], kb * kKBlockBytes, n0, q.e);
            tma_load_2d(sX + stage * Cfg::kXBytes, &tmX, &full[stage], kb * kKBlockBytes, row0);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
      }
    } else if (warp == 1 && leader) {
      // the whole warp walks the loop and one lane issues: the loop's state then stays in uniform
      // registers, which is where the MMA takes its descriptors from
      const bool issue = elect_one();
      constexpr uint32_t idesc = idesc_f16_f32(kNTile, TN);
      const uint64_t b0 = sdesc_kmajor_sw128(smem_u32(sB));
      int unit = 0, buf = 0;
      uint32_t phase = 0, bphase = 0;
      for (long long j = 0; j < mine; ++j) {
        const int units = 2 * (kb_end - ka);
        for (int i = 0, in_chunk = 0; i < units; ++i) {
          const bool first = in_chunk == 0, last = ++in_chunk == kChunkUnits || i == units - 1;
          // both barriers are asked at once, before either is waited for
          bool ready = PAIR ? mbar_test_wait_cluster(&cfull[unit], phase) : mbar_test_wait(&cfull[unit], phase);
          if (first) ready = mbar_test_wait(&tempty[buf], bphase ^ 1) & ready;
          if (!ready) {
            if (first && !mbar_wait_cluster(&tempty[buf], bphase ^ 1, abort_flag, p.status)) goto teardown;
            if (!mbar_wait_cluster(&cfull[unit], phase, abort_flag, p.status)) goto teardown;
          }
          tc_fence_after();
          const uint32_t a = tmem_base + unit * Cfg::kUnitCols, d = tmem_base + Cfg::kDCol + buf * TN;
          const uint64_t b = b0 + unit * (Cfg::kBBytes >> 4);
          if (issue) {
#pragma unroll
            for (int s = 0; s < kUnit / 16; ++s) {   // 16 values: 8 columns of A, 32 bytes of B
              if (PAIR)
                tc_mma_f16_ts_pair(d, a + 8 * s, b + 2 * s, idesc, !first || s > 0);
              else
                tc_mma_f16_ts(d, a + 8 * s, b + 2 * s, idesc, !first || s > 0);
            }
            commit_to(&cempty[unit]);
            if (last) commit_to(&tfull[buf]);
          }
          __syncwarp();
          if (++unit == kUnits) {
            unit = 0;
            phase ^= 1;
          }
          if (last) {
            in_chunk = 0;
            buf ^= 1;
            if (buf == 0) bphase ^= 1;
          }
        }
      }
    }
  } else if (warp < 8) {
    if (PAIR) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsConvert));
    const int quad = warp & 3, id = threadIdx.x - 128;   // id: this thread's weight row
    const uint32_t a0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    int stage = 0, unit = 0;
    uint32_t phase = 0, uphase = 0;
    const long long blocks = mine * (kb_end - ka);
    for (long long k = 0; k < blocks; ++k) {
      if (!mbar_wait(&full[stage], phase, abort_flag, p.status)) goto teardown;
      const uint8_t* w = sW + stage * Cfg::kWBytes + id * kKBlockBytes;
      const uint8_t* x = sX + stage * Cfg::kXBytes;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 wv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) wv[j] = *reinterpret_cast<const uint4*>(w + (((4 * h + j) ^ (id & 7)) << 4));
        // x: 16 bytes a task, a row's four side by side in j
        constexpr int kTasks = Cfg::kXRows * 4, kPer = (kTasks + 127) / 128;
        uint4 xv[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int task = id + 128 * i, row = task % Cfg::kXRows, j = task / Cfg::kXRows;
          if (kTasks % 128 == 0 || task < kTasks)
            xv[i] = *reinterpret_cast<const uint4*>(x + row * kKBlockBytes + (((4 * h + j) ^ (row & 7)) << 4));
        }
        if (!mbar_wait(&cempty[unit], uphase ^ 1, abort_flag, p.status)) goto teardown;
        tc_fence_after();
        uint32_t f[32];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f16_of_int8(wv[j].x, f[8 * j], f[8 * j + 1]);
          f16_of_int8(wv[j].y, f[8 * j + 2], f[8 * j + 3]);
          f16_of_int8(wv[j].z, f[8 * j + 4], f[8 * j + 5]);
          f16_of_int8(wv[j].w, f[8 * j + 6], f[8 * j + 7]);
        }
        tmem_st_32x32b_x32(a0 + unit * Cfg::kUnitCols, f);
        uint8_t* b = sB + unit * Cfg::kBBytes;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int task = id + 128 * i, row = task % Cfg::kXRows, j = task / Cfg::kXRows;
          if (kTasks % 128 == 0 || task < kTasks) {
            uint4 lo, hi;
            f16_of_int8(xv[i].x, lo.x, lo.y);
            f16_of_int8(xv[i].y, lo.z, lo.w);
            f16_of_int8(xv[i].z, hi.x, hi.y);
            f16_of_int8(xv[i].w, hi.z, hi.w);
            *reinterpret_cast<uint4*>(b + row * 128 + (((2 * j) ^ (row & 7)) << 4)) = lo;
            *reinterpret_cast<uint4*>(b + row * 128 + (((2 * j + 1) ^ (row & 7)) << 4)) = hi;
          }
        }
        fence_proxy_async_smem();   // what was stored to shared memory is the MMA's to read
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR)
            mbar_arrive_remote(map_to_rank(smem_u32(&cfull[unit]), 0));
          else
            mbar_arrive(&cfull[unit]);
          if (h == 1) mbar_arrive(&empty[stage]);
        }
        if (++unit == kUnits) {
          unit = 0;
          uphase ^= 1;
        }
      }
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
  } else {
    if (PAIR) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsEpi));
    const int quad = warp & 3;
    const int c0 = (warp - 8) / 4 * kCols;   // this thread's columns
    const uint32_t from0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + Cfg::kDCol + c0;
    int buf = 0;
    uint32_t bphase = 0, rphase = 0;
    constexpr int kHeld = (kCols + 31) / 32;   // row scales that a lane holds for its warp
    for (long long t = t0; t < tiles; t += tstep) {
      const LinearTile q = tile_at<TN, kNTile>(p, prefix, t);
      const int nrow = quad * 32 + lane;   // this thread's weight row of the CTA's tile
      const int n = q.n0 + (PAIR ? rank * 128 : 0) + nrow;
      const long long en = static_cast<long long>(q.e) * p.N + n;
      const float ws = n < p.N ? p.w_scale[en] : 0.f, bias = p.bias && n < p.N ? p.bias[en] : 0.f;
      float held[kHeld];
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const int c = c0 + 32 * i + lane;
        held[i] = 32 * i + lane < kCols && c < q.rows ? p.x_scale[(q.row0 + c) * p.xs_row] : 0.f;
      }
      int acc[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[c] = 0;
#pragma unroll 1
      for (int kb = ka; kb < kb_end; kb += kChunk / kKBlockBytes) {
        if (!mbar_wait(&tfull[buf], bphase, abort_flag, p.status)) goto teardown;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(from0 + buf * TN + c, r);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[c + i] += __float2int_rn(__uint_as_float(r[i]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR)
            mbar_arrive_remote_relaxed(map_to_rank(smem_u32(&tempty[buf]), 0));
          else
            mbar_arrive(&tempty[buf]);
        }
        buf ^= 1;
        if (buf == 0) bphase ^= 1;
      }
      // c: column of the tile; xs: its row's scale
      auto put = [&](int c, int sum, float xs) {
        const float v = act_clamp(__fadd_rn(__fmul_rn(__int2float_rn(sum), __fmul_rn(xs, ws)), bias), p.lo, p.hi);
        if (!CONVF_IN_BOUNDS(q.row0 + c < p.rows && n < p.N, p.status)) return;
        const long long at = static_cast<long long>(q.row0 + c) * p.ldy + n;
        if (p.out_bf16)
          static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v);
        else
          static_cast<float*>(p.y)[at] = v;
      };
      if (PAIR || split == 1) {
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const float xs = __shfl_sync(0xFFFFFFFFu, held[c / 32], c % 32);
          if (c0 + c < q.rows && n < p.N) put(c0 + c, acc[c], xs);
        }
      } else if constexpr (TN <= 64 && !PAIR) {
        // column c is finished by rank c / per: send it there, then finish this rank's own
        const int per = TN / split;
        if (!mbar_wait_cluster(rfree, rphase ^ 1, abort_flag, p.status)) goto teardown;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const int to = c / per;
          if (c < q.rows)
            st_cluster_f32(map_to_rank(smem_u32(red + (rank * per + c - to * per) * 128 + nrow), to), __int_as_float(acc[c]));
        }
        asm volatile("fence.acq_rel.cluster;" ::: "memory");
        __syncwarp();
        if (lane < split) mbar_arrive_remote(map_to_rank(smem_u32(rfull), lane));
        if (!mbar_wait_cluster(rfull, rphase, abort_flag, p.status)) goto teardown;
        const int own = min(per, q.rows - rank * per);
        for (int j = 0; j < own; ++j) {
          int sum = 0;
          for (int s = 0; s < split; ++s) sum += red[(s * per + j) * 128 + nrow];
          const int c = rank * per + j;
          float xs = held[0];
          if (kHeld > 1 && c >= 32) xs = held[kHeld - 1];
          xs = __shfl_sync(0xFFFFFFFFu, xs, c & 31);
          if (n < p.N) put(c, sum, xs);
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
  if (PAIR || split > 1) cluster_sync();   // no CTA leaves while a peer may still write to it or signal it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem_base, Cfg::kTmemCols);
    else
      tmem_dealloc(tmem_base, Cfg::kTmemCols);
  }
}

template <int TN, bool PAIR>
cudaError_t configure() {
  static OncePerDevice once;
  return once([] {
    if (PAIR) {
      // the register split waits for ever if the kernel was given fewer registers than it shares out
      cudaFuncAttributes at;
      const cudaError_t got = cudaFuncGetAttributes(&at, linear_int8_kernel<TN, PAIR>);
      if (got != cudaSuccess) return got;
      if (at.numRegs < Int8Cfg<TN, PAIR>::kRegs) return cudaErrorInvalidKernelImage;
    }
    return cudaFuncSetAttribute(linear_int8_kernel<TN, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Int8Cfg<TN, PAIR>::kSmem);
  });
}

template <int TN, bool PAIR>
cudaError_t launch_t(const LinearParams& p, const LinearPlan& plan, const CUtensorMap& tmW, const CUtensorMap& tmX,
                     cudaStream_t stream) {
  const cudaError_t e = configure<TN, PAIR>();
  if (e != cudaSuccess) return e;
  return launch_pdl(linear_int8_kernel<TN, PAIR>, dim3(plan.grid), dim3(Int8Cfg<TN, PAIR>::kThreads), Int8Cfg<TN, PAIR>::kSmem,
                    stream, PAIR ? 2 : plan.split, p, plan.split, tmW, tmX);
}

template <int TN>
int max_clusters_t(int split, int num_sms) {
  if (split == 1) return num_sms * Int8Cfg<TN, false>::kPerSm;
  if (configure<TN, false>() != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(split);
  cfg.blockDim = dim3(Int8Cfg<TN, false>::kThreads);
  cfg.dynamicSmemBytes = Int8Cfg<TN, false>::kSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  return cudaOccupancyMaxActiveClusters(&n, linear_int8_kernel<TN, false>, &cfg) == cudaSuccess ? n : 0;
}

}  // namespace

cudaError_t launch_linear_int8(const LinearParams& p, const LinearPlan& plan, const CUtensorMap& tmW, const CUtensorMap& tmX,
                               cudaStream_t stream) {
  switch (plan.tile) {
    case 16: return launch_t<16, false>(p, plan, tmW, tmX, stream);
    case 32: return launch_t<32, false>(p, plan, tmW, tmX, stream);
    case 64: return launch_t<64, false>(p, plan, tmW, tmX, stream);
    case kInt8PairRows: return launch_t<kInt8PairRows, true>(p, plan, tmW, tmX, stream);
  }
  return cudaErrorInvalidValue;
}

int linear_int8_max_clusters(int tile, int split, int num_sms) {
  switch (tile) {
    case 16: return max_clusters_t<16>(split, num_sms);
    case 32: return max_clusters_t<32>(split, num_sms);
    case 64: return max_clusters_t<64>(split, num_sms);
  }
  return 0;
}

}  // namespace convf
