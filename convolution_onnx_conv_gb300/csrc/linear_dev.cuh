// Device-side parts shared by the linear kernels: the tile schedule over ragged row groups, the
// e4m3 MMA, and the last step of an output element.
//
// The linear kernels read offsets, scales and biases as ordinary loads after pdl_wait_prior(): the kernel
// before may write them, and still runs when these begin.  Read-only loads (ld.global.nc) ask for data that
// nothing writes while the kernel runs: the compiler may take them above the wait, and L1 may hold lines
// from before it.
#pragma once
#include <cuda_bf16.h>

#include "convf_internal.h"
#include "linear_internal.h"
#include "ptx.cuh"

namespace convf {

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 inputs, fp32 accumulator, one CTA; 32 values of k per call.
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tc_mma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor, kind::f8f6f4 with e4m3 A/B (formats 0), fp32 D, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// true in one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// whether phase `parity` of `bar` has completed, without waiting
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Wait for a phase that arrivals from other CTAs of the cluster complete (their writes to this CTA's
// shared memory are visible after it); bounded as mbar_wait is.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  const uint32_t a = smem_u32(bar);
  const long long t0 = clock64();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(a), "r"(parity)
        : "memory");
    if (ok) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > kWatchdogCycles) {
      *abort_flag = 1;
      if (status) atomicOr(status, kStatusTimeout);
      return false;
    }
  }
}

// Arrive on another CTA's mbarrier without publishing this thread's memory accesses: for handing
// back a TMEM buffer, whose reads tcgen05.wait::ld has completed.  (A release at cluster scope first
// waits for every load and store in flight, the scales' prefetch among them: 2400 cycles per k-block
// instead of 600.)
__device__ __forceinline__ void mbar_arrive_remote_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__device__ __forceinline__ void st_cluster_f32(uint32_t cluster_addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}

// The rows of x that expert e takes: [first, last).  (Read where there are tiles, that is, where build_schedule
// has found the offsets in order.)
struct RowGroup {
  int first, last;
};
__device__ __forceinline__ RowGroup row_group(const LinearParams& p, int e) {
  if (!p.offsets) return RowGroup{0, p.rows};
  return RowGroup{p.offsets[e], p.offsets[e + 1]};
}

// Tiles of `tile` rows over the experts: prefix[i] = row tiles of the experts before the i-th pair of them
// (a prefix for each expert would not leave the room that the stages need).  One warp.  Offsets that
// decrease or pass the rows give no tiles at all (the tiles of such groups can be more than an int counts);
// block_lead tells the CTA that reports them.
__device__ __forceinline__ int expert_pairs(const LinearParams& p) { return (p.experts + 1) >> 1; }
__device__ __forceinline__ void build_schedule(const LinearParams& p, int tile, int* prefix, bool block_lead) {
  const int lane = threadIdx.x & 31, pairs = expert_pairs(p);
  uint32_t sum = 0;
  bool bad = false;
  for (int base = 0; base < pairs; base += 32) {
    const int i = base + lane;
    uint32_t n = 0;
    for (int e = 2 * i; e < min(2 * i + 2, p.experts); ++e) {
      const RowGroup g = row_group(p, e);
      if (g.first < 0 || g.last < g.first || g.last > p.rows)
        bad = true;
      else
        n += (g.last - g.first + tile - 1) / tile;
    }
    uint32_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += t;
    }
    if (i < pairs) prefix[i] = static_cast<int>(sum + incl - n);
    sum += __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
  bad = __any_sync(0xFFFFFFFFu, bad);
  if (lane == 0) {
    prefix[pairs] = bad ? 0 : static_cast<int>(sum);
    if (bad && block_lead) atomicOr(p.status, kStatusOffsets);
  }
}
constexpr int kScheduleBytes = (kMaxExperts / 2 + 4) * 4;   // of prefix

// One output tile: `rows` rows of x from row0, weight rows from n0, of an expert.
struct LinearTile {
  int e, row0, rows, n0;
};
__device__ __forceinline__ long long tile_count(const LinearParams& p, const int* prefix) {
  return static_cast<long long>(prefix[expert_pairs(p)]) * p.n_tiles;
}
// Tile t of tile_count.  Within an expert the row tiles run fastest, in groups of kRasterRows: the CTAs
// of a wave share weight tiles (each is then read from memory once, and again from L2), and a long
// prompt's rows are not all passed over once per weight tile.
constexpr int kRasterRows = 8;
template <int TILE, int NTILE>
__device__ __forceinline__ LinearTile tile_at(const LinearParams& p, const int* prefix, long long t) {
  int lo = 0, hi = expert_pairs(p);   // the last pair whose tiles start at or before t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (static_cast<long long>(prefix[mid]) * p.n_tiles <= t)
      lo = mid;
    else
      hi = mid;
  }
  long long local = t - static_cast<long long>(prefix[lo]) * p.n_tiles;
  LinearTile r;
  r.e = 2 * lo;
  RowGroup g = row_group(p, r.e);
  int mt = (g.last - g.first + TILE - 1) / TILE;
  if (local >= static_cast<long long>(mt) * p.n_tiles) {
    local -= static_cast<long long>(mt) * p.n_tiles;
    g = row_group(p, ++r.e);
    mt = (g.last - g.first + TILE - 1) / TILE;
  }
  const int group = static_cast<int>(local / (static_cast<long long>(kRasterRows) * p.n_tiles));
  const int in_group = static_cast<int>(local - static_cast<long long>(group) * kRasterRows * p.n_tiles);
  const int height = min(kRasterRows, mt - group * kRasterRows);
  const int nt = in_group / height, m = group * kRasterRows + in_group - nt * height;
  r.row0 = g.first + m * TILE;
  r.rows = min(TILE, g.last - r.row0);
  r.n0 = nt * NTILE;
  return r;
}

// 32 lanes x 64 consecutive 32-bit columns as register pairs, and the wait for them in the same
// statement (the values cannot be used before it).  (Loaded as 64 registers and paired outside of it,
// the pairs cost the compiler a move per register.)
__device__ __forceinline__ void tmem_ld_64_wait(uint32_t taddr, unsigned long long (&r)[32]) {
  asm volatile(
      "{\n\t.reg .b32 t<64>;\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{t0, t1, t2, t3, t4, t5, t6, t7, t8, t9, t10, t11, t12, t13, t14, t15, t16, t17, t18, t19, t20, t21, t22, t23, t24, t25, t26, t27, t28, t29, t30, t31, t32, t33, t34, t35, t36, t37, t38, t39, t40, t41, t42, t43, t44, t45, t46, t47, t48, t49, t50, t51, t52, t53, t54, t55, t56, t57, t58, t59, t60, t61, t62, t63}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n\t"
      "mov.b64 %0, {t0, t1};\n\t"
      "mov.b64 %1, {t2, t3};\n\t"
      "mov.b64 %2, {t4, t5};\n\t"
      "mov.b64 %3, {t6, t7};\n\t"
      "mov.b64 %4, {t8, t9};\n\t"
      "mov.b64 %5, {t10, t11};\n\t"
      "mov.b64 %6, {t12, t13};\n\t"
      "mov.b64 %7, {t14, t15};\n\t"
      "mov.b64 %8, {t16, t17};\n\t"
      "mov.b64 %9, {t18, t19};\n\t"
      "mov.b64 %10, {t20, t21};\n\t"
      "mov.b64 %11, {t22, t23};\n\t"
      "mov.b64 %12, {t24, t25};\n\t"
      "mov.b64 %13, {t26, t27};\n\t"
      "mov.b64 %14, {t28, t29};\n\t"
      "mov.b64 %15, {t30, t31};\n\t"
      "mov.b64 %16, {t32, t33};\n\t"
      "mov.b64 %17, {t34, t35};\n\t"
      "mov.b64 %18, {t36, t37};\n\t"
      "mov.b64 %19, {t38, t39};\n\t"
      "mov.b64 %20, {t40, t41};\n\t"
      "mov.b64 %21, {t42, t43};\n\t"
      "mov.b64 %22, {t44, t45};\n\t"
      "mov.b64 %23, {t46, t47};\n\t"
      "mov.b64 %24, {t48, t49};\n\t"
      "mov.b64 %25, {t50, t51};\n\t"
      "mov.b64 %26, {t52, t53};\n\t"
      "mov.b64 %27, {t54, t55};\n\t"
      "mov.b64 %28, {t56, t57};\n\t"
      "mov.b64 %29, {t58, t59};\n\t"
      "mov.b64 %30, {t60, t61};\n\t"
      "mov.b64 %31, {t62, t63};\n\t"
      "}"
      : "=l"(r[0]), "=l"(r[1]), "=l"(r[2]), "=l"(r[3]), "=l"(r[4]), "=l"(r[5]), "=l"(r[6]), "=l"(r[7]),
        "=l"(r[8]), "=l"(r[9]), "=l"(r[10]), "=l"(r[11]), "=l"(r[12]), "=l"(r[13]), "=l"(r[14]),
        "=l"(r[15]), "=l"(r[16]), "=l"(r[17]), "=l"(r[18]), "=l"(r[19]), "=l"(r[20]), "=l"(r[21]),
        "=l"(r[22]), "=l"(r[23]), "=l"(r[24]), "=l"(r[25]), "=l"(r[26]), "=l"(r[27]), "=l"(r[28]),
        "=l"(r[29]), "=l"(r[30]), "=l"(r[31])
      : "r"(taddr)
      : "memory");
}

// the clamp of an activation that keeps a NaN
__device__ __forceinline__ float act_clamp(float v, float lo, float hi) { return v < lo ? lo : (v > hi ? hi : v); }

}  // namespace convf
