// Device-side parts shared by the linear kernels: the tile schedule over ragged row groups, the
// e4m3 MMA, and the last step of an output element.
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

// The rows of x that expert e takes: [first, last), inside [0, rows) whatever the offsets hold.
struct RowGroup {
  int first, last;
};
__device__ __forceinline__ RowGroup row_group(const LinearParams& p, int e) {
  if (!p.offsets) return RowGroup{0, p.rows};
  const int a = min(max(__ldg(p.offsets + e), 0), p.rows);
  const int b = min(max(__ldg(p.offsets + e + 1), a), p.rows);
  return RowGroup{a, b};
}

// Tiles of `tile` rows over the experts: prefix[e] = row tiles of the experts before e.  One warp;
// block_lead tells the CTA that reports offsets that decrease or pass the rows.
__device__ __forceinline__ void build_schedule(const LinearParams& p, int tile, int* prefix, bool block_lead) {
  const int lane = threadIdx.x & 31;
  int sum = 0;
  bool bad = false;
  for (int base = 0; base < p.experts; base += 32) {
    const int e = base + lane;
    int n = 0;
    if (e < p.experts) {
      const RowGroup g = row_group(p, e);
      n = (g.last - g.first + tile - 1) / tile;
      if (block_lead && p.offsets) {
        const int a = __ldg(p.offsets + e), b = __ldg(p.offsets + e + 1);
        bad = bad || a < 0 || b < a || b > p.rows;
      }
    }
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += t;
    }
    if (e < p.experts) prefix[e] = sum + incl - n;
    sum += __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
  if (lane == 0) prefix[p.experts] = sum;
  if (bad) atomicOr(p.status, kStatusOffsets);
}

// One output tile: `rows` rows of x from row0, weight rows from n0, of an expert.
struct LinearTile {
  int e, row0, rows, n0;
};
// Tile t of prefix[experts] * n_tiles.  Within an expert the row tiles run fastest, in groups of
// kRasterRows: the CTAs of a wave share weight tiles (each is then read from memory once, and again
// from L2), and a long prompt's rows are not all passed over once per weight tile.
constexpr int kRasterRows = 8;
template <int TILE, int NTILE>
__device__ __forceinline__ LinearTile tile_at(const LinearParams& p, const int* prefix, long long t) {
  int lo = 0, hi = p.experts;   // the last expert whose tiles start at or before t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (static_cast<long long>(prefix[mid]) * p.n_tiles <= t)
      lo = mid;
    else
      hi = mid;
  }
  const int mt = prefix[lo + 1] - prefix[lo];
  const long long local = t - static_cast<long long>(prefix[lo]) * p.n_tiles;
  const int group = static_cast<int>(local / (static_cast<long long>(kRasterRows) * p.n_tiles));
  const int in_group = static_cast<int>(local - static_cast<long long>(group) * kRasterRows * p.n_tiles);
  const int height = min(kRasterRows, mt - group * kRasterRows);
  const int nt = in_group / height, m = group * kRasterRows + in_group - nt * height;
  const RowGroup g = row_group(p, lo);
  LinearTile r;
  r.e = lo;
  r.row0 = g.first + m * TILE;
  r.rows = min(TILE, g.last - r.row0);
  r.n0 = nt * NTILE;
  return r;
}

// 32 lanes x 64 consecutive 32-bit columns, and the wait for them in the same statement (the values
// cannot be used before it)
__device__ __forceinline__ void tmem_ld_32x32b_x64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]),
        "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]),
        "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]),
        "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
        "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
}

// the clamp of an activation that keeps a NaN
__device__ __forceinline__ float act_clamp(float v, float lo, float hi) { return v < lo ? lo : (v > hi ? hi : v); }

}  // namespace convf
