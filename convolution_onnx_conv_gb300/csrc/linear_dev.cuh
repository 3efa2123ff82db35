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

// tcgen05.wait::ld that the uses of r cannot be moved above
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// the clamp of an activation that keeps a NaN
__device__ __forceinline__ float act_clamp(float v, float lo, float hi) { return v < lo ? lo : (v > hi ? hi : v); }

}  // namespace convf
