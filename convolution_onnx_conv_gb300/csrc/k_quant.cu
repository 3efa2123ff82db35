// Quantising to e4m3 with a float scale per block: s = max|v| / 448, q = e4m3(v / s).
//
// Bound by the bytes: x once in, one byte per value and a scale per block out.  Rows that begin on 8, 16 or
// 32 bytes are read as vectors, others element by element with the lanes side by side.
//
// The definition's quotient is the float32 one, rounded again to e4m3.  A division per value made the
// kernel execute 34 instructions per value and bound it by those; here the block's scale has its
// reciprocal taken once, and each value a product and one correction by its remainder: 9 to 11
// instructions per value, more than half of them per block.  100352 x 256 fp32: 20.8 us, 6.2 TB/s; bf16,
// with half the bytes per value, is bound by the instructions: 8192 x 2048 gated 17.4 us (calls one behind
// another; 20.3 and 15.3 from a graph).
#include <type_traits>

#include "convf_internal.h"
#include "linear_internal.h"
#include "ptx.cuh"
#include "quant_dev.cuh"

namespace convf {

namespace {

// g / (1 + exp(-g)), for negative g as g exp(g) / (1 + exp(g)): the divisor stays within [1, 2], where the
// approximate reciprocal is within an ulp (one of more than 2^126 is zero, which g = -88 would come to)
__device__ __forceinline__ float gate(float g) {
  const float e = expf(-fabsf(g));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return (g >= 0.f ? g : g * e) * r;
}

// CTAs on an SM (gated fp32 rows spill at four: 27.1 us for 8192 x 2048 instead of 24.2)
template <typename T, bool GATED>
constexpr int kRowsPerSm = GATED && sizeof(T) == 4 ? 3 : 4;

// Lanes that share a block.  What a lane does per block and not per value is most of its instructions, so a
// lane takes many values: 32 where they are held as bf16, 16 as fp32 (registers).
template <typename T, bool GATED, bool VEC>
constexpr int kLanes = VEC && !GATED && sizeof(T) == 2 ? 4 : 8;

// Scales per row: a few lanes take a block, and load the next before they work on this one.
template <typename T, bool GATED, bool VEC>
__global__ void __launch_bounds__(256, kRowsPerSm<T, GATED>) quantize_rows_kernel(const QuantParams p) {
  typedef typename RawOf<T>::type Raw;
  typedef typename std::conditional<GATED, RawF32, Raw>::type Held;   // a block's values while its scale is found
  constexpr int kL = kLanes<T, GATED, VEC>, kGroups = 256 / kL, kPairs = 8 / kL;   // kPairs: of 8 values
  pdl_launch_dependents();
  pdl_wait_prior();
  const int sub = threadIdx.x % kL;
  // position (row, block) of this lane group and its step: divisions once, not per block
  const uint32_t first = blockIdx.x * kGroups + threadIdx.x / kL, step = gridDim.x * kGroups;
  uint32_t r = first / p.nblk;
  int b = static_cast<int>(first - r * p.nblk);
  const uint32_t dr = step / p.nblk;
  const int db = static_cast<int>(step - dr * p.nblk);
  const uint32_t rows = p.rows;
  auto advance = [&] {
    r += dr;
    b += db;
    if (b >= p.nblk) {
      b -= p.nblk;
      ++r;
    }
  };
  auto column = [&](int block, int k) { return block * kScaleBlock + (VEC ? (sub * kPairs + k) * 16 : sub); };
  auto source = [&] { return r >= rows ? -1 : p.index ? p.index[r] : static_cast<int>(r); };
  Raw raw[kPairs][2], up[kPairs][2];
  auto fetch = [&](int src, int fb) {
    const bool there = src >= 0 && src < p.x_rows;
    const T* row = static_cast<const T*>(p.x) + static_cast<long long>(there ? src : 0) * p.ldx;
    const int cols = there ? p.cols : 0;
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      load_16<VEC>(row, column(fb, k), cols, p.x_align, raw[k]);
      if (GATED) load_16<VEC>(row + p.cols, column(fb, k), cols, p.x_align, up[k]);
    }
  };
  // in turn: this block's values are here, the next one's row is known, the one's after it is looked up
  uint32_t cr = r;
  int cb = b;
  fetch(source(), b);
  advance();
  int next_src = source();
  // whole warps loop together (the shuffles below name all 32 lanes): the first lane group's row decides
  while (__shfl_sync(0xFFFFFFFFu, cr < rows, 0)) {
    Held v[kPairs][2];
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      if constexpr (GATED) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float g[8], u[8];
          raw[k][h].floats(g);
          up[k][h].floats(u);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[k][h].w[i] = __float_as_uint(gate(g[i]) * u[i]);
        }
      } else {
        v[k][0] = raw[k][0];
        v[k][1] = raw[k][1];
      }
    }
    const uint32_t nr = r;
    const int nb = b;
    // (the loads before the maximum: 100352 x 256 fp32 22.0 us instead of 21.0)
    float m = max_abs(v[0]);
#pragma unroll
    for (int k = 1; k < kPairs; ++k) m = max_nan(m, max_abs(v[k]));
    fetch(next_src, nb);
    advance();
    next_src = source();
#pragma unroll
    for (int o = kL / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const BlockScale bs = scale_of(m);
    if (cr < rows) {
      if (sub == 0) p.scale[cr * p.lds + cb] = bs.s;
#pragma unroll
      for (int k = 0; k < kPairs; ++k) store_16<VEC>(p.q + cr * p.ldq, column(cb, k), p.cols, p.q_align, v[k], bs);
    }
    cr = nr;
    cb = nb;
  }
}

// Scales per 128 x 128 block: a CTA of 512 threads takes one at a time, 2 rows of 16 elements per thread,
// held in registers between the maximum and the division; the next block is on its way meanwhile.  (256
// threads of 64 elements need 120 registers, 16 warps on an SM: 1 us more.  5000 x 4100 bf16: 13.8 us, 11.4
// from a graph.)
template <typename T, bool VEC>
__global__ void __launch_bounds__(512, 2) quantize_tiles_kernel(const QuantParams p) {
  typedef typename RawOf<T>::type Raw;
  constexpr int kRows = 2, kWarps = 16;
  pdl_launch_dependents();
  pdl_wait_prior();
  __shared__ float part[2][kWarps];
  const int items = (p.rows + kScaleBlock - 1) / kScaleBlock;   // blocks of rows, times p.nblk
  const int lane_column = VEC ? (threadIdx.x & 7) * 16 : threadIdx.x & 7, row0 = threadIdx.x >> 3;
  Raw raw[kRows][2];
  // this CTA's block (rb, cb) and its step: divisions once, not per block
  int rb = static_cast<int>(blockIdx.x / p.nblk), cb = static_cast<int>(blockIdx.x - static_cast<unsigned>(rb) * p.nblk);
  const int dr = static_cast<int>(gridDim.x / p.nblk), dc = static_cast<int>(gridDim.x - static_cast<unsigned>(dr) * p.nblk);
  auto fetch = [&] {
    const long long at = static_cast<long long>(rb) * kScaleBlock + row0;
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      load_16<VEC>(static_cast<const T*>(p.x) + (at + 64 * i) * p.ldx, cb * kScaleBlock + lane_column,
                   rb < items && at + 64 * i < p.rows ? p.cols : 0, p.x_align, raw[i]);
  };
  fetch();
  for (int turn = 0; rb < items; turn ^= 1) {
    const int rows = min(p.rows - rb * kScaleBlock, kScaleBlock), c0 = cb * kScaleBlock;
    const long long first = static_cast<long long>(rb) * kScaleBlock + row0, scale_at = rb * p.lds + cb;
    Raw v[kRows][2];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      v[i][0] = raw[i][0];
      v[i][1] = raw[i][1];
    }
    float m = max_nan(max_abs(v[0]), max_abs(v[1]));
    rb += dr;
    cb += dc;
    if (cb >= p.nblk) {
      cb -= p.nblk;
      ++rb;
    }
    if (sizeof(Raw) == 16) fetch();   // (fp32 has no registers for it)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    // two sets of partial maxima in turn: a warp may be a block ahead of one still reading
    if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i) m = max_nan(m, part[turn][i]);
    const BlockScale bs = scale_of(m);
    if (threadIdx.x == 0) p.scale[scale_at] = bs.s;
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (row0 + 64 * i < rows) store_16<VEC>(p.q + (first + 64 * i) * p.ldq, c0 + lane_column, p.cols, p.q_align, v[i], bs);
    if (sizeof(Raw) != 16) fetch();
  }
}

template <typename T, bool GATED, bool VEC>
cudaError_t launch_rows(const QuantParams& p, int num_sms, cudaStream_t stream) {
  constexpr int kGroups = 256 / kLanes<T, GATED, VEC>;
  const long long ctas = (static_cast<long long>(p.rows) * p.nblk + kGroups - 1) / kGroups;
  const long long cap = static_cast<long long>(num_sms) * kRowsPerSm<T, GATED>;   // resident
  return launch_pdl(quantize_rows_kernel<T, GATED, VEC>, dim3(static_cast<unsigned>(ctas < cap ? ctas : cap)), dim3(256), 0,
                    stream, 1, p);
}

template <typename T, bool VEC>
cudaError_t launch_t(const QuantParams& p, bool gated, int block_rows, int num_sms, cudaStream_t stream) {
  if (block_rows != 1) {
    const long long ctas = static_cast<long long>((p.rows + kScaleBlock - 1) / kScaleBlock) * p.nblk;
    const long long cap = static_cast<long long>(num_sms) * 2;   // resident
    return launch_pdl(quantize_tiles_kernel<T, VEC>, dim3(static_cast<unsigned>(ctas < cap ? ctas : cap)), dim3(512), 0,
                      stream, 1, p);
  }
  return gated ? launch_rows<T, true, VEC>(p, num_sms, stream) : launch_rows<T, false, VEC>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_quantize_blocks(const QuantParams& p, bool bf16, bool gated, int block_rows, int num_sms,
                                   cudaStream_t stream) {
  const bool vec = p.x_align >= 8 && p.q_align >= 8;
  if (bf16)
    return vec ? launch_t<__nv_bfloat16, true>(p, gated, block_rows, num_sms, stream)
               : launch_t<__nv_bfloat16, false>(p, gated, block_rows, num_sms, stream);
  return vec ? launch_t<float, true>(p, gated, block_rows, num_sms, stream)
             : launch_t<float, false>(p, gated, block_rows, num_sms, stream);
}

}  // namespace convf
