// Quantising to e4m3 with a float scale per block: s = max|v| / 448, q = e4m3(v / s).
//
// The quotients are IEEE divisions (not products with a reciprocal), so that a stored scale and
// its values are exactly what the definition gives: a tie in the last step is decided by the last
// bit of v / s.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "convf_internal.h"
#include "linear_internal.h"
#include "ptx.cuh"

namespace convf {

namespace {

// max that keeps a NaN (fmaxf drops it): a block that holds one has a NaN scale
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }

// 8 consecutive elements as two (float) or one (bf16) 16-byte loads
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 t = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// columns [c, c + 8) of a row, zero past `cols` (a chunk that ends past the row is read one
// element at a time: the row may be the buffer's last)
template <typename T>
__device__ __forceinline__ void load_chunk(const T* row, int c, int cols, bool vec, float (&v)[8]) {
  if (vec && c + 8 <= cols) {
    load8(row + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? load1(row + c + i) : 0.f;
  }
}

__device__ __forceinline__ void store_chunk(uint8_t* row, int c, int cols, bool vec, const float (&v)[8], float s) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // s == 0: a block of zeros (or one whose scale underflowed): zeros, not 0 / 0
    const float2 t = s == 0.f ? make_float2(0.f, 0.f) : make_float2(v[2 * i] / s, v[2 * i + 1] / s);
    w[i] = __nv_cvt_float2_to_fp8x2(t, __NV_SATFINITE, __NV_E4M3);
  }
  const uint2 o = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
  if (vec && c + 8 <= cols) {
    *reinterpret_cast<uint2*>(row + c) = o;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) row[c + i] = static_cast<uint8_t>((i < 4 ? o.x : o.y) >> (8 * (i & 3)));
  }
}

__device__ __forceinline__ float max8(const float (&v)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(v[i]));
  return m;
}

// Scales per row: 16 lanes take a block of 128 columns, 8 elements each.
template <typename T, bool GATED>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantParams p) {
  pdl_launch_dependents();
  pdl_wait_prior();
  const int sub = threadIdx.x & 15;
  const long long items = static_cast<long long>(p.rows) * p.nblk;
  // whole half-warps loop together (the shuffles below name all 32 lanes): `mine` masks the tail
  for (long long base = static_cast<long long>(blockIdx.x) * 16; base < items; base += static_cast<long long>(gridDim.x) * 16) {
    const long long item = base + (threadIdx.x >> 4);
    const bool mine = item < items;
    const int r = mine ? static_cast<int>(item / p.nblk) : 0;
    const int b = mine ? static_cast<int>(item - static_cast<long long>(r) * p.nblk) : 0;
    const int c = b * kScaleBlock + sub * 8;
    const int src = mine ? (p.index ? __ldg(p.index + r) : r) : -1;
    float v[8] = {};
    if (src >= 0 && src < p.x_rows) {
      const T* row = static_cast<const T*>(p.x) + static_cast<long long>(src) * p.ldx;
      load_chunk(row, c, p.cols, p.vec_x, v);
      if (GATED) {
        float u[8];
        load_chunk(row + p.cols, c, p.cols, p.vec_u, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] / (1.f + expf(-v[i])) * u[i];
      }
    }
    float m = max8(v);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float s = m / kE4m3Max;
    if (mine) {
      if (sub == 0) p.scale[static_cast<long long>(r) * p.lds + b] = s;
      store_chunk(p.q + static_cast<long long>(r) * p.ldq, c, p.cols, p.vec_q, v, s);
    }
  }
}

// Scales per 128 x 128 block: a CTA takes one at a time, 8 rows of 8 elements per thread, held in
// registers between the maximum and the division.
template <typename T>
__global__ void __launch_bounds__(256) quantize_tiles_kernel(const QuantParams p) {
  pdl_launch_dependents();
  pdl_wait_prior();
  __shared__ float part[2][8];
  const long long items = static_cast<long long>((p.rows + kScaleBlock - 1) / kScaleBlock) * p.nblk;
  int turn = 0;
  for (long long item = blockIdx.x; item < items; item += gridDim.x, turn ^= 1) {
    const int rb = static_cast<int>(item / p.nblk);
    const int cb = static_cast<int>(item - static_cast<long long>(rb) * p.nblk);
    const int rows = min(p.rows - rb * kScaleBlock, kScaleBlock);
    const int c = cb * kScaleBlock + (threadIdx.x & 15) * 8;
    const long long first = static_cast<long long>(rb) * kScaleBlock + (threadIdx.x >> 4);
    float v[8][8];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
      if ((threadIdx.x >> 4) + 16 * i < rows)
        load_chunk(static_cast<const T*>(p.x) + (first + 16 * i) * p.ldx, c, p.cols, p.vec_x, v[i]);
      m = max_nan(m, max8(v[i]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    // two sets of partial maxima in turn: a warp may be a block ahead of one still reading
    if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_nan(m, part[turn][i]);
    const float s = m / kE4m3Max;
    if (threadIdx.x == 0) p.scale[rb * p.lds + cb] = s;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((threadIdx.x >> 4) + 16 * i < rows) store_chunk(p.q + (first + 16 * i) * p.ldq, c, p.cols, p.vec_q, v[i], s);
  }
}

template <typename T>
cudaError_t launch_t(const QuantParams& p, bool gated, int block_rows, int num_sms, cudaStream_t stream) {
  const bool tiles = block_rows != 1;
  long long blocks = tiles ? static_cast<long long>((p.rows + kScaleBlock - 1) / kScaleBlock) * p.nblk
                           : (static_cast<long long>(p.rows) * p.nblk + 15) / 16;
  const long long cap = static_cast<long long>(num_sms) * 8;
  if (blocks > cap) blocks = cap;
  const dim3 grid(static_cast<unsigned>(blocks));
  if (tiles) return launch_pdl(quantize_tiles_kernel<T>, grid, dim3(256), 0, stream, 1, p);
  return gated ? launch_pdl(quantize_rows_kernel<T, true>, grid, dim3(256), 0, stream, 1, p)
               : launch_pdl(quantize_rows_kernel<T, false>, grid, dim3(256), 0, stream, 1, p);
}

}  // namespace

cudaError_t launch_quantize_blocks(const QuantParams& p, bool bf16, bool gated, int block_rows, int num_sms,
                                   cudaStream_t stream) {
  return bf16 ? launch_t<__nv_bfloat16>(p, gated, block_rows, num_sms, stream)
              : launch_t<float>(p, gated, block_rows, num_sms, stream);
}

}  // namespace convf
