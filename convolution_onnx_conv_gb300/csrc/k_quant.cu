// Quantising to e4m3 with a float scale per block: s = max|v| / 448, q = e4m3(v / s).
//
// Bound by the bytes: x once in, one byte per value and a scale per block out.  16 lanes hold a block of
// 128 columns, several blocks on their way at once; rows that begin on 8 or 16 bytes are read as
// vectors, others element by element with the lanes side by side.
//
// The definition's quotient is the float32 one, rounded again to e4m3.  A division per value would
// cost more than the bytes, so q comes from v * (1 / s), which is within 2.5 units in the last place
// of the quotient, and from the quotient itself where a tie of e4m3 is that near (or the value is
// below e4m3's normal range): the stored values are the definition's in every case.
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
__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xFFFF0000u);
}

// 8 consecutive elements in 16-byte (wide) or 8-byte loads
__device__ __forceinline__ void load8(const __nv_bfloat16* p, bool wide, float (&v)[8]) {
  uint4 t;
  if (wide) {
    t = __ldg(reinterpret_cast<const uint4*>(p));
  } else {
    const uint2 a = __ldg(reinterpret_cast<const uint2*>(p)), b = __ldg(reinterpret_cast<const uint2*>(p) + 1);
    t = make_uint4(a.x, a.y, b.x, b.y);
  }
  unpack2(t.x, v[0], v[1]);
  unpack2(t.y, v[2], v[3]);
  unpack2(t.z, v[4], v[5]);
  unpack2(t.w, v[6], v[7]);
}
__device__ __forceinline__ void load8(const float* p, bool wide, float (&v)[8]) {
  if (wide) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = __ldg(reinterpret_cast<const float2*>(p) + i);
      v[2 * i] = a.x;
      v[2 * i + 1] = a.y;
    }
  }
}

// This lane's 8 columns of the block that begins at column c0, zero past `cols`.  VEC: columns
// c0 + 8 sub .. (a chunk that ends past the row is read one element at a time: the row may be the
// buffer's last); else columns c0 + sub + 16 i.
template <bool VEC, typename T>
__device__ __forceinline__ void load_lane(const T* row, int c0, int sub, int cols, bool wide, float (&v)[8]) {
  if (VEC) {
    const int c = c0 + sub * 8;
    if (c + 8 <= cols) {
      load8(row + c, wide, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? load1(row + c + i) : 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c0 + sub + 16 * i < cols ? load1(row + c0 + sub + 16 * i) : 0.f;
  }
}

// v / s for the rounding to e4m3, given r = 1 / s: the same result after that rounding
__device__ __forceinline__ float quotient(float v, float s, float r) {
  float t = v * r;
  // e4m3 keeps 3 of the 23 fraction bits: a tie has 0x80000 in the other 20.  Below the normal range
  // (2^-6) ties lie elsewhere; zero is exact.
  const uint32_t a = __float_as_uint(t) & 0x7FFFFFFFu;
  if (((a & 0xFFFFFu) - 0x7FFFCu <= 8u) | (a - 1u < 0x3C7FFFFFu)) t = v / s;
  return t;
}

template <bool VEC>
__device__ __forceinline__ void store_lane(uint8_t* row, int c0, int sub, int cols, const float (&v)[8], float s) {
  // s == 0: a block of zeros (or one whose scale underflowed): zeros, not 0 / 0.  Beside these limits 1 / s
  // could leave float32's normal range, or is no number.
  const bool usual = s > 0x1p-100f && s < 0x1p100f;
  const float r = usual ? 1.f / s : 0.f;
  float t[8];
  if (usual) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = quotient(v[i], s, r);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = s == 0.f ? 0.f : v[i] / s;
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __nv_cvt_float2_to_fp8x2(make_float2(t[2 * i], t[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  const uint2 o = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
  if (VEC) {
    const int c = c0 + sub * 8;
    if (c + 8 <= cols) {
      *reinterpret_cast<uint2*>(row + c) = o;
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = VEC ? c0 + sub * 8 + i : c0 + sub + 16 * i;
    if (c < cols) row[c] = static_cast<uint8_t>((i < 4 ? o.x : o.y) >> (8 * (i & 3)));
  }
}

__device__ __forceinline__ float max8(const float (&v)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(v[i]));
  return m;
}

// Scales per row: 16 lanes take NB consecutive blocks of a row at a time.
template <typename T, bool GATED, bool VEC, int NB>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantParams p) {
  pdl_launch_dependents();
  pdl_wait_prior();
  const int sub = threadIdx.x & 15;
  const int per_row = (p.nblk + NB - 1) / NB;
  const long long items = static_cast<long long>(p.rows) * per_row;
  // whole warps loop together (the shuffles below name all 32 lanes): `mine` masks the tail
  for (long long base = static_cast<long long>(blockIdx.x) * 16; base < items; base += static_cast<long long>(gridDim.x) * 16) {
    const long long item = base + (threadIdx.x >> 4);
    const bool mine = item < items;
    // (a 64-bit division is a subroutine)
    const int r = !mine ? 0 : items < (1LL << 31) ? static_cast<int>(static_cast<uint32_t>(item) / static_cast<uint32_t>(per_row))
                                                  : static_cast<int>(item / per_row);
    const int b0 = mine ? static_cast<int>(item - static_cast<long long>(r) * per_row) * NB : p.nblk;
    const int src = mine ? (p.index ? __ldg(p.index + r) : r) : -1;
    const bool there = src >= 0 && src < p.x_rows;
    const T* row = static_cast<const T*>(p.x) + static_cast<long long>(there ? src : 0) * p.ldx;
    float v[NB][8];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      if (there && b0 + j < p.nblk) {
        load_lane<VEC>(row, (b0 + j) * kScaleBlock, sub, p.cols, p.wide, v[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
      }
    }
    if (GATED) {
      float u[NB][8];
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if (there && b0 + j < p.nblk) {
          load_lane<VEC>(row + p.cols, (b0 + j) * kScaleBlock, sub, p.cols, p.wide, u[j]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) u[j][i] = 0.f;
        }
      }
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] / (1.f + expf(-v[j][i])) * u[j][i];
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      float m = max8(v[j]);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const float s = m / kE4m3Max;
      if (b0 + j < p.nblk) {
        if (sub == 0) p.scale[static_cast<long long>(r) * p.lds + b0 + j] = s;
        store_lane<VEC>(p.q + static_cast<long long>(r) * p.ldq, (b0 + j) * kScaleBlock, sub, p.cols, v[j], s);
      }
    }
  }
}

// Scales per 128 x 128 block: a CTA takes one at a time, 8 rows of 8 elements per thread, held in
// registers between the maximum and the division.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) quantize_tiles_kernel(const QuantParams p) {
  pdl_launch_dependents();
  pdl_wait_prior();
  __shared__ float part[2][8];
  const long long items = static_cast<long long>((p.rows + kScaleBlock - 1) / kScaleBlock) * p.nblk;
  const int sub = threadIdx.x & 15, row0 = threadIdx.x >> 4;
  int turn = 0;
  for (long long item = blockIdx.x; item < items; item += gridDim.x, turn ^= 1) {
    const int rb = static_cast<int>(item / p.nblk);
    const int cb = static_cast<int>(item - static_cast<long long>(rb) * p.nblk);
    const int rows = min(p.rows - rb * kScaleBlock, kScaleBlock);
    const long long first = static_cast<long long>(rb) * kScaleBlock + row0;
    float v[8][8];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (row0 + 16 * i < rows) {
        load_lane<VEC>(static_cast<const T*>(p.x) + (first + 16 * i) * p.ldx, cb * kScaleBlock, sub, p.cols, p.wide, v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_nan(m, max8(v[i]));
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
      if (row0 + 16 * i < rows)
        store_lane<VEC>(p.q + (first + 16 * i) * p.ldq, cb * kScaleBlock, sub, p.cols, v[i], s);
  }
}

template <typename T, bool GATED, bool VEC>
cudaError_t launch_rows(const QuantParams& p, int num_sms, cudaStream_t stream) {
  // more blocks per lane group keep more bytes on the way; fewer spread a small call over more SMs
  const long long half_warps = static_cast<long long>(num_sms) * 8 * 16;
  const long long blocks = static_cast<long long>(p.rows) * p.nblk;
  const int nb = !GATED && p.nblk >= 4 && blocks >= 4 * half_warps ? 4 : p.nblk >= 2 && blocks >= 2 * half_warps ? 2 : 1;
  const long long ctas = (static_cast<long long>(p.rows) * ((p.nblk + nb - 1) / nb) + 15) / 16;
  const long long cap = static_cast<long long>(num_sms) * 8;
  const dim3 grid(static_cast<unsigned>(ctas < cap ? ctas : cap));
  if (nb == 4 && !GATED) return launch_pdl(quantize_rows_kernel<T, false, VEC, 4>, grid, dim3(256), 0, stream, 1, p);
  if (nb == 2) return launch_pdl(quantize_rows_kernel<T, GATED, VEC, 2>, grid, dim3(256), 0, stream, 1, p);
  return launch_pdl(quantize_rows_kernel<T, GATED, VEC, 1>, grid, dim3(256), 0, stream, 1, p);
}

template <typename T, bool VEC>
cudaError_t launch_t(const QuantParams& p, bool gated, int block_rows, int num_sms, cudaStream_t stream) {
  if (block_rows != 1) {
    const long long ctas = static_cast<long long>((p.rows + kScaleBlock - 1) / kScaleBlock) * p.nblk;
    const long long cap = static_cast<long long>(num_sms) * 8;
    return launch_pdl(quantize_tiles_kernel<T, VEC>, dim3(static_cast<unsigned>(ctas < cap ? ctas : cap)), dim3(256), 0,
                      stream, 1, p);
  }
  return gated ? launch_rows<T, true, VEC>(p, num_sms, stream) : launch_rows<T, false, VEC>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_quantize_blocks(const QuantParams& p, bool bf16, bool gated, int block_rows, int num_sms,
                                   cudaStream_t stream) {
  if (bf16)
    return p.vec ? launch_t<__nv_bfloat16, true>(p, gated, block_rows, num_sms, stream)
                 : launch_t<__nv_bfloat16, false>(p, gated, block_rows, num_sms, stream);
  return p.vec ? launch_t<float, true>(p, gated, block_rows, num_sms, stream)
               : launch_t<float, false>(p, gated, block_rows, num_sms, stream);
}

}  // namespace convf
