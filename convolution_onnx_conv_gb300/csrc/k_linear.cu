// Linear layers, simplest form: one thread per output element.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "convf_internal.h"
#include "linear_internal.h"
#include "ptx.cuh"

namespace convf {

namespace {

__device__ __forceinline__ float e4m3_to_float(uint8_t b) {
  __nv_fp8_e4m3 t;
  t.__x = b;
  return static_cast<float>(t);
}

template <bool E4M3>
__global__ void __launch_bounds__(256) linear_simple_kernel(const LinearParams p) {
  pdl_launch_dependents();
  pdl_wait_prior();
  const int n = blockIdx.y * 32 + (threadIdx.x & 31);
  const long long m = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (n >= p.N || m >= p.rows) return;
  int e = 0;
  if (p.offsets) {
    bool found = false;
    for (int i = 0; i < p.experts && !found; ++i)
      if (m >= p.offsets[i] && m < p.offsets[i + 1]) {
        e = i;
        found = true;
      }
    if (m == 0 && n == 0) {
      bool bad = p.offsets[0] < 0 || p.offsets[p.experts] > p.rows;
      for (int i = 0; i < p.experts; ++i) bad = bad || p.offsets[i + 1] < p.offsets[i];
      if (bad) atomicOr(p.status, kStatusOffsets);
    }
    if (!found) return;
  }
  const int kblk = (p.K + kScaleBlock - 1) / kScaleBlock;
  const int nblk = (p.N + kScaleBlock - 1) / kScaleBlock;
  float acc = 0.f;
  if (E4M3) {
    const uint8_t* x = static_cast<const uint8_t*>(p.x) + m * p.ldx;
    const uint8_t* w = static_cast<const uint8_t*>(p.w) + e * p.expert_stride + n * p.ldw;
    const float* ws = p.w_scale + (static_cast<long long>(e) * nblk + n / kScaleBlock) * kblk;
    for (int b = 0; b < kblk; ++b) {
      float t = 0.f;
      const int k1 = min(p.K, (b + 1) * kScaleBlock);
      for (int k = b * kScaleBlock; k < k1; ++k) t = fmaf(e4m3_to_float(x[k]), e4m3_to_float(w[k]), t);
      acc = fmaf(t, p.x_scale[m * p.xs_row + b * p.xs_blk] * ws[b], acc);
    }
  } else {
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + m * p.ldx;
    const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(p.w) + e * p.expert_stride + n * p.ldw;
    for (int k = 0; k < p.K; ++k) acc = fmaf(__bfloat162float(x[k]), __bfloat162float(w[k]), acc);
  }
  if (p.bias) acc += p.bias[static_cast<long long>(e) * p.N + n];
  // a NaN stays a NaN (fminf and fmaxf would drop it)
  acc = acc < p.lo ? p.lo : (acc > p.hi ? p.hi : acc);
  if (p.out_bf16)
    static_cast<__nv_bfloat16*>(p.y)[m * p.ldy + n] = __float2bfloat16_rn(acc);
  else
    static_cast<float*>(p.y)[m * p.ldy + n] = acc;
}

}  // namespace

cudaError_t launch_linear_simple(const LinearParams& p, bool e4m3, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((static_cast<long long>(p.rows) + 7) / 8), (p.N + 31) / 32);
  return e4m3 ? launch_pdl(linear_simple_kernel<true>, grid, dim3(256), 0, stream, 1, p)
              : launch_pdl(linear_simple_kernel<false>, grid, dim3(256), 0, stream, 1, p);
}

}  // namespace convf
