// Device-side parts shared by the int8 linear kernels: fp16 MMAs whose first operand is in TMEM, int8 -> fp16, and
// the last step of an output element.
//
// sm_103a's tcgen05.mma has no integer kind, and its warp-level int8 MMA (25 cycles of an SM for 16 x 8 x 32) reaches a
// twenty-fifth of the fp16 rate: enough for a handful of rows only (linear_int8_direct.cu).  For more: an
// int8 value is an fp16 number, the product of two is at most 2^14 and fp32 holds every integer up to 2^24: fp16
// MMAs add kInt8Chunk products exactly, and the chunks' sums are added as int32 in registers.  So every sum is the
// integer, whatever the order, and all forms give the same bits.
//
// The bytes stay int8 up to shared memory (TMA); converting warps make fp16 of them there: a byte in the low bits
// of an fp16 number 1024 + .. and a subtraction (Kim, Henry, Fahim and Awadalla, "Who Says Elephants Can't Run: Bringing
// Large Scale MoE Models into Cloud Scale Production", 2022), 3 integer instructions (half rate: what bounds the conversion) and
// 2 packed additions for 4 values.  Converted weights, the MMA's 128 rows, go to TMEM, from where the MMA can read
// its first operand, and not back to shared memory (reading 1 byte, writing 2 and the MMA reading those would be 5
// bytes of its bandwidth a value); rows of x are the MMA's columns and go back to shared memory.  Values keep no
// order within four of them: both operands are permuted alike.
#pragma once
#include <cuda_fp16.h>

#include "linear_dev.cuh"

namespace convf {

constexpr int kUnit = 64;            // values of a unit, what is converted at a time: an fp16 row of 128 bytes
constexpr int kUnitCols = kUnit / 2; // TMEM columns of a unit of weights
constexpr int kInt8Chunk = 1024;     // values that an accumulator sums: 2^24 at most

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
// Arrive on another CTA's mbarrier and publish, in the cluster, what this thread has written to its CTA's shared memory or
// has seen written there (behind a wait for those who wrote it).  The fence is for shared memory alone.
__device__ __forceinline__ void mbar_arrive_remote_shared(uint32_t cluster_addr) {
  asm volatile(
      "fence.release.sync_restrict::shared::cta.cluster;\n\t"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
      : "memory");
}
// Four int8 values as fp16: {0, 2} and {1, 3}.  0x6400 | (b ^ 0x80) is 1024 + 128 + b.  (Each mask and bias in one
// three-input operation: from C++ the compiler made two of them, 200 instead of 140 cycles for 64 values a thread.)
__device__ __forceinline__ uint32_t int8_magic(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x00FF00FF, %2, 0x6A;" : "=r"(r) : "r"(w), "r"(0x64806480u));   // (w & mask) ^ bias
  return r;
}
__device__ __forceinline__ void f16_of_int8(uint32_t w, uint32_t& even, uint32_t& odd) {
  const __half2 bias = __half2half2(__ushort_as_half(0xE480));   // -1152
  const uint32_t e = int8_magic(w), o = int8_magic(w >> 8);
  const __half2 he = __hadd2(*reinterpret_cast<const __half2*>(&e), bias), ho = __hadd2(*reinterpret_cast<const __half2*>(&o), bias);
  even = *reinterpret_cast<const uint32_t*>(&he);
  odd = *reinterpret_cast<const uint32_t*>(&ho);
}

// 16 int8 values as 8 words of fp16
__device__ __forceinline__ void f16_of_int8_16(const uint4& v, uint32_t* f) {
  f16_of_int8(v.x, f[0], f[1]);
  f16_of_int8(v.y, f[2], f[3]);
  f16_of_int8(v.z, f[4], f[5]);
  f16_of_int8(v.w, f[6], f[7]);
}

// What is behind a sum: its weight row's scale and bias, the clamp.  Without a bias nothing is added, and -0 is what leaves
// every product as it is: adding 0 would turn a product of -0 (a negative sum times a scale that underflows) into 0.
constexpr float kNoBias = -0.f;
struct Int8Finish {
  float ws, bias, lo, hi;
  __device__ __forceinline__ float operator()(int sum, float xs) const {
    return act_clamp(__fadd_rn(__fmul_rn(__int2float_rn(sum), __fmul_rn(xs, ws)), bias), lo, hi);
  }
};
// Weight row n of output row m.  Lanes are adjacent weight rows.
__device__ __forceinline__ void int8_put(const LinearParams& p, long long m, int n, float v) {
  if (!CONVF_IN_BOUNDS(m < p.rows && n < p.N, p.status)) return;
  const long long at = m * p.ldy + n;
  if (p.out_bf16)
    static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(p.y)[at] = v;
}
// kCols columns of a tile (rows of x from m0, `rows` of them there), eight at a time: their values first, then the
// stores one behind another.  held: the scale of column 32 i + lane.
template <int kCols>
__device__ __forceinline__ void int8_put_columns(const LinearParams& p, const Int8Finish& finish, const int (&acc)[kCols],
                                                 const float* held, long long m0, int rows, int n) {
#pragma unroll
  for (int c = 0; c < kCols; c += 8) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = finish(acc[c + i], __shfl_sync(0xFFFFFFFFu, held[c / 32], (c + i) % 32));
    if (n < p.N) {
      if (c + 8 <= rows) {
#pragma unroll
        for (int i = 0; i < 8; ++i) int8_put(p, m0 + c + i, n, v[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + i < rows) int8_put(p, m0 + c + i, n, v[i]);
      }
    }
  }
}
// 16 columns of the accumulator, and the wait for them in the same statement: in a statement of its own it would keep the
// compiler from moving memory accesses above it, but not a use of the registers.
__device__ __forceinline__ void tmem_ld_16_wait(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// acc += the accumulator's columns from `from`
template <int kCols>
__device__ __forceinline__ void int8_add_columns(int (&acc)[kCols], uint32_t from) {
#pragma unroll
  for (int c = 0; c < kCols; c += 16) {
    uint32_t r[16];
    tmem_ld_16_wait(from + c, r);
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[c + i] += __float2int_rn(__uint_as_float(r[i]));
  }
}

}  // namespace convf
