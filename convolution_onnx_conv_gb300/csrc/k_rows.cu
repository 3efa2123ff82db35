// Rows to 8 bits with what a whole row has in common: int8 with one scale per row, and the root-mean-square
// norm (after the residual's addition) in front of int8 rows or of e4m3 blocks.
//
// With h the row (x, gathered or gated, or x + residual) and t = h * weight (t = h without a norm):
//   s = max|t| / 127 over the row, q = rint(t / s)                (int8)
//   s = max|t| / 448 over 128 columns, q = e4m3(t / s)            (e4m3)
//   scale = s * r, r = 1 / sqrt(mean(h^2) + eps)                  (r = 1 without a norm)
// The factor r of a row is positive, so quantising h * r * weight gives the same 8-bit values: they need no r,
// and a row takes one reduction, of its maximum and its sum of squares together, instead of two in turn.
//
// Bound by the bytes: each row is read once, a thread holds 16 values of it, the next row's loads are on
// their way while this one is reduced and written.  A row takes 32 to 512 threads by its width; wider rows are
// read twice, the second time from L2.
//
// int8 values come from the correctly rounded float32 quotient, which a product by the scale's reciprocal and
// two corrections by the remainder give: the first leaves an error below a unit in the last place, and the
// second is then the rounded quotient (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990: a reciprocal to nearest and a quotient within a unit).
#include <type_traits>

#include "convf_internal.h"
#include "linear_internal.h"
#include "ptx.cuh"
#include "quant_dev.cuh"

#ifndef CONVF_ROWS_KIND
#error "compile with -DCONVF_ROWS_KIND=0 (rows), 1 (gated rows), 2 (norm, int8) or 3 (norm, e4m3)"
#endif

namespace convf {

namespace {

constexpr int kKind = CONVF_ROWS_KIND;
constexpr bool kGated = kKind == kRowsGated, kNorm = kKind >= kRowsNormInt8, kInt8 = kKind != kRowsNormE4m3;

// g / (1 + exp(-g)), each operation rounded to nearest
__device__ __forceinline__ float gate_rn(float g) { return __fdiv_rn(g, 1.f + expf(-g)); }

// the row's scale for int8, and the reciprocal for quotients(), or 0 where a remainder could be subnormal or
// the scale is no number
__device__ __forceinline__ BlockScale int8_scale_of(float m) {
  const float s = __fdiv_rn(m, 127.f);
  return BlockScale{s, m > 0x1p-50f && m < 0x1p60f ? __frcp_rn(s) : 0.f};
}

// t / s rounded to nearest, and rounded to an integer: the low byte of the results is the int8 value.  Adding
// 1.5 * 2^23 rounds to an integer, ties to even.
__device__ __forceinline__ void int8_pair(float t0, float t1, BlockScale bs, uint32_t& b0, uint32_t& b1) {
  asm("{\n\t.reg .b64 t, r, s, q, e, m;\n\t"
      "mov.b64 t, {%2, %3};\n\tmov.b64 r, {%5, %5};\n\tmov.b64 s, {%4, %4};\n\tmov.b64 m, {%6, %6};\n\t"
      "mul.rn.f32x2 q, t, r;\n\t"
      "fma.rn.f32x2 e, q, s, t;\n\t"
      "fma.rn.f32x2 q, e, r, q;\n\t"
      "fma.rn.f32x2 e, q, s, t;\n\t"
      "fma.rn.f32x2 q, e, r, q;\n\t"
      "add.rn.f32x2 q, q, m;\n\t"
      "mov.b64 {%0, %1}, q;\n\t}"
      : "=r"(b0), "=r"(b1)
      : "f"(t0), "f"(t1), "f"(-bs.s), "f"(bs.r), "f"(12582912.f));
}
__device__ __forceinline__ uint32_t int8_slow(float t, float s) {
  const float q = __fdiv_rn(t, s);
  // a scale of 0 (a row of zeros, or one whose scale underflowed) or none: zeros
  if (s == 0.f || !(q >= -1e9f && q <= 1e9f)) return 0;
  return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(rintf(q), -127.f), 127.f))) & 0xFFu;
}
[[maybe_unused]] __device__ __forceinline__ uint2 int8_8(const uint32_t* w, BlockScale bs) {
  uint32_t o[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t b[4];
    if (bs.r != 0.f) {
#pragma unroll
      for (int j = 0; j < 4; j += 2)
        int8_pair(__uint_as_float(w[4 * i + j]), __uint_as_float(w[4 * i + j + 1]), bs, b[j], b[j + 1]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = int8_slow(__uint_as_float(w[4 * i + j]), bs.s);
    }
    o[i] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  }
  return make_uint2(o[0], o[1]);
}

// 16 columns of a row of q
template <bool VEC>
__device__ __forceinline__ void store_int8_16(uint8_t* row, int c, int cols, int align, const RawF32 (&t)[2], BlockScale bs) {
  const uint2 o[2] = {int8_8(t[0].w, bs), int8_8(t[1].w, bs)};
  store_bytes_16<VEC>(row, c, cols, align, o);
}

// 16 columns of a row of h, at the columns that load_16 reads
template <bool VEC, typename R>
__device__ __forceinline__ void store_h_16(R* row, int c, int cols, int align, const RawF32 (&h)[2]) {
  constexpr bool BF16 = sizeof(R) == 2;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int first = c + (VEC ? 8 : 64) * k;
    if (VEC && first + 8 <= cols) {
      if constexpr (BF16) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 two = __floats2bfloat162_rn(__uint_as_float(h[k].w[2 * i]), __uint_as_float(h[k].w[2 * i + 1]));
          w[i] = *reinterpret_cast<const uint32_t*>(&two);
        }
        if (align >= 16) {
          *reinterpret_cast<uint4*>(row + first) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          reinterpret_cast<uint2*>(row + first)[0] = make_uint2(w[0], w[1]);
          reinterpret_cast<uint2*>(row + first)[1] = make_uint2(w[2], w[3]);
        }
      } else if (align >= 16) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          reinterpret_cast<uint4*>(row + first)[i] = make_uint4(h[k].w[4 * i], h[k].w[4 * i + 1], h[k].w[4 * i + 2], h[k].w[4 * i + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) reinterpret_cast<uint2*>(row + first)[i] = make_uint2(h[k].w[2 * i], h[k].w[2 * i + 1]);
      }
    } else if (!VEC || first < cols) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = VEC ? first + i : first + 8 * i;
        if (at < cols) {
          if constexpr (BF16)
            row[at] = __float2bfloat16_rn(__uint_as_float(h[k].w[i]));
          else
            row[at] = __uint_as_float(h[k].w[i]);
        }
      }
    }
  }
}

struct NoResidual {};

// What a thread holds of a row as it is in memory
template <typename T, typename R>
struct RowRaw {
  typedef typename RawOf<T>::type X;
  typedef typename RawOf<typename std::conditional<std::is_same<R, NoResidual>::value, __nv_bfloat16, R>::type>::type Second;
  X x[2];
  typename std::conditional<kGated, X, Second>::type second[2];   // the gated row's other half, or the residual
};

// Threads on an SM: 512 to 1024 rows' threads with 32 to 64 KB of the next rows on their way.  (With 1024 the kernels
// of more than 16 words a thread spilled up to 400 bytes.)
template <typename T, typename R>
constexpr int kThreadsPerSm = sizeof(RowRaw<T, R>) - (kGated || !std::is_same<R, NoResidual>::value ? 0 : sizeof(RowRaw<T, R>::second)) <= 64 ? 1024 : 512;

// G threads take a row: 16 columns each (columns 16 i .. of thread i; VEC false: load_16's columns between
// its 8 lanes').  WIDE: the row is longer, and passed over in steps of 16 G columns, twice.
template <typename T, typename R, bool VEC, int G, bool WIDE>
__global__ void __launch_bounds__(G < 128 ? 128 : G, kThreadsPerSm<T, R> / (G < 128 ? 128 : G)) rows_kernel(const RowsParams p) {
  constexpr bool RES = !std::is_same<R, NoResidual>::value;
  constexpr int kCta = G < 128 ? 128 : G, kPerCta = kCta / G, kWarps = G / 32;
  typedef RowRaw<T, R> Raw;
  pdl_launch_dependents();
  pdl_wait_prior();
  __shared__ float part[2][2][kWarps];   // by row parity: sums and maxima of a row's warps
  const int tid = kPerCta > 1 ? threadIdx.x % G : threadIdx.x;
  const long long step = static_cast<long long>(gridDim.x) * kPerCta;
  long long r = static_cast<long long>(blockIdx.x) * kPerCta + (kPerCta > 1 ? threadIdx.x / G : 0);
  const int first = VEC ? tid * 16 : tid / 8 * kScaleBlock + tid % 8;   // this thread's columns

  auto source = [&](long long row) -> int { return row >= p.rows ? -1 : p.index ? p.index[row] : static_cast<int>(row); };
  auto fetch = [&](Raw& raw, int src, int c) {
    const bool there = src >= 0 && src < p.x_rows;
    const long long at = there ? src : 0;
    const int cols = there ? p.cols : 0;
    const T* row = static_cast<const T*>(p.x) + at * p.ldx;
    load_16<VEC>(row, c, cols, p.x_align, raw.x);
    if constexpr (kGated) load_16<VEC>(row + p.cols, c, cols, p.x_align, raw.second);
    if constexpr (RES) load_16<VEC>(static_cast<const R*>(p.residual) + at * p.ldr, c, cols, p.r_align, raw.second);
  };
  // the values of one thread: h is what the norm takes the squares of, t what is quantised
  auto values = [&](const Raw& raw, RawF32 (&h)[2]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float a[8];
      raw.x[k].floats(a);
      if constexpr (kGated || RES) {
        float b[8];
        raw.second[k].floats(b);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = kGated ? gate_rn(a[i]) * b[i] : a[i] + b[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k].w[i] = __float_as_uint(a[i]);
    }
  };
  auto weigh = [&](RawF32 (&h)[2], int c) {   // h -> t
    if constexpr (kNorm) {
      if (p.weight_bf16) {
        RawBf16 w[2];
        load_16<VEC>(static_cast<const __nv_bfloat16*>(p.weight), c, p.cols, p.w_align, w);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float f[8];
          w[k].floats(f);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[k].w[i] = __float_as_uint(__uint_as_float(h[k].w[i]) * f[i]);
        }
      } else if (p.weight) {
        RawF32 w[2];
        load_16<VEC>(static_cast<const float*>(p.weight), c, p.cols, p.w_align, w);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) h[k].w[i] = __float_as_uint(__uint_as_float(h[k].w[i]) * __uint_as_float(w[k].w[i]));
      }
    }
  };
  auto squares = [&](const RawF32 (&h)[2], float sum) {
    float a[4] = {sum, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i & 3] = fmaf(__uint_as_float(h[k].w[i]), __uint_as_float(h[k].w[i]), a[i & 3]);
    return (a[0] + a[1]) + (a[2] + a[3]);
  };
  // sum and maximum over the row's threads
  auto reduce = [&](float& sum, float& m, int turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (kNorm) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      if (kInt8) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    }
    if constexpr (kWarps > 1) {
      // (two sets in turn: a warp may be a row ahead of one still reading)
      if ((threadIdx.x & 31) == 0) {
        part[turn][0][threadIdx.x >> 5] = sum;
        part[turn][1][threadIdx.x >> 5] = m;
      }
      __syncthreads();
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        if (kNorm) sum += part[turn][0][i];
        if (kInt8) m = max_nan(m, part[turn][1][i]);
      }
    }
  };
  auto factor = [&](float sum) { return kNorm ? __frsqrt_rn(sum / static_cast<float>(p.cols) + p.eps) : 1.f; };
  // columns from c of row `row`: int8 by the row's scale, e4m3 by each block's (8 lanes)
  auto put = [&](long long row, const RawF32 (&t)[2], int c, BlockScale bs, float f) {
    if constexpr (kInt8) {
      store_int8_16<VEC>(p.q + row * p.ldq, c, p.cols, p.q_align, t, bs);
    } else {
      store_16<VEC>(p.q + row * p.ldq, c, p.cols, p.q_align, t, bs);
      const int block = c / kScaleBlock;
      if ((tid & 7) == 0 && block < p.nblk) p.scale[row * p.lds + block] = bs.s * f;
    }
  };
  auto block_scale = [&](const RawF32 (&t)[2]) {
    float m = max_abs(t);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    return scale_of(m);
  };

  // (whole warps, and for G > 32 whole CTAs, share a row: they leave the loops together)
  if constexpr (!WIDE) {
    Raw raw;
    fetch(raw, source(r), first);
    int next_src = source(r + step);
    for (int turn = 0; r < p.rows; turn ^= 1) {
      RawF32 t[2];
      values(raw, t);
      if (r + step < p.rows) fetch(raw, next_src, first);
      next_src = source(r + 2 * step);
      if constexpr (RES)
        if (p.h) store_h_16<VEC>(static_cast<R*>(p.h) + r * p.ldh, first, p.cols, p.r_align, t);
      float sum = kNorm ? squares(t, 0.f) : 0.f, m = 0.f;
      weigh(t, first);
      BlockScale bs{};
      if constexpr (kInt8)
        m = max_abs(t);
      else
        bs = block_scale(t);
      reduce(sum, m, turn);
      if constexpr (kInt8) {
        bs = int8_scale_of(m);
        if (tid == 0) p.scale[r] = bs.s * factor(sum);
      }
      put(r, t, first, bs, factor(sum));
      r += step;
    }
  } else {
    // (a thread reads the same elements in both passes, and h is written in the second: it may lie on the residual)
    for (int turn = 0; r < p.rows; turn ^= 1) {
      const int src = source(r);
      float sum = 0.f, m = 0.f;
      for (int c = first; c - first < p.cols; c += 16 * G) {
        Raw raw;
        RawF32 t[2];
        fetch(raw, src, c);
        values(raw, t);
        if (kNorm) sum = squares(t, sum);
        if (kInt8) {
          weigh(t, c);
          m = max_nan(m, max_abs(t));
        }
      }
      reduce(sum, m, turn);
      BlockScale bs{};
      const float f = factor(sum);
      if constexpr (kInt8) {
        bs = int8_scale_of(m);
        if (tid == 0) p.scale[r] = bs.s * f;
      }
      for (int c = first; c - first < p.cols; c += 16 * G) {
        Raw raw;
        RawF32 t[2];
        fetch(raw, src, c);
        values(raw, t);
        if constexpr (RES)
          if (p.h) store_h_16<VEC>(static_cast<R*>(p.h) + r * p.ldh, c, p.cols, p.r_align, t);
        weigh(t, c);
        if constexpr (!kInt8) bs = block_scale(t);
        put(r, t, c, bs, f);
      }
      r += step;
    }
  }
}

template <typename T, typename R, bool VEC, int G, bool WIDE>
cudaError_t launch_g(const RowsParams& p, int num_sms, cudaStream_t stream) {
  constexpr int kCta = G < 128 ? 128 : G, kPerCta = kCta / G;
  const long long ctas = (p.rows + kPerCta - 1LL) / kPerCta, cap = static_cast<long long>(num_sms) * (kThreadsPerSm<T, R> / kCta);
  return launch_pdl(rows_kernel<T, R, VEC, G, WIDE>, dim3(static_cast<unsigned>(ctas < cap ? ctas : cap)), dim3(kCta), 0, stream,
                    1, p);
}

template <typename T, typename R, bool VEC>
cudaError_t launch_v(const RowsParams& p, int num_sms, cudaStream_t stream) {
  if (p.cols <= 16 * 32) return launch_g<T, R, VEC, 32, false>(p, num_sms, stream);
  if (p.cols <= 16 * 128) return launch_g<T, R, VEC, 128, false>(p, num_sms, stream);
  if (p.cols <= 16 * 256) return launch_g<T, R, VEC, 256, false>(p, num_sms, stream);
  if (p.cols <= 16 * 512) return launch_g<T, R, VEC, 512, false>(p, num_sms, stream);
  return launch_g<T, R, VEC, 512, true>(p, num_sms, stream);
}

template <typename T, typename R>
cudaError_t launch_r(const RowsParams& p, int num_sms, cudaStream_t stream) {
  const bool vec = p.x_align >= 8 && p.r_align >= 8 && p.q_align >= 8 && p.w_align >= 8;
  return vec ? launch_v<T, R, true>(p, num_sms, stream) : launch_v<T, R, false>(p, num_sms, stream);
}

template <typename T>
cudaError_t launch_t(const RowsParams& p, int num_sms, cudaStream_t stream) {
  if constexpr (kNorm) {
    if (p.residual) {
      return p.residual_bf16 ? launch_r<T, __nv_bfloat16>(p, num_sms, stream) : launch_r<T, float>(p, num_sms, stream);
    }
  }
  return launch_r<T, NoResidual>(p, num_sms, stream);
}

}  // namespace

template <>
cudaError_t launch_rows<kKind>(const RowsParams& p, bool bf16, int num_sms, cudaStream_t stream) {
  return bf16 ? launch_t<__nv_bfloat16>(p, num_sms, stream) : launch_t<float>(p, num_sms, stream);
}

}  // namespace convf
