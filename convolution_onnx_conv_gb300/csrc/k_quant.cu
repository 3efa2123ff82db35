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
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <type_traits>

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

// x and the index are read as ordinary loads: they may be the output of the kernel before, which still runs
// when this one begins.  Read-only loads ask for data that nothing writes while the kernel runs: the compiler
// may take them above the wait for that kernel, and L1 may hold lines from before it.

// 8 elements as they are in memory, and as floats
struct RawBf16 {
  uint32_t w[4];
  __device__ __forceinline__ void floats(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
struct RawF32 {
  uint32_t w[8];
  __device__ __forceinline__ void floats(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  }
};
template <typename T> struct RawOf;
template <> struct RawOf<__nv_bfloat16> { typedef RawBf16 type; };
template <> struct RawOf<float> { typedef RawF32 type; };
__device__ __forceinline__ void set(RawBf16& r, int i, const __nv_bfloat16* p) {
  const uint32_t b = *reinterpret_cast<const uint16_t*>(p);
  if (i & 1)
    r.w[i >> 1] |= b << 16;
  else
    r.w[i >> 1] = b;
}
__device__ __forceinline__ void set(RawF32& r, int i, const float* p) { r.w[i] = __float_as_uint(*p); }

// 8 values of a row, zero past `cols`.  VEC: columns c .. c + 7, in 16-byte or 8-byte loads (a chunk that
// ends past the row is read one element at a time: the row may be the buffer's last); else columns c,
// c + 8, .., which lie side by side with the other lanes'.
template <bool VEC, typename T>
__device__ __forceinline__ typename RawOf<T>::type load_8(const T* row, int c, int cols, int align) {
  typedef typename RawOf<T>::type Raw;
  constexpr int kWords = sizeof(Raw) / 4;
  Raw r;
  if (VEC && c + 8 <= cols) {
    const T* p = row + c;
    if (align >= 16) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 t = reinterpret_cast<const uint4*>(p)[i / 4];
        r.w[i] = t.x;
        r.w[i + 1] = t.y;
        r.w[i + 2] = t.z;
        r.w[i + 3] = t.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 2) {
        const uint2 t = reinterpret_cast<const uint2*>(p)[i / 2];
        r.w[i] = t.x;
        r.w[i + 1] = t.y;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kWords; ++i) r.w[i] = 0;
    if (!VEC || c < cols) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = VEC ? c + i : c + 8 * i;
        if (at < cols) set(r, i, row + at);
      }
    }
  }
  return r;
}
__device__ __forceinline__ void load_32_bytes(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
      : "l"(p));
}

// 16 values of a row.  VEC: columns c .. c + 15, by 32 bytes where rows begin on 32; else (h, i) is column
// c + 64 h + 8 i, between the other lanes'.
template <bool VEC, typename Raw, typename T>
__device__ __forceinline__ void load_16(const T* row, int c, int cols, int align, Raw (&r)[2]) {
  if (VEC && align == 32 && (c + 16 <= cols || c >= cols)) {
    uint32_t w[2 * sizeof(Raw) / 4] = {};
    if (c < cols) {
      load_32_bytes(row + c, w);
      if (sizeof(Raw) == 32) load_32_bytes(row + c + 8, w + sizeof(Raw) / 4);
    }
#pragma unroll
    for (int i = 0; i < 2 * sizeof(Raw) / 4; ++i) r[i / (sizeof(Raw) / 4)].w[i % (sizeof(Raw) / 4)] = w[i];
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) r[h] = load_8<VEC>(row, c + (VEC ? 8 : 64) * h, cols, align);
}

// A block's scale s = m / 448, rounded to nearest, and r = -1 / s for minus_quotients(), or 0 where a remainder
// could be subnormal or s is no number.  m / 448 is m * (1/448) in two parts (Brisebarre, Muller and Raina,
// "Accelerating correctly rounded floating-point division when the divisor is known in advance", 2004);
// equal to the quotient for every one of the 2^23 fractions where nothing is subnormal.
struct BlockScale {
  float s, r;
};
__device__ __forceinline__ BlockScale scale_of(float m) {
  if (m > 0x1p-50f && m < 0x1p60f) {
    const float s = fmaf(m, 0x1.24924ap-9f, m * -0x1.b6db6ep-34f);
    return BlockScale{s, -__frcp_rn(s)};
  }
  return BlockScale{m / kE4m3Max, 0.f};
}

// -(v / s) given r = -1 / s rounded to nearest: v r is within 1.5 units in the last place, and the correction
// by its remainder (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990) is, before its rounding, within 2^-46 of the quotient.  So it is the float32 quotient
// unless that lies so close to the middle between two floats; for e4m3 only the middles next to a boundary
// between two e4m3 values matter, and all 5696 pairs of significands whose quotient is within 2^-41 of one
// of those come out right (enumerated).  Where v's remainder is subnormal the quotient is zero in e4m3.
// The sign is turned so that a zero keeps its own: an exact remainder is +0, and +0 times r adds -0 to the
// product v r of either sign (with 1 / s it would add +0, and -0 would become +0).  Two values at a time
// (packed multiply-adds).
__device__ __forceinline__ float2 minus_quotients(float v0, float v1, float s, float r) {
  float2 t;
  asm("{\n\t.reg .b64 v, r, s, t, e;\n\t"
      "mov.b64 v, {%2, %3};\n\tmov.b64 r, {%4, %4};\n\tmov.b64 s, {%5, %5};\n\t"
      "mul.rn.f32x2 t, v, r;\n\t"
      "fma.rn.f32x2 e, t, s, v;\n\t"
      "fma.rn.f32x2 t, e, r, t;\n\t"
      "mov.b64 {%0, %1}, t;\n\t}"
      : "=f"(t.x), "=f"(t.y)
      : "f"(v0), "f"(v1), "f"(r), "f"(s));
  return t;
}

// 8 quotients as e4m3; FAST: r is minus the scale's reciprocal
template <bool FAST>
__device__ __forceinline__ uint2 e4m3_8(const float (&v)[8], BlockScale bs) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // s == 0: a block of zeros (or one whose scale underflowed): zeros, not 0 / 0
    const float2 t = FAST ? minus_quotients(v[2 * i], v[2 * i + 1], bs.s, bs.r)
                          : bs.s == 0.f ? make_float2(0.f, 0.f) : make_float2(v[2 * i] / bs.s, v[2 * i + 1] / bs.s);
    w[i] = __nv_cvt_float2_to_fp8x2(t, __NV_SATFINITE, __NV_E4M3);
  }
  const uint32_t flip = FAST ? 0x80808080u : 0u;   // (negating the floats instead: gathered rows 15.4 us, not 15.1)
  return make_uint2((w[0] | (w[1] << 16)) ^ flip, (w[2] | (w[3] << 16)) ^ flip);
}

// the same columns of a row of q
template <bool VEC, typename Held>
__device__ __forceinline__ void store_16(uint8_t* row, int c, int cols, int align, const Held (&held)[2], BlockScale bs) {
  float v[2][8];
  held[0].floats(v[0]);
  held[1].floats(v[1]);
  uint2 o[2];
  if (bs.r != 0.f) {
    o[0] = e4m3_8<true>(v[0], bs);
    o[1] = e4m3_8<true>(v[1], bs);
  } else {
    o[0] = e4m3_8<false>(v[0], bs);
    o[1] = e4m3_8<false>(v[1], bs);
  }
  if (VEC && align >= 16 && c + 16 <= cols) {
    *reinterpret_cast<uint4*>(row + c) = make_uint4(o[0].x, o[0].y, o[1].x, o[1].y);
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int first = c + (VEC ? 8 : 64) * h;
    if (VEC && first + 8 <= cols) {
      *reinterpret_cast<uint2*>(row + first) = o[h];
    } else if (!VEC || first < cols) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = VEC ? first + i : first + 8 * i;
        if (at < cols) row[at] = static_cast<uint8_t>((i < 4 ? o[h].x : o[h].y) >> (8 * (i & 3)));
      }
    }
  }
}

// g / (1 + exp(-g)), for negative g as g exp(g) / (1 + exp(g)): the divisor stays within [1, 2], where the
// approximate reciprocal is within an ulp (one of more than 2^126 is zero, which g = -88 would come to)
__device__ __forceinline__ float gate(float g) {
  const float e = expf(-fabsf(g));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return (g >= 0.f ? g : g * e) * r;
}

// max|v| of 16 values (a NaN stays one)
__device__ __forceinline__ float max_abs(const RawF32 (&v)[2]) {
  float m[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 8; i += 2)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m[h]) : "f"(__uint_as_float(v[h].w[i])), "f"(__uint_as_float(v[h].w[i + 1])));
  return max_nan(m[0], m[1]);
}
__device__ __forceinline__ float max_abs(const RawBf16 (&v)[2]) {
  uint32_t m[2] = {0, 0};   // two values at a time, as they are
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      asm("{\n\t.reg .b32 a;\n\tabs.bf16x2 a, %1;\n\tmax.NaN.bf16x2 %0, %0, a;\n\t}" : "+r"(m[h]) : "r"(v[h].w[i]));
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m[0]) : "r"(m[1]));
  return max_nan(__uint_as_float(m[0] << 16), __uint_as_float(m[0] & 0xFFFF0000u));
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
