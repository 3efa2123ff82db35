// Device-side parts shared by the kernels that quantise rows (to e4m3 with a scale per block, to int8 with a
// scale per row): values as they are in memory, the maximum, a block's scale, and quotients by it.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "linear_internal.h"

namespace convf {

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

// 16 bytes of a row of q, at the columns that load_16 reads
template <bool VEC>
__device__ __forceinline__ void store_bytes_16(uint8_t* row, int c, int cols, int align, const uint2 (&o)[2]) {
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

// the same columns of a row of q in e4m3
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
  store_bytes_16<VEC>(row, c, cols, align, o);
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

}  // namespace convf
