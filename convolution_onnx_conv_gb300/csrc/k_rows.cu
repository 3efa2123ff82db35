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
// Bound by the bytes: each row is read once, a thread holds 16 columns of it, the next row's loads are on
// their way while this one is reduced and written.  A row takes a warp, or a CTA of as many warps as it has
// columns for; rows wider than a CTA are read twice, the second time from L2.
//
// 8192 x 4096 bf16 with a bf16 residual, e4m3: 41.3 us, 5.7 TB/s (84% of a copy's rate); int8 39.5; without a residual
// 8192 x 4096 to int8 17.3 to 18.5 us, 5.5 to 5.8 TB/s.  Gated 8192 x 2 * 2048 bf16 19.6 us (floor 12.4; issue slots 53%, ALU
// 40%), fp32 24.2 for 2 * 2048 of 8192 rows (22.3).  Below 4096 columns, above 8192 and for gated bf16 rows what bounds it
// is waiting: a CTA has a row in flight and one asked for, and a row ends at a barrier.  4095 x 2000 with an fp32 residual
// 19.8 to 21.2 us, 4.3 TB/s.  Rows gathered by an index take the form with bounds tests: a permutation of 8192 x 4096 bf16 20.8 us
// (17.3 in order), 16380 rows of 4095 x 2000 20.1 (floor 7.3, each row four times).
//
// Rows that do not begin on 16 bytes (any odd number of bf16 columns) are read and written by 16 bytes all the
// same: aligned units that hold a thread's columns, shifted into place in registers by what is the same for the
// whole row.  (8191 x 1001 bf16 with a residual 22.9 us, element by element 31.6.)
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

// g / (1 + exp(-g)) of 8 values, each operation rounded to nearest.  Where no |g| is large the quotient is the
// reciprocal, refined once (to nearest), and a product with two corrections, as above and two at a time.
__device__ __forceinline__ void gate_8(float (&g)[8]) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(g[i]));
  if (top < 64.f) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float d0 = 1.f + expf(-g[i]), d1 = 1.f + expf(-g[i + 1]);
      float r0, r1;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(d0));
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(d1));
      asm("{\n\t.reg .b64 g, d, r, q, e, one;\n\t"
          "mov.b64 g, {%0, %1};\n\tmov.b64 d, {%2, %3};\n\tmov.b64 r, {%4, %5};\n\tmov.b64 one, {%6, %6};\n\t"
          "fma.rn.f32x2 e, d, r, one;\n\t"   // (d: minus the divisor)
          "fma.rn.f32x2 r, e, r, r;\n\t"
          "mul.rn.f32x2 q, g, r;\n\t"
          "fma.rn.f32x2 e, d, q, g;\n\t"
          "fma.rn.f32x2 q, e, r, q;\n\t"
          "fma.rn.f32x2 e, d, q, g;\n\t"
          "fma.rn.f32x2 q, e, r, q;\n\t"
          "mov.b64 {%0, %1}, q;\n\t}"
          : "+f"(g[i]), "+f"(g[i + 1])
          : "f"(-d0), "f"(-d1), "f"(r0), "f"(r1), "f"(1.f));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = __fdiv_rn(g[i], 1.f + expf(-g[i]));
  }
}

// the row's scale for int8, and the reciprocal for quotients(), or 0 where a remainder could be subnormal or
// the scale is no number
__device__ __forceinline__ BlockScale int8_scale_of(float m) {
  if (m > 0x1p-50f && m < 0x1p60f) {
    // m * (1/127) in two parts, as scale_of(); equal to the quotient for every one of the 2^23 fractions
    const float s = fmaf(m, 0x1.020408p-7f, m * 0x1.020408p-35f);
    return BlockScale{s, __frcp_rn(s)};
  }
  return BlockScale{m / 127.f, 0.f};
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

// ------------------------------------------------------------------------------ 16 columns of a row

// What a thread has asked for of a row: 16 columns as they are in memory.  ALIGN: bytes on which rows begin, 16, 8,
// or 0 for fewer: then from the 16-byte unit that holds the first column; 32: also, every thread has its 16 columns,
// of a row that is there, and nothing is checked.
template <typename T, int ALIGN>
struct Piece {
  static constexpr int kWords = 4 * sizeof(T);   // of 16 columns
  uint32_t w[kWords + (ALIGN ? 0 : 4)];
  int first;   // ALIGN = 0: bytes before the first column
};

template <int BYTES>
__device__ __forceinline__ void load_unit(const uint8_t* at, uint32_t* w) {
  if constexpr (BYTES == 32) {
    load_32_bytes(at, w);
  } else if constexpr (BYTES == 16) {
    const uint4 t = *reinterpret_cast<const uint4*>(at);
    w[0] = t.x;
    w[1] = t.y;
    w[2] = t.z;
    w[3] = t.w;
  } else {
    const uint2 t = *reinterpret_cast<const uint2*>(at);
    w[0] = t.x;
    w[1] = t.y;
  }
}

// Asks for 16 columns of a row in whole units, which may reach past the row's end but not out of the buffer,
// [begin, end): returns whether they lie inside.  Where they do not, or where there is nothing to ask for, `spare` is
// read, units of the same buffer: no branches around the loads, so that nothing waits for them at the end of one
// (with branches the next row's loads were waited for before this row's work).
template <typename T, int ALIGN>
__device__ __forceinline__ bool ask(Piece<T, ALIGN>& v, const T* at, bool any, const uint8_t* begin, const uint8_t* end,
                                    const uint8_t* spare, int align) {
  constexpr int kBytes = sizeof(v.w);
  const uint8_t* from = reinterpret_cast<const uint8_t*>(at);
  if constexpr (ALIGN == 32) {
#pragma unroll
    for (int k = 0; k < kBytes; k += 32) load_unit<32>(from + k, v.w + k / 4);
    return true;
  }
  v.first = 0;
  if constexpr (!ALIGN) {
    v.first = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15);
    from -= v.first;
  }
  const bool inside = from + kBytes <= end && (ALIGN || from >= begin);
  from = any && inside ? from : spare;
  auto units = [&](auto bytes) {
    constexpr int U = decltype(bytes)::value;
#pragma unroll
    for (int k = 0; k < kBytes; k += U) load_unit<U>(from + k, v.w + k / 4);
  };
  if (ALIGN == 16 && align == 32)
    units(std::integral_constant<int, 32>{});
  else
    units(std::integral_constant<int, ALIGN == 8 ? 8 : 16>{});
  return inside || !any;
}
// the same by the elements
template <typename T, int ALIGN>
__device__ __forceinline__ void ask_elements(Piece<T, ALIGN>& v, const T* at, int n) {
  v.first = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (i < n) {
      if constexpr (sizeof(T) == 2)
        v.w[i >> 1] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(at + i)) << (16 * (i & 1));
      else
        v.w[i] = __float_as_uint(at[i]);
    }
  }
}

// The first KEEP words from the byte `by` on (a multiple of an element's size, at most 15; the same for a whole row:
// its lanes take the same case).
template <typename T, int KEEP, int N>
__device__ __forceinline__ void shift_down(uint32_t (&w)[N], int by) {
  const int odd = sizeof(T) == 2 ? 8 * (by & 2) : 0;
  auto from = [&](auto words) {
    constexpr int k = decltype(words)::value;
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
      if constexpr (sizeof(T) == 2)
        w[i] = __funnelshift_r(w[i + k], i + k + 1 < N ? w[i + k + 1] : 0u, odd);
      else
        w[i] = w[i + k];
    }
  };
  switch (by >> 2) {
    case 0: if (odd) from(std::integral_constant<int, 0>{}); break;
    case 1: from(std::integral_constant<int, 1>{}); break;
    case 2: from(std::integral_constant<int, 2>{}); break;
    default: from(std::integral_constant<int, 3>{}); break;
  }
}

// The 16 columns as floats, zeros past the n-th.
template <typename T, int ALIGN>
__device__ __forceinline__ void settle(Piece<T, ALIGN>& v, int n, float (&f)[16]) {
  if constexpr (!ALIGN) shift_down<T, Piece<T, ALIGN>::kWords>(v.w, v.first);
  if (ALIGN != 32 && n < 16) {
#pragma unroll
    for (int i = 0; i < Piece<T, ALIGN>::kWords; ++i) {
      if constexpr (sizeof(T) == 2)
        v.w[i] = 2 * i + 1 < n ? v.w[i] : 2 * i < n ? v.w[i] & 0xFFFFu : 0u;
      else
        v.w[i] = i < n ? v.w[i] : 0u;
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if constexpr (sizeof(T) == 2)
      f[i] = __uint_as_float(i & 1 ? v.w[i >> 1] & 0xFFFF0000u : v.w[i >> 1] << 16);
    else
      f[i] = __uint_as_float(v.w[i]);
  }
}

// Writes the 16 columns of each lane of a warp, from the row's column c on (`n` of the lane's there): 16 bytes at a
// time.  ALIGN = 0: a lane writes the aligned units that end in its columns, with the lane before's last bytes in the
// first; units that are not all of this warp's or this row's go element by element.
template <typename R, int ALIGN>
__device__ __forceinline__ void put_16(R* at, int n, const float (&f)[16]) {
  constexpr int kWords = 4 * sizeof(R), kEach = 16 / sizeof(R);   // of a unit
  const int lane = threadIdx.x & 31;
  uint32_t w[kWords + 4];
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    if constexpr (sizeof(R) == 2) {
      const __nv_bfloat162 two = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[4 + i] = *reinterpret_cast<const uint32_t*>(&two);
    } else {
      w[4 + i] = __float_as_uint(f[i]);
    }
  }
  typedef typename std::conditional<sizeof(R) == 2, uint16_t, uint32_t>::type Bits;
  const int by = !ALIGN ? static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15) : 0;   // the same for the whole row
  const int before = by / static_cast<int>(sizeof(R));   // elements of the lane before in this lane's first unit
  if (by) {
    if (lane == 31) {   // the warp's last elements, which are in no lane's units
#pragma unroll
      for (int i = 16 - kEach + 1; i < 16; ++i)
        if (i >= 16 - before && i < n) {
          const uint32_t word = w[4 + i * static_cast<int>(sizeof(R)) / 4];
          reinterpret_cast<Bits*>(at)[i] = static_cast<Bits>(sizeof(R) == 2 && (i & 1) ? word >> 16 : word);
        }
    }
    uint32_t last[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) last[i] = __shfl_up_sync(0xFFFFFFFFu, w[kWords + i], 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = last[i];
    shift_down<R, kWords>(w, 16 - by);
  } else {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = w[4 + i];
  }
  auto unit = [&](int k) {   // whole
    R* to = at + kEach * k - before;
    if (ALIGN != 8) {
      *reinterpret_cast<uint4*>(to) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    } else {
      reinterpret_cast<uint2*>(to)[0] = make_uint2(w[4 * k], w[4 * k + 1]);
      reinterpret_cast<uint2*>(to)[1] = make_uint2(w[4 * k + 2], w[4 * k + 3]);
    }
  };
  if (ALIGN == 32 || (n >= 16 && (!by || lane > 0))) {
#pragma unroll
    for (int k = 0; k < kWords / 4; ++k) unit(k);
    return;
  }
  if constexpr (ALIGN != 32) {
#pragma unroll
    for (int k = 0; k < kWords / 4; ++k) {
      const int e0 = kEach * k - before;   // the unit's first element, counted from this lane's first
      if ((e0 >= 0 || lane > 0) && e0 + kEach <= n) {
        unit(k);
      } else {
#pragma unroll
        for (int i = 0; i < kEach; ++i)
          if ((e0 + i >= 0 || lane > 0) && e0 + i < n) {
            const uint32_t word = w[4 * k + i * static_cast<int>(sizeof(R)) / 4];
            reinterpret_cast<Bits*>(at)[e0 + i] = static_cast<Bits>(sizeof(R) == 2 && (i & 1) ? word >> 16 : word);
          }
      }
    }
  }
}

// 16 bytes of a row of q, `n` of them there
__device__ __forceinline__ void put_bytes_16(uint8_t* at, int n, int align, const uint2 (&o)[2]) {
  if (n >= 16 && align >= 16) {
    *reinterpret_cast<uint4*>(at) = make_uint4(o[0].x, o[0].y, o[1].x, o[1].y);
    return;
  }
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const uint32_t w = i < 8 ? (i < 4 ? o[0].x : o[0].y) : (i < 12 ? o[1].x : o[1].y);
    if (align >= 4 && i + 4 <= n) {
      *reinterpret_cast<uint32_t*>(at + i) = w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < n) at[i + j] = static_cast<uint8_t>(w >> (8 * j));
    }
  }
}

struct NoResidual {};
template <typename R>
constexpr bool kHasResidual = !std::is_same<R, NoResidual>::value;

// What a thread has asked for of a row
template <typename T, typename R, int ALIGN>
struct RowPieces {
  typedef typename std::conditional<kGated, T, typename std::conditional<kHasResidual<R>, R, T>::type>::type Second;
  Piece<T, ALIGN> x;
  Piece<Second, ALIGN> second;   // the gated row's other half, or the residual (else not used)
  int row, n;                    // of x; columns from the first on that are there
  bool whole;                    // all of it has been asked for
};

// Threads on an SM, by the registers that a row's bytes on their way take.
template <typename T, typename R, int ALIGN>
constexpr int kBytesPerColumn = sizeof(T) * (kGated ? 2 : 1) + (kHasResidual<R> ? sizeof(typename std::conditional<kHasResidual<R>, R, T>::type) : 0) + (ALIGN ? 0 : 2);
template <typename T, typename R, int ALIGN>
constexpr int kThreadsPerSm = kBytesPerColumn<T, R, ALIGN> <= 4 ? 1024 : kBytesPerColumn<T, R, ALIGN> <= 8 ? 768 : 512;
// Two CTAs of the two-pass form on an SM: 64 registers a thread, too few for a row's bytes and a second operand's (a
// residual's, a gate's other half), with which it spills 16 to 1116 bytes.  3000 x 9001 fp32 with an fp32 residual 427 us
// (floor 52), 3000 x 20000 508 (115), bf16 with bf16 182 (62); gated fp32 4096 x 2 * 12001 386 (65).  Without a second
// operand it spills up to 164 bytes: 4096 x 20000 bf16 74 us (36), fp32 90 (61).
constexpr int kWideThreads = 512;

// How a row is shared out: to a warp (up to 512 columns), to a CTA of as many warps as 512 columns each take, or to a
// CTA that passes over it twice.
enum Share : int { kWarpRow = 0, kCtaRow = 1, kWideRow = 2 };

template <typename T, typename R, int ALIGN, int SHARE>
__global__ void __launch_bounds__(SHARE == kWarpRow ? 128 : SHARE == kWideRow ? kWideThreads : kThreadsPerSm<T, R, ALIGN>,
                                  SHARE == kWarpRow ? kThreadsPerSm<T, R, ALIGN> / 128 : SHARE == kWideRow ? 2 : 1)
    rows_kernel(const RowsParams p) {
  constexpr bool RES = kHasResidual<R>, WHOLE = ALIGN == 32;
  typedef RowPieces<T, R, ALIGN> Pieces;
  typedef typename Pieces::Second Second;
  pdl_launch_dependents();
  pdl_wait_prior();
  __shared__ float2 part[2][32];   // by row parity: sum and maximum of each of a row's warps
  const int lane = threadIdx.x & 31, warps = SHARE == kWarpRow ? 1 : static_cast<int>(blockDim.x) >> 5;
  const int tid = SHARE == kWarpRow ? lane : static_cast<int>(threadIdx.x);
  const long long step = static_cast<long long>(gridDim.x) * (SHARE == kWarpRow ? 4 : 1);
  long long r = SHARE == kWarpRow ? static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5) : blockIdx.x;
  const int first = tid * 16;   // this thread's columns

  auto source = [&](long long row) -> int {
    if constexpr (WHOLE) return static_cast<int>(row < p.rows ? row : p.rows - 1);   // (a last row is asked for once more)
    return row >= p.rows ? -1 : p.index ? p.index[row] : static_cast<int>(row);
  };
  auto x_of = [&](int src, int c) { return static_cast<const T*>(p.x) + static_cast<long long>(src) * p.ldx + c; };
  auto res_of = [&](int src, int c) {
    if constexpr (RES)
      return static_cast<const R*>(p.residual) + static_cast<long long>(src) * p.ldr + c;
    else
      return static_cast<const Second*>(nullptr);
  };
  // columns c .. of row `src`; a source outside of x is a row of zeros
  const uint8_t *x_begin = static_cast<const uint8_t*>(p.x), *r_begin = static_cast<const uint8_t*>(p.residual);
  auto fetch = [&](Pieces& v, int src, int c) {
    const bool there = WHOLE || (src >= 0 && src < p.x_rows);
    v.row = there ? src : 0;
    v.n = WHOLE ? 16 : there ? p.cols - c : 0;
    if (!WHOLE && p.small) {
      v.x.first = v.second.first = 0;
      v.whole = v.n <= 0;
      return;
    }
    const bool any = v.n > 0;
    v.whole = ask<T, ALIGN>(v.x, x_of(v.row, c), any, x_begin, p.x_end, p.x_spare, p.x_align);
    if constexpr (kGated) v.whole = ask<Second, ALIGN>(v.second, x_of(v.row, c) + p.cols, any, x_begin, p.x_end, p.x_spare, p.x_align) && v.whole;
    if constexpr (RES) v.whole = ask<Second, ALIGN>(v.second, res_of(v.row, c), any, r_begin, p.r_end, p.r_spare, p.r_align) && v.whole;
  };
  // h of columns c .. (what the norm takes the squares of)
  auto values = [&](Pieces& v, int c, float (&h)[16]) {
    const int n = v.n;
    if (!WHOLE && !v.whole) {   // a buffer's first or last columns
#pragma unroll
      for (int i = 0; i < sizeof(v.x.w) / 4; ++i) v.x.w[i] = 0;
      ask_elements<T, ALIGN>(v.x, x_of(v.row, c), n);
      if constexpr (kGated || RES) {
#pragma unroll
        for (int i = 0; i < sizeof(v.second.w) / 4; ++i) v.second.w[i] = 0;
        ask_elements<Second, ALIGN>(v.second, kGated ? reinterpret_cast<const Second*>(x_of(v.row, c) + p.cols) : res_of(v.row, c), n);
      }
    }
    settle<T, ALIGN>(v.x, n, h);
    if constexpr (kGated) {
      float u[16], g[2][8];
      settle<Second, ALIGN>(v.second, n, u);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[k][i] = h[8 * k + i];
        gate_8(g[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[8 * k + i] = __fmul_rn(g[k][i], u[8 * k + i]);
      }
    }
    if constexpr (RES) {
      float u[16];
      settle<Second, ALIGN>(v.second, n, u);
#pragma unroll
      for (int i = 0; i < 16; ++i) h[i] = __fadd_rn(h[i], u[i]);
    }
  };
  auto keep = [&](long long row, int c, const float (&h)[16]) {
    if constexpr (RES)
      if (p.h) put_16<R, ALIGN>(static_cast<R*>(p.h) + row * p.ldh + c, WHOLE ? 16 : p.cols - c, h);
  };
  auto weigh = [&](float (&h)[16], int c) {   // h -> t
    if constexpr (kNorm) {
      if (!p.weight) return;
      const int n = p.cols - c;
      if (WHOLE || (n >= 16 && p.w_align >= 16)) {
        const uint4* w = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.weight) + static_cast<long long>(c) * (p.weight_bf16 ? 2 : 4));
        if (p.weight_bf16) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint4 v = w[k];
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              h[8 * k + 2 * i] = __fmul_rn(h[8 * k + 2 * i], __uint_as_float(u[i] << 16));
              h[8 * k + 2 * i + 1] = __fmul_rn(h[8 * k + 2 * i + 1], __uint_as_float(u[i] & 0xFFFF0000u));
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 v = w[k];
            h[4 * k] = __fmul_rn(h[4 * k], __uint_as_float(v.x));
            h[4 * k + 1] = __fmul_rn(h[4 * k + 1], __uint_as_float(v.y));
            h[4 * k + 2] = __fmul_rn(h[4 * k + 2], __uint_as_float(v.z));
            h[4 * k + 3] = __fmul_rn(h[4 * k + 3], __uint_as_float(v.w));
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < n)
            h[i] = __fmul_rn(h[i], p.weight_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.weight)[c + i])
                                                 : static_cast<const float*>(p.weight)[c + i]);
      }
    }
  };
  auto squares = [&](const float (&h)[16], float sum) {
    float a[4] = {sum, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 16; ++i) a[i & 3] = fmaf(h[i], h[i], a[i & 3]);
    return (a[0] + a[1]) + (a[2] + a[3]);
  };
  auto max_abs_16 = [&](const float (&t)[16]) {
    float m[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 16; i += 4)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m[k]) : "f"(t[i + 2 * k]), "f"(t[i + 2 * k + 1]));
    return max_nan(m[0], m[1]);
  };
  // sum and maximum over the row's threads
  auto reduce = [&](float& sum, float& m, int turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (kNorm) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    }
    // (floats of one sign compare as integers, a NaN above the infinity)
    if (kInt8) m = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m)));
    if constexpr (SHARE != kWarpRow) {
      // (two sets in turn: a warp may be a row ahead of one still reading)
      if (lane == 0) {
        part[turn][threadIdx.x >> 5] = make_float2(sum, m);
      }
      __syncthreads();
      sum = m = 0.f;
#pragma unroll 4
      for (int i = 0; i < warps; ++i) {
        const float2 t = part[turn][i];
        if (kNorm) sum += t.x;
        if (kInt8) m = max_nan(m, t.y);
      }
    }
  };
  // (rsqrtf is within 2 units in the last place; only scales have it in them)
  auto factor = [&](float sum) { return kNorm ? rsqrtf(fmaf(sum, p.inv_cols, p.eps)) : 1.f; };
  // columns from c of row `row`: int8 by the row's scale, e4m3 by each block's (8 lanes)
  auto put = [&](long long row, const float (&t)[16], int c, BlockScale bs, float f) {
    const int n = WHOLE ? 16 : p.cols - c;
    uint32_t w[2][8];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i >> 3][i & 7] = __float_as_uint(t[i]);
    uint2 o[2];
    if constexpr (kInt8) {
      o[0] = int8_8(w[0], bs);
      o[1] = int8_8(w[1], bs);
    } else {
      const float v[2][8] = {{t[0], t[1], t[2], t[3], t[4], t[5], t[6], t[7]}, {t[8], t[9], t[10], t[11], t[12], t[13], t[14], t[15]}};
#pragma unroll
      for (int k = 0; k < 2; ++k) o[k] = bs.r != 0.f ? e4m3_8<true>(v[k], bs) : e4m3_8<false>(v[k], bs);
      const int block = c / kScaleBlock;
      if ((lane & 7) == 0 && (WHOLE || block < p.nblk)) p.scale[row * p.lds + block] = bs.s * f;
    }
    if (n > 0) put_bytes_16(p.q + row * p.ldq + c, n, WHOLE ? 16 : p.q_align, o);
  };
  auto block_scale = [&](const float (&t)[16]) {
    float m = max_abs_16(t);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    return scale_of(m);
  };

  // (whole warps, or whole CTAs, share a row: they leave the loops together)
  if constexpr (SHARE != kWideRow) {
    Pieces v;
    fetch(v, source(r), first);
    int next_src = source(r + step);
    for (int turn = 0; r < p.rows; turn ^= 1) {
      float t[16];
      values(v, first, t);
      if (WHOLE || r + step < p.rows) fetch(v, next_src, first);
      next_src = source(r + 2 * step);
      keep(r, first, t);
      float sum = kNorm ? squares(t, 0.f) : 0.f, m = 0.f;
      weigh(t, first);
      BlockScale bs{};
      if constexpr (kInt8)
        m = max_abs_16(t);
      else
        bs = block_scale(t);
      reduce(sum, m, turn);
      if constexpr (kInt8) {
        bs = int8_scale_of(m);
        if (tid == 0) p.scale[r] = bs.s * factor(sum);
        put(r, t, first, bs, 0.f);
      } else {
        put(r, t, first, bs, factor(sum));
      }
      r += step;
    }
  } else {
    // (a thread reads the same elements in both passes, and h is written in the second: it may lie on the residual)
    const int wide = 16 * static_cast<int>(blockDim.x);
    for (int turn = 0; r < p.rows; turn ^= 1) {
      const int src = source(r);
      float sum = 0.f, m = 0.f;
      for (int c = first; c - first < p.cols; c += wide) {
        Pieces v;
        float t[16];
        fetch(v, src, c);
        values(v, c, t);
        if (kNorm) sum = squares(t, sum);
        if (kInt8) {
          weigh(t, c);
          m = max_nan(m, max_abs_16(t));
        }
      }
      reduce(sum, m, turn);
      BlockScale bs{};
      const float f = factor(sum);
      if constexpr (kInt8) {
        bs = int8_scale_of(m);
        if (tid == 0) p.scale[r] = bs.s * f;
      }
      for (int c = first; c - first < p.cols; c += wide) {
        Pieces v;
        float t[16];
        fetch(v, src, c);
        values(v, c, t);
        keep(r, c, t);
        weigh(t, c);
        if constexpr (!kInt8) bs = block_scale(t);
        put(r, t, c, bs, f);
      }
      r += step;
    }
  }
}

template <typename T, typename R, int ALIGN>
cudaError_t launch_s(const RowsParams& p, int num_sms, cudaStream_t stream) {
  constexpr int kThreads = kThreadsPerSm<T, R, ALIGN>;
  auto go = [&](void (*kernel)(RowsParams), int threads, int rows_per_cta, int per_sm) {
    const long long ctas = (p.rows + rows_per_cta - 1LL) / rows_per_cta, cap = static_cast<long long>(num_sms) * per_sm;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas < cap ? ctas : cap)), dim3(threads), 0, stream, 1, p);
  };
  if constexpr (ALIGN == 32) {
    return go(rows_kernel<T, R, 32, kCtaRow>, p.cols / 16, 1, kThreads / (p.cols / 16));
  } else {
    if (p.cols <= 512) return go(rows_kernel<T, R, ALIGN, kWarpRow>, 128, 4, kThreads / 128);
    const int threads = (p.cols - 1) / 512 * 32 + 32;
    if (threads <= kThreads) return go(rows_kernel<T, R, ALIGN, kCtaRow>, threads, 1, kThreads / threads);
    return go(rows_kernel<T, R, ALIGN, kWideRow>, kWideThreads, 1, 2);
  }
}

template <typename T, typename R>
cudaError_t launch_r(const RowsParams& p, int num_sms, cudaStream_t stream) {
  const int align = p.x_align < p.r_align ? p.x_align : p.r_align;
  if (align == 32 && p.q_align >= 16 && p.w_align >= 16 && p.cols % 512 == 0 && p.cols / 16 <= kThreadsPerSm<T, R, 32> && !p.index)
    return launch_s<T, R, 32>(p, num_sms, stream);
  return align >= 16 ? launch_s<T, R, 16>(p, num_sms, stream)
         : align == 8 ? launch_s<T, R, 8>(p, num_sms, stream)
                      : launch_s<T, R, 0>(p, num_sms, stream);
}

template <typename T>
cudaError_t launch_t(const RowsParams& p, int num_sms, cudaStream_t stream) {
  if constexpr (kNorm) {
    if (p.residual)
      return p.residual_bf16 ? launch_r<T, __nv_bfloat16>(p, num_sms, stream) : launch_r<T, float>(p, num_sms, stream);
  }
  return launch_r<T, NoResidual>(p, num_sms, stream);
}

}  // namespace

template <>
cudaError_t launch_rows<kKind>(const RowsParams& p, bool bf16, int num_sms, cudaStream_t stream) {
  return bf16 ? launch_t<__nv_bfloat16>(p, num_sms, stream) : launch_t<float>(p, num_sms, stream);
}

}  // namespace convf
