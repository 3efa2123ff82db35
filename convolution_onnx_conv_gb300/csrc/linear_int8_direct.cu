// Linear layers on int8 operands for a handful of rows per weight matrix: y = x W^T with integer sums, from operands that
// go from memory to registers and nowhere else.
//
// With few rows of x a weight byte takes part in few products: its way from memory is what the layer costs.  The tcgen05
// form for few rows (tc_linear_int8_few.cu) takes it through shared memory, a conversion to fp16, TMEM, the MMAs, their
// sums' way back and a cluster's exchange, one behind the other: 10 us for 1 x 4096 x 4096, whose bytes take 2.5.  Here a
// lane asks at once for all that its next products read, and integers stay integers.
//
// Up to 4 rows: dp4a (four products of 8 bits added to an integer; an SM does 16 a cycle, so a row takes 64 bytes of
// weights per cycle, and memory brings 23).  A warp takes 2 weight rows whole, 512 bytes of each per load, and adds its
// lanes' sums by one instruction each (redux); of short rows it takes 4 or 8, so that a lane still has 8 loads on their
// way.  Warps share nothing but the schedule, wait for nothing but loads, and have tiles one behind another: one search
// of the schedule, and the next tile's rows are known and come to L2 meanwhile.  Bound by memory: 16384 x 16384, 1 row
// 40.3 us (6.7 TB/s, 98% of a copy's rate), 24 experts of 2048 x 2048, a row each, 14.2 (through the tensor cores 24.1);
// 4096 x 4096, 1 row 2.8 us, 4 rows 3.8.  (The same with 5 CTAs of 102 registers on an SM, not 4 of 128: 3.0 and 4.7.)  With 4
// and 8 weight rows a warp a tile of 4 rows spills (84 and 248 bytes): 20000 x 1024, 1 row 4.5 us, 4 rows 6.2; 20000 x 512
// 3.9 and 4.9.
//
// Up to 16 rows: mma.sync m16n8k32, 25 cycles of an SM for 512 bytes of weights and 8 rows (20 bytes per cycle, which is
// what bounds it; with both operands as fp16 the MMAs take 16 cycles, but the conversion 12 more).  A CTA takes 16 weight
// rows and its warps share their bytes: 16 bytes of each of two rows are a lane's part of two MMAs' first operands (which
// 32 of the 64 values are an MMA's, and in which order, is the same for both operands and otherwise free).  The warps'
// sums meet in shared memory once a tile.  4096 x 4096, 8 rows 5.3 us (11.7), 16 rows 7.9 (12.5); 8192 x 8192, 8 rows 13.8.
#include "linear_int8_dev.cuh"

namespace convf {

namespace {

__device__ __forceinline__ uint4 load_weights(const int8_t* at) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(at));
  return v;
}

// ------------------------------------------------------------------------------ up to 4 rows

constexpr int kDotRows = kInt8DotRows;   // of x, of a warp's tile
constexpr int kDotUnits = 8;             // 16-byte units of weights that a lane asks for at once
constexpr int kDotThreads = 32 * kInt8DotWarps;

__device__ __forceinline__ int dot_16(const uint4& a, const uint4& b, int sum) {
  sum = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), sum);
  sum = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), sum);
  sum = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), sum);
  return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), sum);
}

// A warp's tile of R rows at most (rows past q.rows are the last one again, and not stored).
template <int R, int COLS>
__device__ __forceinline__ void dot_tile(const LinearParams& p, const Int8Operands& o, const LinearTile& q) {
  constexpr int kAhead = kDotUnits / COLS;   // of each row
  const int lane = threadIdx.x & 31, units = o.K >> 4;
  const int8_t* w[COLS];
  const int8_t* x[R];
#pragma unroll
  for (int i = 0; i < COLS; ++i) w[i] = o.w + q.e * o.w_stride + min(q.n0 + i, p.N - 1) * o.ldw;
#pragma unroll
  for (int r = 0; r < R; ++r) x[r] = o.x + (q.row0 + min(r, q.rows - 1)) * o.ldx;
  // the lane's element: its scales are on their way meanwhile
  const int mr = lane / COLS, n = q.n0 + lane % COLS;
  const bool mine = mr < q.rows && mr < R && n < p.N;
  float ws = 0.f, bias = 0.f, xs = 0.f;
  if (mine) {
    const long long en = static_cast<long long>(q.e) * p.N + n;
    ws = p.w_scale[en];
    bias = p.bias ? p.bias[en] : kNoBias;
    xs = p.x_scale[(q.row0 + mr) * p.xs_row];
  }
  int acc[R][COLS];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < COLS; ++i) acc[r][i] = 0;
  for (int u0 = lane; u0 - lane < units; u0 += 32 * kAhead) {
    uint4 v[kAhead][COLS];
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
#pragma unroll
      for (int i = 0; i < COLS; ++i) {
        v[a][i] = make_uint4(0, 0, 0, 0);
        if (u0 + 32 * a < units) v[a][i] = load_weights(w[i] + 16LL * (u0 + 32 * a));
      }
    constexpr int kX = R <= 2 || kAhead < 2 ? kAhead : 2;   // units of x asked for at once
#pragma unroll
    for (int a0 = 0; a0 < kAhead; a0 += kX) {
      uint4 h[kX][R];
#pragma unroll
      for (int a = 0; a < kX; ++a)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          h[a][r] = make_uint4(0, 0, 0, 0);
          if (u0 + 32 * (a0 + a) < units) h[a][r] = *reinterpret_cast<const uint4*>(x[r] + 16LL * (u0 + 32 * (a0 + a)));
        }
#pragma unroll
      for (int a = 0; a < kX; ++a)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < COLS; ++i) acc[r][i] = dot_16(v[a0 + a][i], h[a][r], acc[r][i]);
    }
  }
  if (lane < (o.K & 15)) {   // what is behind the last whole unit (there may be no more bytes than that)
    const long long at = 16LL * units + lane;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < COLS; ++i) acc[r][i] += w[i][at] * x[r][at];
  }
  int sum = 0;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < COLS; ++i) {
      const int s = __reduce_add_sync(0xFFFFFFFFu, acc[r][i]);
      if (lane == r * COLS + i) sum = s;
    }
  if (mine) int8_put(p, q.row0 + mr, n, Int8Finish{ws, bias, p.lo, p.hi}(sum, xs));
}

// A warp's tiles one behind another: an expert's row tiles, then the next weight rows, then the next expert with rows.
template <int COLS>
struct DotWalk {
  RowGroup g;
  int e, m, mt, n0;   // mt: row tiles of the expert
  __device__ __forceinline__ void open(const LinearParams& p) {
    g = row_group(p, e);
    mt = (g.last - g.first + kDotRows - 1) / kDotRows;
  }
  // tile t of all
  __device__ __forceinline__ void start(const LinearParams& p, const int* prefix, long long t) {
    e = 0;
    if (p.offsets) {
      int lo = 0, hi = expert_pairs(p);   // the last pair whose tiles start at or before t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (static_cast<long long>(prefix[mid]) * p.n_tiles <= t)
          lo = mid;
        else
          hi = mid;
      }
      t -= static_cast<long long>(prefix[lo]) * p.n_tiles;
      e = 2 * lo;
    }
    open(p);
    if (t >= static_cast<long long>(mt) * p.n_tiles) {
      t -= static_cast<long long>(mt) * p.n_tiles;
      ++e;
      open(p);
    }
    const int nt = static_cast<int>(t / mt);
    m = static_cast<int>(t - static_cast<long long>(nt) * mt);
    n0 = nt * COLS;
  }
  __device__ __forceinline__ void next(const LinearParams& p) {   // (there is one)
    if (++m < mt) return;
    m = 0;
    n0 += COLS;
    if (n0 < p.N) return;
    n0 = 0;
    do {
      ++e;
      open(p);
    } while (mt == 0);
  }
  __device__ __forceinline__ LinearTile tile() const {
    const int row0 = g.first + m * kDotRows;
    return LinearTile{e, row0, min(kDotRows, g.last - row0), n0};
  }
  // this tile's weights to L2
  __device__ __forceinline__ void prefetch(const LinearParams& p, const Int8Operands& o) const {
    const int8_t* w = o.w + e * o.w_stride + n0 * o.ldw;
    for (int at = (threadIdx.x & 31) * 128; at < o.K; at += 4096)
#pragma unroll
      for (int i = 0; i < COLS; ++i)
        if (n0 + i < p.N) asm volatile("prefetch.global.L2 [%0];" ::"l"(w + i * o.ldw + at));
  }
};

template <int COLS>
__global__ void __launch_bounds__(kDotThreads, 4) linear_int8_dot_kernel(const LinearParams p, const Int8Operands o) {
  __shared__ int prefix[kScheduleBytes / 4];
  const int warp = blockIdx.x * kInt8DotWarps + (threadIdx.x >> 5);
  const long long warps = static_cast<long long>(gridDim.x) * kInt8DotWarps;
  long long tiles = 0, t = 0, end = 0;
  auto share = [&] {   // of the tiles, this warp's
    t = tiles * warp / warps;
    end = tiles * (warp + 1) / warps;
  };
  DotWalk<COLS> walk;
  pdl_launch_dependents();
  if (!p.offsets) {   // one layer: its tiles are known, and its weights can come to L2, before the kernel before has ended
    tiles = (p.rows + kDotRows - 1LL) / kDotRows * p.n_tiles;
    share();
    if (t < end) {
      walk.start(p, prefix, t);
      walk.prefetch(p, o);
    }
  }
  pdl_wait_prior();
  if (p.offsets) {
    if (threadIdx.x < 32) build_schedule(p, kDotRows, prefix, blockIdx.x == 0);
    __syncthreads();
    tiles = tile_count(p, prefix);
    share();
    if (t < end) walk.start(p, prefix, t);
  }
  while (t < end) {
    const LinearTile q = walk.tile();
    if (++t < end) {
      walk.next(p);
      // (Rows of 1 to 8 KB: 64 experts of 2048 x 2048 36.1 us, 42.8 without; 4096 x 1024 40.0, 45.3.  A warp's longer
      // rows keep memory busy by themselves, 16384 x 16384 38.5 us without and 46.6 with; shorter ones' time is too short.)
      if (walk.m == 0 && o.K >= 1024 && o.K <= 8192) walk.prefetch(p, o);
    }
    if (q.rows == 1)
      dot_tile<1, COLS>(p, o, q);
    else if (q.rows == 2)
      dot_tile<2, COLS>(p, o, q);
    else
      dot_tile<4, COLS>(p, o, q);
  }
}

// ------------------------------------------------------------------------------ up to 16 rows

constexpr int kRows = kInt8MmaRows, kCols = kInt8MmaCols;   // of a CTA's tile: rows of x, weight rows
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kSegment = 128;   // bytes of a row that a warp takes at a time, then the next warp the next
constexpr int kAhead = 2;       // such segments that a warp asks for at once
constexpr int kPitch = kRows + 1;

__device__ __forceinline__ uint4 load_bytes(const int8_t* at, int n) {
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 15; ++i)
    if (i < n) w[i >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(at[i])) << (8 * (i & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// acc (16 x 8) += A (16 x 32) B (32 x 8)
__device__ __forceinline__ void mma_int8(int (&acc)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(acc[0]), "+r"(acc[1]), "+r"(acc[2]), "+r"(acc[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 64 values of k: `lo` and `hi` 16 of each of the lane's weight rows, `b` of its row of x
__device__ __forceinline__ void mma_64(int (&acc)[4], const uint4& lo, const uint4& hi, const uint4& b) {
  mma_int8(acc, lo.x, hi.x, lo.y, hi.y, b.x, b.y);
  mma_int8(acc, lo.z, hi.z, lo.w, hi.w, b.z, b.w);
}

// This warp's part of a tile's sums, of NB groups of 8 rows of x: at `red`, [kCols][kPitch].
template <int NB>
__device__ __forceinline__ void sums_of(const LinearParams& p, const Int8Operands& o, const LinearTile& q, int* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, units = o.K >> 4, row = lane >> 2;
  const int8_t* w0 = o.w + q.e * o.w_stride;
  const int8_t* lo = w0 + min(q.n0 + row, p.N - 1) * o.ldw;
  const int8_t* hi = w0 + min(q.n0 + row + 8, p.N - 1) * o.ldw;
  const int8_t* x[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) x[b] = o.x + (q.row0 + min(row + 8 * b, q.rows - 1)) * o.ldx;
  int acc[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b][0] = acc[b][1] = acc[b][2] = acc[b][3] = 0;
  constexpr int kUnits = kSegment / 16;
  for (int s = warp; s * kUnits < units; s += kWarps * kAhead) {
    uint4 vl[kAhead][2], vh[kAhead][2], vx[kAhead][2][NB];
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int u = (s + a * kWarps) * kUnits + 4 * h + (lane & 3);
        const bool here = u < units;
        vl[a][h] = vh[a][h] = make_uint4(0, 0, 0, 0);
        if (here) {
          vl[a][h] = load_weights(lo + 16LL * u);
          vh[a][h] = load_weights(hi + 16LL * u);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          vx[a][h][b] = make_uint4(0, 0, 0, 0);
          if (here) vx[a][h][b] = *reinterpret_cast<const uint4*>(x[b] + 16LL * u);
        }
      }
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < NB; ++b) mma_64(acc[b], vl[a][h], vh[a][h], vx[a][h][b]);
  }
  if ((o.K & 15) && warp == units / kUnits % kWarps) {   // what is behind the last whole unit (there may be no more bytes)
    const int n = (lane & 3) == 0 ? o.K & 15 : 0;
    const uint4 l = load_bytes(lo + 16LL * units, n), h = load_bytes(hi + 16LL * units, n);
#pragma unroll
    for (int b = 0; b < NB; ++b) mma_64(acc[b], l, h, load_bytes(x[b] + 16LL * units, n));
  }
  red += row * kPitch + 2 * (lane & 3);
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    red[8 * b] = acc[b][0];
    red[8 * b + 1] = acc[b][1];
    red[8 * kPitch + 8 * b] = acc[b][2];
    red[8 * kPitch + 8 * b + 1] = acc[b][3];
  }
}

__global__ void __launch_bounds__(kThreads, 2) linear_int8_mma_kernel(const LinearParams p, const Int8Operands o) {
  __shared__ int prefix[kScheduleBytes / 4];
  __shared__ int red[2][kWarps][kCols * kPitch];   // by tile parity
  pdl_launch_dependents();
  pdl_wait_prior();
  if (threadIdx.x < 32) build_schedule(p, kRows, prefix, blockIdx.x == 0);
  __syncthreads();
  const long long tiles = tile_count(p, prefix);
  const int nr = threadIdx.x % kCols, mr = threadIdx.x / kCols;   // this thread's element of a tile
  int turn = 0;
  for (long long t = blockIdx.x; t < tiles; t += gridDim.x, turn ^= 1) {
    const LinearTile q = tile_at<kRows, kCols>(p, prefix, t);
    const int n = q.n0 + nr;
    const bool mine = mr < q.rows && n < p.N;
    float ws = 0.f, bias = 0.f, xs = 0.f;
    if (mine) {
      const long long en = static_cast<long long>(q.e) * p.N + n;
      ws = p.w_scale[en];
      bias = p.bias ? p.bias[en] : kNoBias;
      xs = p.x_scale[(q.row0 + mr) * p.xs_row];
    }
    if (q.rows <= 8)
      sums_of<1>(p, o, q, red[turn][threadIdx.x >> 5]);
    else
      sums_of<2>(p, o, q, red[turn][threadIdx.x >> 5]);
    __syncthreads();   // (one a tile: the other set is written before the next)
    if (mine) {
      int sum = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += red[turn][w][nr * kPitch + mr];
      int8_put(p, q.row0 + mr, n, Int8Finish{ws, bias, p.lo, p.hi}(sum, xs));
    }
  }
}

}  // namespace

cudaError_t launch_linear_int8_direct(const LinearParams& p, const LinearPlan& plan, const Int8Operands& o, cudaStream_t stream) {
  if (plan.tile == kInt8MmaRows) return launch_pdl(linear_int8_mma_kernel, dim3(plan.grid), dim3(kThreads), 0, stream, 1, p, o);
  auto go = [&](void (*kernel)(LinearParams, Int8Operands)) { return launch_pdl(kernel, dim3(plan.grid), dim3(kDotThreads), 0, stream, 1, p, o); };
  switch (int8_dot_cols(o.K)) {
    case 2: return go(linear_int8_dot_kernel<2>);
    case 4: return go(linear_int8_dot_kernel<4>);
    default: return go(linear_int8_dot_kernel<8>);
  }
}

int linear_int8_direct_ctas(int tile, int num_sms) {
  int n = 0;   // (the dot kernels are built for the same number)
  const cudaError_t e = tile == kInt8DotRows ? cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, linear_int8_dot_kernel<2>, kDotThreads, 0)
                                             : cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, linear_int8_mma_kernel, kThreads, 0);
  return e == cudaSuccess ? n * num_sms : 0;
}

}  // namespace convf
