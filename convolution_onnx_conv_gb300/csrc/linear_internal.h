// Interface between the host side of the linear layers and the 8-bit rows (linear.cu, rows.cu) and their kernels.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace convf {

// Bit set in a layer's status word when a run's row offsets decreased or passed the rows.
constexpr int kStatusOffsets = 4;
constexpr int kScaleBlock = 128;    // columns (and weight rows) that share a scale
constexpr float kE4m3Max = 448.0f;
constexpr int kMaxExtent = 0x7FFFFF00;   // rows, columns, N and K: the last tile's end is still an int
constexpr int kMaxExperts = 1024;   // the tile schedule keeps a prefix of them in shared memory
constexpr int kKBlockBytes = 128;   // bytes of a k-block's operand row: 128 e4m3 or 64 bf16 values

// What is set or looked up once for each device, not once for a process, by the current device (an
// attribute of a kernel, the dynamic shared memory that it may ask for, belongs to a device).
constexpr int kMaxDevices = 64;
struct OncePerDevice {
  bool done[kMaxDevices] = {};
  // runs set() unless it has succeeded on the current device before
  template <typename Set>
  cudaError_t operator()(Set set) {
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < kMaxDevices;
    if (known && done[dev]) return cudaSuccess;
    e = set();
    if (e == cudaSuccess && known) done[dev] = true;
    return e;
  }
};

// Memory of a call: `rows` rows of `row` bytes, `stride` bytes apart.
struct Region {
  const void* p;
  long long rows, row, stride;
};
// Whether two of them share a byte.  Rows at the same distance may lie between each other's (columns of one
// buffer); other pairs go by the bytes from their first to their last.
inline bool overlap(Region a, Region b) {
  if (!a.p || !b.p || a.rows < 1 || b.rows < 1 || a.row < 1 || b.row < 1) return false;
  const long long d = static_cast<long long>(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
  if (d >= (a.rows - 1) * a.stride + a.row || -d >= (b.rows - 1) * b.stride + b.row) return false;
  if (a.rows == 1) a.stride = b.stride;
  if (b.rows == 1) b.stride = a.stride;
  const long long s = a.stride;
  if (s != b.stride || s < a.row || s < b.row) return true;
  // row i of a and row j of b are d + (j - i) s apart: of the differences that can share a byte, there are
  // two at most, around -d / s
  const long long r = (d % s + s) % s, m = (r - d) / s;   // d + m s = r, in [0, s)
  auto there = [&](long long k) { return k > -a.rows && k < b.rows; };
  return (r < a.row && there(m)) || (s - r < b.row && there(m - 1));
}

struct QuantParams {
  const void* x;
  long long ldx;
  int x_rows;
  const int32_t* index;
  int rows, cols, nblk;      // nblk = ceil(cols / 128)
  uint8_t* q;
  long long ldq;
  float* scale;
  long long lds;
  int x_align, q_align;      // bytes on which rows of x (and its second half, gated) and of q begin: 32, 16, 8, or less
};
cudaError_t launch_quantize_blocks(const QuantParams& p, bool bf16, bool gated, int block_rows, int num_sms,
                                   cudaStream_t stream);

// Rows to 8 bits with a scale, or a norm's factor, of the whole row (k_rows.cu).
enum RowsKind : int { kRowsPlain = 0, kRowsGated = 1, kRowsNormInt8 = 2, kRowsNormE4m3 = 3 };
struct RowsParams {
  const void* x;
  long long ldx;
  int x_rows;
  const int32_t* index;
  int rows, cols, nblk;      // nblk = ceil(cols / 128)
  const void* residual;      // added to x, or null; residual_bf16: its type and h's
  long long ldr;
  int residual_bf16;
  void* h;                   // where x + residual goes, or null; may be the residual or x themselves
  long long ldh;
  const void* weight;        // [cols] or null
  int weight_bf16;
  float eps, inv_cols;       // inv_cols: 1 / cols
  uint8_t* q;
  long long ldq;
  float* scale;              // [rows]; e4m3: [rows][lds]
  long long lds;
  int x_align, r_align, w_align, q_align;   // as QuantParams' (r_align: the residual's and h's, 32 without them)
  const uint8_t *x_end, *r_end;             // behind the last bytes of x and the residual
  const uint8_t *x_spare, *r_spare;         // 80 bytes of each from a multiple of 32 on; small: one of them has no such
  int small;
};
template <int KIND>
cudaError_t launch_rows(const RowsParams& p, bool bf16, int num_sms, cudaStream_t stream);
template <> cudaError_t launch_rows<kRowsPlain>(const RowsParams&, bool, int, cudaStream_t);
template <> cudaError_t launch_rows<kRowsGated>(const RowsParams&, bool, int, cudaStream_t);
template <> cudaError_t launch_rows<kRowsNormInt8>(const RowsParams&, bool, int, cudaStream_t);
template <> cudaError_t launch_rows<kRowsNormE4m3>(const RowsParams&, bool, int, cudaStream_t);

struct LinearParams {
  int rows, N, experts;
  int num_kb;                // k-blocks of 128 bytes
  int chunk_kb;              // k-blocks that an MMA accumulator sums before its sum goes to the registers'
  int vec_y;                 // y's rows begin on 16 bytes
  int whole_units;           // and end on 16 bytes too
  int n_tiles;               // weight-row tiles of the chosen form
  const float* x_scale;
  long long xs_row, xs_blk;
  const float* w_scale;      // [experts][nblk][num_kb]; int8 [experts][N]
  const float* bias;         // [experts][N] or null
  const int32_t* offsets;    // [experts + 1] or null
  void* y;
  long long ldy;
  int out_bf16;
  float lo, hi;
  int clamp;                 // [lo, hi] is not all numbers
  int* status;
};

// What a run launches (linear_plan): the form, its row tile, and how many CTAs share a tile's k.
enum LinearForm : int { kLinearFew = 0, kLinearMany = 1, kLinearInt8 = 2, kLinearInt8Direct = 3 };
struct LinearPlan {
  int form;
  int tile;     // rows of x per tile: kLinearFew 16, 32 or 64; kLinearMany 128, or 256 on CTA pairs;
                // kLinearInt8 16 or 64, or kInt8PairRows on CTA pairs; kLinearInt8Direct kInt8DotRows or kInt8MmaRows
  int split;    // kLinearFew, kLinearInt8: CTAs of a cluster that share a tile's reduction (1, 2, 4 or 8)
  int grid;     // CTAs
};

// tmW: {K, N, experts}, boxes of 128 bytes x 128 rows; tmX: {K, rows}, boxes of 128 bytes x plan.tile
// rows; both in the 128-byte swizzle.
cudaError_t launch_linear_few(const LinearParams& p, const LinearPlan& plan, bool e4m3, const CUtensorMap& tmW,
                              const CUtensorMap& tmX, cudaStream_t stream);
// clusters of `split` CTAs that run at once on the current device (0 on an error)
int linear_few_max_clusters(bool e4m3, int tile, int split, int num_sms);


// tmW: boxes of 128 bytes x 256 rows (on CTA pairs x 64 for e4m3, x 128 for bf16);
// tmX: boxes of 128 bytes x 128 rows; tmY (used where vec_y): {N, rows} of y, boxes of 128 bytes x 32 rows.
cudaError_t launch_linear_many(const LinearParams& p, const LinearPlan& plan, bool e4m3, const CUtensorMap& tmW,
                               const CUtensorMap& tmX, const CUtensorMap& tmY, cudaStream_t stream);
// Few rows: tmW: boxes of 128 bytes x 128 rows; tmX: boxes of 128 bytes x plan.tile rows.  Many: tmW: boxes of 128
// bytes x 96 rows; tmX: of 128 bytes x 128 rows; tmY (used where vec_y): {N, rows} of y, boxes of 64 bytes x 32 rows
// in the 64-byte swizzle.
constexpr int kInt8PairRows = 256, kInt8PairCols = 192;
constexpr int kInt8MaxK = (1 << 17) - 1;   // products of 2^14 at most: sums stay within 32 bits
cudaError_t launch_linear_int8_few(const LinearParams& p, const LinearPlan& plan, const CUtensorMap& tmW, const CUtensorMap& tmX,
                                   cudaStream_t stream);
cudaError_t launch_linear_int8_many(const LinearParams& p, const LinearPlan& plan, const CUtensorMap& tmW, const CUtensorMap& tmX,
                                    const CUtensorMap& tmY, cudaStream_t stream);
int linear_int8_max_clusters(int tile, int split, int num_sms);
// A handful of rows, from the operands as they are: no tensor maps.
constexpr int kInt8DotRows = 4, kInt8DotWarps = 4;   // of x, of a warp's tile; warps of a CTA
// weight rows of a warp's tile: as many as fill a lane's loads
constexpr int int8_dot_cols(int K) { return K <= 512 ? 8 : K <= 1024 ? 4 : 2; }
constexpr int kInt8MmaRows = 16, kInt8MmaCols = 16;   // of a CTA's tile
struct Int8Operands {
  const int8_t *w, *x;
  long long ldw, w_stride, ldx;   // w_stride: between experts
  int K;
};
cudaError_t launch_linear_int8_direct(const LinearParams& p, const LinearPlan& plan, const Int8Operands& o, cudaStream_t stream);
int linear_int8_direct_ctas(int tile, int num_sms);   // that run at once on the current device (0 on an error)

constexpr int kManyCols = 256;   // weight rows of a kLinearMany tile

}  // namespace convf
