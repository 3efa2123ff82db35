// Interface between the host side of the block-scaled operators (linear.cu) and their kernels.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace convf {

// Bit set in a layer's status word when a run's row offsets decreased or passed the rows.
constexpr int kStatusOffsets = 4;
constexpr int kScaleBlock = 128;    // columns (and weight rows) that share a scale
constexpr float kE4m3Max = 448.0f;
constexpr int kMaxExperts = 1024;   // the tile schedule keeps a prefix of them in shared memory

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
  // vector accesses: x's (and, gated, the second half's) 16-byte and q's 8-byte ones are aligned
  int vec_x, vec_u, vec_q;
};
cudaError_t launch_quantize_blocks(const QuantParams& p, bool bf16, bool gated, int block_rows, int num_sms,
                                   cudaStream_t stream);

struct LinearParams {
  int rows, N, K, experts;
  const void* x;
  long long ldx;
  const float* x_scale;
  long long xs_row, xs_blk;
  const void* w;
  long long ldw, expert_stride;
  const float* w_scale;      // [experts][nblk][kblk]
  const float* bias;         // [experts][N] or null
  const int32_t* offsets;    // [experts + 1] or null
  void* y;
  long long ldy;
  int out_bf16;
  float lo, hi;
  int* status;
};
cudaError_t launch_linear_simple(const LinearParams& p, bool e4m3, cudaStream_t stream);

}  // namespace convf
