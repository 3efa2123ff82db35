// Host side of conv_fused_quantize_rows and conv_fused_rms_norm_quantize: validates every argument (refuse,
// never guess) and launches on the caller's stream (kernels: k_rows.cu).
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/conv_fused.h"
#include "api_internal.h"
#include "linear_host.h"
#include "linear_internal.h"

using namespace convf;

namespace {

constexpr int kMaxCols = 1 << 30;   // a thread's last columns are still an int

bool is_out_dtype(int t) { return t == CONVF_OUT_F32 || t == CONVF_OUT_BF16; }
int size_of(int t) { return t == CONVF_OUT_BF16 ? 2 : 4; }

convf_status check_extent(int rows, int cols) {
  if (rows < 0) return record_error(CONVF_ERR_INVALID_ARG, "rows=%d must be >= 0", rows);
  if (cols < 1) return record_error(CONVF_ERR_INVALID_ARG, "cols=%d must be >= 1", cols);
  if (rows > kMaxExtent || cols > kMaxCols)
    return record_error(CONVF_ERR_UNSUPPORTED, "rows=%d, cols=%d: at most %d and %d are served", rows, cols, kMaxExtent, kMaxCols);
  return CONVF_OK;
}

template <int KIND>
convf_status launch(const RowsParams& p, int x_dtype, void* stream) {
  int dev = -1, sms = 0;
  const convf_status st = current_device(&dev, &sms);
  if (st != CONVF_OK) return st;
  const cudaError_t e = launch_rows<KIND>(p, x_dtype == CONVF_OUT_BF16, sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return record_error(CONVF_ERR_CUDA, "quantising launch failed: %s", cudaGetErrorString(e));
  return record_ok();
}

// behind the last of `rows` rows of `row` bytes, `stride` bytes apart
const uint8_t* end_of(const void* p, long long rows, long long row, long long stride) {
  return p && rows > 0 ? static_cast<const uint8_t*>(p) + (rows - 1) * stride + row : static_cast<const uint8_t*>(p);
}
// 80 bytes that a thread without columns may read, or null
const uint8_t* spare_of(const void* p, const uint8_t* end) {
  const uint8_t* from = reinterpret_cast<const uint8_t*>((reinterpret_cast<uintptr_t>(p) + 31) & ~static_cast<uintptr_t>(31));
  return end - static_cast<const uint8_t*>(p) >= 31 + 80 ? from : nullptr;
}

uintptr_t bits(const void* p) { return reinterpret_cast<uintptr_t>(p); }

}  // namespace

extern "C" {

convf_status conv_fused_quantize_rows(const convf_quant_rows_args* a, void* stream) {
  if (!a) return record_error(CONVF_ERR_INVALID_ARG, "args is NULL");
  const convf_status st = check_extent(a->rows, a->cols);
  if (st != CONVF_OK) return st;
  if (a->x_rows < 0) return record_error(CONVF_ERR_INVALID_ARG, "x_rows=%d must be >= 0", a->x_rows);
  if (!is_out_dtype(a->x_dtype))
    return record_error(CONVF_ERR_INVALID_ARG, "x_dtype=%d is not CONVF_OUT_F32 or CONVF_OUT_BF16", a->x_dtype);
  if (a->gated != 0 && a->gated != 1) return record_error(CONVF_ERR_INVALID_ARG, "gated=%d is not 0 or 1", a->gated);
  if (!a->index && a->x_rows != a->rows)
    return record_error(CONVF_ERR_INVALID_ARG, "x_rows=%d must be rows=%d without an index", a->x_rows, a->rows);
  const long long wide = static_cast<long long>(a->cols) * (a->gated ? 2 : 1);
  const int esz = size_of(a->x_dtype);
  if (a->ldx < wide) return record_error(CONVF_ERR_INVALID_ARG, "ldx=%lld is less than the row's %lld", a->ldx, wide);
  if (a->ldq < a->cols) return record_error(CONVF_ERR_INVALID_ARG, "ldq=%lld is less than cols=%d", a->ldq, a->cols);
  if (too_far(a->x_rows, a->ldx, 4) || too_far(a->rows, a->ldq, 1))
    return record_error(CONVF_ERR_INVALID_ARG, "ldx=%lld, ldq=%lld: the rows pass the address space", a->ldx, a->ldq);
  if (a->rows == 0) return record_ok();
  if (!a->q || !a->scale || (!a->x && a->x_rows > 0)) return record_error(CONVF_ERR_INVALID_ARG, "x, q or scale is NULL");
  if (!aligned(a->x, esz) || !aligned(a->scale, 4) || !aligned(a->index, 4))
    return record_error(CONVF_ERR_INVALID_ARG, "x, index and scale must be aligned to their elements");
  const Region x_at{a->x, a->x_rows, wide * esz, a->ldx * esz}, q_at{a->q, a->rows, a->cols, a->ldq};
  const Region scale_at{a->scale, 1, a->rows * 4LL, 0}, index_at{a->index, 1, a->rows * 4LL, 0};
  if (overlap(x_at, q_at) || overlap(x_at, scale_at) || overlap(q_at, scale_at))
    return record_error(CONVF_ERR_INVALID_ARG, "x, q and scale overlap");
  if (overlap(index_at, q_at) || overlap(index_at, scale_at))   // (rows are looked up while others are written)
    return record_error(CONVF_ERR_INVALID_ARG, "index and q or scale overlap");
  RowsParams p{};
  p.x = a->x; p.ldx = a->ldx; p.x_rows = a->x_rows; p.index = a->index;
  p.rows = a->rows; p.cols = a->cols; p.nblk = (a->cols - 1) / kScaleBlock + 1;
  p.q = static_cast<uint8_t*>(a->q); p.ldq = a->ldq; p.scale = a->scale;
  p.x_align = common_alignment(bits(a->x) | a->ldx * esz | (a->gated ? static_cast<long long>(a->cols) * esz : 0));
  p.q_align = common_alignment(bits(a->q) | a->ldq);
  p.r_align = p.w_align = 32;
  p.x_end = end_of(a->x, a->x_rows, wide * esz, a->ldx * esz);
  p.x_spare = spare_of(a->x, p.x_end);
  p.small = !p.x_spare;
  return a->gated ? launch<kRowsGated>(p, a->x_dtype, stream) : launch<kRowsPlain>(p, a->x_dtype, stream);
}

convf_status conv_fused_rms_norm_quantize(const convf_norm_args* a, void* stream) {
  if (!a) return record_error(CONVF_ERR_INVALID_ARG, "args is NULL");
  const convf_status st = check_extent(a->rows, a->cols);
  if (st != CONVF_OK) return st;
  if (!is_out_dtype(a->x_dtype))
    return record_error(CONVF_ERR_INVALID_ARG, "x_dtype=%d is not CONVF_OUT_F32 or CONVF_OUT_BF16", a->x_dtype);
  if (a->residual && !is_out_dtype(a->residual_dtype))
    return record_error(CONVF_ERR_INVALID_ARG, "residual_dtype=%d is not CONVF_OUT_F32 or CONVF_OUT_BF16", a->residual_dtype);
  if (a->weight && !is_out_dtype(a->weight_dtype))
    return record_error(CONVF_ERR_INVALID_ARG, "weight_dtype=%d is not CONVF_OUT_F32 or CONVF_OUT_BF16", a->weight_dtype);
  if (a->out != CONVF_LINEAR_E4M3 && a->out != CONVF_LINEAR_INT8)
    return record_error(CONVF_ERR_INVALID_ARG, "out=%d is not CONVF_LINEAR_E4M3 or CONVF_LINEAR_INT8", a->out);
  if (!(a->eps > 0.f) || !std::isfinite(a->eps))
    return record_error(CONVF_ERR_INVALID_ARG, "eps=%g must be positive and finite", a->eps);
  if (a->h && !a->residual) return record_error(CONVF_ERR_INVALID_ARG, "h goes with a residual (without one it is x)");
  const bool int8 = a->out == CONVF_LINEAR_INT8;
  const int nblk = (a->cols - 1) / kScaleBlock + 1;
  if (a->ldx < a->cols) return record_error(CONVF_ERR_INVALID_ARG, "ldx=%lld is less than cols=%d", a->ldx, a->cols);
  if (a->residual && a->ldr < a->cols) return record_error(CONVF_ERR_INVALID_ARG, "ldr=%lld is less than cols=%d", a->ldr, a->cols);
  if (a->h && a->ldh < a->cols) return record_error(CONVF_ERR_INVALID_ARG, "ldh=%lld is less than cols=%d", a->ldh, a->cols);
  if (a->ldq < a->cols) return record_error(CONVF_ERR_INVALID_ARG, "ldq=%lld is less than cols=%d", a->ldq, a->cols);
  if (!int8 && a->lds < nblk) return record_error(CONVF_ERR_INVALID_ARG, "lds=%lld is less than the row's %d scales", a->lds, nblk);
  if (too_far(a->rows, a->ldx, 4) || too_far(a->rows, a->ldq, 1) || (a->residual && too_far(a->rows, a->ldr, 4)) ||
      (a->h && too_far(a->rows, a->ldh, 4)) || (!int8 && too_far(a->rows, a->lds, 4)))
    return record_error(CONVF_ERR_INVALID_ARG, "ldx=%lld, ldr=%lld, ldh=%lld, ldq=%lld, lds=%lld: the rows pass the address space",
                        a->ldx, a->ldr, a->ldh, a->ldq, a->lds);
  if (a->rows == 0) return record_ok();
  if (!a->x || !a->q || !a->scale) return record_error(CONVF_ERR_INVALID_ARG, "x, q or scale is NULL");
  const int xsz = size_of(a->x_dtype), rsz = size_of(a->residual_dtype), wsz = size_of(a->weight_dtype);
  if (!aligned(a->x, xsz) || !aligned(a->residual, rsz) || !aligned(a->h, rsz) || !aligned(a->weight, wsz) || !aligned(a->scale, 4))
    return record_error(CONVF_ERR_INVALID_ARG, "x, residual, h, weight and scale must be aligned to their elements");
  const long long cols = a->cols;
  const Region x_at{a->x, a->rows, cols * xsz, a->ldx * xsz}, r_at{a->residual, a->rows, cols * rsz, a->ldr * rsz};
  const Region h_at{a->h, a->rows, cols * rsz, a->ldh * rsz}, w_at{a->weight, 1, cols * wsz, 0};
  const Region q_at{a->q, a->rows, cols, a->ldq};
  const Region scale_at = int8 ? Region{a->scale, 1, a->rows * 4LL, 0} : Region{a->scale, a->rows, nblk * 4LL, a->lds * 4};
  // (an element of h is written by the thread that has read it of x and the residual)
  const bool on_r = a->h == a->residual && (a->ldh == a->ldr || a->rows == 1);
  const bool on_x = a->h == a->x && a->residual_dtype == a->x_dtype && (a->ldh == a->ldx || a->rows == 1);
  if ((!on_r && overlap(h_at, r_at)) || (!on_x && overlap(h_at, x_at)))
    return record_error(CONVF_ERR_INVALID_ARG, "h overlaps x or the residual and is not the same rows");
  for (const Region& in : {x_at, r_at, w_at, h_at})
    if (overlap(in, q_at) || overlap(in, scale_at))
      return record_error(CONVF_ERR_INVALID_ARG, "q or scale overlaps x, residual, h or weight");
  if (overlap(q_at, scale_at)) return record_error(CONVF_ERR_INVALID_ARG, "q and scale overlap");
  if (overlap(h_at, w_at)) return record_error(CONVF_ERR_INVALID_ARG, "h and weight overlap");
  RowsParams p{};
  p.x = a->x; p.ldx = a->ldx; p.x_rows = a->rows;
  p.rows = a->rows; p.cols = a->cols; p.nblk = nblk;
  p.residual = a->residual; p.ldr = a->ldr; p.residual_bf16 = a->residual_dtype == CONVF_OUT_BF16;
  p.h = a->h; p.ldh = a->ldh;
  p.weight = a->weight; p.weight_bf16 = a->weight && a->weight_dtype == CONVF_OUT_BF16; p.eps = a->eps;
  p.inv_cols = 1.f / static_cast<float>(a->cols);
  p.q = static_cast<uint8_t*>(a->q); p.ldq = a->ldq; p.scale = a->scale; p.lds = a->lds;
  p.x_align = common_alignment(bits(a->x) | a->ldx * xsz);
  p.r_align = common_alignment((a->residual ? bits(a->residual) | a->ldr * rsz : 0) | (a->h ? bits(a->h) | a->ldh * rsz : 0));
  p.w_align = common_alignment(bits(a->weight));
  p.x_end = end_of(a->x, a->rows, cols * xsz, a->ldx * xsz);
  p.r_end = end_of(a->residual, a->rows, cols * rsz, a->ldr * rsz);
  p.x_spare = spare_of(a->x, p.x_end);
  p.r_spare = spare_of(a->residual, p.r_end);
  p.small = !p.x_spare || (a->residual && !p.r_spare);
  p.q_align = common_alignment(bits(a->q) | a->ldq);
  return int8 ? launch<kRowsNormInt8>(p, a->x_dtype, stream) : launch<kRowsNormE4m3>(p, a->x_dtype, stream);
}

}  // extern "C"
