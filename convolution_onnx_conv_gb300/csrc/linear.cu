// Host side of conv_fused_quantize_blocks and the linear layers (conv_fused_linear_*: block-scaled, bf16, int8):
// validates every argument (refuse, never guess) and launches on the caller's stream.  Weights
// and scales are read where they are; nothing of a run is kept for the next.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdio>
#include <new>

#include "../../include/conv_fused.h"
#include "api_internal.h"
#include "convf_internal.h"
#include "linear_host.h"
#include "linear_internal.h"
#include "live_handles.h"

using namespace convf;

namespace {

constexpr uint32_t kLinearMagic = 0x11EA4001u;
constexpr uint32_t kLinearDead = 0xDEAD11EAu;

}  // namespace

struct convf_linear {
  LiveHandleCount live;
  uint32_t magic;
  CUtensorMap tmW64, tmW128, tmW256;   // boxes of 64 (int8: 96), 128 and 256 weight rows
  int device, num_sms;
  convf_linear_desc d;
  const void* w;
  const float* w_scale;
  const float* bias;
  float lo, hi;
  int* status;   // device
};

namespace {

convf_status check_linear(const convf_linear* l) {
  if (!l) return record_error(CONVF_ERR_INVALID_ARG, "layer is NULL");
  if (l->magic == kLinearDead) return record_error(CONVF_ERR_INVALID_ARG, "layer was destroyed");
  if (l->magic != kLinearMagic) return record_error(CONVF_ERR_INVALID_ARG, "not a convf linear layer");
  return CONVF_OK;
}

convf_status check_linear_desc(const convf_linear_desc* d) {
  if (!d) return record_error(CONVF_ERR_INVALID_ARG, "desc is NULL");
  if (d->N < 1 || d->K < 1) return record_error(CONVF_ERR_INVALID_ARG, "N=%d and K=%d must be >= 1", d->N, d->K);
  if (d->N > kMaxExtent || d->K > kMaxExtent)
    return record_error(CONVF_ERR_UNSUPPORTED, "N=%d, K=%d: at most %d are served", d->N, d->K, kMaxExtent);
  if (d->experts < 1) return record_error(CONVF_ERR_INVALID_ARG, "experts=%d must be >= 1", d->experts);
  if (d->experts > kMaxExperts)
    return record_error(CONVF_ERR_UNSUPPORTED, "experts=%d: at most %d are served", d->experts, kMaxExperts);
  if (d->dtype != CONVF_LINEAR_BF16 && d->dtype != CONVF_LINEAR_E4M3 && d->dtype != CONVF_LINEAR_INT8)
    return record_error(CONVF_ERR_INVALID_ARG, "dtype=%d is not CONVF_LINEAR_BF16, CONVF_LINEAR_E4M3 or CONVF_LINEAR_INT8", d->dtype);
  if (d->dtype == CONVF_LINEAR_INT8 && d->K > kInt8MaxK)
    return record_error(CONVF_ERR_UNSUPPORTED, "K=%d: int8 sums of more than %d products may pass 32 bits", d->K, kInt8MaxK);
  const long long esz = d->dtype == CONVF_LINEAR_BF16 ? 2 : 1;
  if (d->ldw < d->K) return record_error(CONVF_ERR_INVALID_ARG, "ldw=%lld is less than K=%d", d->ldw, d->K);
  if (too_far(d->N, d->ldw, 2)) return record_error(CONVF_ERR_INVALID_ARG, "ldw=%lld: W passes the address space", d->ldw);
  if (d->ldw * esz % 16)
    return record_error(CONVF_ERR_UNSUPPORTED, "ldw=%lld: weight rows must be a multiple of 16 bytes apart", d->ldw);
  if (d->experts > 1) {
    if (d->expert_stride < (d->N - 1LL) * d->ldw + d->K)
      return record_error(CONVF_ERR_INVALID_ARG, "expert_stride=%lld: the experts' weights overlap", d->expert_stride);
    if (too_far(d->experts, d->expert_stride, 2))
      return record_error(CONVF_ERR_INVALID_ARG, "expert_stride=%lld: W passes the address space", d->expert_stride);
    if (d->expert_stride * esz % 16)
      return record_error(CONVF_ERR_UNSUPPORTED, "expert_stride=%lld: experts must be a multiple of 16 bytes apart",
                          d->expert_stride);
  }
  if (d->act < CONVF_ACT_NONE || d->act > CONVF_ACT_CLIP)
    return record_error(CONVF_ERR_INVALID_ARG, "act=%d is not a convf_act", d->act);
  if (d->act == CONVF_ACT_CLIP && !(d->clip_lo <= d->clip_hi))
    return record_error(CONVF_ERR_INVALID_ARG, "clip bounds (%g, %g) need lo <= hi", d->clip_lo, d->clip_hi);
  if (d->out_dtype != CONVF_OUT_F32 && d->out_dtype != CONVF_OUT_BF16)
    return record_error(CONVF_ERR_INVALID_ARG, "out_dtype=%d is not CONVF_OUT_F32 or CONVF_OUT_BF16", d->out_dtype);
  return CONVF_OK;
}

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// clusters of `split` CTAs of a few-rows kernel (of operands `dtype`) that run at once (looked up once per
// process and device; every writer stores the same value)
int few_clusters(int dev, int num_sms, int dtype, int tile, int split) {
  static int known[kMaxDevices][4][3][4];
  int ti = 0, si = 0;
  while ((16 << ti) < tile) ++ti;
  while ((1 << si) < split) ++si;
  int* at = dev >= 0 && dev < kMaxDevices ? &known[dev][dtype][ti][si] : nullptr;
  if (at && *at) return *at;
  const int n = dtype == CONVF_LINEAR_INT8 ? linear_int8_max_clusters(tile, split, num_sms)
                                           : linear_few_max_clusters(dtype == CONVF_LINEAR_E4M3, tile, split, num_sms);
  if (at) *at = n;
  return n;
}

// CTAs of a direct int8 kernel that run at once (as few_clusters)
int direct_ctas(int dev, int num_sms, int tile) {
  static int known[kMaxDevices][2];
  int* at = dev >= 0 && dev < kMaxDevices ? &known[dev][tile == kInt8MmaRows] : nullptr;
  if (at && *at) return *at;
  const int n = linear_int8_direct_ctas(tile, num_sms);
  if (at) *at = n;
  return n;
}

// weight rows of a plan's tile
int tile_columns(const LinearPlan& plan, int K) {
  if (plan.form == kLinearInt8Direct) return plan.tile == kInt8DotRows ? int8_dot_cols(K) : kInt8MmaCols;
  return plan.tile < 128 ? 128 : plan.form == kLinearInt8 ? kInt8PairCols : kManyCols;
}

// What a run of `rows` rows launches: the form with the least estimated time.  How the rows fall on
// the experts is known on the device only, so the estimate goes by their mean, with half a tile per
// expert lost at the groups' ends (any offsets are right with any plan).
LinearPlan make_plan(const convf_linear_desc& d, int dev, int num_sms, int rows) {
  const bool e4m3 = d.dtype == CONVF_LINEAR_E4M3, int8 = d.dtype == CONVF_LINEAR_INT8;
  const long long taken = rows < d.experts ? rows : d.experts;   // experts that can have rows
  const long long esz = d.dtype == CONVF_LINEAR_BF16 ? 2 : 1;
  const int num_kb = static_cast<int>(ceil_div(d.K * esz, kKBlockBytes));
  auto row_tiles = [&](int tile) {
    if (d.experts == 1) return ceil_div(rows, tile);
    const long long n = (2LL * rows / tile + taken) / 2;
    return n > taken ? n : taken;
  };
  // Estimated nanoseconds, fitted to runs of every form at 1 to 24576 rows, 1 to 64 experts and N, K from
  // 1024 to 4096: waves of tiles, each its k-blocks' time and a start and end, behind a launch; or the
  // bytes, at 6.3 TB/s, if that is more.  (2048 x 2048 layers, 16 experts, e4m3: 64 rows few/16 15.4 us,
  // many/128 16.2; 512 rows 21.3, 16.6; 4096 x 4096 layer: 48 rows few/16 12.5 us, few/64 14.0, many/256
  // 15.7; 2048 rows of 2048 x 2048 few/64 29 us, many/128 12.5.)  Over 34 sizes the choice takes at most 5%
  // more than the best form.
  LinearPlan plan{};
  long long best = -1;
  const long long bytes = taken * d.N * d.K * esz + static_cast<long long>(rows) * (d.K * esz + d.N * 2LL);
  auto take = [&](int form, int tile, int split, long long units, long long n_tiles, long long model, long long memory) {
    const long long ns = (model > memory ? model : memory) + model / 8;
    if (best >= 0 && ns >= best) return;
    best = ns;
    const long long most = (d.experts > 1 ? rows / tile + taken : ceil_div(rows, tile)) * n_tiles;
    const int ctas = (form == kLinearMany && tile == 256) || (form == kLinearInt8 && tile == kInt8PairRows) ? 2 : split;
    plan = LinearPlan{form, tile, split, ctas * static_cast<int>(most < units ? most : units)};
  };
  auto offer = [&](int form, int tile, int split, long long units, long long n_tiles, long long per_kb, long long ends) {
    const long long waves = ceil_div(row_tiles(tile) * n_tiles, units);
    take(form, tile, split, units, n_tiles, 3500 + waves * (ceil_div(num_kb, split) * per_kb + ends), 3500 + bytes / 6300);
  };
  const long long nt = ceil_div(d.N, 128), nt_many = ceil_div(d.N, kManyCols);
  if (int8) {
    // Fitted to runs of every form at 1 to 8192 rows, 1 to 64 experts and N, K from 300 to 16384.  The tensor cores'
    // forms, over 150 sizes: 0.4% more than the best of them on the average and 9% at most (64 rows of 4096 x 4096: 64
    // columns, split 4 15.0 us, unsplit 16.4, 16 columns 19.4, pairs 21.3; 1024 rows over 8 experts of 2048 x 2048: pairs
    // 24.3, 64 columns 27.6, 16 columns 48.0; over 32 experts 58.4, 38.7 and 54.5; the k-blocks' times are from later runs).  With the direct forms, over 230 sizes
    // of few rows, 1.3% and 32% (a row count says nothing of how it falls on the experts): 4096 x 4096, 1 row: by dot
    // products 2.8 us, direct MMAs 5.2, 16 columns 10.3; 4 rows 3.8, 5.2, 11.6; 8 rows 7, 5.3, 11.7; 32 rows 19, 14.4,
    // 18.6, 64 columns 14.9; 64 rows 35, 22.5, 22.3, 15.7; 64 rows over 64 experts of 2048 x 2048 26.1, 33.3, 28.5.  Those
    // 32% are the worst of the groups that were run, not of all: where one expert takes every row, the choice by the mean loses
    // more.  64 rows of one of 64 experts of 4096 x 4096 40.0 us (dot products; one layer of 64 rows 15.0), 256 rows 38.8
    // (17.4), 1024 rows 56.7 (38.4); of 2048 x 2048 13.1 (8.0), 13.4 (10.9), 19.2 (16.2).
    const long long dot_cols = int8_dot_cols(d.K), dot = direct_ctas(dev, num_sms, kInt8DotRows), mma = direct_ctas(dev, num_sms, kInt8MmaRows);
    const long long mean = ceil_div(rows, taken);   // rows of an expert
    const long long kilos = d.N * static_cast<long long>(d.K) / 1000;
    if (dot > 0 && mean <= 64) {
      const long long tiles = row_tiles(kInt8DotRows) * ceil_div(d.N, dot_cols), warps = dot * kInt8DotWarps;
      const long long loads = ceil_div(tiles, warps) * (ceil_div(d.K * dot_cols, 4096) * 800 + 800);
      const long long products = row_tiles(kInt8DotRows) * kilos * (mean > 2 ? 4 : mean) * 15 / 1000;
      take(kLinearInt8Direct, kInt8DotRows, 1, warps, ceil_div(d.N, dot_cols), 1300 + (loads > products ? loads : products), 1300 + bytes / 6800);
      plan.grid = static_cast<int>(ceil_div(plan.grid, kInt8DotWarps));   // (the first to offer: it has been taken)
    }
    if (mma > 0 && mean <= 64) {
      const long long tiles = row_tiles(kInt8MmaRows) * ceil_div(d.N, kInt8MmaCols), groups = mean > 8 ? 2 : 1;
      const long long loads = ceil_div(tiles, mma) * (ceil_div(d.K, 2048) * 1030 * groups + 600);
      const long long products = row_tiles(kInt8MmaRows) * kilos * groups * 150 / 1000;
      take(kLinearInt8Direct, kInt8MmaRows, 1, mma, ceil_div(d.N, kInt8MmaCols), 2500 + (loads > products ? loads : products), 2500 + bytes / 6300);
    }
    for (int tile = 16; tile <= (rows > 16 ? 64 : 16); tile *= 4) {
      for (int split = 1; split <= 8 && split <= num_kb; split *= 2) {
        const int units = few_clusters(dev, num_sms, d.dtype, tile, split);
        const long long tiles = row_tiles(tile) * nt;
        if (units < 1 || (split > 1 && tiles > units)) continue;   // sharing a tile pays in a single wave
        const long long per_kb = tile == 64 ? 285 : tiles * split <= num_sms ? 380 : 500;
        const long long ends = split == 1 ? (tile == 64 ? 1340 : 230) : (tile == 64 ? 6800 : 3210) + 70 * split;
        offer(kLinearInt8, tile, split, units, nt, per_kb, ends);
      }
    }
    if (num_sms >= 2) offer(kLinearInt8, kInt8PairRows, 1, num_sms / 2, ceil_div(d.N, kInt8PairCols), 380, 3410);
    return plan;
  }
  for (int tile = 16; tile <= 64; tile *= 2) {
    // with two CTAs on an SM (16 and 32 columns), and alone
    const long long shared = tile == 16 ? (e4m3 ? 330 : 240) : (e4m3 ? 480 : 280);
    const long long alone = tile == 16 ? (e4m3 ? 230 : 160) : tile == 32 ? (e4m3 ? 330 : 200) : (e4m3 ? 430 : 245);
    for (int split = 1; split <= 8 && split <= num_kb; split *= 2) {
      const long long tiles = row_tiles(tile) * nt;
      const int units = few_clusters(dev, num_sms, d.dtype, tile, split);
      if (units < 1 || (split > 1 && tiles > units)) continue;   // sharing a tile pays in a single wave
      const bool one_each = tiles * split <= num_sms;
      offer(kLinearFew, tile, split, units, nt, one_each || tile == 64 ? (tile == 64 && one_each && e4m3 ? 330 : alone) : shared,
            split == 1 ? 700 : 1000 + 500 * split + 75 * tile);
    }
  }
  offer(kLinearMany, 128, 1, num_sms, nt_many, e4m3 ? 420 : 360, 1800);
  if (num_sms >= 2) offer(kLinearMany, 256, 1, num_sms / 2, nt_many, e4m3 ? 390 : 290, 1800);
  return plan;
}

// boxes of box_bytes (128 or 64) x box_rows rows, in the swizzle of as many bytes
convf_status encode_map(CUtensorMap* m, CUtensorMapDataType type, int esz, int dims, const void* p, const cuuint64_t* size,
                        const cuuint64_t* strides, int box_rows, const char* what, int box_bytes = kKBlockBytes) {
  EncodeTiledFn tiled;
  EncodeIm2colFn im2col;
  if (!tensor_map_encoders(&tiled, &im2col)) return record_error(CONVF_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_bytes / esz),
                             static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t es[3] = {1, 1, 1};
  const CUresult r = tiled(m, type, dims, const_cast<void*>(p), size, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           box_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return record_error(CONVF_ERR_CUDA, "encoding the tensor map of %s failed (%d)", what, (int)r);
  return CONVF_OK;
}

}  // namespace

extern "C" {

convf_status conv_fused_quantize_blocks(const convf_quant_args* a, void* stream) {
  if (!a) return record_error(CONVF_ERR_INVALID_ARG, "args is NULL");
  if (a->rows < 0) return record_error(CONVF_ERR_INVALID_ARG, "rows=%d must be >= 0", a->rows);
  if (a->cols < 1) return record_error(CONVF_ERR_INVALID_ARG, "cols=%d must be >= 1", a->cols);
  if (a->rows > kMaxExtent || a->cols > kMaxExtent)
    return record_error(CONVF_ERR_UNSUPPORTED, "rows=%d, cols=%d: at most %d are served", a->rows, a->cols, kMaxExtent);
  if (a->x_rows < 0) return record_error(CONVF_ERR_INVALID_ARG, "x_rows=%d must be >= 0", a->x_rows);
  if (a->x_dtype != CONVF_OUT_F32 && a->x_dtype != CONVF_OUT_BF16)
    return record_error(CONVF_ERR_INVALID_ARG, "x_dtype=%d is not CONVF_OUT_F32 or CONVF_OUT_BF16", a->x_dtype);
  if (a->gated != 0 && a->gated != 1) return record_error(CONVF_ERR_INVALID_ARG, "gated=%d is not 0 or 1", a->gated);
  if (a->block_rows != 1 && a->block_rows != kScaleBlock)
    return record_error(CONVF_ERR_INVALID_ARG, "block_rows=%d is not 1 or %d", a->block_rows, kScaleBlock);
  if (a->block_rows != 1 && (a->index || a->gated))
    return record_error(CONVF_ERR_UNSUPPORTED, "an index or gated values are quantised with block_rows = 1 only");
  if (!a->index && a->x_rows != a->rows)
    return record_error(CONVF_ERR_INVALID_ARG, "x_rows=%d must be rows=%d without an index", a->x_rows, a->rows);
  const long long wide = static_cast<long long>(a->cols) * (a->gated ? 2 : 1);
  const int nblk = (a->cols - 1) / kScaleBlock + 1;
  if (a->ldx < wide) return record_error(CONVF_ERR_INVALID_ARG, "ldx=%lld is less than the row's %lld", a->ldx, wide);
  if (a->ldq < a->cols) return record_error(CONVF_ERR_INVALID_ARG, "ldq=%lld is less than cols=%d", a->ldq, a->cols);
  if (a->lds < nblk) return record_error(CONVF_ERR_INVALID_ARG, "lds=%lld is less than the row's %d scales", a->lds, nblk);
  if (too_far(a->x_rows, a->ldx, 4) || too_far(a->rows, a->ldq, 1) || too_far(a->rows, a->lds, 4))
    return record_error(CONVF_ERR_INVALID_ARG, "ldx=%lld, ldq=%lld, lds=%lld: the rows pass the address space", a->ldx,
                        a->ldq, a->lds);
  if (a->rows == 0) return record_ok();
  if (!a->q || !a->scale || (!a->x && a->x_rows > 0)) return record_error(CONVF_ERR_INVALID_ARG, "x, q or scale is NULL");
  const int esz = a->x_dtype == CONVF_OUT_BF16 ? 2 : 4;
  if (!aligned(a->x, esz) || !aligned(a->scale, 4) || !aligned(a->index, 4))
    return record_error(CONVF_ERR_INVALID_ARG, "x, index and scale must be aligned to their elements");
  const Region x_at{a->x, a->x_rows, wide * esz, a->ldx * esz}, q_at{a->q, a->rows, a->cols, a->ldq};
  const Region scale_at{a->scale, (a->rows - 1LL) / a->block_rows + 1, nblk * 4LL, a->lds * 4};
  const Region index_at{a->index, 1, a->rows * 4LL, a->rows * 4LL};
  if (overlap(x_at, q_at) || overlap(x_at, scale_at) || overlap(q_at, scale_at))
    return record_error(CONVF_ERR_INVALID_ARG, "x, q and scale overlap");
  if (overlap(index_at, q_at) || overlap(index_at, scale_at))   // (rows are looked up while others are written)
    return record_error(CONVF_ERR_INVALID_ARG, "index and q or scale overlap");
  int dev = -1, sms = 0;
  convf_status st = current_device(&dev, &sms);
  if (st != CONVF_OK) return st;
  QuantParams p{};
  p.x = a->x; p.ldx = a->ldx; p.x_rows = a->x_rows; p.index = a->index;
  p.rows = a->rows; p.cols = a->cols; p.nblk = nblk;
  p.q = static_cast<uint8_t*>(a->q); p.ldq = a->ldq; p.scale = a->scale; p.lds = a->lds;
  const uintptr_t x_bits = reinterpret_cast<uintptr_t>(a->x) | a->ldx * esz | (a->gated ? static_cast<long long>(a->cols) * esz : 0);
  const uintptr_t q_bits = reinterpret_cast<uintptr_t>(a->q) | a->ldq;
  p.x_align = common_alignment(x_bits);
  p.q_align = common_alignment(q_bits);
  const cudaError_t e = launch_quantize_blocks(p, esz == 2, a->gated != 0, a->block_rows, sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return record_error(CONVF_ERR_CUDA, "quantising launch failed: %s", cudaGetErrorString(e));
  return record_ok();
}

convf_status conv_fused_linear_create(const convf_linear_desc* desc, const void* W, const float* w_scale,
                                      const float* bias, convf_linear** out) {
  if (!out) return record_error(CONVF_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  convf_status st = check_linear_desc(desc);
  if (st != CONVF_OK) return st;
  if (!W) return record_error(CONVF_ERR_INVALID_ARG, "W is NULL");
  if (!aligned(W, 16)) return record_error(CONVF_ERR_INVALID_ARG, "W must be 16-byte aligned");
  if ((desc->dtype != CONVF_LINEAR_BF16) != (w_scale != nullptr))
    return record_error(CONVF_ERR_INVALID_ARG, "w_scale goes with e4m3 weights or int8 ones, and with those only");
  if (!aligned(w_scale, 4) || !aligned(bias, 4))
    return record_error(CONVF_ERR_INVALID_ARG, "w_scale and bias must be aligned to their elements");
  const bool host_injected = take_injected_alloc_failure();
  convf_linear* l = host_injected ? nullptr : new (std::nothrow) convf_linear();
  if (!l) return record_error(CONVF_ERR_OOM, "allocation of the layer failed%s", host_injected ? " (injected)" : "");
  l->magic = kLinearMagic;
  l->d = *desc;
  l->w = W;
  l->w_scale = w_scale;
  l->bias = bias;
  switch (desc->act) {
    case CONVF_ACT_RELU: l->lo = 0.f; l->hi = INFINITY; break;
    case CONVF_ACT_RELU6: l->lo = 0.f; l->hi = 6.f; break;
    case CONVF_ACT_CLIP: l->lo = desc->clip_lo; l->hi = desc->clip_hi; break;
    default: l->lo = -INFINITY; l->hi = INFINITY; break;
  }
  st = current_device(&l->device, &l->num_sms);
  if (st != CONVF_OK) {
    delete l;
    return st;
  }
  {
    const bool bytes = desc->dtype != CONVF_LINEAR_BF16;
    const cuuint64_t esz = bytes ? 1 : 2;
    const cuuint64_t size[3] = {static_cast<cuuint64_t>(desc->K), static_cast<cuuint64_t>(desc->N),
                                static_cast<cuuint64_t>(desc->experts)};
    const cuuint64_t strides[2] = {desc->ldw * esz,
                                   (desc->experts > 1 ? desc->expert_stride : desc->N * desc->ldw) * esz};
    const CUtensorMapDataType type = bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    st = encode_map(&l->tmW64, type, esz, 3, W, size, strides, desc->dtype == CONVF_LINEAR_INT8 ? 96 : 64, "W");
    if (st == CONVF_OK) st = encode_map(&l->tmW128, type, esz, 3, W, size, strides, 128, "W");
    if (st == CONVF_OK) st = encode_map(&l->tmW256, type, esz, 3, W, size, strides, 256, "W");
    if (st != CONVF_OK) {
      delete l;
      return st;
    }
  }
  const bool dev_injected = take_injected_alloc_failure();
  cudaError_t e = dev_injected ? cudaErrorMemoryAllocation : cudaMalloc(&l->status, 256);
  if (e != cudaSuccess) {
    delete l;
    return record_error(CONVF_ERR_OOM, "device allocation of 256 bytes failed%s", dev_injected ? " (injected)" : "");
  }
  e = cudaMemset(l->status, 0, 256);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    cudaFree(l->status);
    delete l;
    return record_error(CONVF_ERR_CUDA, "clearing the layer's status failed: %s", cudaGetErrorString(e));
  }
  *out = l;
  return record_ok();
}

convf_status conv_fused_linear_run(convf_linear* l, const convf_linear_args* a, void* stream) {
  convf_status st = check_linear(l);
  if (st != CONVF_OK) return st;
  if (!a) return record_error(CONVF_ERR_INVALID_ARG, "args is NULL");
  const convf_linear_desc& d = l->d;
  const bool e4m3 = d.dtype == CONVF_LINEAR_E4M3, int8 = d.dtype == CONVF_LINEAR_INT8, scaled = e4m3 || int8;
  const long long esz = scaled ? 1 : 2, osz = d.out_dtype == CONVF_OUT_BF16 ? 2 : 4;
  if (a->rows < 0) return record_error(CONVF_ERR_INVALID_ARG, "rows=%d must be >= 0", a->rows);
  if (a->rows > kMaxExtent) return record_error(CONVF_ERR_UNSUPPORTED, "rows=%d: at most %d are served", a->rows, kMaxExtent);
  if (too_far(a->rows, a->ldx, 2) || too_far(a->rows, a->ldy, 4) || too_far(a->rows, a->xs_row, 4) ||
      (!int8 && too_far(d.K, a->xs_blk, 4)))
    return record_error(CONVF_ERR_INVALID_ARG, "ldx=%lld, ldy=%lld, x_scale strides (%lld, %lld): the rows pass the address space",
                        a->ldx, a->ldy, a->xs_row, a->xs_blk);
  if (a->ldx < d.K) return record_error(CONVF_ERR_INVALID_ARG, "ldx=%lld is less than K=%d", a->ldx, d.K);
  if (a->ldx * esz % 16)
    return record_error(CONVF_ERR_UNSUPPORTED, "ldx=%lld: rows of x must be a multiple of 16 bytes apart", a->ldx);
  if (a->ldy < d.N) return record_error(CONVF_ERR_INVALID_ARG, "ldy=%lld is less than N=%d", a->ldy, d.N);
  if (scaled && (a->xs_row < 0 || (e4m3 && a->xs_blk < 0)))
    return record_error(CONVF_ERR_INVALID_ARG, "x_scale strides (%lld, %lld) must be >= 0", a->xs_row, a->xs_blk);
  if (!a->offsets && d.experts > 1) return record_error(CONVF_ERR_INVALID_ARG, "%d experts need row offsets", d.experts);
  if (a->rows == 0) return record_ok();
  if (!a->x || !a->y) return record_error(CONVF_ERR_INVALID_ARG, "x or y is NULL");
  if (scaled != (a->x_scale != nullptr))
    return record_error(CONVF_ERR_INVALID_ARG, "x_scale goes with e4m3 layers or int8 ones, and with those only");
  if (!aligned(a->x, 16)) return record_error(CONVF_ERR_INVALID_ARG, "x must be 16-byte aligned");
  if (!aligned(a->y, osz) || !aligned(a->x_scale, 4) || !aligned(a->offsets, 4))
    return record_error(CONVF_ERR_INVALID_ARG, "y, x_scale and offsets must be aligned to their elements");
  // y against all that the run reads (its tiles are written while others are read)
  const Region y_at{a->y, a->rows, d.N * osz, a->ldy * osz};
  const long long nblk = ceil_div(d.K, kScaleBlock), wblk = ceil_div(d.N, kScaleBlock);
  const long long apart = d.experts > 1 ? d.expert_stride * esz : 0;
  const Region w_at = d.experts == 1 || apart == d.N * d.ldw * esz
                          ? Region{l->w, static_cast<long long>(d.experts) * d.N, d.K * esz, d.ldw * esz}
                          : Region{l->w, 1, (d.experts - 1) * apart + ((d.N - 1) * d.ldw + d.K) * esz, 0};
  const Region xs_at = !scaled ? Region{}
                       : int8 ? (a->xs_row ? Region{a->x_scale, a->rows, 4, a->xs_row * 4} : Region{a->x_scale, 1, 4, 0})
                       : a->xs_blk == 1 ? Region{a->x_scale, a->rows, nblk * 4, a->xs_row * 4}
                       : a->xs_row == 1 ? Region{a->x_scale, nblk, a->rows * 4LL, a->xs_blk * 4}
                                        : Region{a->x_scale, 1, ((a->rows - 1) * a->xs_row + (nblk - 1) * a->xs_blk + 1) * 4, 0};
  if (overlap(Region{a->x, a->rows, d.K * esz, a->ldx * esz}, y_at))
    return record_error(CONVF_ERR_INVALID_ARG, "x and y overlap");
  if (overlap(w_at, y_at)) return record_error(CONVF_ERR_INVALID_ARG, "the weights and y overlap");
  if (overlap(xs_at, y_at)) return record_error(CONVF_ERR_INVALID_ARG, "x_scale and y overlap");
  if (overlap(Region{l->w_scale, 1, (int8 ? static_cast<long long>(d.experts) * d.N : d.experts * wblk * nblk) * 4, 0}, y_at) ||
      overlap(Region{l->bias, 1, static_cast<long long>(d.experts) * d.N * 4, 0}, y_at) ||
      overlap(Region{a->offsets, 1, (d.experts + 1) * 4LL, 0}, y_at))
    return record_error(CONVF_ERR_INVALID_ARG, "w_scale, bias or offsets overlap y");
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != l->device)
    return record_error(CONVF_ERR_INVALID_ARG, "the current device (%d) is not the layer's device (%d)", dev, l->device);
  const LinearPlan plan = make_plan(d, l->device, l->num_sms, a->rows);
  CUtensorMap tmX{};
  const cuuint64_t size[2] = {static_cast<cuuint64_t>(d.K), static_cast<cuuint64_t>(a->rows)};
  const cuuint64_t stride = a->ldx * esz;
  const int x_box = plan.tile < 128 ? plan.tile : 128;
  if (plan.form != kLinearInt8Direct)   // (which reads its operands as they are)
    st = encode_map(&tmX, scaled ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<int>(esz), 2,
                    a->x, size, &stride, x_box, "x");
  if (st != CONVF_OK) return st;
  LinearParams p{};
  p.rows = a->rows; p.N = d.N; p.experts = d.experts;
  p.num_kb = static_cast<int>(ceil_div(d.K * esz, kKBlockBytes));
  p.n_tiles = static_cast<int>(ceil_div(d.N, tile_columns(plan, d.K)));
  // bf16 operands: the MMA's own accumulator truncates, so its sums go to registers every 256 values where
  // the result is fp32 (1.2e-6 of the result at K = 1000 without it, 3e-7 with it), and every 4096 values
  // where it is bf16: terms of one sign then lose 1e-5 of their sum at most, whatever K is (without it 8e-4
  // at K = 131072, and a whole step of bf16 from about 10^6)
  p.chunk_kb = e4m3 ? 1 : osz == 2 ? 64 : 4;
  p.vec_y = aligned(a->y, 16) && a->ldy * osz % 16 == 0;
  p.whole_units = p.vec_y && d.N * osz % 16 == 0;
  p.x_scale = a->x_scale; p.xs_row = a->xs_row; p.xs_blk = a->xs_blk; p.w_scale = l->w_scale; p.bias = l->bias;
  p.offsets = a->offsets; p.y = a->y; p.ldy = a->ldy; p.out_bf16 = d.out_dtype == CONVF_OUT_BF16;
  p.lo = l->lo; p.hi = l->hi; p.status = l->status;
  p.clamp = l->lo != -INFINITY || l->hi != INFINITY;
  CUtensorMap tmY = tmX;   // (not used without vec_y)
  if (plan.tile >= 128 && p.vec_y) {
    const cuuint64_t ysize[2] = {static_cast<cuuint64_t>(d.N), static_cast<cuuint64_t>(a->rows)};
    const cuuint64_t ystride = a->ldy * osz;
    st = encode_map(&tmY, osz == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                    static_cast<int>(osz), 2, a->y, ysize, &ystride, 32, "y", int8 ? 64 : kKBlockBytes);
    if (st != CONVF_OK) return st;
  }
  const cudaStream_t strm = static_cast<cudaStream_t>(stream);
  const Int8Operands int8_operands{static_cast<const int8_t*>(l->w), static_cast<const int8_t*>(a->x), d.ldw, d.expert_stride, a->ldx, d.K};
  const cudaError_t e = plan.form == kLinearInt8Direct ? launch_linear_int8_direct(p, plan, int8_operands, strm)
                        : plan.form == kLinearInt8 ? (plan.tile == kInt8PairRows ? launch_linear_int8_many(p, plan, l->tmW64, tmX, tmY, strm)
                                                                               : launch_linear_int8_few(p, plan, l->tmW128, tmX, strm))
                        : plan.form == kLinearFew
                            ? launch_linear_few(p, plan, e4m3, l->tmW128, tmX, strm)
                            : launch_linear_many(p, plan, e4m3, plan.tile != 256 ? l->tmW256 : e4m3 ? l->tmW64 : l->tmW128,
                                                 tmX, tmY, strm);
  if (e != cudaSuccess) return record_error(CONVF_ERR_CUDA, "linear launch failed: %s", cudaGetErrorString(e));
  return record_ok();
}

convf_status conv_fused_linear_status(convf_linear* l) {
  convf_status st = check_linear(l);
  if (st != CONVF_OK) return st;
  int v = 0;
  if (cudaMemcpy(&v, l->status, sizeof v, cudaMemcpyDeviceToHost) != cudaSuccess)
    return record_error(CONVF_ERR_CUDA, "reading the layer's status failed");
  if (v & kStatusTimeout)
    return record_error(CONVF_ERR_TIMEOUT, "a bounded device wait ran out in an earlier run of the layer");
  if (v & kStatusBounds)
    return record_error(CONVF_ERR_BOUNDS, "a linear kernel computed an out-of-range index (bounds-checking build)");
  if (v & kStatusOffsets)
    return record_error(CONVF_ERR_INVALID_ARG, "an earlier run's offsets decreased or passed its rows");
  return record_ok();
}

convf_status conv_fused_linear_clear_status(convf_linear* l) {
  convf_status st = check_linear(l);
  if (st != CONVF_OK) return st;
  if (cudaMemset(l->status, 0, sizeof(int)) != cudaSuccess)
    return record_error(CONVF_ERR_CUDA, "clearing the layer's status failed");
  return record_ok();
}

convf_status conv_fused_linear_describe(const convf_linear* l, int rows, char* buf, size_t len) {
  convf_status st = check_linear(l);
  if (st != CONVF_OK) return st;
  if (!buf || len == 0) return record_error(CONVF_ERR_INVALID_ARG, "buf is NULL or len is 0");
  if (rows < 0) return record_error(CONVF_ERR_INVALID_ARG, "rows=%d must be >= 0", rows);
  const int n = snprintf(buf, len, "N=%d K=%d experts=%d %s rows=%d out=%s", l->d.N, l->d.K, l->d.experts,
                         l->d.dtype == CONVF_LINEAR_E4M3 ? "e4m3" : l->d.dtype == CONVF_LINEAR_INT8 ? "int8" : "bf16", rows,
                         l->d.out_dtype == CONVF_OUT_BF16 ? "bf16" : "f32");
  if (rows > 0 && n > 0 && static_cast<size_t>(n) < len) {
    int dev = -1;   // the plan asks the current device how many clusters it runs at once
    if (cudaGetDevice(&dev) != cudaSuccess || dev != l->device)
      return record_error(CONVF_ERR_INVALID_ARG, "the current device (%d) is not the layer's device (%d)", dev, l->device);
    const LinearPlan plan = make_plan(l->d, l->device, l->num_sms, rows);
    snprintf(buf + n, len - n, " form=%s tile=%dx%d split=%d grid=%d", plan.form == kLinearInt8Direct ? "direct" : plan.tile < 128 ? "few_rows" : "many_rows",
             plan.tile, tile_columns(plan, l->d.K), plan.split, plan.grid);
  }
  return record_ok();
}

void conv_fused_linear_destroy(convf_linear* l) {
  if (!l || l->magic != kLinearMagic) return;
  cudaFree(l->status);
  l->magic = kLinearDead;
  delete l;
}

}  // extern "C"
