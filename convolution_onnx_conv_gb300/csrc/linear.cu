// Host side of the block-scaled operators (conv_fused_quantize_blocks, conv_fused_linear_*):
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
#include "linear_internal.h"
#include "live_handles.h"

using namespace convf;

namespace {

constexpr uint32_t kLinearMagic = 0x11EA4001u;
constexpr uint32_t kLinearDead = 0xDEAD11EAu;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// whether `rows` rows `ld` elements apart pass the address space (their products then pass 64 bits)
bool too_far(long long rows, long long ld, int esz) { return ld > ((1LL << 48) / esz) / (rows > 1 ? rows : 1); }

// SMs of the current device (looked up once per device), or an error
convf_status current_device(int* dev, int* num_sms) {
  static int sms[kMaxDevices];   // 0 = not looked up; every writer stores the same value
  if (cudaGetDevice(dev) != cudaSuccess) return record_error(CONVF_ERR_CUDA, "no current CUDA device");
  const bool known = *dev >= 0 && *dev < kMaxDevices;
  *num_sms = known ? sms[*dev] : 0;
  if (*num_sms == 0) {
    if (cudaDeviceGetAttribute(num_sms, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess || *num_sms < 1)
      return record_error(CONVF_ERR_CUDA, "the SM count of device %d could not be read", *dev);
    if (known) sms[*dev] = *num_sms;
  }
  return CONVF_OK;
}

}  // namespace

struct convf_linear {
  LiveHandleCount live;
  uint32_t magic;
  CUtensorMap tmW64, tmW128, tmW256;   // boxes of 64, 128 and 256 weight rows
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
  if (d->dtype != CONVF_LINEAR_BF16 && d->dtype != CONVF_LINEAR_E4M3)
    return record_error(CONVF_ERR_INVALID_ARG, "dtype=%d is not CONVF_LINEAR_BF16 or CONVF_LINEAR_E4M3", d->dtype);
  const long long esz = d->dtype == CONVF_LINEAR_E4M3 ? 1 : 2;
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

// clusters of `split` CTAs of the few-rows kernel that run at once (looked up once per process and
// device; every writer stores the same value)
int few_clusters(int dev, int num_sms, bool e4m3, int tile, int split) {
  static int known[kMaxDevices][2][3][4];
  int ti = 0, si = 0;
  while ((16 << ti) < tile) ++ti;
  while ((1 << si) < split) ++si;
  int* at = dev >= 0 && dev < kMaxDevices ? &known[dev][e4m3][ti][si] : nullptr;
  if (at && *at) return *at;
  const int n = linear_few_max_clusters(e4m3, tile, split, num_sms);
  if (at) *at = n;
  return n;
}

// What a run of `rows` rows launches: the form with the least estimated time.  How the rows fall on
// the experts is known on the device only, so the estimate goes by their mean, with half a tile per
// expert lost at the groups' ends (any offsets are right with any plan).
LinearPlan make_plan(const convf_linear_desc& d, int dev, int num_sms, int rows) {
  const bool e4m3 = d.dtype == CONVF_LINEAR_E4M3;
  const long long taken = rows < d.experts ? rows : d.experts;   // experts that can have rows
  const int num_kb = static_cast<int>(ceil_div(static_cast<long long>(d.K) * (e4m3 ? 1 : 2), kKBlockBytes));
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
  const long long esz = e4m3 ? 1 : 2;
  const long long bytes = taken * d.N * d.K * esz + static_cast<long long>(rows) * (d.K * esz + d.N * 2LL);
  auto offer = [&](int form, int tile, int split, long long units, long long n_tiles, long long per_kb, long long ends) {
    const long long waves = ceil_div(row_tiles(tile) * n_tiles, units);
    const long long model = 3500 + waves * (ceil_div(num_kb, split) * per_kb + ends), memory = 3500 + bytes / 6300;
    const long long ns = (model > memory ? model : memory) + model / 8;
    if (best >= 0 && ns >= best) return;
    best = ns;
    const long long most = (d.experts > 1 ? rows / tile + taken : ceil_div(rows, tile)) * n_tiles;
    const int ctas = form == kLinearMany && tile == 256 ? 2 : split;
    plan = LinearPlan{form, tile, split, ctas * static_cast<int>(most < units ? most : units)};
  };
  const long long nt = ceil_div(d.N, 128), nt_many = ceil_div(d.N, kManyCols);
  for (int tile = 16; tile <= 64; tile *= 2) {
    // with two CTAs on an SM (16 and 32 columns), and alone
    const long long shared = tile == 16 ? (e4m3 ? 330 : 240) : (e4m3 ? 480 : 280);
    const long long alone = tile == 16 ? (e4m3 ? 230 : 160) : tile == 32 ? (e4m3 ? 330 : 200) : (e4m3 ? 430 : 245);
    for (int split = 1; split <= 8 && split <= num_kb; split *= 2) {
      const long long tiles = row_tiles(tile) * nt;
      const int units = few_clusters(dev, num_sms, e4m3, tile, split);
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

// boxes of 128 bytes x box_rows rows in the 128-byte swizzle
convf_status encode_map(CUtensorMap* m, CUtensorMapDataType type, int esz, int dims, const void* p, const cuuint64_t* size,
                        const cuuint64_t* strides, int box_rows, const char* what) {
  EncodeTiledFn tiled;
  EncodeIm2colFn im2col;
  if (!tensor_map_encoders(&tiled, &im2col)) return record_error(CONVF_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(kKBlockBytes / esz),
                             static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t es[3] = {1, 1, 1};
  const CUresult r = tiled(m, type, dims, const_cast<void*>(p), size, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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
  auto common = [](uintptr_t v) { return static_cast<int>((v | 32) & (~(v | 32) + 1)); };   // largest power of two of v, up to 32
  p.x_align = common(x_bits);
  p.q_align = common(q_bits);
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
  if ((desc->dtype == CONVF_LINEAR_E4M3) != (w_scale != nullptr))
    return record_error(CONVF_ERR_INVALID_ARG, "w_scale goes with e4m3 weights, and with those only");
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
    const bool e4m3 = desc->dtype == CONVF_LINEAR_E4M3;
    const cuuint64_t esz = e4m3 ? 1 : 2;
    const cuuint64_t size[3] = {static_cast<cuuint64_t>(desc->K), static_cast<cuuint64_t>(desc->N),
                                static_cast<cuuint64_t>(desc->experts)};
    const cuuint64_t strides[2] = {desc->ldw * esz,
                                   (desc->experts > 1 ? desc->expert_stride : desc->N * desc->ldw) * esz};
    const CUtensorMapDataType type = e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    st = encode_map(&l->tmW64, type, esz, 3, W, size, strides, 64, "W");
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
  const bool e4m3 = d.dtype == CONVF_LINEAR_E4M3;
  const long long esz = e4m3 ? 1 : 2, osz = d.out_dtype == CONVF_OUT_BF16 ? 2 : 4;
  if (a->rows < 0) return record_error(CONVF_ERR_INVALID_ARG, "rows=%d must be >= 0", a->rows);
  if (a->rows > kMaxExtent) return record_error(CONVF_ERR_UNSUPPORTED, "rows=%d: at most %d are served", a->rows, kMaxExtent);
  if (too_far(a->rows, a->ldx, 2) || too_far(a->rows, a->ldy, 4) || too_far(a->rows, a->xs_row, 4) || too_far(d.K, a->xs_blk, 4))
    return record_error(CONVF_ERR_INVALID_ARG, "ldx=%lld, ldy=%lld, x_scale strides (%lld, %lld): the rows pass the address space",
                        a->ldx, a->ldy, a->xs_row, a->xs_blk);
  if (a->ldx < d.K) return record_error(CONVF_ERR_INVALID_ARG, "ldx=%lld is less than K=%d", a->ldx, d.K);
  if (a->ldx * esz % 16)
    return record_error(CONVF_ERR_UNSUPPORTED, "ldx=%lld: rows of x must be a multiple of 16 bytes apart", a->ldx);
  if (a->ldy < d.N) return record_error(CONVF_ERR_INVALID_ARG, "ldy=%lld is less than N=%d", a->ldy, d.N);
  if (e4m3 && (a->xs_row < 0 || a->xs_blk < 0))
    return record_error(CONVF_ERR_INVALID_ARG, "x_scale strides (%lld, %lld) must be >= 0", a->xs_row, a->xs_blk);
  if (!a->offsets && d.experts > 1) return record_error(CONVF_ERR_INVALID_ARG, "%d experts need row offsets", d.experts);
  if (a->rows == 0) return record_ok();
  if (!a->x || !a->y) return record_error(CONVF_ERR_INVALID_ARG, "x or y is NULL");
  if (e4m3 != (a->x_scale != nullptr))
    return record_error(CONVF_ERR_INVALID_ARG, "x_scale goes with e4m3 layers, and with those only");
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
  const Region xs_at = !e4m3 ? Region{}
                       : a->xs_blk == 1 ? Region{a->x_scale, a->rows, nblk * 4, a->xs_row * 4}
                       : a->xs_row == 1 ? Region{a->x_scale, nblk, a->rows * 4LL, a->xs_blk * 4}
                                        : Region{a->x_scale, 1, ((a->rows - 1) * a->xs_row + (nblk - 1) * a->xs_blk + 1) * 4, 0};
  if (overlap(Region{a->x, a->rows, d.K * esz, a->ldx * esz}, y_at))
    return record_error(CONVF_ERR_INVALID_ARG, "x and y overlap");
  if (overlap(w_at, y_at)) return record_error(CONVF_ERR_INVALID_ARG, "the weights and y overlap");
  if (overlap(xs_at, y_at)) return record_error(CONVF_ERR_INVALID_ARG, "x_scale and y overlap");
  if (overlap(Region{l->w_scale, 1, d.experts * wblk * nblk * 4, 0}, y_at) ||
      overlap(Region{l->bias, 1, static_cast<long long>(d.experts) * d.N * 4, 0}, y_at) ||
      overlap(Region{a->offsets, 1, (d.experts + 1) * 4LL, 0}, y_at))
    return record_error(CONVF_ERR_INVALID_ARG, "w_scale, bias or offsets overlap y");
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != l->device)
    return record_error(CONVF_ERR_INVALID_ARG, "the current device (%d) is not the layer's device (%d)", dev, l->device);
  const LinearPlan plan = make_plan(d, l->device, l->num_sms, a->rows);
  CUtensorMap tmX;
  const cuuint64_t size[2] = {static_cast<cuuint64_t>(d.K), static_cast<cuuint64_t>(a->rows)};
  const cuuint64_t stride = a->ldx * esz;
  st = encode_map(&tmX, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<int>(esz), 2,
                  a->x, size, &stride, plan.tile < 128 ? plan.tile : 128, "x");
  if (st != CONVF_OK) return st;
  LinearParams p{};
  p.rows = a->rows; p.N = d.N; p.experts = d.experts;
  p.num_kb = static_cast<int>(ceil_div(d.K * esz, kKBlockBytes));
  p.n_tiles = static_cast<int>(ceil_div(d.N, plan.form == kLinearMany ? kManyCols : 128));
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
  if (plan.form == kLinearMany && p.vec_y) {
    const cuuint64_t ysize[2] = {static_cast<cuuint64_t>(d.N), static_cast<cuuint64_t>(a->rows)};
    const cuuint64_t ystride = a->ldy * osz;
    st = encode_map(&tmY, osz == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                    static_cast<int>(osz), 2, a->y, ysize, &ystride, 32, "y");
    if (st != CONVF_OK) return st;
  }
  const cudaStream_t strm = static_cast<cudaStream_t>(stream);
  const cudaError_t e = plan.form == kLinearFew
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
                         l->d.dtype == CONVF_LINEAR_E4M3 ? "e4m3" : "bf16", rows,
                         l->d.out_dtype == CONVF_OUT_BF16 ? "bf16" : "f32");
  if (rows > 0 && n > 0 && static_cast<size_t>(n) < len) {
    int dev = -1;   // the plan asks the current device how many clusters it runs at once
    if (cudaGetDevice(&dev) != cudaSuccess || dev != l->device)
      return record_error(CONVF_ERR_INVALID_ARG, "the current device (%d) is not the layer's device (%d)", dev, l->device);
    const LinearPlan plan = make_plan(l->d, l->device, l->num_sms, rows);
    snprintf(buf + n, len - n, " form=%s tile=%dx%d split=%d grid=%d", plan.form == kLinearFew ? "few_rows" : "many_rows",
             plan.tile, plan.form == kLinearFew ? 128 : kManyCols, plan.split, plan.grid);
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
