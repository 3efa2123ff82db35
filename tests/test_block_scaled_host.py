"""The block-scaled operators without a GPU: what the kernels' sources must not hold, and the host side on
stand-ins for CUDA tensors and for the CUDA runtime."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "convolution_onnx_conv_gb300", "csrc")


def source(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", ["k_quant.cu", "linear_dev.cuh", "tc_linear_few.cu", "tc_linear_many.cu"])
def test_no_read_only_loads_of_what_the_kernel_before_may_write(name):
    """The kernels begin while the kernel before them in the stream still runs and wait for it inside.  A
    read-only load (ld.global.nc) asks for data that nothing writes while the kernel runs, and an asm statement
    that is not volatile may be moved above the wait: neither may read x, an index, scales, offsets or biases."""
    text = source(name)
    assert not re.search(r"__ldg\b|\.nc\b|__ldcg|__ldca", text)
    assert not re.search(r"asm\s*\(\s*\"ld\.", text)


# ------------------------------------------------------------------------------ tensors of several devices

class FakeCuda:
    """What the binding asks of a CUDA tensor."""
    is_cuda = True

    def __init__(self, shape, dtype, device=0, strides=None):
        self.shape, self.dtype, self._device = tuple(shape), dtype, device
        self.device = f"cuda:{device}"
        if strides is None:
            strides, n = [], 1
            for d in reversed(self.shape):
                strides.insert(0, n)
                n *= d
        self._strides = tuple(strides)

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self._strides if i is None else self._strides[i]

    def get_device(self):
        return self._device

    def data_ptr(self):
        return 1 << 28

    def is_contiguous(self):
        return True

    def contiguous(self):
        return self

    def __getitem__(self, _):   # t[None]
        return FakeCuda((1,) + self.shape, self.dtype, self._device, (0,) + self._strides)


@pytest.fixture
def calls(monkeypatch):
    """The library's calls, recorded instead of made; the current device is 0."""
    from convolution_onnx_conv_gb300 import _binding, _build
    _build.build()
    names, made = _binding._Torch, []
    names.bind()
    monkeypatch.setattr(names, "stream", lambda index: 0)
    monkeypatch.setattr(names, "current_device", lambda: 0, raising=False)
    monkeypatch.setattr(names, "empty", lambda shape, dtype, device: FakeCuda(shape, dtype))
    monkeypatch.setattr(names, "quantize", lambda args, stream: made.append(args._obj) or 0)
    monkeypatch.setattr(names, "run", lambda layer, args, stream: made.append(args._obj) or 0)
    monkeypatch.setattr(_binding, "conv_fused_linear_create", lambda d, *tensors: made.append(d) or 0)   # (no handle to free)
    return made


def test_quantise_takes_tensors_of_the_current_device_only(calls):
    import torch
    import convolution_onnx_conv_gb300 as cf
    x = FakeCuda((4, 256), torch.bfloat16)
    cf.quantize_blocks(x)
    assert len(calls) == 1
    for kw in (dict(x=FakeCuda((4, 256), torch.bfloat16, 1)), dict(index=FakeCuda((4,), torch.int32, 1)),
               dict(q=FakeCuda((4, 256), torch.float8_e4m3fn, 1)), dict(scale=FakeCuda((4, 2), torch.float32, 1))):
        with pytest.raises(ValueError, match="device 1"):
            cf.quantize_blocks(**{"x": x, **kw})
    assert len(calls) == 1


def test_layers_take_tensors_of_their_device_only(calls):
    import torch
    import convolution_onnx_conv_gb300 as cf
    e4m3, f32 = torch.float8_e4m3fn, torch.float32

    def operands(device=0):
        return dict(w=FakeCuda((3, 96, 256), e4m3, device), w_scale=FakeCuda((3, 1, 2), f32, device),
                    bias=FakeCuda((3, 96), f32, device))

    layer = cf.ExpertLinear(**operands())
    assert len(calls) == 1
    for name in ("w", "w_scale", "bias"):
        with pytest.raises(ValueError, match="device 1"):
            cf.ExpertLinear(**{**operands(), name: operands(1)[name]})
    with pytest.raises(ValueError, match="device 1"):
        cf.ExpertLinear(**operands(1))
    assert len(calls) == 1

    def run(device=0):
        return dict(x=FakeCuda((4, 256), e4m3, device), offsets=FakeCuda((4,), torch.int32, device),
                    x_scale=FakeCuda((4, 2), f32, device), y=FakeCuda((4, 96), f32, device))

    layer(**run())
    assert len(calls) == 2
    for name in ("x", "offsets", "x_scale", "y"):
        with pytest.raises(ValueError, match="device 1"):
            layer(**{**run(), name: run(1)[name]})
    assert len(calls) == 2


# ------------------------------------------------------------------------------ two devices in a process

TWO_DEVICES = r"""
#include <cuda_runtime.h>
#include <cstdio>
#include <cstring>
#include <map>
#include <utility>
// a runtime of two devices, each with its own limit of dynamic shared memory per kernel (48 KB at first)
static int device = 0;
static std::map<std::pair<int, const void*>, size_t> limit;
template <typename F> const void* address(F f) { const void* p; memcpy(&p, &f, sizeof p); return p; }
static cudaError_t fake_get_device(int* d) { *d = device; return cudaSuccess; }
template <typename F> cudaError_t fake_set(F f, cudaFuncAttribute, int bytes) {
  limit[{device, address(f)}] = bytes;
  return cudaSuccess;
}
template <typename F> cudaError_t fake_attributes(cudaFuncAttributes* a, F) { a->numRegs = 168; return cudaSuccess; }
template <typename F> bool fits(size_t bytes, F f) {
  const auto at = limit.find({device, address(f)});
  return bytes <= (at == limit.end() ? 49152 : at->second);
}
template <typename F, typename... A> cudaError_t fake_launch(const cudaLaunchConfig_t* c, F f, A&&...) {
  return fits(c->dynamicSmemBytes, f) ? cudaSuccess : cudaErrorInvalidValue;
}
template <typename F> cudaError_t fake_clusters(int* n, F f, const cudaLaunchConfig_t* c) {
  *n = 18;
  return fits(c->dynamicSmemBytes, f) ? cudaSuccess : cudaErrorInvalidValue;
}
#define cudaGetDevice fake_get_device
#define cudaFuncSetAttribute fake_set
#define cudaFuncGetAttributes fake_attributes
#define cudaLaunchKernelEx fake_launch
#define cudaOccupancyMaxActiveClusters fake_clusters
#include SOURCE
int main() {
  convf::LinearParams p{};
  CUtensorMap m{};
  int bad = 0;
  for (device = 0; device < 2; ++device)
    for (int e4m3 = 0; e4m3 < 2; ++e4m3)
      for (int turn = 0; turn < 2; ++turn)
        for (int i = 0; i < 3; ++i) {
#ifdef FEW
          const convf::LinearPlan plan{convf::kLinearFew, 16 << i, 1, 152};
          bad += convf::launch_linear_few(p, plan, e4m3, m, m, nullptr) != cudaSuccess;
          bad += convf::linear_few_max_clusters(e4m3, 16 << i, 4, 152) != 18;
#else
          const convf::LinearPlan plan{convf::kLinearMany, i ? 256 : 128, 1, 152};
          p.vec_y = i == 2;
          bad += convf::launch_linear_many(p, plan, e4m3, m, m, m, nullptr) != cudaSuccess;
#endif
        }
  printf("%d refused\n", bad);
  return bad != 0;
}
"""


@pytest.mark.parametrize("name", ["tc_linear_few", "tc_linear_many"])
def test_kernels_are_set_up_on_every_device(name, tmp_path):
    """The host side of the launches, on a runtime that keeps a kernel's shared-memory limit per device."""
    import subprocess
    from convolution_onnx_conv_gb300 import _build
    main = tmp_path / "main.cu"
    main.write_text(TWO_DEVICES)
    exe = str(tmp_path / "main")
    subprocess.run([_build._nvcc(), "-gencode", "arch=compute_103a,code=compute_103a", "-Xcicc", "-O0", "-std=c++17",
                    "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    f'-DSOURCE="{name}.cu"', *(["-DFEW"] if name == "tc_linear_few" else []), str(main), "-o", exe, "-lcuda"],
                   check=True, capture_output=True)
    res = subprocess.run([exe], capture_output=True, text=True)
    assert res.returncode == 0 and res.stdout == "0 refused\n", res.stdout + res.stderr


# ------------------------------------------------------------------------------ operands that overlap

REGIONS = r"""
#include "linear_internal.h"
#include <cstdio>
#include <cstdlib>
#include <vector>
using convf::Region;
static void mark(std::vector<int>& bytes, Region g, int bit) {
  for (long long i = 0; i < g.rows; ++i)
    for (long long k = 0; k < g.row; ++k) bytes[reinterpret_cast<uintptr_t>(g.p) + i * g.stride + k] |= bit;
}
int main() {
  srand(1);
  int met = 0, free_inside = 0, wrong = 0;
  for (int n = 0; n < 200000; ++n) {
    auto any = [&](bool same, long long stride) {
      const long long row = 1 + rand() % 8, rows = rand() % 5;
      return Region{reinterpret_cast<const void*>(uintptr_t(1 + rand() % 60)), rows, row,
                    same ? stride : row + rand() % 8};
    };
    const bool same = rand() % 4 != 0;
    const long long stride = 8 + rand() % 8;
    const Region a = any(same, stride), b = any(same, stride);
    std::vector<int> bytes(400);
    mark(bytes, a, 1);
    mark(bytes, b, 2);
    bool share = false;
    for (int v : bytes) share |= v == 3;
    const bool said = convf::overlap(a, b);
    // exact at equal strides; else what shares a byte is never let through
    wrong += (same || a.rows == 1 || b.rows == 1) && a.row <= b.stride && b.row <= a.stride ? said != share : share && !said;
    wrong += said != convf::overlap(b, a);
    met += share;
    free_inside += !said && same && a.rows > 1 && b.rows > 1;
  }
  printf("%d wrong, %d\n", wrong, met > 1000 && free_inside > 1000);
  return wrong;
}
"""


def test_overlap_of_strided_rows_against_their_bytes(tmp_path):
    import subprocess
    from convolution_onnx_conv_gb300 import _build
    main, exe = tmp_path / "main.cpp", str(tmp_path / "main")
    main.write_text(REGIONS)
    subprocess.run([_build._nvcc(), "-std=c++17", "-I", CSRC, str(main), "-o", exe], check=True, capture_output=True)
    res = subprocess.run([exe], capture_output=True, text=True)
    assert res.stdout == "0 wrong, 1\n"


@pytest.mark.parametrize("where", ["q", "scale"])
def test_an_index_that_overlaps_an_output_is_refused(where):
    import convolution_onnx_conv_gb300 as cf
    from convolution_onnx_conv_gb300 import _build
    from convolution_onnx_conv_gb300._binding import QuantArgs
    _build.build()
    P = 0x10000000   # addresses that nothing reads: the call is refused before any CUDA call
    a = QuantArgs(rows=4, cols=200, x=P, x_dtype=cf.CONVF_OUT_BF16, x_rows=9, ldx=200, index=4 * P, gated=0, block_rows=1,
                  q=2 * P, ldq=208, scale=3 * P, lds=2)
    setattr(a, where, 4 * P + 8)
    with pytest.raises(cf.ConvFusedError) as e:
        cf.conv_fused_quantize_blocks(a)
    assert e.value.status == cf.CONVF_ERR_INVALID_ARG and "index and q or scale overlap" in str(e.value)


# ------------------------------------------------------------------------------ one row has no stride

def test_the_stride_of_one_row_is_not_asked_about(calls):
    """A row out of a wider buffer, whose rows are an odd number of elements apart."""
    import torch
    import convolution_onnx_conv_gb300 as cf
    bf16 = torch.bfloat16
    layer = cf.BlockLinear(FakeCuda((1, 17), bf16, strides=(33, 1)))           # N = 1
    assert calls[-1].ldw >= 17 and calls[-1].ldw * 2 % 16 == 0
    layer(FakeCuda((1, 17), bf16, strides=(35, 1)), y=FakeCuda((1, 1), torch.float32, strides=(7, 1)))
    assert calls[-1].ldx >= 17 and calls[-1].ldx * 2 % 16 == 0
    cf.quantize_blocks(FakeCuda((1, 256), bf16, strides=(257, 1)), q=FakeCuda((1, 256), torch.float8_e4m3fn, strides=(259, 1)))
    assert calls[-1].ldx * 2 % 32 == 0 and calls[-1].ldq % 16 == 0             # (read and written as vectors)
