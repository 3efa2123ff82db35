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
