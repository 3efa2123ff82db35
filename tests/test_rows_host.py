"""Refusals of the int8 row quantiser and the norm that need no GPU: every malformed argument is named before any
CUDA call, and tensors are looked at on stand-ins."""
import pytest

import convolution_onnx_conv_gb300 as cf
from convolution_onnx_conv_gb300 import _binding, _build
from convolution_onnx_conv_gb300._binding import NormArgs, QuantRowsArgs
from test_block_scaled_host import FakeCuda, source

P = 0x10000000   # an aligned address that nothing reads
BAD, NOT = cf.CONVF_ERR_INVALID_ARG, cf.CONVF_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return cf.load_library()


def rows_args(**kw):
    v = dict(rows=4, cols=200, x=P, x_dtype=cf.CONVF_OUT_BF16, x_rows=4, ldx=200, index=None, gated=0, q=2 * P, ldq=208, scale=3 * P)
    v.update(kw)
    return QuantRowsArgs(*[v[n] for n, _ in QuantRowsArgs._fields_])


@pytest.mark.parametrize("kw,status,needle", [
    (dict(rows=-1), BAD, "rows=-1"),
    (dict(cols=0), BAD, "cols=0"),
    (dict(cols=2 ** 30 + 1), NOT, "cols=1073741825"),
    (dict(rows=2 ** 31 - 1), NOT, "rows=2147483647"),
    (dict(x_rows=-2), BAD, "x_rows=-2"),
    (dict(x_rows=5), BAD, "x_rows=5"),
    (dict(x_dtype=2), BAD, "x_dtype=2"),
    (dict(gated=2), BAD, "gated=2"),
    (dict(ldx=199), BAD, "ldx=199"),
    (dict(gated=1, ldx=399), BAD, "ldx=399"),
    (dict(ldq=199), BAD, "ldq=199"),
    (dict(ldx=2 ** 62), BAD, "address space"),
    (dict(rows=2 ** 30, x_rows=2 ** 30, ldq=2 ** 40), BAD, "address space"),
    (dict(x=None), BAD, "NULL"),
    (dict(q=None), BAD, "NULL"),
    (dict(scale=None), BAD, "NULL"),
    (dict(x=P + 1), BAD, "aligned"),
    (dict(scale=3 * P + 2), BAD, "aligned"),
    (dict(index=4 * P + 1), BAD, "aligned"),
    (dict(q=P + 1500), BAD, "overlap"),
    (dict(scale=2 * P + 700), BAD, "overlap"),
    (dict(scale=P + 40), BAD, "overlap"),
    (dict(index=2 * P + 4, x_rows=9), BAD, "index and q or scale overlap"),
    (dict(index=3 * P + 8, x_rows=9), BAD, "index and q or scale overlap"),
])
def test_rows_refusals(kw, status, needle):
    with pytest.raises(cf.ConvFusedError) as e:
        cf.conv_fused_quantize_rows(rows_args(**kw))
    assert e.value.status == status and needle in str(e.value)


def norm_args(**kw):
    v = dict(rows=4, cols=200, x=P, x_dtype=cf.CONVF_OUT_BF16, ldx=200, residual=2 * P, residual_dtype=cf.CONVF_OUT_F32, ldr=200,
             h=3 * P, ldh=200, weight=4 * P, weight_dtype=cf.CONVF_OUT_F32, eps=1e-6, out=cf.CONVF_LINEAR_E4M3, q=5 * P, ldq=208,
             scale=6 * P, lds=2)
    v.update(kw)
    return NormArgs(*[v[n] for n, _ in NormArgs._fields_])


@pytest.mark.parametrize("kw,status,needle", [
    (dict(rows=-1), BAD, "rows=-1"),
    (dict(cols=0), BAD, "cols=0"),
    (dict(cols=2 ** 30 + 1), NOT, "cols=1073741825"),
    (dict(x_dtype=3), BAD, "x_dtype=3"),
    (dict(residual_dtype=-1), BAD, "residual_dtype=-1"),
    (dict(weight_dtype=2), BAD, "weight_dtype=2"),
    (dict(out=0), BAD, "out=0"),
    (dict(out=2), BAD, "out=2"),
    (dict(eps=0.0), BAD, "eps=0"),
    (dict(eps=-1.0), BAD, "eps=-1"),
    (dict(eps=float("nan")), BAD, "eps=nan"),
    (dict(eps=float("inf")), BAD, "eps=inf"),
    (dict(residual=None), BAD, "h goes with a residual"),
    (dict(ldx=199), BAD, "ldx=199"),
    (dict(ldr=199), BAD, "ldr=199"),
    (dict(ldh=199), BAD, "ldh=199"),
    (dict(ldq=199), BAD, "ldq=199"),
    (dict(lds=1), BAD, "lds=1"),
    (dict(ldh=2 ** 60), BAD, "address space"),
    (dict(lds=2 ** 60), BAD, "address space"),
    (dict(x=None), BAD, "NULL"),
    (dict(q=None), BAD, "NULL"),
    (dict(scale=None), BAD, "NULL"),
    (dict(x=P + 1), BAD, "aligned"),
    (dict(residual=2 * P + 2), BAD, "aligned"),
    (dict(h=3 * P + 2), BAD, "aligned"),
    (dict(weight=4 * P + 2), BAD, "aligned"),
    (dict(scale=6 * P + 1), BAD, "aligned"),
    (dict(h=2 * P, ldh=204), BAD, "not the same rows"),            # over the residual, at another stride
    (dict(h=2 * P + 400), BAD, "not the same rows"),
    (dict(h=P), BAD, "not the same rows"),                         # over x, which has another type
    (dict(h=P + 800, residual_dtype=cf.CONVF_OUT_BF16), BAD, "not the same rows"),
    (dict(q=P + 8), BAD, "q or scale overlaps"),
    (dict(q=2 * P + 8), BAD, "q or scale overlaps"),
    (dict(q=3 * P + 8), BAD, "q or scale overlaps"),
    (dict(q=4 * P + 8), BAD, "q or scale overlaps"),
    (dict(scale=3 * P + 8), BAD, "q or scale overlaps"),
    (dict(scale=5 * P + 8), BAD, "q and scale overlap"),
    (dict(weight=3 * P + 8), BAD, "h and weight overlap"),
])
def test_norm_refusals(kw, status, needle):
    with pytest.raises(cf.ConvFusedError) as e:
        cf.conv_fused_rms_norm_quantize(norm_args(**kw))
    assert e.value.status == status and needle in str(e.value)


def test_no_rows_is_no_launch():
    cf.conv_fused_quantize_rows(rows_args(rows=0, x_rows=0, x=None, q=None, scale=None))
    cf.conv_fused_rms_norm_quantize(norm_args(rows=0, x=None, q=None, scale=None))
    for call in ("conv_fused_quantize_rows", "conv_fused_rms_norm_quantize"):
        assert getattr(cf.load_library(), call)(None, None) == BAD


@pytest.mark.parametrize("name", ["k_rows.cu", "quant_dev.cuh"])
def test_no_read_only_loads_of_what_the_kernel_before_may_write(name):
    import re
    text = source(name)
    assert not re.search(r"__ldg\b|\.nc\b|__ldcg|__ldca", text)
    assert not re.search(r"asm\s*\(\s*\"ld\.", text)


# ------------------------------------------------------------------------------ tensors

@pytest.fixture
def calls(monkeypatch):
    names, made = _binding._Torch, []
    names.bind()
    monkeypatch.setattr(names, "stream", lambda index: 0)
    monkeypatch.setattr(names, "current_device", lambda: 0, raising=False)
    monkeypatch.setattr(names, "empty", lambda shape, dtype, device: FakeCuda(shape, dtype))
    monkeypatch.setattr(names, "empty_strided", lambda shape, strides, dtype, device: FakeCuda(shape, dtype, strides=strides))
    monkeypatch.setattr(names, "quantize_rows", lambda args, stream: made.append(args._obj) or 0)
    monkeypatch.setattr(names, "norm", lambda args, stream: made.append(args._obj) or 0)
    return made


def test_rows_tensors_are_looked_at(calls):
    import torch
    bf16, f32, i8 = torch.bfloat16, torch.float32, torch.int8
    x = FakeCuda((4, 250), bf16)
    q, s = cf.quantize_rows(x)
    assert q.dtype is i8 and q.shape == (4, 250) and q.stride(0) == 256 and s.shape == (4,) and len(calls) == 1
    for kw, words in ((dict(x=FakeCuda((4, 250), torch.float16)), "bf16 or fp32"),
                      (dict(x=FakeCuda((4, 250), bf16, 1)), "device 1"),
                      (dict(x=FakeCuda((4, 250), bf16, strides=(1, 4))), "adjacent"),
                      (dict(x=FakeCuda((4, 251), bf16), gated=True), "even number"),
                      (dict(index=FakeCuda((4,), torch.int64)), "int32"),
                      (dict(index=FakeCuda((4,), torch.int32, 1)), "device 1"),
                      (dict(q=FakeCuda((4, 250), torch.uint8)), "q must be"),
                      (dict(q=FakeCuda((4, 249), i8)), "q must be"),
                      (dict(q=FakeCuda((4, 250), i8, 1)), "device 1"),
                      (dict(scale=FakeCuda((4, 2), f32)), "vector of 4"),
                      (dict(scale=FakeCuda((4,), bf16)), "vector of 4"),
                      (dict(scale=FakeCuda((4,), f32, 1)), "device 1")):
        with pytest.raises(ValueError, match=words):
            cf.quantize_rows(**{"x": x, **kw})
    assert len(calls) == 1


def test_norm_tensors_are_looked_at(calls):
    import torch
    bf16, f32, i8, e4m3 = torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn
    x, r = FakeCuda((4, 250), bf16), FakeCuda((4, 250), f32)
    q, s = cf.rms_norm_quantize(x)
    assert q.dtype is e4m3 and s.shape == (4, 2)
    q, s, h = cf.rms_norm_quantize(x, FakeCuda((250,), bf16), residual=r, int8=True)
    assert q.dtype is i8 and s.shape == (4,) and h.dtype is f32 and h.shape == (4, 250) and len(calls) == 2
    assert calls[1].weight_dtype == cf.CONVF_OUT_BF16 and calls[1].residual_dtype == cf.CONVF_OUT_F32 and calls[1].out == cf.CONVF_LINEAR_INT8
    for kw, words in ((dict(x=FakeCuda((4, 250), torch.float16)), "bf16 or fp32"),
                      (dict(x=FakeCuda((250,), bf16)), "two dimensions"),
                      (dict(x=FakeCuda((4, 250), bf16, 1)), "device 1"),
                      (dict(weight=FakeCuda((249,), f32)), "vector of 250"),
                      (dict(weight=FakeCuda((250,), torch.float16)), "bf16 or fp32"),
                      (dict(weight=FakeCuda((250,), f32, 1)), "device 1"),
                      (dict(residual=FakeCuda((4, 249), f32)), "residual must be"),
                      (dict(residual=FakeCuda((4, 250), torch.float64)), "bf16 or fp32"),
                      (dict(residual=FakeCuda((4, 250), f32, 1)), "device 1"),
                      (dict(residual=r, h=FakeCuda((4, 250), bf16)), "h must be"),
                      (dict(residual=r, h=FakeCuda((5, 250), f32)), "h must be"),
                      (dict(residual=r, h=FakeCuda((4, 250), f32, 1)), "device 1"),
                      (dict(h=FakeCuda((4, 250), bf16)), "h goes with a residual"),
                      (dict(q=FakeCuda((4, 250), i8)), "q must be"),
                      (dict(int8=True, q=FakeCuda((4, 250), e4m3)), "q must be"),
                      (dict(scale=FakeCuda((4,), f32)), "two dimensions"),
                      (dict(scale=FakeCuda((4, 3), f32)), "scale must be"),
                      (dict(int8=True, scale=FakeCuda((4, 2), f32)), "vector of 4")):
        with pytest.raises(ValueError, match=words):
            cf.rms_norm_quantize(**{"x": x, **kw})
    assert len(calls) == 2
