"""Refusals of the block-scaled operators that need no GPU: every malformed argument is named before
any CUDA call."""
import ctypes

import pytest

import convolution_onnx_conv_gb300 as cf
from convolution_onnx_conv_gb300 import _build
from convolution_onnx_conv_gb300._binding import LinearArgs, LinearDesc, QuantArgs


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return cf.load_library()


P = 0x10000000   # an aligned address that nothing reads


def quant(**kw):
    v = dict(rows=4, cols=200, x=P, x_dtype=cf.CONVF_OUT_BF16, x_rows=4, ldx=200, index=None, gated=0, block_rows=1,
             q=2 * P, ldq=208, scale=3 * P, lds=2)
    v.update(kw)
    return QuantArgs(*[v[n] for n, _ in QuantArgs._fields_])


@pytest.mark.parametrize("kw,status,needle", [
    (dict(rows=-1), cf.CONVF_ERR_INVALID_ARG, "rows=-1"),
    (dict(cols=0), cf.CONVF_ERR_INVALID_ARG, "cols=0"),
    (dict(x_rows=-2), cf.CONVF_ERR_INVALID_ARG, "x_rows=-2"),
    (dict(x_rows=5), cf.CONVF_ERR_INVALID_ARG, "x_rows=5"),
    (dict(x_dtype=2), cf.CONVF_ERR_INVALID_ARG, "x_dtype=2"),
    (dict(cols=2 ** 31 - 200), cf.CONVF_ERR_UNSUPPORTED, "cols=2147483448"),
    (dict(rows=2 ** 31 - 1), cf.CONVF_ERR_UNSUPPORTED, "rows=2147483647"),
    (dict(ldx=2 ** 62), cf.CONVF_ERR_INVALID_ARG, "address space"),
    (dict(rows=2 ** 30, x_rows=2 ** 30, ldq=2 ** 40), cf.CONVF_ERR_INVALID_ARG, "address space"),
    (dict(gated=2), cf.CONVF_ERR_INVALID_ARG, "gated=2"),
    (dict(block_rows=64), cf.CONVF_ERR_INVALID_ARG, "block_rows=64"),
    (dict(block_rows=128, index=4 * P), cf.CONVF_ERR_UNSUPPORTED, "block_rows = 1"),
    (dict(block_rows=128, gated=1), cf.CONVF_ERR_UNSUPPORTED, "block_rows = 1"),
    (dict(ldx=199), cf.CONVF_ERR_INVALID_ARG, "ldx=199"),
    (dict(gated=1, ldx=399), cf.CONVF_ERR_INVALID_ARG, "ldx=399"),
    (dict(ldq=199), cf.CONVF_ERR_INVALID_ARG, "ldq=199"),
    (dict(lds=1), cf.CONVF_ERR_INVALID_ARG, "lds=1"),
    (dict(x=None), cf.CONVF_ERR_INVALID_ARG, "NULL"),
    (dict(q=None), cf.CONVF_ERR_INVALID_ARG, "NULL"),
    (dict(scale=None), cf.CONVF_ERR_INVALID_ARG, "NULL"),
    (dict(x=P + 1), cf.CONVF_ERR_INVALID_ARG, "aligned"),
    (dict(scale=3 * P + 2), cf.CONVF_ERR_INVALID_ARG, "aligned"),
    (dict(q=P + 1500), cf.CONVF_ERR_INVALID_ARG, "overlap"),
    (dict(scale=2 * P + 700), cf.CONVF_ERR_INVALID_ARG, "overlap"),
])
def test_quantise_refusals(kw, status, needle):
    with pytest.raises(cf.ConvFusedError) as e:
        cf.conv_fused_quantize_blocks(quant(**kw))
    assert e.value.status == status and needle in str(e.value)


def test_quantise_no_rows_is_no_launch(lib):
    cf.conv_fused_quantize_blocks(quant(rows=0, x_rows=0, x=None, q=None, scale=None))
    assert lib.conv_fused_quantize_blocks(None, None) == cf.CONVF_ERR_INVALID_ARG


def linear(**kw):
    v = dict(N=96, K=200, experts=3, dtype=cf.CONVF_LINEAR_E4M3, ldw=208, expert_stride=96 * 208, act=cf.CONVF_ACT_NONE,
             clip_lo=0.0, clip_hi=6.0, out_dtype=cf.CONVF_OUT_F32)
    v.update(kw)
    return LinearDesc(*[v[n] for n, _ in LinearDesc._fields_])


@pytest.mark.parametrize("kw,status,needle", [
    (dict(N=0), cf.CONVF_ERR_INVALID_ARG, "N=0"),
    (dict(K=0), cf.CONVF_ERR_INVALID_ARG, "K=0"),
    (dict(N=2 ** 31 - 255), cf.CONVF_ERR_UNSUPPORTED, "N=2147483393"),
    (dict(K=2 ** 31 - 1, ldw=2 ** 31), cf.CONVF_ERR_UNSUPPORTED, "K=2147483647"),
    (dict(ldw=2 ** 61), cf.CONVF_ERR_INVALID_ARG, "address space"),
    (dict(expert_stride=2 ** 61), cf.CONVF_ERR_INVALID_ARG, "address space"),
    (dict(experts=0), cf.CONVF_ERR_INVALID_ARG, "experts=0"),
    (dict(experts=1025), cf.CONVF_ERR_UNSUPPORTED, "experts=1025"),
    (dict(dtype=2), cf.CONVF_ERR_INVALID_ARG, "dtype=2"),
    (dict(ldw=192), cf.CONVF_ERR_INVALID_ARG, "ldw=192"),
    (dict(ldw=204), cf.CONVF_ERR_UNSUPPORTED, "16 bytes"),
    (dict(dtype=cf.CONVF_LINEAR_BF16, ldw=204), cf.CONVF_ERR_UNSUPPORTED, "16 bytes"),
    (dict(expert_stride=95 * 208), cf.CONVF_ERR_INVALID_ARG, "overlap"),
    (dict(expert_stride=96 * 208 + 8), cf.CONVF_ERR_UNSUPPORTED, "16 bytes"),
    (dict(act=4), cf.CONVF_ERR_INVALID_ARG, "act=4"),
    (dict(act=cf.CONVF_ACT_CLIP, clip_lo=2.0, clip_hi=1.0), cf.CONVF_ERR_INVALID_ARG, "clip"),
    (dict(act=cf.CONVF_ACT_CLIP, clip_lo=float("nan")), cf.CONVF_ERR_INVALID_ARG, "clip"),
    (dict(out_dtype=2), cf.CONVF_ERR_INVALID_ARG, "out_dtype=2"),
])
def test_linear_refusals(kw, status, needle):
    with pytest.raises(cf.ConvFusedError) as e:
        cf.conv_fused_linear_create(linear(**kw), P, 2 * P)
    assert e.value.status == status and needle in str(e.value)


@pytest.mark.parametrize("w,ws,dtype,needle", [
    (None, P, cf.CONVF_LINEAR_E4M3, "W is NULL"), (P + 8, P, cf.CONVF_LINEAR_E4M3, "16-byte"),
    (P, None, cf.CONVF_LINEAR_E4M3, "w_scale"), (P, P, cf.CONVF_LINEAR_BF16, "w_scale"),
    (P, P + 2, cf.CONVF_LINEAR_E4M3, "aligned"),
])
def test_linear_pointer_refusals(w, ws, dtype, needle):
    with pytest.raises(cf.ConvFusedError) as e:
        cf.conv_fused_linear_create(linear(dtype=dtype), w, ws)
    assert e.value.status == cf.CONVF_ERR_INVALID_ARG and needle in str(e.value)


def test_layer_checks(lib):
    assert lib.conv_fused_linear_create(ctypes.byref(linear()), P, P, None, None) == cf.CONVF_ERR_INVALID_ARG
    assert lib.conv_fused_linear_run(None, ctypes.byref(LinearArgs()), None) == cf.CONVF_ERR_INVALID_ARG
    junk = (ctypes.c_uint32 * 64)()
    assert lib.conv_fused_linear_run(ctypes.addressof(junk), ctypes.byref(LinearArgs()), None) == cf.CONVF_ERR_INVALID_ARG
    assert "not a convf linear layer" in cf.conv_fused_last_error()
    assert lib.conv_fused_linear_status(None) == cf.CONVF_ERR_INVALID_ARG
    lib.conv_fused_linear_destroy(None)   # no-op


def test_create_reports_an_injected_host_allocation_failure():
    cf.conv_fused_debug_fail_alloc(1)
    with pytest.raises(cf.ConvFusedError) as e:
        cf.conv_fused_linear_create(linear(), P, 2 * P)
    assert e.value.status == cf.CONVF_ERR_OOM and "(injected)" in str(e.value)
