"""ctypes binding of ``libconvfused.so`` (argument marshalling only).

The Python names are the C names; every compute step runs in the library's CUDA
kernels.  There is no fallback: if the library is missing this module raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

from . import _build

# --- enums (mirror include/conv_fused.h)
CONVF_OK, CONVF_ERR_INVALID_ARG, CONVF_ERR_UNSUPPORTED, CONVF_ERR_OOM, CONVF_ERR_CUDA, \
    CONVF_ERR_TIMEOUT, CONVF_ERR_BOUNDS = 0, -1, -2, -3, -4, -5, -6
CONVF_BF16, CONVF_S8, CONVF_Q8 = 0, 1, 2
CONVF_OUT_F32, CONVF_OUT_BF16 = 0, 1
CONVF_NCHW, CONVF_NHWC = 0, 1
CONVF_ACT_NONE, CONVF_ACT_RELU, CONVF_ACT_RELU6, CONVF_ACT_CLIP = 0, 1, 2, 3
CONVF_AUTO_PAD_NOTSET, CONVF_AUTO_PAD_SAME_UPPER, CONVF_AUTO_PAD_SAME_LOWER, \
    CONVF_AUTO_PAD_VALID = 0, 1, 2, 3
CONVF_VARIANT_AUTO, CONVF_VARIANT_IMPLICIT_GEMM, CONVF_VARIANT_GEMM_1X1, CONVF_VARIANT_DEPTHWISE, \
    CONVF_VARIANT_INT8, CONVF_VARIANT_IMPLICIT_GEMM_GATHER, CONVF_VARIANT_IMPLICIT_GEMM_WINDOW, \
    CONVF_VARIANT_IMPLICIT_GEMM_HALO, CONVF_VARIANT_INT8_TC, CONVF_VARIANT_GROUPED_DIRECT, \
    CONVF_VARIANT_MBV2_BLOCK = 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10
VARIANT_NAMES = {0: "auto", 1: "implicit_gemm_im2col", 2: "gemm_1x1", 3: "depthwise",
                 4: "int8_mma", 5: "implicit_gemm_gather", 6: "implicit_gemm_window", 7: "implicit_gemm_halo",
                 8: "int8_tcgen05_exact", 9: "grouped_direct", 10: "mbv2_block"}
CONVF_LINEAR_BF16, CONVF_LINEAR_E4M3, CONVF_LINEAR_INT8 = 0, 1, 3
AUTO_PAD = {"NOTSET": 0, "SAME_UPPER": 1, "SAME_LOWER": 2, "VALID": 3}

EXPORTED = ["conv_fused_output_shape", "conv_fused_resolve_pads", "conv_bn_scale_shift",
            "conv_fused_plan", "conv_fused_pack_weights", "conv_fused_create", "conv_fused_run",
            "conv_fused_status", "conv_fused_clear_status", "conv_fused_destroy",
            "conv_fused_variant", "conv_fused_describe", "conv_fused_last_error",
            "conv_fused_watchdog_selftest", "conv_fused_run_noalloc", "conv_fused_measure_int8_mma_rate",
            "conv_fused_run_residual", "conv_fused_create_qlinear", "conv_fused_create_preact",
            "conv_fused_create_mbv2_block", "conv_fused_debug_fail_alloc", "conv_fused_debug_live_handles",
            "conv_fused_chain_create", "conv_fused_chain_create_ex", "conv_fused_chain_run", "conv_fused_chain_status",
            "conv_fused_chain_clear_status", "conv_fused_chain_describe", "conv_fused_chain_destroy",
            "conv_fused_quantize_blocks", "conv_fused_linear_create", "conv_fused_linear_run",
            "conv_fused_linear_status", "conv_fused_linear_clear_status", "conv_fused_linear_describe",
            "conv_fused_linear_destroy", "conv_fused_quantize_rows", "conv_fused_rms_norm_quantize"]


class ConvDesc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("C", ctypes.c_int), ("H", ctypes.c_int), ("W", ctypes.c_int),
                ("K", ctypes.c_int), ("R", ctypes.c_int), ("S", ctypes.c_int),
                ("stride", ctypes.c_int * 2), ("dilation", ctypes.c_int * 2),
                ("pads", ctypes.c_int * 4), ("auto_pad", ctypes.c_int), ("group", ctypes.c_int),
                ("dtype", ctypes.c_int), ("x_layout", ctypes.c_int), ("y_layout", ctypes.c_int),
                ("act", ctypes.c_int), ("clip_lo", ctypes.c_float), ("clip_hi", ctypes.c_float),
                ("variant", ctypes.c_int), ("tile_n", ctypes.c_int), ("cta_pair", ctypes.c_int),
                ("stream_k", ctypes.c_int), ("kblocks_per_step", ctypes.c_int),
                ("out_dtype", ctypes.c_int), ("residual", ctypes.c_int)]


class BlockDesc(ctypes.Structure):
    """convf_block_desc: one MobileNetV2 inverted-residual block."""
    _fields_ = [("N", ctypes.c_int), ("H", ctypes.c_int), ("W", ctypes.c_int), ("Cin", ctypes.c_int),
                ("Ch", ctypes.c_int), ("Cout", ctypes.c_int), ("stride", ctypes.c_int), ("expand", ctypes.c_int),
                ("residual", ctypes.c_int)]


class ChainStep(ctypes.Structure):
    """convf_chain_step: one conv run of a chain (handle, x, residual or NULL, y)."""
    _fields_ = [("conv", ctypes.c_void_p), ("x", ctypes.c_void_p), ("r", ctypes.c_void_p), ("y", ctypes.c_void_p)]


class QuantArgs(ctypes.Structure):
    """convf_quant_args: what conv_fused_quantize_blocks reads and writes."""
    _fields_ = [("rows", ctypes.c_int), ("cols", ctypes.c_int), ("x", ctypes.c_void_p), ("x_dtype", ctypes.c_int),
                ("x_rows", ctypes.c_int), ("ldx", ctypes.c_longlong), ("index", ctypes.c_void_p),
                ("gated", ctypes.c_int), ("block_rows", ctypes.c_int), ("q", ctypes.c_void_p),
                ("ldq", ctypes.c_longlong), ("scale", ctypes.c_void_p), ("lds", ctypes.c_longlong)]


class QuantRowsArgs(ctypes.Structure):
    """convf_quant_rows_args: what conv_fused_quantize_rows reads and writes."""
    _fields_ = [("rows", ctypes.c_int), ("cols", ctypes.c_int), ("x", ctypes.c_void_p), ("x_dtype", ctypes.c_int),
                ("x_rows", ctypes.c_int), ("ldx", ctypes.c_longlong), ("index", ctypes.c_void_p),
                ("gated", ctypes.c_int), ("q", ctypes.c_void_p), ("ldq", ctypes.c_longlong), ("scale", ctypes.c_void_p)]


class NormArgs(ctypes.Structure):
    """convf_norm_args: what conv_fused_rms_norm_quantize reads and writes."""
    _fields_ = [("rows", ctypes.c_int), ("cols", ctypes.c_int), ("x", ctypes.c_void_p), ("x_dtype", ctypes.c_int),
                ("ldx", ctypes.c_longlong), ("residual", ctypes.c_void_p), ("residual_dtype", ctypes.c_int),
                ("ldr", ctypes.c_longlong), ("h", ctypes.c_void_p), ("ldh", ctypes.c_longlong),
                ("weight", ctypes.c_void_p), ("weight_dtype", ctypes.c_int), ("eps", ctypes.c_float),
                ("out", ctypes.c_int), ("q", ctypes.c_void_p), ("ldq", ctypes.c_longlong), ("scale", ctypes.c_void_p),
                ("lds", ctypes.c_longlong)]


class LinearDesc(ctypes.Structure):
    """convf_linear_desc: a linear layer, or one per expert."""
    _fields_ = [("N", ctypes.c_int), ("K", ctypes.c_int), ("experts", ctypes.c_int), ("dtype", ctypes.c_int),
                ("ldw", ctypes.c_longlong), ("expert_stride", ctypes.c_longlong), ("act", ctypes.c_int),
                ("clip_lo", ctypes.c_float), ("clip_hi", ctypes.c_float), ("out_dtype", ctypes.c_int)]


class LinearArgs(ctypes.Structure):
    """convf_linear_args: one run's rows."""
    _fields_ = [("rows", ctypes.c_int), ("x", ctypes.c_void_p), ("ldx", ctypes.c_longlong),
                ("x_scale", ctypes.c_void_p), ("xs_row", ctypes.c_longlong), ("xs_blk", ctypes.c_longlong),
                ("offsets", ctypes.c_void_p), ("y", ctypes.c_void_p), ("ldy", ctypes.c_longlong)]


class QParams(ctypes.Structure):
    """convf_qparams: ONNX QLinearConv scales and zero points (host arrays for w's)."""
    _fields_ = [("x_signed", ctypes.c_int), ("w_signed", ctypes.c_int), ("y_signed", ctypes.c_int),
                ("x_zero_point", ctypes.c_int32), ("w_zero_point", ctypes.c_void_p), ("x_scale", ctypes.c_float),
                ("w_scale", ctypes.c_void_p), ("y_scale", ctypes.c_float), ("y_zero_point", ctypes.c_int32),
                ("relu", ctypes.c_int)]


def make_desc(N, C, H, W, K, R, S, stride=(1, 1), pads=(0, 0, 0, 0), dilation=(1, 1), group=1,
              dtype=CONVF_BF16, act=CONVF_ACT_NONE, clip=(0.0, 6.0), auto_pad="NOTSET",
              variant=CONVF_VARIANT_AUTO, layout=CONVF_NHWC, tile_n=0, cta_pair=0, stream_k=0,
              kblocks_per_step=0, out_dtype=CONVF_OUT_F32, residual=0) -> ConvDesc:
    d = ConvDesc()
    d.N, d.C, d.H, d.W, d.K, d.R, d.S = N, C, H, W, K, R, S
    d.stride[:] = list(stride)
    d.dilation[:] = list(dilation)
    d.pads[:] = list(pads)
    d.auto_pad = AUTO_PAD[auto_pad] if isinstance(auto_pad, str) else int(auto_pad)
    d.group = group
    d.dtype = dtype
    d.x_layout = d.y_layout = layout
    d.act = act
    d.clip_lo, d.clip_hi = float(clip[0]), float(clip[1])
    d.variant = variant
    d.tile_n = tile_n
    d.cta_pair = cta_pair
    d.stream_k = stream_k
    d.kblocks_per_step = kblocks_per_step
    d.out_dtype = out_dtype
    d.residual = residual
    return d


class ConvFusedError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"status {status}: {msg}")
        self.status = status


_LIB = None


def _bounds_build() -> bool:
    return os.environ.get("CONVF_DEBUG_BOUNDS", "") not in ("", "0")


def library_path() -> str:
    """The library this process loads: libconvfused.so, or the bounds-checking build when the
    environment sets CONVF_DEBUG_BOUNDS=1."""
    return _build.LIB_BOUNDS if _bounds_build() else _build.LIB


def load_library(build_if_missing: bool = False):
    """Load the CUDA library (building it first only when asked)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if build_if_missing:
        _build.build(debug_bounds=_bounds_build())
    if not os.path.exists(path):
        raise ImportError(f"{os.path.basename(path)} is not built ({path}); run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER
    dptr = P(ConvDesc)
    vp = ctypes.c_void_p
    lib.conv_fused_output_shape.argtypes = [dptr, P(ctypes.c_int)]
    lib.conv_fused_resolve_pads.argtypes = [dptr, P(ctypes.c_int)]
    lib.conv_bn_scale_shift.argtypes = [ctypes.c_int] + [P(ctypes.c_float)] * 4 + [ctypes.c_float] + \
        [P(ctypes.c_float)] * 2
    lib.conv_fused_plan.argtypes = [dptr, ctypes.c_int, P(ctypes.c_int), P(ctypes.c_int), P(ctypes.c_int),
                                    P(ctypes.c_int)]
    lib.conv_fused_pack_weights.argtypes = [dptr, ctypes.c_int, vp, vp, ctypes.c_size_t]
    lib.conv_fused_create.argtypes = [dptr, vp, vp, vp, vp, vp, vp, ctypes.c_int32, P(vp)]
    lib.conv_fused_create_qlinear.argtypes = [dptr, vp, vp, P(QParams), P(vp)]
    lib.conv_fused_create_preact.argtypes = [dptr, vp, vp, vp, vp, vp, vp, ctypes.c_int, P(vp)]
    lib.conv_fused_create_mbv2_block.argtypes = [P(BlockDesc)] + [vp] * 9 + [P(vp)]
    lib.conv_fused_run.argtypes = [vp, vp, vp, vp]
    lib.conv_fused_run_residual.argtypes = [vp, vp, vp, vp, vp]
    lib.conv_fused_status.argtypes = [vp]
    lib.conv_fused_clear_status.argtypes = [vp]
    lib.conv_fused_destroy.argtypes = [vp]
    lib.conv_fused_destroy.restype = None
    lib.conv_fused_variant.argtypes = [vp]
    lib.conv_fused_describe.argtypes = [vp, ctypes.c_char_p, ctypes.c_size_t]
    lib.conv_fused_last_error.argtypes = []
    lib.conv_fused_last_error.restype = ctypes.c_char_p
    lib.conv_fused_watchdog_selftest.argtypes = [vp, ctypes.c_longlong, vp]
    lib.conv_fused_run_noalloc.argtypes = [dptr, vp, vp, vp, vp, vp, vp, vp]
    lib.conv_fused_measure_int8_mma_rate.argtypes = [vp, P(ctypes.c_double)]
    lib.conv_fused_debug_fail_alloc.argtypes = [ctypes.c_int]
    lib.conv_fused_debug_live_handles.argtypes = []
    lib.conv_fused_chain_create.argtypes = [P(ChainStep), ctypes.c_int, P(vp)]
    lib.conv_fused_chain_create_ex.argtypes = [P(ChainStep), ctypes.c_int, ctypes.c_int, P(vp)]
    lib.conv_fused_chain_run.argtypes = [vp, vp]
    lib.conv_fused_chain_status.argtypes = [vp]
    lib.conv_fused_chain_clear_status.argtypes = [vp]
    lib.conv_fused_chain_describe.argtypes = [vp, ctypes.c_char_p, ctypes.c_size_t]
    lib.conv_fused_chain_destroy.argtypes = [vp]
    lib.conv_fused_chain_destroy.restype = None
    lib.conv_fused_quantize_blocks.argtypes = [P(QuantArgs), vp]
    lib.conv_fused_quantize_rows.argtypes = [P(QuantRowsArgs), vp]
    lib.conv_fused_rms_norm_quantize.argtypes = [P(NormArgs), vp]
    lib.conv_fused_linear_create.argtypes = [P(LinearDesc), vp, vp, vp, P(vp)]
    lib.conv_fused_linear_run.argtypes = [vp, P(LinearArgs), vp]
    lib.conv_fused_linear_status.argtypes = [vp]
    lib.conv_fused_linear_clear_status.argtypes = [vp]
    lib.conv_fused_linear_describe.argtypes = [vp, ctypes.c_int, ctypes.c_char_p, ctypes.c_size_t]
    lib.conv_fused_linear_destroy.argtypes = [vp]
    lib.conv_fused_linear_destroy.restype = None
    for name in EXPORTED:
        if name not in ("conv_fused_destroy", "conv_fused_last_error", "conv_fused_chain_destroy",
                        "conv_fused_linear_destroy"):
            getattr(lib, name).restype = ctypes.c_int
    _LIB = lib
    return lib


def _check(status: int):
    if status != CONVF_OK:
        raise ConvFusedError(status, conv_fused_last_error())


def _addr(a) -> Optional[int]:
    """Host address of a numpy array / CPU tensor, device address of a CUDA tensor, or an int."""
    if a is None:
        return None
    if isinstance(a, int):
        return a
    if hasattr(a, "data_ptr"):
        return a.data_ptr()
    return a.ctypes.data


# --------------------------------------------------------------------------- C entry points

def conv_fused_last_error() -> str:
    return load_library().conv_fused_last_error().decode()


def conv_fused_output_shape(desc: ConvDesc):
    out = (ctypes.c_int * 4)()
    _check(load_library().conv_fused_output_shape(ctypes.byref(desc), out))
    return tuple(out)


def conv_fused_resolve_pads(desc: ConvDesc):
    out = (ctypes.c_int * 4)()
    _check(load_library().conv_fused_resolve_pads(ctypes.byref(desc), out))
    return tuple(out)


def conv_bn_scale_shift(gamma, beta, mean, var, eps: float = 1e-5):
    """Returns (scale, shift) as float32 numpy arrays."""
    import numpy as np
    arrs = [np.ascontiguousarray(np.asarray(a, dtype=np.float32)) for a in (gamma, beta, mean, var)]
    K = arrs[0].shape[0]
    scale = np.empty(K, np.float32)
    shift = np.empty(K, np.float32)
    fp = lambda a: a.ctypes.data_as(ctypes.POINTER(ctypes.c_float))
    _check(load_library().conv_bn_scale_shift(K, *[fp(a) for a in arrs], float(eps), fp(scale), fp(shift)))
    return scale, shift


def conv_fused_plan(desc: ConvDesc, num_sms: int = 152, with_pair: bool = False):
    """(variant, tile_n, ktot) or, with with_pair, (variant, tile_n, ktot, cta_pair)."""
    v, bn, kt, pr = ctypes.c_int(), ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check(load_library().conv_fused_plan(ctypes.byref(desc), num_sms, ctypes.byref(v), ctypes.byref(bn),
                                          ctypes.byref(kt), ctypes.byref(pr)))
    return (v.value, bn.value, kt.value, pr.value) if with_pair else (v.value, bn.value, kt.value)


def conv_fused_pack_weights(desc: ConvDesc, variant: int, W_bits, out):
    _check(load_library().conv_fused_pack_weights(ctypes.byref(desc), variant, _addr(W_bits), _addr(out),
                                                  out.size if hasattr(out, "size") and not callable(out.size)
                                                  else out.numel()))


def conv_fused_create(desc: ConvDesc, W, bias=None, bn_scale=None, bn_shift=None, requant_mult=None,
                      requant_shift=None, out_zero_point: int = 0) -> int:
    """Host arrays (numpy or CPU tensors, contiguous) in, handle (int) out."""
    h = ctypes.c_void_p()
    _check(load_library().conv_fused_create(ctypes.byref(desc), _addr(W), _addr(bias), _addr(bn_scale),
                                            _addr(bn_shift), _addr(requant_mult), _addr(requant_shift),
                                            int(out_zero_point), ctypes.byref(h)))
    return h.value


def conv_fused_create_preact(desc: ConvDesc, W, bias=None, bn_scale=None, bn_shift=None, pre_scale=None,
                             pre_shift=None, pre_act: int = CONVF_ACT_RELU) -> int:
    """Handle with a pre-activation prologue: the conv reads clamp(pre_scale*x + pre_shift)."""
    h = ctypes.c_void_p()
    _check(load_library().conv_fused_create_preact(ctypes.byref(desc), _addr(W), _addr(bias), _addr(bn_scale),
                                                   _addr(bn_shift), _addr(pre_scale), _addr(pre_shift),
                                                   int(pre_act), ctypes.byref(h)))
    return h.value


def conv_fused_create_mbv2_block(d: BlockDesc, w_expand, e_scale, e_shift, w_dw, d_scale, d_shift, w_project,
                                 p_scale, p_shift) -> int:
    """Fused MobileNetV2 block handle (host arrays: bf16 bits for weights, float32 affines)."""
    h = ctypes.c_void_p()
    _check(load_library().conv_fused_create_mbv2_block(ctypes.byref(d), _addr(w_expand), _addr(e_scale),
                                                       _addr(e_shift), _addr(w_dw), _addr(d_scale), _addr(d_shift),
                                                       _addr(w_project), _addr(p_scale), _addr(p_shift),
                                                       ctypes.byref(h)))
    return h.value


def conv_fused_create_qlinear(desc: ConvDesc, W, bias, q: QParams) -> int:
    """QLinearConv handle: desc.dtype == CONVF_Q8, W host int8/uint8 [K][C/group][R][S], bias host
    int32[K] or None, q the scales and zero points (its w arrays host pointers)."""
    h = ctypes.c_void_p()
    _check(load_library().conv_fused_create_qlinear(ctypes.byref(desc), _addr(W), _addr(bias), ctypes.byref(q),
                                                    ctypes.byref(h)))
    return h.value


def conv_fused_run(handle: int, x, y, stream=None):
    """x, y: device pointers (ints) or CUDA tensors; stream: cudaStream_t int, torch stream or None."""
    s = stream
    if s is not None and hasattr(s, "cuda_stream"):
        s = s.cuda_stream
    _check(load_library().conv_fused_run(handle, _addr(x), _addr(y), s))


def conv_fused_run_residual(handle: int, x, r, y, stream=None):
    """conv_fused_run for residual handles: y = act(scale * conv(x) + bias' + r)."""
    s = stream
    if s is not None and hasattr(s, "cuda_stream"):
        s = s.cuda_stream
    _check(load_library().conv_fused_run_residual(handle, _addr(x), _addr(r), _addr(y), s))


def conv_fused_status(handle: int) -> int:
    return load_library().conv_fused_status(handle)


def conv_fused_clear_status(handle: int):
    _check(load_library().conv_fused_clear_status(handle))


def conv_fused_destroy(handle: int):
    load_library().conv_fused_destroy(handle)


def conv_fused_variant(handle: int) -> int:
    v = load_library().conv_fused_variant(handle)
    if v < 0:
        _check(v)
    return v


def conv_fused_describe(handle: int) -> str:
    buf = ctypes.create_string_buffer(512)
    _check(load_library().conv_fused_describe(handle, buf, 512))
    return buf.value.decode()


def conv_fused_watchdog_selftest(status_dev, budget_cycles: int, stream=None):
    s = stream.cuda_stream if stream is not None and hasattr(stream, "cuda_stream") else stream
    _check(load_library().conv_fused_watchdog_selftest(_addr(status_dev), int(budget_cycles), s))


def conv_fused_debug_fail_alloc(n: int):
    """Test hook: the n-th allocation the create calls make from now on fails (0 disarms)."""
    _check(load_library().conv_fused_debug_fail_alloc(int(n)))


def conv_fused_debug_live_handles() -> int:
    """Number of handles created and not yet destroyed."""
    return int(load_library().conv_fused_debug_live_handles())


def conv_fused_measure_int8_mma_rate(stream=None) -> float:
    """TOP/s of back-to-back int8 mma.sync on this GPU (register operands)."""
    s = stream.cuda_stream if stream is not None and hasattr(stream, "cuda_stream") else stream
    out = ctypes.c_double()
    _check(load_library().conv_fused_measure_int8_mma_rate(s, ctypes.byref(out)))
    return out.value


def conv_fused_run_noalloc(desc: ConvDesc, x, w_packed, scale, bias, y, status=None, stream=None):
    """Allocation-free run: every argument a device pointer (int) or CUDA tensor."""
    s = stream.cuda_stream if stream is not None and hasattr(stream, "cuda_stream") else stream
    _check(load_library().conv_fused_run_noalloc(ctypes.byref(desc), _addr(x), _addr(w_packed), _addr(scale),
                                                 _addr(bias), _addr(y), _addr(status), s))


def conv_fused_chain_create(steps, cta_pairs: int = 0) -> int:
    """steps: sequence of (handle, x, r or None, y) with device pointers (ints) or CUDA tensors;
    cta_pairs: 0 automatic, 1 single CTAs, 2 CTA pairs (conv_fused_chain_create_ex)."""
    arr = (ChainStep * len(steps))()
    for i, (h, x, r, y) in enumerate(steps):
        arr[i] = ChainStep(h, _addr(x), _addr(r), _addr(y))
    c = ctypes.c_void_p()
    _check(load_library().conv_fused_chain_create_ex(arr, len(steps), cta_pairs, ctypes.byref(c)))
    return c.value


def conv_fused_chain_run(chain: int, stream=None):
    s = stream
    if s is not None and hasattr(s, "cuda_stream"):
        s = s.cuda_stream
    _check(load_library().conv_fused_chain_run(chain, s))


def conv_fused_chain_status(chain: int) -> int:
    return load_library().conv_fused_chain_status(chain)


def conv_fused_chain_clear_status(chain: int):
    _check(load_library().conv_fused_chain_clear_status(chain))


def conv_fused_chain_describe(chain: int) -> str:
    buf = ctypes.create_string_buffer(65536)
    _check(load_library().conv_fused_chain_describe(chain, buf, 65536))
    return buf.value.decode()


def conv_fused_chain_destroy(chain: int):
    load_library().conv_fused_chain_destroy(chain)


def conv_fused_quantize_blocks(args: QuantArgs, stream=None):
    s = stream.cuda_stream if stream is not None and hasattr(stream, "cuda_stream") else stream
    _check(load_library().conv_fused_quantize_blocks(ctypes.byref(args), s))


def conv_fused_quantize_rows(args: QuantRowsArgs, stream=None):
    s = stream.cuda_stream if stream is not None and hasattr(stream, "cuda_stream") else stream
    _check(load_library().conv_fused_quantize_rows(ctypes.byref(args), s))


def conv_fused_rms_norm_quantize(args: NormArgs, stream=None):
    s = stream.cuda_stream if stream is not None and hasattr(stream, "cuda_stream") else stream
    _check(load_library().conv_fused_rms_norm_quantize(ctypes.byref(args), s))


def conv_fused_linear_create(desc: LinearDesc, W, w_scale=None, bias=None) -> int:
    """Device pointers (ints) or CUDA tensors, which must outlive the layer; returns its handle."""
    out = ctypes.c_void_p()
    _check(load_library().conv_fused_linear_create(ctypes.byref(desc), _addr(W), _addr(w_scale), _addr(bias),
                                                   ctypes.byref(out)))
    return out.value


def conv_fused_linear_run(layer: int, args: LinearArgs, stream=None):
    s = stream.cuda_stream if stream is not None and hasattr(stream, "cuda_stream") else stream
    _check(load_library().conv_fused_linear_run(layer, ctypes.byref(args), s))


def conv_fused_linear_status(layer: int) -> int:
    return load_library().conv_fused_linear_status(layer)


def conv_fused_linear_clear_status(layer: int):
    _check(load_library().conv_fused_linear_clear_status(layer))


def conv_fused_linear_describe(layer: int, rows: int) -> str:
    buf = ctypes.create_string_buffer(512)
    _check(load_library().conv_fused_linear_describe(layer, int(rows), buf, 512))
    return buf.value.decode()


def conv_fused_linear_destroy(layer: int):
    load_library().conv_fused_linear_destroy(layer)


# --------------------------------------------------------------------------- torch convenience

class FusedConv:
    """One prepared conv node over torch tensors.

    ``w`` (bf16 KCRS or int8), ``bias`` and the BN affine are CPU tensors; they are copied
    to the device once here.  Calling the object runs the kernel on the current torch stream
    with ``x`` a CUDA tensor in channels-last storage (logical NCHW) and returns y (fp32 or
    int8, channels-last).
    """

    def __init__(self, N, C, H, W, K, R, S, w, bias=None, bn_scale=None, bn_shift=None, stride=(1, 1),
                 pads=(0, 0, 0, 0), dilation=(1, 1), group=1, act=CONVF_ACT_NONE, clip=(0.0, 6.0),
                 auto_pad="NOTSET", variant=CONVF_VARIANT_AUTO, requant_mult=None, requant_shift=None,
                 out_zero_point=0, tile_n=0, cta_pair=0, stream_k=0, kblocks_per_step=0,
                 out_bf16=False, residual=False, pre_scale=None, pre_shift=None, pre_act=None):
        import torch
        s8 = w.dtype == torch.int8
        self.desc = make_desc(N, C, H, W, K, R, S, stride, pads, dilation, group,
                              CONVF_S8 if s8 else CONVF_BF16, act, clip, auto_pad, variant, tile_n=tile_n,
                              cta_pair=cta_pair, stream_k=stream_k, kblocks_per_step=kblocks_per_step,
                              out_dtype=CONVF_OUT_BF16 if out_bf16 else CONVF_OUT_F32, residual=int(bool(residual)))
        self.out_bf16 = bool(out_bf16)
        self.residual = bool(residual)
        wc = w.contiguous().cpu()
        wbits = wc if s8 else wc.view(torch.int16)
        keep = [wbits]

        def host(t, dt):
            if t is None:
                return None
            t = torch.as_tensor(t).to(dt).contiguous().cpu()
            keep.append(t)
            return t

        if pre_act is not None:
            # pre-activation prologue (bf16 convs): the conv reads clamp(pre_scale*x + pre_shift)
            self.handle = conv_fused_create_preact(self.desc, wbits, host(bias, torch.float32),
                                                   host(bn_scale, torch.float32), host(bn_shift, torch.float32),
                                                   host(pre_scale, torch.float32), host(pre_shift, torch.float32),
                                                   pre_act)
        else:
            self.handle = conv_fused_create(self.desc, wbits, host(bias, torch.int32 if s8 else torch.float32),
                                            host(bn_scale, torch.float32), host(bn_shift, torch.float32),
                                            host(requant_mult, torch.int32), host(requant_shift, torch.int32),
                                            out_zero_point)
        self.out_shape = conv_fused_output_shape(self.desc)
        self.s8 = s8

    @property
    def variant(self) -> int:
        return conv_fused_variant(self.handle)

    def describe(self) -> str:
        return conv_fused_describe(self.handle)

    def new_output(self):
        import torch
        N, K, Ho, Wo = self.out_shape
        dt = torch.int8 if self.s8 else (torch.bfloat16 if self.out_bf16 else torch.float32)
        return torch.empty((N, Ho, Wo, K), dtype=dt, device="cuda").permute(0, 3, 1, 2)

    def __call__(self, x, y=None, stream=None, r=None):
        """Runs on the current torch stream; ``r`` is the residual (y's shape, dtype and
        channels-last storage) for handles made with ``residual=True``."""
        import torch
        if not x.is_cuda:
            raise ValueError("x must be a CUDA tensor")
        if not x.is_contiguous(memory_format=torch.channels_last) and x.numel() > 0:
            raise ValueError("x must use channels-last storage")
        if y is None:
            y = self.new_output()
        s = stream if stream is not None else torch.cuda.current_stream().cuda_stream
        if self.residual:
            if r is None:
                raise ValueError("this conv adds a residual: pass r")
            conv_fused_run_residual(self.handle, x.data_ptr(), r.data_ptr(), y.data_ptr(), s)
        else:
            conv_fused_run(self.handle, x.data_ptr(), y.data_ptr(), s)
        return y

    def status(self) -> int:
        return conv_fused_status(self.handle)

    def close(self):
        if self.handle:
            conv_fused_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class QLinearConv(FusedConv):
    """ONNX QLinearConv over torch tensors: ``w`` int8 or uint8 (KCRS, CPU), ``bias`` int32[K] or
    None, per-channel ``w_scale`` / ``w_zero_point`` (or scalars).  Calling it with an 8-bit
    channels-last CUDA tensor x returns the 8-bit y (uint8 or int8 per ``y_signed``)."""

    def __init__(self, N, C, H, W, K, R, S, w, bias=None, x_scale=1.0, x_zero_point=0, w_scale=1.0,
                 w_zero_point=0, y_scale=1.0, y_zero_point=0, x_signed=False, y_signed=False, relu=False,
                 stride=(1, 1), pads=(0, 0, 0, 0), dilation=(1, 1), group=1, auto_pad="NOTSET",
                 variant=CONVF_VARIANT_AUTO, tile_n=0, kblocks_per_step=0):
        import numpy as np
        import torch
        self.desc = make_desc(N, C, H, W, K, R, S, stride, pads, dilation, group, CONVF_Q8, CONVF_ACT_NONE,
                              (0.0, 6.0), auto_pad, variant, tile_n=tile_n, kblocks_per_step=kblocks_per_step)
        self.out_bf16 = False
        self.residual = False
        self.s8 = True
        self.y_signed = bool(y_signed)
        wc = w.contiguous().cpu()
        ws = np.ascontiguousarray(np.broadcast_to(np.asarray(w_scale, dtype=np.float32).reshape(-1), (K,)))
        wz = np.ascontiguousarray(np.broadcast_to(np.asarray(w_zero_point, dtype=np.int32).reshape(-1), (K,)))
        b = None if bias is None else torch.as_tensor(bias).to(torch.int32).contiguous().cpu()
        self._keep = [wc, ws, wz, b]
        q = QParams()
        q.x_signed, q.w_signed, q.y_signed = int(bool(x_signed)), int(wc.dtype == torch.int8), int(bool(y_signed))
        q.x_zero_point, q.y_zero_point = int(x_zero_point), int(y_zero_point)
        q.x_scale, q.y_scale = float(x_scale), float(y_scale)
        q.w_zero_point, q.w_scale = wz.ctypes.data, ws.ctypes.data
        q.relu = int(bool(relu))
        self.handle = conv_fused_create_qlinear(self.desc, wc, b, q)
        self.out_shape = conv_fused_output_shape(self.desc)

    def new_output(self):
        import torch
        N, K, Ho, Wo = self.out_shape
        dt = torch.int8 if self.y_signed else torch.uint8
        return torch.empty((N, Ho, Wo, K), dtype=dt, device="cuda").permute(0, 3, 1, 2)


class InvertedResidualBlock(FusedConv):
    """A MobileNetV2 block as one fused kernel over torch tensors: ``w_expand`` (bf16 [Ch][Cin][1][1]
    or None), ``w_dw`` (bf16 [Ch][1][3][3]), ``w_project`` (bf16 [Cout][Ch][1][1]) and each stage's
    folded BN affine (scale, shift) as float arrays.  Calling it with x (bf16, channels-last) returns
    y (fp32, channels-last)."""

    def __init__(self, N, Cin, H, W, Ch, Cout, stride, w_expand, e_affine, w_dw, d_affine, w_project, p_affine,
                 residual=False):
        import numpy as np
        import torch
        d = BlockDesc()
        d.N, d.H, d.W, d.Cin, d.Ch, d.Cout, d.stride = N, H, W, Cin, Ch, Cout, stride
        d.expand = int(w_expand is not None)
        d.residual = int(bool(residual))
        self.block = d

        def bits(t):
            return None if t is None else t.contiguous().cpu().view(torch.int16)

        def f32(a):
            return None if a is None else np.ascontiguousarray(np.asarray(a, dtype=np.float32))

        es, et = (f32(e_affine[0]), f32(e_affine[1])) if e_affine is not None else (None, None)
        keep = [bits(w_expand), es, et, bits(w_dw), f32(d_affine[0]), f32(d_affine[1]), bits(w_project),
                f32(p_affine[0]), f32(p_affine[1])]
        self._keep = keep
        self.handle = conv_fused_create_mbv2_block(d, *keep)
        Ho = (H + 2 - 3) // stride + 1
        Wo = (W + 2 - 3) // stride + 1
        self.out_shape = (N, Cout, Ho, Wo)
        self.s8 = False
        self.out_bf16 = False
        self.residual = False


class ConvChain:
    """A sequence of FusedConv runs as one persistent launch (conv_fused_chain_*).

    ``steps`` is a sequence of ``(conv, x, y)`` or ``(conv, x, y, r)`` with ``conv`` a FusedConv
    (1x1-GEMM or im2col implicit-GEMM variant) and ``x``, ``y``, ``r`` CUDA tensors in
    channels-last storage.  A step whose ``x`` (or ``r``) is an earlier step's ``y`` reads that
    output.  The tensors and the convs must outlive the chain; calling it runs every step on the
    current torch stream."""

    def __init__(self, steps, cta_pairs: int = 0):
        self._keep = [tuple(st) for st in steps]
        items = []
        for st in self._keep:
            conv, x, y = st[0], st[1], st[2]
            r = st[3] if len(st) > 3 else None
            items.append((conv.handle, x.data_ptr(), None if r is None else r.data_ptr(), y.data_ptr()))
        self.handle = conv_fused_chain_create(items, cta_pairs)

    def describe(self) -> str:
        return conv_fused_chain_describe(self.handle)

    def __call__(self, stream=None):
        import torch
        s = stream if stream is not None else torch.cuda.current_stream().cuda_stream
        conv_fused_chain_run(self.handle, s)

    def status(self) -> int:
        return conv_fused_chain_status(self.handle)

    def clear_status(self):
        conv_fused_chain_clear_status(self.handle)

    def close(self):
        if self.handle:
            conv_fused_chain_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class _Torch:
    """Names of torch that every call uses (the package imports torch only where it is used)."""
    ready = False

    @classmethod
    def bind(cls):
        import torch
        cls.bf16, cls.f32, cls.e4m3, cls.i32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32
        cls.i8 = torch.int8
        cls.empty, cls.empty_strided, cls.cuda = torch.empty, torch.empty_strided, torch.cuda
        # the public call builds a Stream object (2 us of a 10 us call)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        cls.stream = raw if raw is not None else lambda index: torch.cuda.current_stream(index).cuda_stream
        raw = getattr(torch._C, "_cuda_getDevice", None)
        cls.current_device = raw if raw is not None else torch.cuda.current_device
        cls.quantize = load_library().conv_fused_quantize_blocks
        cls.quantize_rows = load_library().conv_fused_quantize_rows
        cls.norm = load_library().conv_fused_rms_norm_quantize
        cls.run = load_library().conv_fused_linear_run
        cls.ready = True

    @staticmethod
    def refuse_apart(device, **tensors):
        """Refuses tensors of another device than `device`: a kernel would use their addresses as its own."""
        for name, t in tensors.items():
            if t is not None and t.get_device() != device:
                raise ValueError(f"{name} is on device {t.get_device()}, the other operands on device {device}")

    @classmethod
    def on(cls, stream, device):
        """Context in which torch allocates for `stream` (a torch stream or a cudaStream_t)."""
        if not hasattr(stream, "cuda_stream"):
            # (torch takes an external stream 0 for a new one)
            stream = cls.cuda.ExternalStream(stream, device) if stream else cls.cuda.default_stream(device)
        return cls.cuda.stream(stream)


def _rows_2d(t, name):
    """(rows, cols, row stride) of a CUDA tensor [rows][cols] whose columns are adjacent."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    r, c = t.shape
    ld, adjacent = t.stride()
    if adjacent != 1 and c > 1:
        raise ValueError(f"{name}'s columns must be adjacent (stride 1)")
    return r, c, (ld if r > 1 else (c + 31) // 32 * 32)   # one row has no stride of its own: an aligned one


def quantize_blocks(x, index=None, gated=False, block_rows=1, q=None, scale=None, stream=None):
    """(q, scale): the rows of ``x`` (CUDA, bf16 or fp32, [rows][cols], any row stride) as e4m3 values
    and a float scale per row and 128 columns (``block_rows=1``), or per 128 x 128 block
    (``block_rows=128``, as a layer's weights have them); x is about q * scale.

    ``index`` (int32, CUDA) takes the rows x[index] instead (an entry outside x gives a row of zeros);
    ``gated=True`` takes x as [rows][2*cols] and quantises g / (1 + exp(-g)) * u of its halves g and
    u.  Rows of q lie a multiple of 16 bytes apart, as the layers read them; ``q`` and ``scale`` may
    be given; all tensors are on the current device.  Runs on the current torch stream, or on ``stream``
    (a torch stream or a cudaStream_t)."""
    T = _Torch
    if not T.ready:
        T.bind()
    if stream is not None and x.is_cuda and (q is None or scale is None):
        # outputs belong to the stream that writes them
        with T.on(stream, x.device):
            return quantize_blocks(x, index, gated, block_rows, q, scale)
    rows, cols, ldx = _rows_2d(x, "x")
    on = x.get_device()
    if on != T.current_device():
        raise ValueError(f"x is on device {on}, the current device is {T.current_device()}")
    if (q is not None and q.get_device() != on) or (scale is not None and scale.get_device() != on) \
            or (index is not None and index.get_device() != on):
        T.refuse_apart(on, index=index, q=q, scale=scale)
    xr = rows
    kind = x.dtype
    if kind is T.bf16:
        kind = CONVF_OUT_BF16
    elif kind is T.f32:
        kind = CONVF_OUT_F32
    else:
        raise ValueError("x must be bf16 or fp32")
    if gated:
        if cols % 2:
            raise ValueError("gated rows have an even number of columns")
        cols //= 2
    where = None
    if index is not None:
        if not index.is_cuda or index.dtype is not T.i32 or index.dim() != 1 or not index.is_contiguous():
            raise ValueError("index must be a contiguous int32 CUDA vector")
        rows, where = index.shape[0], index.data_ptr()
    nblk = (cols + 127) // 128
    srows = rows if block_rows == 1 else (rows + 127) // 128
    device = x.device
    if q is None:
        ldq = (cols + 15) // 16 * 16
        q = T.empty((rows, cols), dtype=T.e4m3, device=device) if ldq == cols else \
            T.empty_strided((rows, cols), (ldq, 1), dtype=T.e4m3, device=device)
    else:
        qr, qc, ldq = _rows_2d(q, "q")
        if q.dtype is not T.e4m3 or qr != rows or qc != cols:
            raise ValueError(f"q must be float8_e4m3fn of shape ({rows}, {cols})")
    if scale is None:
        lds = nblk
        scale = T.empty((srows, nblk), dtype=T.f32, device=device)
    else:
        sr, sc, lds = _rows_2d(scale, "scale")
        if scale.dtype is not T.f32 or sr != srows or sc != nblk:
            raise ValueError(f"scale must be float32 of shape ({srows}, {nblk})")
    if stream is None:
        stream = T.stream(on)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    st = T.quantize(ctypes.byref(QuantArgs(rows, cols, x.data_ptr(), kind, xr, ldx, where, 1 if gated else 0, block_rows,
                                           q.data_ptr(), ldq, scale.data_ptr(), lds)), stream)
    if st != CONVF_OK:
        _check(st)
    return q, scale


def _kind(t, name):
    """convf_out_dtype of a tensor."""
    if t.dtype is _Torch.bf16:
        return CONVF_OUT_BF16
    if t.dtype is _Torch.f32:
        return CONVF_OUT_F32
    raise ValueError(f"{name} must be bf16 or fp32")


def _bytes_like(q, rows, cols, dtype, device):
    """(tensor, row stride) of the 8-bit values [rows][cols]: `q` if given, or new rows a multiple of 16 bytes apart."""
    if q is None:
        ldq = (cols + 15) // 16 * 16
        return (_Torch.empty((rows, cols), dtype=dtype, device=device) if ldq == cols else
                _Torch.empty_strided((rows, cols), (ldq, 1), dtype=dtype, device=device)), ldq
    qr, qc, ldq = _rows_2d(q, "q")
    if q.dtype is not dtype or qr != rows or qc != cols:
        raise ValueError(f"q must be {dtype} of shape ({rows}, {cols})")
    return q, ldq


def _row_scales(scale, rows, device):
    """A scale per row: `scale` if given, or a new vector."""
    if scale is None:
        return _Torch.empty((rows,), dtype=_Torch.f32, device=device)
    if not scale.is_cuda or scale.dtype is not _Torch.f32 or scale.shape != (rows,) or not scale.is_contiguous():
        raise ValueError(f"scale must be a contiguous CUDA float32 vector of {rows}")
    return scale


def quantize_rows(x, index=None, gated=False, q=None, scale=None, stream=None):
    """(q, scale): the rows of ``x`` (CUDA, bf16 or fp32, [rows][cols], any row stride) as int8 values in
    -127 .. 127 and a float scale per row; x is about q * scale[:, None].  A layer's weights [N][K] are
    quantised by the same call: a scale per output channel.

    ``index``, ``gated``, ``q`` and ``stream`` as for quantize_blocks; ``scale`` [rows] may be given."""
    T = _Torch
    if not T.ready:
        T.bind()
    if stream is not None and x.is_cuda and (q is None or scale is None):
        with T.on(stream, x.device):   # outputs belong to the stream that writes them
            return quantize_rows(x, index, gated, q, scale)
    rows, cols, ldx = _rows_2d(x, "x")
    on = x.get_device()
    if on != T.current_device():
        raise ValueError(f"x is on device {on}, the current device is {T.current_device()}")
    if (q is not None and q.get_device() != on) or (scale is not None and scale.get_device() != on) \
            or (index is not None and index.get_device() != on):
        T.refuse_apart(on, index=index, q=q, scale=scale)
    xr, kind = rows, _kind(x, "x")
    if gated:
        if cols % 2:
            raise ValueError("gated rows have an even number of columns")
        cols //= 2
    where = None
    if index is not None:
        if not index.is_cuda or index.dtype is not T.i32 or index.dim() != 1 or not index.is_contiguous():
            raise ValueError("index must be a contiguous int32 CUDA vector")
        rows, where = index.shape[0], index.data_ptr()
    device = x.device
    q, ldq = _bytes_like(q, rows, cols, T.i8, device)
    scale = _row_scales(scale, rows, device)
    if stream is None:
        stream = T.stream(on)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    st = T.quantize_rows(ctypes.byref(QuantRowsArgs(rows, cols, x.data_ptr(), kind, xr, ldx, where, 1 if gated else 0,
                                                    q.data_ptr(), ldq, scale.data_ptr())), stream)
    if st != CONVF_OK:
        _check(st)
    return q, scale


def rms_norm_quantize(x, weight=None, eps=1e-6, residual=None, int8=False, q=None, scale=None, h=None, stream=None):
    """(q, scale), or (q, scale, h) with a ``residual``: with h = x + residual (x without one), the rows
    h / sqrt(mean(h^2) + eps) * weight as e4m3 values with a scale per row and 128 columns, or with
    ``int8=True`` as int8 values with a scale per row; h, in the residual's type, is the sum for the next
    residual.

    ``x`` and ``residual``: CUDA, bf16 or fp32 (each its own), [rows][cols], any row stride; ``weight``
    [cols] bf16 or fp32, or None.  ``q``, ``scale`` and ``h`` may be given; ``h`` may be the residual itself
    (or x, of the residual's type), to be overwritten.  All tensors are on the current device.  Runs on the
    current torch stream, or on ``stream``."""
    T = _Torch
    if not T.ready:
        T.bind()
    if stream is not None and x.is_cuda and (q is None or scale is None or (residual is not None and h is None)):
        with T.on(stream, x.device):   # outputs belong to the stream that writes them
            return rms_norm_quantize(x, weight, eps, residual, int8, q, scale, h)
    rows, cols, ldx = _rows_2d(x, "x")
    on = x.get_device()
    if on != T.current_device():
        raise ValueError(f"x is on device {on}, the current device is {T.current_device()}")
    if (weight is not None and weight.get_device() != on) or (residual is not None and residual.get_device() != on) \
            or (q is not None and q.get_device() != on) or (scale is not None and scale.get_device() != on) \
            or (h is not None and h.get_device() != on):
        T.refuse_apart(on, weight=weight, residual=residual, q=q, scale=scale, h=h)
    device, kind = x.device, _kind(x, "x")
    wp = wk = rp = rk = hp = ldr = ldh = 0
    if weight is not None:
        if not weight.is_cuda or weight.shape != (cols,) or not weight.is_contiguous():
            raise ValueError(f"weight must be a contiguous CUDA vector of {cols}")
        wp, wk = weight.data_ptr(), _kind(weight, "weight")
    if residual is not None:
        rr, rc, ldr = _rows_2d(residual, "residual")
        if rr != rows or rc != cols:
            raise ValueError(f"residual must be of shape ({rows}, {cols})")
        rp, rk = residual.data_ptr(), _kind(residual, "residual")
        if h is None:
            h, ldh = T.empty((rows, cols), dtype=residual.dtype, device=device), cols
        elif h is residual:
            ldh = ldr
        else:
            hr, hc, ldh = _rows_2d(h, "h")
            if h.dtype is not residual.dtype or hr != rows or hc != cols:
                raise ValueError(f"h must be {residual.dtype} of shape ({rows}, {cols})")
        hp = h.data_ptr()
    elif h is not None:
        raise ValueError("h goes with a residual (without one it is x)")
    if int8:
        q, ldq = _bytes_like(q, rows, cols, T.i8, device)
        scale, lds = _row_scales(scale, rows, device), 1
    else:
        q, ldq = _bytes_like(q, rows, cols, T.e4m3, device)
        lds = nblk = (cols + 127) // 128
        if scale is None:
            scale = T.empty((rows, nblk), dtype=T.f32, device=device)
        else:
            sr, sc, lds = _rows_2d(scale, "scale")
            if scale.dtype is not T.f32 or sr != rows or sc != nblk:
                raise ValueError(f"scale must be float32 of shape ({rows}, {nblk})")
    if stream is None:
        stream = T.stream(on)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    st = T.norm(ctypes.byref(NormArgs(rows, cols, x.data_ptr(), kind, ldx, rp, rk, ldr, hp, ldh, wp, wk, eps,
                                      CONVF_LINEAR_INT8 if int8 else CONVF_LINEAR_E4M3, q.data_ptr(), ldq,
                                      scale.data_ptr(), lds)), stream)
    if st != CONVF_OK:
        _check(st)
    return (q, scale) if residual is None else (q, scale, h)


class ExpertLinear:
    """Linear layers, one per expert, over rows sorted by expert: rows offsets[e] up to offsets[e+1]
    of x times ``w[e]``.

    ``w``: CUDA [experts][N][K], bf16, float8_e4m3fn or int8, read in place (rows and experts a multiple
    of 16 bytes apart); ``w_scale`` fp32 [experts][ceil(N/128)][ceil(K/128)] (e4m3) or [experts][N]
    (int8: K at most 131071); ``bias`` fp32 [experts][N] or None (both in place too where they are contiguous); all on the current device; ``act`` and ``clip`` as for a conv; y is fp32, or bf16 with ``out_bf16``.
    Calling it runs on the current torch stream."""

    def __init__(self, w, w_scale=None, bias=None, act=CONVF_ACT_NONE, clip=(0.0, 6.0), out_bf16=False):
        import torch
        if not _Torch.ready:
            _Torch.bind()
        if not w.is_cuda or w.dim() != 3:
            raise ValueError("w must be a CUDA tensor [experts][N][K]")
        if w.dtype not in (torch.bfloat16, torch.float8_e4m3fn, torch.int8):
            raise ValueError("w must be bf16, float8_e4m3fn or int8")
        E, N, K = w.shape
        if K > 1 and w.stride(2) != 1:
            raise ValueError("w's columns must be adjacent (stride 1)")
        self.e4m3, self.int8 = w.dtype == torch.float8_e4m3fn, w.dtype == torch.int8
        if (self.e4m3 or self.int8) != (w_scale is not None):
            raise ValueError("w_scale goes with float8_e4m3fn or int8 weights, and with those only")
        blocks = (E, -(-N // 128), -(-K // 128))
        for name, t, shape in (("w_scale", w_scale, (E, N) if self.int8 else blocks), ("bias", bias, (E, N))):
            if t is not None and (not t.is_cuda or t.dtype != torch.float32 or tuple(t.shape) != shape):
                raise ValueError(f"{name} must be a CUDA fp32 tensor of shape {shape}")
        self.device = w.get_device()
        if self.device != _Torch.current_device():
            raise ValueError(f"w is on device {self.device}, the current device is {_Torch.current_device()}")
        _Torch.refuse_apart(self.device, w_scale=w_scale, bias=bias)
        w_scale = None if w_scale is None else w_scale.contiguous()
        bias = None if bias is None else bias.contiguous()
        self._keep = (w, w_scale, bias)   # the layer reads them in place
        self.experts, self.N, self.K, self.kblk, self.dtype = E, N, K, blocks[2], w.dtype
        self.out_dtype = torch.bfloat16 if out_bf16 else torch.float32
        d = LinearDesc(N, K, E, CONVF_LINEAR_E4M3 if self.e4m3 else CONVF_LINEAR_INT8 if self.int8 else CONVF_LINEAR_BF16,
                       w.stride(1) if N > 1 else -(-K // 16) * 16, w.stride(0), act, float(clip[0]), float(clip[1]),
                       CONVF_OUT_BF16 if out_bf16 else CONVF_OUT_F32)
        self.handle = conv_fused_linear_create(d, w, w_scale, bias)

    def _run(self, x, offsets, x_scale, y, stream):
        if stream is not None and x.is_cuda and y is None:
            with _Torch.on(stream, x.device):   # y belongs to the stream that writes it
                return self._run(x, offsets, x_scale, None, None)
        rows, K, ldx = _rows_2d(x, "x")
        if K != self.K:
            raise ValueError(f"x must have {self.K} columns")
        if x.dtype is not self.dtype:
            raise ValueError(f"x must be {self.dtype}")
        if x.get_device() != self.device:   # (the library compares it with the current one)
            raise ValueError(f"x is on device {x.get_device()}, the layer on device {self.device}")
        if (y is not None and y.get_device() != self.device) \
                or (x_scale is not None and x_scale.get_device() != self.device):
            _Torch.refuse_apart(self.device, x_scale=x_scale, y=y)
        xs = xs_row = xs_blk = 0
        if self.e4m3:
            if x_scale is None or not x_scale.is_cuda or x_scale.dtype is not _Torch.f32 \
                    or x_scale.shape != (rows, self.kblk):
                raise ValueError(f"x_scale must be a CUDA fp32 tensor of shape {(rows, self.kblk)}")
            xs = x_scale.data_ptr()
            xs_row, xs_blk = x_scale.stride()
        elif self.int8:
            if x_scale is None or not x_scale.is_cuda or x_scale.dtype is not _Torch.f32 or x_scale.shape != (rows,):
                raise ValueError(f"x_scale must be a CUDA fp32 tensor of shape {(rows,)}")
            xs = x_scale.data_ptr()
            xs_row = x_scale.stride(0)
        elif x_scale is not None:
            raise ValueError("x_scale goes with float8_e4m3fn or int8 layers only")
        if y is None:
            y, ldy = _Torch.empty((rows, self.N), dtype=self.out_dtype, device=x.device), self.N
        else:
            yr, yc, ldy = _rows_2d(y, "y")
            if y.dtype is not self.out_dtype or yr != rows or yc != self.N:
                raise ValueError(f"y must be {self.out_dtype} of shape ({rows}, {self.N})")
        if stream is None:
            stream = _Torch.stream(self.device)
        elif hasattr(stream, "cuda_stream"):
            stream = stream.cuda_stream
        st = _Torch.run(self.handle, ctypes.byref(LinearArgs(rows, x.data_ptr(), ldx, xs, xs_row, xs_blk, offsets,
                                                             y.data_ptr(), ldy)), stream)
        if st != CONVF_OK:
            _check(st)
        return y

    def __call__(self, x, offsets, x_scale=None, y=None, stream=None):
        """y [rows][N] for ``x`` [rows][K] (w's type; rows a multiple of 16 bytes apart), ``offsets``
        int32 CUDA [experts+1] and ``x_scale`` fp32, for e4m3 [rows][ceil(K/128)] and for int8 [rows] (any
        strides).
        Rows that no expert takes are not written, and none at all with offsets that decrease or pass
        the rows (``status`` reports those)."""
        if not offsets.is_cuda or offsets.dtype is not _Torch.i32 or offsets.shape != (self.experts + 1,) \
                or not offsets.is_contiguous():
            raise ValueError(f"offsets must be a contiguous int32 CUDA vector of {self.experts + 1}")
        if offsets.get_device() != self.device:
            raise ValueError(f"offsets is on device {offsets.get_device()}, the layer on device {self.device}")
        return self._run(x, offsets.data_ptr(), x_scale, y, stream)

    def describe(self, rows: int) -> str:
        return conv_fused_linear_describe(self.handle, rows)

    def status(self) -> int:
        return conv_fused_linear_status(self.handle)

    def clear_status(self):
        conv_fused_linear_clear_status(self.handle)

    def close(self):
        if getattr(self, "handle", None):
            conv_fused_linear_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class BlockLinear(ExpertLinear):
    """One linear layer on block-scaled e4m3 operands: ``w`` float8_e4m3fn [N][K] with ``w_scale``
    [ceil(N/128)][ceil(K/128)] (or bf16 without scales), ``bias`` fp32 [N] or None; the rest as
    ExpertLinear.  Calling it with x and x_scale, as quantize_blocks gives them, returns y."""

    def __init__(self, w, w_scale=None, bias=None, act=CONVF_ACT_NONE, clip=(0.0, 6.0), out_bf16=False):
        if w.dim() != 2:
            raise ValueError("w must be a CUDA tensor [N][K]")
        super().__init__(w[None], None if w_scale is None else w_scale[None], None if bias is None else bias[None], act,
                         clip, out_bf16)

    def __call__(self, x, x_scale=None, y=None, stream=None):
        return self._run(x, None, x_scale, y, stream)


class Int8Linear(BlockLinear):
    """One linear layer on int8 operands: ``w`` int8 [N][K] with ``w_scale`` fp32 [N] (a scale per output
    channel, as quantize_rows gives them), ``bias`` fp32 [N] or None; the rest as ExpertLinear.  Calling it
    with x (int8 [rows][K]) and x_scale [rows], as quantize_rows or rms_norm_quantize give them, returns
    y = act(sum * (x_scale * w_scale) + bias), the sums exact integers."""

    def __init__(self, w, w_scale, bias=None, act=CONVF_ACT_NONE, clip=(0.0, 6.0), out_bf16=False):
        import torch
        if w.dtype != torch.int8:
            raise ValueError("w must be int8")
        super().__init__(w, w_scale, bias, act, clip, out_bf16)
