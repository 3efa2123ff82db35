"""The int8 linear layers without a GPU: refusals before any CUDA call, tensors on stand-ins, what the kernels' sources
must not hold, and their set-up on a runtime of two devices."""
import os
import re
import subprocess

import pytest

import convolution_onnx_conv_gb300 as cf
from convolution_onnx_conv_gb300 import _binding, _build
from convolution_onnx_conv_gb300._binding import LinearArgs, LinearDesc
from test_block_scaled_host import CSRC, ROOT, TWO_DEVICES, FakeCuda, source

P = 0x10000000   # an aligned address that nothing reads
BAD, NOT = cf.CONVF_ERR_INVALID_ARG, cf.CONVF_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return cf.load_library()


def linear(**kw):
    v = dict(N=96, K=200, experts=3, dtype=cf.CONVF_LINEAR_INT8, ldw=208, expert_stride=96 * 208, act=cf.CONVF_ACT_NONE,
             clip_lo=0.0, clip_hi=6.0, out_dtype=cf.CONVF_OUT_F32)
    v.update(kw)
    return LinearDesc(*[v[n] for n, _ in LinearDesc._fields_])


@pytest.mark.parametrize("kw,status,needle", [
    (dict(K=131072, ldw=131072, expert_stride=96 * 131072), NOT, "K=131072"),
    (dict(K=0), BAD, "K=0"),
    (dict(ldw=192), BAD, "ldw=192"),
    (dict(ldw=200), NOT, "16 bytes"),
    (dict(ldw=216), NOT, "16 bytes"),
    (dict(expert_stride=95 * 208), BAD, "overlap"),
    (dict(expert_stride=96 * 208 + 8), NOT, "16 bytes"),
    (dict(dtype=4), BAD, "dtype=4"),
])
def test_create_refusals(kw, status, needle):
    with pytest.raises(cf.ConvFusedError) as e:
        cf.conv_fused_linear_create(linear(**kw), P, 2 * P)
    assert e.value.status == status and needle in str(e.value)


@pytest.mark.parametrize("w,ws,bias,needle", [(None, P, None, "W is NULL"), (P + 8, P, None, "16-byte"), (P, None, None, "w_scale"),
                                              (P, P + 2, None, "aligned"), (P, P, P + 1, "aligned")])
def test_create_refuses_operands(w, ws, bias, needle):
    with pytest.raises(cf.ConvFusedError) as e:
        cf.conv_fused_linear_create(linear(), w, ws, bias)
    assert e.value.status == BAD and needle in str(e.value)


@pytest.mark.parametrize("name", ["linear_int8_dev.cuh", "linear_int8_direct.cu", "tc_linear_int8_few.cu", "tc_linear_int8_many.cu"])
def test_no_read_only_loads_of_what_the_kernel_before_may_write(name):
    text = source(name)
    assert not re.search(r"__ldg\b|\.nc\b|__ldcg|__ldca", text)
    assert not re.search(r"asm\s*\(\s*\"ld\.", text)


def test_every_wait_is_bounded():
    """The kernels wait through the bounded helpers only."""
    for name in ("tc_linear_int8_few.cu", "tc_linear_int8_many.cu"):
        assert not re.search(r"try_wait|while\s*\(\s*(true|1|!)", source(name))


@pytest.mark.parametrize("name", ["tc_linear_int8_few", "tc_linear_int8_many"])
def test_kernels_are_set_up_on_every_device(name, tmp_path):
    """The host side of the launches, on a runtime that keeps a kernel's shared-memory limit per device."""
    few = name.endswith("few")
    head, body = TWO_DEVICES.split("int main() {")
    launches = """
          const convf::LinearPlan plan{convf::kLinearInt8, tile, 1, 152};
          bad += convf::launch_linear_int8_few(p, plan, m, m, nullptr) != cudaSuccess;
          bad += convf::linear_int8_max_clusters(tile, 4, 152) != 18;""" if few else """
          const convf::LinearPlan plan{convf::kLinearInt8, convf::kInt8PairRows, 1, 152};
          bad += convf::launch_linear_int8_many(p, plan, m, m, m, nullptr) != cudaSuccess;"""
    main = tmp_path / "main.cu"
    main.write_text(head.replace("a->numRegs = 168", "a->numRegs = 72") + """int main() {
  convf::LinearParams p{};
  CUtensorMap m{};
  int bad = 0;
  for (device = 0; device < 2; ++device)
    for (int turn = 0; turn < 2; ++turn)
      for (int tile = 16; tile <= 64; tile *= 4) {""" + launches + """
      }
  printf("%d refused\\n", bad);
  return bad != 0;
}
""")
    exe = str(tmp_path / "main")
    subprocess.run([_build._nvcc(), "-gencode", "arch=compute_103a,code=compute_103a", "-Xcicc", "-O0", "-std=c++17",
                    "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include"), "-I", CSRC, f'-DSOURCE="{name}.cu"',
                    str(main), "-o", exe, "-lcuda"], check=True, capture_output=True)
    res = subprocess.run([exe], capture_output=True, text=True)
    assert res.returncode == 0 and res.stdout == "0 refused\n", res.stdout + res.stderr


# ------------------------------------------------------------------------------ tensors

@pytest.fixture
def calls(monkeypatch):
    names, made = _binding._Torch, []
    names.bind()
    monkeypatch.setattr(names, "stream", lambda index: 0)
    monkeypatch.setattr(names, "current_device", lambda: 0, raising=False)
    monkeypatch.setattr(names, "empty", lambda shape, dtype, device: FakeCuda(shape, dtype))
    monkeypatch.setattr(names, "run", lambda layer, args, stream: made.append(args._obj) or 0)
    monkeypatch.setattr(_binding, "conv_fused_linear_create", lambda d, *tensors: made.append(d) or 0)   # (no handle to free)
    return made


def test_layer_tensors_are_looked_at(calls):
    import torch
    i8, f32, bf16 = torch.int8, torch.float32, torch.bfloat16
    w, ws = FakeCuda((96, 256), i8), FakeCuda((96,), f32)
    layer = cf.Int8Linear(w, ws, out_bf16=True)
    assert calls[-1].dtype == cf.CONVF_LINEAR_INT8 and calls[-1].N == 96 and calls[-1].K == 256
    y = layer(FakeCuda((4, 256), i8), FakeCuda((4,), f32))
    assert y.dtype is bf16 and calls[-1].xs_row == 1
    layer(FakeCuda((4, 256), i8), FakeCuda((4,), f32, strides=(0,)))
    assert calls[-1].xs_row == 0 and len(calls) == 3
    for kw, words in ((dict(w=FakeCuda((96, 256), bf16)), "w must be int8"),
                      (dict(w_scale=None), "w_scale goes with"),
                      (dict(w_scale=FakeCuda((1, 2), f32)), "w_scale must be"),
                      (dict(w_scale=FakeCuda((96,), f32, 1)), "device 1"),
                      (dict(bias=FakeCuda((95,), f32)), "bias must be")):
        with pytest.raises(ValueError, match=words):
            cf.Int8Linear(**{"w": w, "w_scale": ws, **kw})
    for kw, words in ((dict(x=FakeCuda((4, 256), torch.uint8)), "x must be torch.int8"),
                      (dict(x=FakeCuda((4, 255), i8)), "256 columns"),
                      (dict(x=FakeCuda((4, 256), i8, 1)), "device 1"),
                      (dict(x_scale=None), "x_scale must be"),
                      (dict(x_scale=FakeCuda((4, 2), f32)), "x_scale must be"),
                      (dict(x_scale=FakeCuda((4,), bf16)), "x_scale must be"),
                      (dict(x_scale=FakeCuda((4,), f32, 1)), "device 1"),
                      (dict(y=FakeCuda((4, 96), f32)), "y must be"),
                      (dict(y=FakeCuda((4, 96), bf16, 1)), "device 1")):
        with pytest.raises(ValueError, match=words):
            layer(**{"x": FakeCuda((4, 256), i8), "x_scale": FakeCuda((4,), f32), **kw})
    assert len(calls) == 3
    experts = cf.ExpertLinear(FakeCuda((3, 96, 256), i8), FakeCuda((3, 96), f32))
    assert calls[-1].experts == 3
    experts(FakeCuda((4, 256), i8), FakeCuda((4,), torch.int32), FakeCuda((4,), f32))
    with pytest.raises(ValueError, match="w_scale must be"):
        cf.ExpertLinear(FakeCuda((3, 96, 256), i8), FakeCuda((3, 1, 2), f32))
    assert len(calls) == 5
