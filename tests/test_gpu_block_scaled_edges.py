"""Edges of the block-scaled operators on the GPU: stored bytes rather than values, runs that share memory with
their neighbours, long reductions, and every split of the few-rows kernel."""
import pytest
import torch

import convolution_onnx_conv_gb300 as cf

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------------------ the quantiser's bytes

def bytes_64(v, scale, tall=1):
    """The e4m3 bytes of double values by the definition: the float32 quotient's nearest, zeros with the
    quotient's sign, 0x00 where the scale is 0.  (Rounding on the host; |v| / scale is at most 448.)"""
    rows, cols = v.shape
    wide = scale.double().repeat_interleave(tall, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    q = (v / wide).float().clamp(-448, 448).cpu().to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    return torch.where(wide == 0, torch.zeros_like(q), q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -60, 2.0 ** 70])
@pytest.mark.parametrize("cols", [256, 203])
def test_zeros_keep_their_sign(dtype, block_rows, size, cols):
    """-0 beside other values, and values too small for e4m3, in blocks of ordinary and of extreme scales."""
    x = torch.randn((130, cols), generator=gen(cols), device="cuda") * size
    x[:, 1::3] = -0.0
    x[:, 2::9] = 0.0
    x[:, 5::9] *= 2.0 ** -20
    x[7] = -0.0                 # a row of them: its scale is 0
    x = x.to(dtype)
    q, s = cf.quantize_blocks(x, block_rows=block_rows)
    want = bytes_64(x.double(), s, block_rows)
    assert bool((want == 0x80).any()) and torch.equal(q.view(torch.uint8), want)


def test_gated_zeros_keep_their_sign():
    x = torch.ones((3, 256), device="cuda")
    x[0, :4] = torch.tensor([-0.0, 0.0, -0.0, 0.0])
    x[0, 128:132] = torch.tensor([1.0, -1.0, -1.0, 1.0])
    q, _ = cf.quantize_blocks(x, gated=True)
    assert q.view(torch.uint8)[0, :4].tolist() == [0x80, 0x80, 0, 0]
