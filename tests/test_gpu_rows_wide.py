"""Rows to 8 bits on both sides of the widths at which the kernels change, on the GPU against the definitions in 64 bits
(equal and near as in test_gpu_rows.py).

A row takes one pass up to 16 columns for each thread that its form has on an SM: 16384 columns where they take 4 bytes of
a thread's loads or fewer, 12288 up to 8, 8192 for more (two bytes more each where rows begin anywhere).  Wider rows are
read twice, and what is written over the residual or over x is written in the second pass."""
import pytest
import torch

import convolution_onnx_conv_gb300 as cf
from test_gpu_rows import BF16, F32, check_norm, gen, int8_64, randn

pytestmark = pytest.mark.gpu
COLS = [8191, 8192, 8193, 8200, 12288, 12289, 12296, 16384, 16385, 16392, 20000, 20001]


def rows_of(seed, rows, cols, ld, dtype):
    """Rows `ld` elements apart: at addresses of their own alignment."""
    return torch.as_strided(randn(seed, rows * ld, dtype=dtype), (rows, cols), (ld, 1))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", COLS)
def test_rows(cols, dtype):
    for rows, ld in ((2, cols), (3, -(-cols // 32) * 32), (700, cols)):
        x = rows_of(cols + rows, rows, cols, ld, dtype)
        x[rows // 2] = 0
        q, s = cf.quantize_rows(x)
        rq, rs = int8_64(x.double())
        assert torch.equal(s.double(), rs) and torch.equal(q.double(), rq)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", COLS)
def test_rows_gathered(cols, dtype):
    x = randn(cols, 40, cols, dtype=dtype)
    index = torch.randint(0, 40, (650,), generator=gen(5), device="cuda", dtype=torch.int32)
    index[3:6], index[640:] = -1, 40
    q, s = cf.quantize_rows(x, index=index)
    ok = (index >= 0) & (index < 40)
    rq, rs = int8_64(torch.where(ok[:, None], x.double()[index.long().clamp(0, 39)], 0.0))
    assert torch.equal(s.double(), rs) and torch.equal(q.double(), rq)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", COLS)
def test_rows_gated(cols, dtype):
    x = (randn(cols, 330, 2 * cols) * 4).to(dtype)
    x[0, :cols] = -200   # gates that are shut
    index = torch.randint(0, 330, (9,), generator=gen(6), device="cuda", dtype=torch.int32)
    for where in (None, index):
        q, s = cf.quantize_rows(x, index=where, gated=True)
        xs = (x if where is None else x[where.long()]).double()
        v = xs[:, :cols] * torch.sigmoid(xs[:, :cols]) * xs[:, cols:]
        m = v.abs().amax(1)
        live = m > 1e-30
        assert bool(((s.double() - m / 127).abs() <= 2.0 ** -20 * m / 127 + 1e-35).all())
        off = (q.double() - v / (m / 127)[:, None]).abs()[live]
        assert bool((off <= 0.5 + 127 * 2.0 ** -19).all())


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("dtype,res", [(BF16, None), (BF16, BF16), (BF16, F32), (F32, None), (F32, F32)])
@pytest.mark.parametrize("cols", COLS)
def test_norm(cols, dtype, res, int8):
    for rows, ld in ((3, -(-cols // 32) * 32), (400, cols)):
        x = rows_of(cols + rows, rows, cols, ld, dtype) * torch.exp(randn(rows, rows, 1)).to(dtype)
        r = None if res is None else rows_of(cols, rows, cols, ld, res)
        w = 1 + randn(7, cols) / 4
        check_norm(x, w, 1e-6, r, int8, cf.rms_norm_quantize(x, w, 1e-6, residual=r, int8=int8))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("res", [BF16, F32])
@pytest.mark.parametrize("cols", COLS)
def test_norm_in_place(cols, res, int8):
    """h over the residual and over x, rows side by side and apart, each CTA with several of them."""
    w = randn(11, cols)
    for rows, ld in ((700, cols), (330, -(-cols // 32) * 32), (5, cols + 3)):
        x, r = (rows_of(seed, rows, cols, ld, res) for seed in (9, 10))
        a = r.clone() if ld == cols else torch.as_strided(r.as_strided((rows * ld,), (1,)).clone(), (rows, cols), (ld, 1))
        check_norm(x, w, 1e-6, r, int8, cf.rms_norm_quantize(x, w, residual=a, int8=int8, h=a))
        b = torch.as_strided(x.as_strided((rows * ld,), (1,)).clone(), (rows, cols), (ld, 1))
        check_norm(x, w, 1e-6, r, int8, cf.rms_norm_quantize(b, w, residual=r, int8=int8, h=b))


def test_gates_next_to_zero():
    """Gates whose remainders are subnormal: where 1 + exp(-g) is 2 in float32 the gate is g / 2 rounded to nearest, down
    to the smallest numbers.  One column a row, so that the scale is the value over 127."""
    e = torch.randint(-149, -25, (20000,), generator=gen(30), device="cuda")
    g = torch.ldexp(1 + torch.rand((20000,), generator=gen(31), device="cuda", dtype=torch.float64), e).float()
    g = g * torch.where(torch.rand((20000,), generator=gen(32), device="cuda") < 0.5, -1.0, 1.0)
    x = torch.stack([g, torch.ones_like(g)], 1)
    _, s = cf.quantize_rows(x, gated=True)
    v = (g.double() / 2).float().double().abs()
    assert torch.equal(s.double(), (v / 127).float().double())
