"""The int8 linear layers' kernel for many rows, on the GPU: calls of several sizes again and again, several behind one
another and beside other work.  Results are exact, so every call has to give the definition's bits.

Sizes are such that the plan takes this kernel; each test asks the layer's description for it, so that a plan fitted anew
cannot take them elsewhere unseen."""
import pytest
import torch

import convolution_onnx_conv_gb300 as cf
from test_gpu_linear_int8 import BF16, F32, I8, done, expected, operands, rows16

pytestmark = pytest.mark.gpu


def many(layer, rows):
    assert "form=many_rows tile=256x192" in layer.describe(rows), layer.describe(rows)


class Noise:
    """Copies on a stream of their own while the calls of a test run."""

    def __init__(self, on):
        self.on, self.stream = on, torch.cuda.Stream()
        self.a = torch.zeros((1 << 28,), dtype=torch.uint8, device="cuda")
        self.b = torch.zeros_like(self.a)
        self.stream.wait_stream(torch.cuda.current_stream())   # (their memory was other work's of that stream)

    def some(self):
        if self.on:
            with torch.cuda.stream(self.stream):
                for _ in range(6):
                    self.b.copy_(self.a)


def repeat(calls, turns, noise):
    """calls: (layer, call into y, the expected y).  Three calls at a time, one behind another with nothing between them, into
    buffers that held other values; every value of every result counts."""
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    ys = [torch.empty_like(calls[i % len(calls)][2]) for i in range(3)]
    for _ in range(turns):
        for y in ys:
            y.fill_(float("nan"))
        noise.some()
        for i, y in enumerate(ys):
            calls[i % len(calls)][1](y)
        for i, y in enumerate(ys):
            wrong += (y.view(torch.int16) != calls[i % len(calls)][2].view(torch.int16)).sum()
    for layer, _, _ in calls:
        done(layer)
    assert int(wrong) == 0, f"{int(wrong)} wrong values in {3 * turns} calls"


@pytest.mark.parametrize("busy", [False, True], ids=["alone", "busy"])
@pytest.mark.parametrize("rows,n,k,turns", [(1100, 4000, 1100, 100), (4096, 4096, 8192, 50), (8192, 8192, 8192, 50)])
def test_calls_repeat(rows, n, k, turns, busy):
    """Rings of stages and units that stay full over many tiles and a long reduction."""
    calls = []
    for seed in (1, 2):
        x, w, xs, ws = operands(100 * seed + k, rows, 1, n, k)
        lin = cf.Int8Linear(rows16(w)[0], ws[0], out_bf16=True)
        many(lin, rows)
        calls.append((lin, lambda y, lin=lin, x=rows16(x), xs=xs: lin(x, xs, y=y), expected(x, w[0], xs, ws[0], out=BF16)))
        del x, w
    repeat(calls, turns, Noise(busy))


@pytest.mark.parametrize("busy", [False, True], ids=["alone", "busy"])
def test_calls_of_experts_repeat(busy):
    counts = [700, 0, 1500, 513, 1, 900, 1280, 260]
    rows, n, k = sum(counts), 2000, 4096
    calls = []
    for seed in (3, 4):
        x, w, xs, ws = operands(seed, rows, len(counts), n, k)
        off = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
        lin = cf.ExpertLinear(rows16(w), ws, out_bf16=True)
        many(lin, rows)
        want = torch.cat([expected(x[a:b], w[e], xs[a:b], ws[e], out=BF16) for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:]))])
        calls.append((lin, lambda y, lin=lin, x=rows16(x), xs=xs, off=off: lin(x, off, xs, y=y), want))
    repeat(calls, 100, Noise(busy))


FORMS = [(17, 1024, 1000, "direct tile=4x", 1), (48, 1500, 1500, "direct tile=16x", 1), (64, 2048, 520, "few_rows tile=16x", 1),
         (40, 2048, 3000, "few_rows tile=16x", 2), (128, 136, 8192, "few_rows tile=16x", 4), (80, 264, 3000, "few_rows tile=16x", 8),
         (64, 6000, 1000, "few_rows tile=64x", 1), (17, 6000, 8192, "few_rows tile=64x", 2), (400, 520, 6000, "few_rows tile=64x", 4),
         (200, 136, 16384, "few_rows tile=64x", 8), (1000, 3000, 1000, "many_rows tile=256x", 1)]


def of_form(layer, rows, form, split):
    text = layer.describe(rows)
    assert f"form={form}" in text and f"split={split} " in text, text


@pytest.mark.parametrize("rows,n,k,form,split", FORMS)
def test_zeros_keep_their_sign(rows, n, k, form, split):
    """Scales whose product underflows leave a zero of the sum's sign, in every form; with a bias of 0 added it is 0."""
    x, w, xs, ws = operands(rows + n, rows, 1, n, k)
    xs, ws = xs * 0 + 1e-30, ws * 0 + 1e-30
    s = x.double() @ w[0].double().T
    for bias in (None, torch.zeros(n, device="cuda")):
        lin = cf.Int8Linear(rows16(w)[0], ws[0], bias=bias)
        of_form(lin, rows, form, split)
        y = lin(rows16(x), xs)
        done(lin)
        assert not y.any() and torch.equal(torch.signbit(y), (s < 0) if bias is None else torch.zeros_like(y, dtype=torch.bool))
