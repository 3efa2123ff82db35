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


@pytest.mark.parametrize("n", [4099, 4100])
@pytest.mark.parametrize("out", [F32, BF16])
def test_every_way_out(n, out):
    """Results by whole tiles, by 16-byte units and by the elements: rows of y that begin and end on 16 bytes or do not, and
    what lies beside them; with a bias and a clamp, and without."""
    rows, k = 1500, 2100
    x, w, xs, ws = operands(n, rows, 1, n, k)
    bias = torch.randn((n,), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    for b, act, lo, hi in ((None, cf.CONVF_ACT_NONE, -float("inf"), float("inf")), (bias, cf.CONVF_ACT_NONE, -float("inf"), float("inf")),
                           (bias, cf.CONVF_ACT_RELU, 0.0, float("inf")), (None, cf.CONVF_ACT_CLIP, -2.5, 3.0)):
        lin = cf.Int8Linear(rows16(w)[0], ws[0], bias=b, act=act, clip=(-2.5, 3.0), out_bf16=out == BF16)
        many(lin, rows)
        want = expected(x, w[0], xs, ws[0], b, lo, hi, out)
        for offset, ld in ((0, n), (0, 4128), (1, n + 5), (3, 4128)):
            buf = torch.full((rows * ld + 8,), -7.0, dtype=out, device="cuda")
            y = torch.as_strided(buf, (rows, n), (ld, 1), offset)
            lin(rows16(x, pad=1), xs, y=y)
            done(lin)
            assert torch.equal(y, want), (offset, ld)
            y.fill_(-7)
            assert bool((buf == -7).all()), (offset, ld)


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("k", [1030, 4096])
def test_experts(k, out):
    """Groups of a part of a tile, of several, of none; rows that no expert takes; a bias for each and a clamp."""
    counts = [700, 0, 1500, 513, 1, 900, 1280, 260]
    n, before, after = 2000, 3, 5
    rows = sum(counts) + before + after
    x, w, xs, ws = operands(k, rows, len(counts), n, k)
    bias = torch.randn(ws.shape, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    off = torch.tensor([0] + counts).cumsum(0) + before
    lin = cf.ExpertLinear(rows16(w), ws, bias=bias, act=cf.CONVF_ACT_RELU, out_bf16=out == BF16)
    many(lin, rows)
    y = torch.full((rows, n + 8), -7.0, dtype=out, device="cuda")
    lin(rows16(x), off.to(torch.int32).cuda(), xs, y=y[:, :n])
    done(lin)
    want = torch.full_like(y, -7.0)
    for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        want[a:b, :n] = expected(x[a:b], w[e], xs[a:b], ws[e], bias[e], lo=0.0, out=out)
    assert torch.equal(y, want)


def test_many_tiles_of_a_short_reduction():
    """More tiles for a pair than the scheduler has places for, an accumulator of less than one stage."""
    rows, n = 40000, 4096
    for k in (100, 300):
        x, w, xs, ws = operands(k, rows, 1, n, k)
        lin = cf.Int8Linear(rows16(w)[0], ws[0], out_bf16=True)
        many(lin, rows)
        y = lin(rows16(x), xs)
        done(lin)
        assert torch.equal(y, expected(x, w[0], xs, ws[0], out=BF16))


@pytest.mark.parametrize("rows,n,k,form,split", FORMS + [(16, 8192, 32768, "few_rows tile=16x", 2), (512, 4096, 131071, "many_rows tile=256x", 1)])
def test_the_largest_sums_in_every_form(rows, n, k, form, split):
    """Terms of one sign and the largest size, which fill an accumulator's 24 bits and, at the largest K, all of int32."""
    x = torch.full((rows, k), -128, dtype=I8, device="cuda")
    w = torch.full((n, k), -128, dtype=I8, device="cuda")
    w[::3] = 127
    x[0, -1] = 1
    xs, ws = torch.ones(rows, device="cuda"), torch.ones(n, device="cuda")
    lin = cf.Int8Linear(rows16(w), ws)
    of_form(lin, rows, form, split)
    y = lin(rows16(x), xs)
    done(lin)
    assert torch.equal(y, expected(x, w, xs, ws))


def test_every_form_at_once_with_many_rows():
    """Layers of every form, two of them for many rows, on streams of their own, side by side, many times."""
    cases = []
    for seed, (rows, n, k, form, split) in enumerate(FORMS + [(1100, 4000, 1100, "many_rows tile=256x", 1)]):
        x, w, xs, ws = operands(50 + seed, rows, 1, n, k)
        lin = cf.Int8Linear(rows16(w)[0], ws[0], out_bf16=True)
        of_form(lin, rows, form, split)
        cases.append((lin, rows16(x), xs, expected(x, w[0], xs, ws[0], out=BF16), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [[lin(a, s, stream=st) for _ in range(4)] for lin, a, s, _, st in cases]
        torch.cuda.synchronize()
        for (lin, _, _, y, _), got in zip(cases, outs):
            assert all(torch.equal(g, y) for g in got) and lin.status() == cf.CONVF_OK
