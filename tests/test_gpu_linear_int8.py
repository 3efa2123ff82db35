"""Linear layers on int8 operands, one and one per expert, on the GPU.  The sums are integers of less than 2^31,
which 64-bit floating-point sums give exactly, and what follows them is a handful of float32 operations, each rounded
to nearest: results are equal to the definition's, bit for bit, at every size and in every form."""
import re

import pytest
import torch

import convolution_onnx_conv_gb300 as cf

pytestmark = pytest.mark.gpu
BF16, F32, I8 = torch.bfloat16, torch.float32, torch.int8


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows16(t, pad=0):
    """t (int8) with rows a multiple of 16 bytes apart (and `pad` such steps more), 77 between the rows."""
    wide = (-(-t.shape[-1] // 16) + pad) * 16
    b = torch.full((*t.shape[:-1], wide), 77, dtype=I8, device=t.device)
    b[..., : t.shape[-1]] = t
    return b[..., : t.shape[-1]]


def operands(seed, rows, experts, n, k, scaled=True):
    g = gen(seed)
    x = torch.randint(-128, 128, (rows, k), generator=g, device="cuda", dtype=I8)
    w = torch.randint(-128, 128, (experts, n, k), generator=g, device="cuda", dtype=I8)
    xs = torch.rand((rows,), generator=g, device="cuda") / 50 + 1e-4
    ws = torch.rand((experts, n), generator=g, device="cuda") / 50 + 1e-4
    return x, w, xs, ws


def expected(x, w, xs, ws, bias=None, lo=-float("inf"), hi=float("inf"), out=F32):
    y = (x.double() @ w.double().T).float() * (xs[:, None] * ws[None])
    if bias is not None:
        y = y + bias
    return y.clamp(lo, hi).to(out)


def done(layer):
    torch.cuda.synchronize()
    assert layer.status() == cf.CONVF_OK, cf.conv_fused_last_error()


SIZES = [(1, 1, 1), (1, 128, 128), (1, 1000, 2048), (2, 130, 129), (7, 5, 16), (16, 256, 640), (17, 100, 100),
         (33, 129, 2100), (64, 64, 64), (65, 1000, 257), (129, 300, 1000), (191, 256, 513), (193, 257, 1025), (300, 513, 384),
         (1025, 136, 520), (515, 1040, 4096), (2050, 2100, 300)]


@pytest.mark.parametrize("rows,n,k", SIZES)
def test_linear(rows, n, k):
    x, w, xs, ws = operands(rows * 7 + n + k, rows, 1, n, k)
    bias = torch.randn((n,), generator=gen(1), device="cuda")
    for out in (F32, BF16):
        for b in (bias, None):
            lin = cf.Int8Linear(rows16(w)[0], ws[0], bias=b, out_bf16=out == BF16)
            y = lin(rows16(x), xs)
            done(lin)
            assert y.dtype is out and torch.equal(y, expected(x, w[0], xs, ws[0], b, out=out)), lin.describe(rows)
            assert torch.equal(y, lin(rows16(x), xs))
            lin.close()


def test_every_form():
    """Every tile and every split of the reduction is launched and gives the same integers."""
    seen = {}
    for rows in (1, 3, 16, 20, 32, 40, 64, 100, 150, 200, 400, 700, 1500, 4000):
        for n, k in ((64, 16384), (128, 4000), (640, 3000), (1024, 2049), (4096, 512), (8192, 130), (20000, 128)):
            x, w, xs, ws = operands(rows + n, rows, 1, n, k)
            lin = cf.Int8Linear(rows16(w)[0], ws[0])
            form = re.search(r"form=(\w+) tile=(\d+)x\d+ split=(\d+)", lin.describe(rows)).groups()
            if seen.get(form, 0) < 3:
                seen[form] = seen.get(form, 0) + 1
                y = lin(rows16(x), xs)
                done(lin)
                assert torch.equal(y, expected(x, w[0], xs, ws[0])), lin.describe(rows)
            lin.close()
    assert {(f, t) for f, t, _ in seen} == {("direct", "4"), ("direct", "16"), ("few_rows", "16"), ("few_rows", "64"), ("many_rows", "256")}, sorted(seen)
    assert {s for _, _, s in seen} >= {"1", "2", "4"}, sorted(seen)


@pytest.mark.parametrize("rows", [1, 40, 260])
@pytest.mark.parametrize("a,b", [(-128, -128), (-128, 127), (127, 127)])
def test_the_largest_sums(rows, a, b):
    """Terms of one sign and the largest size up to the largest K; ends at which an accumulator's chunk ends and does not."""
    for k in (511, 512, 513, 1024, 65536, 131071):
        w = torch.full((136, k), b, dtype=I8, device="cuda")
        w[::3] = 127
        x = torch.full((rows, k), a, dtype=I8, device="cuda")
        x[0, -1] = 1
        one = torch.ones(136, device="cuda")
        lin = cf.Int8Linear(rows16(w), one)
        y = lin(rows16(x), torch.ones(rows, device="cuda"))
        done(lin)
        assert torch.equal(y, expected(x, w, torch.ones(rows, device="cuda"), one)), k
        lin.close()


COUNTS = [[5], [0, 0, 0], [0, 9, 0], [1, 1, 1, 1], [130, 0, 1, 0, 64, 300], [16, 17, 15, 33, 0, 191, 192, 193],
          [700, 3, 0, 0, 900], [1] * 70, [0] * 200 + [40] + [0] * 100, [2, 0, 1, 3] * 16, [400, 0, 380, 777]]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}e{sum(c)}r")
@pytest.mark.parametrize("n,k", [(130, 200), (264, 1100)])
def test_experts(counts, n, k):
    before, after = 3, 5   # rows that no expert takes
    e, rows = len(counts), sum(counts) + before + after
    x, w, xs, ws = operands(sum(counts) + n, rows, e, n, k)
    off = torch.tensor([0] + counts).cumsum(0) + before
    bias = torch.randn((e, n), generator=gen(2), device="cuda")
    lin = cf.ExpertLinear(rows16(w), ws, bias=bias, out_bf16=len(counts) % 2 == 0, act=cf.CONVF_ACT_RELU)
    y = torch.full((rows, n + 3), -7.0, dtype=lin.out_dtype, device="cuda")
    lin(rows16(x, pad=1), off.to(torch.int32).cuda(), xs, y=y[:, :n])
    done(lin)
    assert bool((y[:, n:] == -7).all()) and bool((y[:before] == -7).all()) and bool((y[rows - after:] == -7).all())
    for i in range(e):
        a, b = int(off[i]), int(off[i + 1])
        assert torch.equal(y[a:b, :n], expected(x[a:b], w[i], xs[a:b], ws[i], bias[i], lo=0.0, out=lin.out_dtype)), i
    lin.close()


def test_bad_offsets_write_nothing():
    x, w, xs, ws = operands(3, 50, 3, 64, 96)
    lin = cf.ExpertLinear(w, ws)
    for off in ([0, 30, 20, 50], [0, 10, 20, 51], [-1, 10, 20, 50]):
        y = torch.full((50, 64), 9.0, device="cuda")
        lin(x, torch.tensor(off, dtype=torch.int32, device="cuda"), xs, y=y)
        torch.cuda.synchronize()
        assert bool((y == 9).all()) and lin.status() == cf.CONVF_ERR_INVALID_ARG
        lin.clear_status()
    lin(x, torch.tensor([0, 10, 20, 50], dtype=torch.int32, device="cuda"), xs)
    done(lin)


@pytest.mark.parametrize("act,clip,lo,hi", [(cf.CONVF_ACT_RELU, (0, 0), 0.0, float("inf")), (cf.CONVF_ACT_RELU6, (0, 0), 0.0, 6.0),
                                            (cf.CONVF_ACT_CLIP, (-2.5, 3.0), -2.5, 3.0)])
def test_activation_clamps(act, clip, lo, hi):
    for rows in (3, 300):
        x, w, xs, ws = operands(4, rows, 1, 70, 256)
        for out in (F32, BF16):
            lin = cf.Int8Linear(rows16(w)[0], ws[0], act=act, clip=clip, out_bf16=out == BF16)
            assert torch.equal(lin(rows16(x), xs), expected(x, w[0], xs, ws[0], lo=lo, hi=hi, out=out))


@pytest.mark.parametrize("rows,n,k", [(5, 131, 300), (61, 257, 700), (450, 515, 500)])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_strides_and_what_lies_beside(rows, n, k, offset):
    """y at any address and stride, columns of a wider buffer; scales at any stride, one for all rows among them."""
    x, w, xs, ws = operands(rows + n, rows, 1, n, k)
    for out in (F32, BF16):
        lin = cf.Int8Linear(rows16(w, pad=2)[0], ws[0], out_bf16=out == BF16)
        buf = torch.full((rows * (n + 5) + 8,), -7.0, dtype=out, device="cuda")
        y = torch.as_strided(buf, (rows, n), (n + 5, 1), offset)
        every = torch.zeros((rows, 3), device="cuda")
        every[:, 1] = xs
        lin(rows16(x, pad=3), every[:, 1], y=y)
        done(lin)
        assert torch.equal(y, expected(x, w[0], xs, ws[0], out=out))
        keep = torch.ones_like(buf, dtype=torch.bool)
        torch.as_strided(keep, (rows, n), (n + 5, 1), offset).fill_(False)
        assert bool((buf[keep] == -7).all())
        same = xs[:1].expand(rows)
        assert torch.equal(lin(rows16(x), same), expected(x, w[0], same, ws[0], out=out))


def test_scales_that_are_no_numbers():
    """NaN and infinite scales stay in their rows and columns; a zero scale gives the bias."""
    x, w, xs, ws = operands(5, 20, 1, 150, 300)
    xs[3], xs[5], ws[0, 7] = float("nan"), 0.0, float("inf")
    bias = torch.randn((150,), generator=gen(6), device="cuda")
    y = cf.Int8Linear(rows16(w)[0], ws[0], bias=bias)(rows16(x), xs)
    assert torch.equal(torch.nan_to_num(y, 1e9), torch.nan_to_num(expected(x, w[0], xs, ws[0], bias), 1e9))


def test_no_rows():
    x, w, xs, ws = operands(6, 0, 1, 32, 64)
    assert cf.Int8Linear(w[0], ws[0])(x, xs).shape == (0, 32)


def test_streams_and_graphs():
    """Two graphs of one layer, replayed at once on streams of their own, and calls on a given stream."""
    x, w, xs, ws = operands(7, 300, 1, 520, 1000)
    lin = cf.Int8Linear(rows16(w)[0], ws[0], out_bf16=True)
    x16 = rows16(x)
    want = {r: expected(x[:r], w[0], xs[:r], ws[0], out=BF16) for r in (4, 300)}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        for r in want:
            y = lin(x16[:r], xs[:r], stream=stream)
            side.synchronize()
            assert torch.equal(y, want[r])
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for r in want:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(lin(x16[:r], xs[:r]))
        graphs.append(g)
    for _ in range(20):
        for y in outs:
            y.fill_(-1)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, want[r]) for y, r in zip(outs, want))
    done(lin)


def test_every_form_at_once():
    """Layers of every form on streams of their own, side by side, many times: none takes what another waits for."""
    cases = []
    for seed, (rows, n, k) in enumerate([(1, 2048, 2048), (12, 1040, 4096), (60, 4096, 300), (128, 2048, 2048), (900, 1000, 1100)]):
        x, w, xs, ws = operands(20 + seed, rows, 1, n, k)
        lin = cf.Int8Linear(rows16(w)[0], ws[0], out_bf16=True)
        cases.append((lin, rows16(x), xs, expected(x, w[0], xs, ws[0], out=BF16), torch.cuda.Stream()))
    counts = [0, 1, 7, 2, 30, 3, 1, 0]
    x, w, xs, ws = operands(30, sum(counts), len(counts), 520, 1500)
    off = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
    experts = cf.ExpertLinear(rows16(w), ws, out_bf16=True)
    want = torch.cat([expected(x[a:b], w[e], xs[a:b], ws[e], out=BF16) for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:]))])
    x16, side = rows16(x), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [[lin(a, s, stream=st) for _ in range(4)] for lin, a, s, _, st in cases]
        ragged = [experts(x16, off, xs, stream=side) for _ in range(4)]
        torch.cuda.synchronize()
        for (lin, _, _, y, _), got in zip(cases, outs):
            assert all(torch.equal(g, y) for g in got) and lin.status() == cf.CONVF_OK
        assert all(torch.equal(g, want) for g in ragged) and experts.status() == cf.CONVF_OK


@pytest.mark.parametrize("k", [500, 1000, 2048, 2055])
def test_groups_of_a_few_rows(k):
    """Groups of no rows to nine, some of them one behind another empty, of a warp's tiles over the groups' borders."""
    counts = [0, 0, 1, 2, 0, 3, 4, 5, 0, 0, 0, 6, 8, 9, 1, 0, 1, 0, 0]
    n = 37
    x, w, xs, ws = operands(k, sum(counts) + 3, len(counts), n, k)
    off = torch.tensor([1] + counts, device="cuda").cumsum(0).to(torch.int32)
    lin = cf.ExpertLinear(rows16(w), ws)
    y = torch.full((x.shape[0], n), -7.0, device="cuda")
    lin(rows16(x), off, xs, y=y)
    done(lin)
    want = torch.full_like(y, -7.0)
    for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        want[a:b] = expected(x[a:b], w[e], xs[a:b], ws[e])
    assert torch.equal(y, want), lin.describe(x.shape[0])


def test_offsets_past_32_bits():
    """Weights, rows and results whose last elements are more than 2^32 elements from their first."""
    n, k = 5, 300
    far = 1_100_000_000 // 16 * 16
    x, w, xs, ws = operands(8, 5, 1, n, k)
    wb, xb = (torch.empty((4 * far + 512,), dtype=I8, device="cuda") for _ in range(2))
    wf, xf = torch.as_strided(wb, (n, k), (far, 1)), torch.as_strided(xb, (5, k), (far, 1))
    wf.copy_(w[0])
    xf.copy_(x)
    yf = torch.as_strided(torch.empty((4 * far + 16,), dtype=BF16, device="cuda"), (5, n), (far, 1))
    lin = cf.Int8Linear(wf, ws[0], out_bf16=True)
    lin(xf, xs, y=yf)
    done(lin)
    assert torch.equal(yf, expected(x, w[0], xs, ws[0], out=BF16))


def test_norm_product_gate_product_as_a_layer_uses_them():
    """A feed-forward layer in int8 from residual to residual, all on one stream, and the same captured: norm and
    quantise, [gate | up], gate and quantise, down, and the next norm adds the residual."""
    g = gen(9)
    rows, width, hidden = 70, 640, 328
    x = torch.randn((rows, width), generator=g, device="cuda").to(BF16)
    r = torch.randn((rows, width), generator=g, device="cuda")
    w1 = torch.randn((2 * hidden, width), generator=g, device="cuda") / width ** 0.5
    w2 = torch.randn((width, hidden), generator=g, device="cuda") / hidden ** 0.5
    nw = 1 + torch.randn((width,), generator=g, device="cuda") / 8
    up = cf.Int8Linear(*cf.quantize_rows(w1), out_bf16=True)
    down = cf.Int8Linear(*cf.quantize_rows(w2), out_bf16=True)

    def layer(x, r):
        q, s, h = cf.rms_norm_quantize(x, nw, residual=r, int8=True)
        q, s = cf.quantize_rows(up(q, s), gated=True)
        return cf.rms_norm_quantize(down(q, s), nw, residual=h, int8=True)

    def plain(x, r):
        def back(q, s):
            return q.double() * s.double()[:, None]

        h = x.double() + r.double()
        q, s, _ = cf.rms_norm_quantize(x, nw, residual=r, int8=True)
        v = h / torch.sqrt(h.pow(2).mean(1, keepdim=True) + 1e-6) * nw.double()
        assert bool(((back(q, s) - v).abs() <= s.double()[:, None] * 0.501).all())   # half a step
        a = (back(q, s) @ back(*cf.quantize_rows(w1)).T).to(BF16)
        gate, u = a.double().chunk(2, 1)
        v = gate * torch.sigmoid(gate) * u
        q, s = cf.quantize_rows(a, gated=True)
        assert bool(((back(q, s) - v).abs() <= s.double()[:, None] * 0.501).all())
        return h + (back(q, s) @ back(*cf.quantize_rows(w2)).T).to(BF16).double()

    q, s, h = layer(x, r)
    # a bf16 result next to a border may be rounded the other way; each of those moves a sum by a step of it
    ref = plain(x, r)
    assert float((h.double() - ref).norm() / ref.norm()) < 2.0 ** -9
    graph = torch.cuda.CUDAGraph()
    xs = torch.zeros_like(x)
    with torch.cuda.graph(graph):
        got = layer(xs, r)
    xs.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (q, s, h)))
