"""The block-scaled operators on the GPU against the formulas in 64 bits: quantising to e4m3, the
linear layer, and one layer per expert over ragged rows.

Tolerances of the products.  Every product of two e4m3 or two bf16 values is exact in float32.  A
sum of n terms in float32, each step off by at most 2^-23 of what it adds up (truncation included),
is off by at most n 2^-23 S with S the sum of the terms' magnitudes; e4m3 sums take 128 terms, then
the blocks, two scales and a bias, bf16 sums K terms and a bias.  A bf16 result (8 significant
bits) is rounded once, to nearest: 2^-8 of its magnitude more.  Integer cases, whose every sum is exact, have to be equal."""
import pytest
import torch

import convolution_onnx_conv_gb300 as cf
from convolution_onnx_conv_gb300 import _binding

pytestmark = pytest.mark.gpu
U = 2.0 ** -23


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows16(t, pad=0):
    """t with rows a multiple of 16 bytes apart (and `pad` such steps more), NaN between the rows."""
    step = 16 // t.element_size()
    wide = (-(-t.shape[-1] // step) + pad) * step
    if t.element_size() == 1:
        b = torch.full((*t.shape[:-1], wide), 0x7F, dtype=torch.uint8, device=t.device)
        b[..., : t.shape[-1]] = t.view(torch.uint8)
        return b.view(t.dtype)[..., : t.shape[-1]]
    b = torch.full((*t.shape[:-1], wide), float("nan"), dtype=t.dtype, device=t.device)
    b[..., : t.shape[-1]] = t
    return b[..., : t.shape[-1]]


def e4m3_64(t):
    t = t.clamp(-448, 448)
    _, e = torch.frexp(t)
    step = ((e.long() - 1).clamp(min=-6) - 3 + 1023 << 52).view(torch.float64)   # 2^(exponent - 3)
    return torch.round(t / step) * step


def quantised_64(v, tall=1):
    """(values, scales) by the definition: the scale and the quotient are float32 numbers."""
    rows, cols = v.shape
    nb = -(-cols // 128)
    q = torch.zeros_like(v)
    s = torch.zeros((-(-rows // tall), nb), dtype=torch.float64, device=v.device)
    for b in range(nb):
        c = v[:, b * 128:(b + 1) * 128]
        m = c.abs().amax(1)
        m = torch.nn.functional.pad(m, (0, -rows % tall)).view(-1, tall).amax(1)
        m = (m / 448).float().double()
        s[:, b] = m
        m = m.repeat_interleave(tall)[:rows, None]
        q[:, b * 128:(b + 1) * 128] = torch.where(m == 0, 0.0, e4m3_64((c / m).float().double()))
    return q, s


def e4m3_randn(g, *shape):
    return (torch.randn(shape, generator=g, device="cuda") * 40).clamp(-448, 448).to(torch.float8_e4m3fn)


def spread(s, k):
    return s.double().repeat_interleave(128, -1)[..., :k]


# ------------------------------------------------------------------------------ quantising

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 129), (5, 2048), (17, 7), (128, 200), (1000, 1000), (40001, 64)])
def test_quantise_rows(rows, cols, dtype):
    x = (torch.randn((rows, cols), generator=gen(rows + cols), device="cuda") * 3).to(dtype)
    x[rows // 2] = 0
    q, s = cf.quantize_blocks(x)
    rq, rs = quantised_64(x.double())
    assert q.stride(0) % 16 == 0 or rows == 1
    assert torch.equal(s.double(), rs) and torch.equal(q.double(), rq)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (127, 128), (128, 129), (129, 127), (300, 1000), (1025, 2056)])
def test_quantise_tiles(rows, cols, dtype):
    x = torch.randn((rows, cols), generator=gen(rows), device="cuda").to(dtype)
    q, s = cf.quantize_blocks(x, block_rows=128)
    rq, rs = quantised_64(x.double(), 128)
    assert torch.equal(s.double(), rs) and torch.equal(q.double(), rq)


@pytest.mark.parametrize("offset,ld", [(0, 300), (1, 300), (8, 304), (3, 301)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantise_any_alignment_and_stride(offset, ld, dtype, block_rows):
    rows, cols = 37, 280
    buf = torch.randn(rows * ld + 16, generator=gen(ld), device="cuda").to(dtype)
    x = torch.as_strided(buf, (rows, cols), (ld, 1), offset)
    qb = torch.full((rows * ld + 16,), 0x55, dtype=torch.uint8, device="cuda")
    q = torch.as_strided(qb, (rows, cols), (ld, 1), offset).view(torch.float8_e4m3fn)
    sb = torch.full((rows, 5), -1.0, device="cuda")
    n = -(-rows // block_rows)
    cf.quantize_blocks(x, q=q, scale=sb[:n, :3], block_rows=block_rows)
    rq, rs = quantised_64(x.double(), block_rows)
    assert torch.equal(sb[:n, :3].double(), rs) and torch.equal(q.double(), rq)
    assert bool((sb[:, 3:] == -1).all()) and bool((sb[n:] == -1).all())   # nothing past the outputs
    keep = torch.ones_like(qb, dtype=torch.bool)
    torch.as_strided(keep, (rows, cols), (ld, 1), offset).fill_(False)
    assert bool((qb[keep] == 0x55).all())


def test_quantise_gathers_and_pads():
    x = torch.randn((50, 300), generator=gen(1), device="cuda").to(torch.bfloat16)
    index = torch.randint(0, 50, (333,), generator=gen(2), device="cuda", dtype=torch.int32)
    bad = torch.tensor([-1, 50, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    index[[0, 7, 100, 332]] = bad
    q, s = cf.quantize_blocks(x, index=index)
    ok = (index >= 0) & (index < 50)
    v = torch.where(ok[:, None], x[index.long().clamp(0, 49)].double(), 0.0)
    rq, rs = quantised_64(v)
    assert torch.equal(q.double(), rq) and torch.equal(s.double(), rs)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (9, 130), (300, 515), (64, 2048)])
def test_quantise_gated(rows, cols, dtype):
    x = (torch.randn((rows, 2 * cols), generator=gen(rows), device="cuda") * 4).to(dtype)
    x[0, 0] = -300.0   # exp overflows: the gate is shut
    q, s = cf.quantize_blocks(x, gated=True)
    g, u = x.double().chunk(2, 1)
    v = g / (1 + torch.exp(-g)) * u
    _, rs = quantised_64(v)
    # float32: exp within 2 ulp, a sum, a quotient and a product; the value then moves by at most
    # half a step of e4m3 (2^-4 of it, or 2^-10 below the smallest normal) and those few ulp; what
    # is below float32's smallest number is zero
    assert bool(((s.double() - rs).abs() <= 8 * U * rs).all())
    back = q.double() * spread(s, cols)
    half = torch.maximum(v.abs() * 2.0 ** -4, spread(s, cols) * 2.0 ** -10)
    assert bool(((back - v).abs() <= half * (1 + 2.0 ** -10) + 16 * U * v.abs() + 2.0 ** -149).all())


def test_quantise_gated_where_the_gate_is_almost_shut():
    # exp(-g) between 2^126 and 2^128; the other factor makes normal numbers of the products
    x = torch.empty((4, 256), device="cuda")
    x[:, :128] = torch.linspace(-88.6, -87.4, 512, device="cuda").view(4, 128)
    x[:, 128:] = 1e30
    q, s = cf.quantize_blocks(x, gated=True)
    g, u = x.double().chunk(2, 1)
    v = g / (1 + torch.exp(-g)) * u
    _, rs = quantised_64(v)
    # exp(g) is held in steps of 2^-149, at least 2^21 of them; its 2 ulp, and a few roundings
    assert bool(((s.double() - rs).abs() <= 2.0 ** -19 * rs).all())
    back = q.double() * spread(s, 128)
    half = torch.maximum(v.abs() * 2.0 ** -4, spread(s, 128) * 2.0 ** -10)
    assert bool(((back - v).abs() <= half * (1 + 2.0 ** -10) + 2.0 ** -19 * v.abs()).all())


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantise_extremes(block_rows):
    x = torch.zeros((130, 256), device="cuda")
    x[0, 5] = float("nan")
    x[129, 200] = float("inf")
    x[1, :128] = 1e-45          # the scale underflows to zero
    x[2, :128] = -3.0e38
    x[3, 130] = -0.0
    q, s = cf.quantize_blocks(x, block_rows=block_rows)
    back = q.float() * (s.repeat_interleave(128, 1) if block_rows == 1 else
                        s.repeat_interleave(128, 0)[:130].repeat_interleave(128, 1))
    assert bool(back[0, :128].isnan().all())
    assert bool(back[129, 128:].isnan().any()) and bool(s[-1, 1].isinf())
    if block_rows == 1:
        assert bool((q[1].float() == 0).all()) and float(s[1, 0]) == 0
        assert bool((q[2, :128].float() == -448).all())
        assert bool((back[3:129] == 0).all())


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantise_tiny_bf16(block_rows):
    """Values and scales among float32's subnormal numbers."""
    x = (torch.randn((130, 300), generator=gen(3), device="cuda").double() * 2.0 ** torch.arange(-130, 0, device="cuda")[:, None])
    x = x.to(torch.bfloat16)
    x[0, :128] = 2.0 ** -133   # bf16's smallest
    q, s = cf.quantize_blocks(x, block_rows=block_rows)
    rq, rs = quantised_64(x.double(), block_rows)
    assert torch.equal(q.double(), rq) and torch.equal(s.double(), rs)


def test_quantise_next_to_the_boundaries():
    """Every value v whose quotient by a scale that occurs is within 2^-41 of the middle between two
    floats next to a boundary between two e4m3 values (a quotient that is off rounds to the wrong one)."""
    m = torch.arange(1 << 23, 1 << 24, device="cuda").double()
    scale = (m / 448).float().double()
    f, e = torch.frexp(scale)
    S, unit = (f * 2.0 ** 24).long(), torch.ldexp(torch.ones((), dtype=torch.float64), (e - 24).cpu()).cuda()
    rows = []
    for top in range(16, 32):                                # e4m3 values and their middles, in sixteenths
        for side in (2, -2 if top > 16 else -1):             # half a float's step up and down
            P = S * ((top << 21) + side)                     # scale times the middle
            j = torch.where(P < 1 << 49, 25, 26)
            V = (P + (torch.ones_like(P) << (j - 1))) >> j   # the nearest float v
            at = ((P - (V << j)).abs() <= 512).nonzero()[:, 0]
            v = V[at].double() * (1 << (j[at] - 25)).double() * unit[at]
            rows.append(torch.stack([m[at], v], 1))
    rows = torch.cat(rows)
    assert len(rows) > 1000 and bool((rows == rows.float().double()).all())
    x = rows.float()
    x = torch.cat([x, torch.nextafter(x[:, 1:], x[:, :1]), torch.nextafter(x[:, 1:], 0 * x[:, :1]), -x[:, 1:]], 1)
    q, s = cf.quantize_blocks(x)
    rq, rs = quantised_64(x.double())
    assert torch.equal(q.double(), rq) and torch.equal(s.double(), rs)


def test_quantise_no_rows():
    q, s = cf.quantize_blocks(torch.empty((0, 200), device="cuda"))
    assert q.shape == (0, 200) and s.shape == (0, 2)


# ------------------------------------------------------------------------------ products

def layer_inputs(g, rows, experts, n, k, e4m3):
    if e4m3:
        x, w = e4m3_randn(g, rows, k), e4m3_randn(g, experts, n, k)
        kb = -(-k // 128)
        xs = torch.rand((rows, kb), generator=g, device="cuda") + 0.01
        ws = torch.rand((experts, -(-n // 128), kb), generator=g, device="cuda") / 64 + 1e-4
    else:
        x = torch.randn((rows, k), generator=g, device="cuda").to(torch.bfloat16)
        w = torch.randn((experts, n, k), generator=g, device="cuda").to(torch.bfloat16)
        xs = ws = None
    return x, w, xs, ws


def real64(x, w, xs, ws):
    """Double operands: x [rows][k], w [experts][n][k]."""
    n, k = w.shape[1:]
    x, w = x.double(), w.double()
    if xs is not None:
        x = x * spread(xs, k)
        w = w * spread(ws, k).repeat_interleave(128, 1)[:, :n]
    return x, w


def check(y, ref, size, k, e4m3, out_bf16):
    n = (128 + -(-k // 128) + 4) if e4m3 else k + 2
    tol = n * U * size
    if out_bf16:
        tol = tol + (ref.abs() + tol) * 2.0 ** -8
    else:
        tol = tol + ref.abs() * 2.0 ** -24
    d = (y.double() - ref).abs()
    assert bool((d <= tol).all()), f"worst {float((d / tol).max()):.3g} of its allowance"


SIZES = [(1, 1, 1), (1, 128, 128), (1, 1000, 2048), (2, 130, 129), (7, 5, 16), (16, 256, 640), (17, 100, 100),
         (33, 129, 2100), (64, 64, 64), (65, 1000, 257), (129, 300, 1000), (300, 513, 384), (1025, 136, 520),
         (515, 1040, 4096), (2050, 2100, 300)]


@pytest.mark.parametrize("rows,n,k", SIZES)
@pytest.mark.parametrize("e4m3", [True, False])
def test_linear(rows, n, k, e4m3):
    g = gen(rows * 7 + n + k)
    x, w, xs, ws = layer_inputs(g, rows, 1, n, k, e4m3)
    bias = torch.randn((n,), generator=g, device="cuda")
    rx, rw = real64(x, w, xs, ws)
    ref = rx @ rw[0].T + bias.double()
    size = rx.abs() @ rw[0].abs().T + bias.abs().double()
    ws0 = None if ws is None else ws[0]
    for out_bf16 in (False, True):
        lin = cf.BlockLinear(rows16(w)[0], ws0, bias=bias, out_bf16=out_bf16)
        y = lin(rows16(x), xs)
        torch.cuda.synchronize()
        assert lin.status() == cf.CONVF_OK, cf.conv_fused_last_error()
        check(y, ref, size, k, e4m3, out_bf16)
        assert torch.equal(y, lin(rows16(x), xs))   # bit for bit
        lin.close()


@pytest.mark.parametrize("rows,n,k", [(1, 40, 256), (12, 200, 384), (70, 260, 1000), (400, 520, 640), (1030, 600, 1152)])
@pytest.mark.parametrize("e4m3", [True, False])
def test_linear_is_exact_on_integers(rows, n, k, e4m3):
    g = gen(rows + n)
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    x = torch.randint(-8, 9, (rows, k), generator=g, device="cuda").float()
    w = torch.randint(-4, 5, (n, k), generator=g, device="cuda").float()
    kb = -(-k // 128)
    xs = 2.0 ** torch.randint(-2, 3, (rows, kb), generator=g, device="cuda").float() if e4m3 else None
    ws = 2.0 ** torch.randint(-2, 3, (-(-n // 128), kb), generator=g, device="cuda").float() if e4m3 else None
    rx, rw = real64(x, w[None], xs, None if ws is None else ws[None])
    lin = cf.BlockLinear(rows16(w.to(dt)), ws)
    assert torch.equal(lin(rows16(x.to(dt)), xs).double(), rx @ rw[0].T)


COUNTS = [[5], [0, 0, 0], [0, 9, 0], [1, 1, 1, 1], [130, 0, 1, 0, 64, 300], [16, 17, 15, 33, 0, 128, 129],
          [700, 3, 0, 0, 900], [1] * 70, [0] * 200 + [40] + [0] * 100, [2, 0, 1, 3] * 16]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}e{sum(c)}r")
@pytest.mark.parametrize("n,k", [(130, 200), (264, 1100)])
@pytest.mark.parametrize("e4m3", [True, False])
def test_experts(counts, n, k, e4m3):
    before, after = 3, 5   # rows that no expert takes
    e, rows = len(counts), sum(counts) + before + after
    g = gen(sum(counts) + n)
    x, w, xs, ws = layer_inputs(g, rows, e, n, k, e4m3)
    off = torch.tensor([0] + counts).cumsum(0) + before
    bias = torch.randn((e, n), generator=g, device="cuda")
    rx, rw = real64(x, w, xs, ws)
    out_bf16 = len(counts) % 2 == 0
    lin = cf.ExpertLinear(rows16(w), ws, bias=bias, out_bf16=out_bf16, act=cf.CONVF_ACT_RELU)
    y = torch.full((rows, n + 3), -7.0, dtype=lin.out_dtype, device="cuda")
    x16 = rows16(x, pad=1)
    doff = off.to(torch.int32).cuda()
    lin(x16, doff, xs, y=y[:, :n])
    torch.cuda.synchronize()
    assert lin.status() == cf.CONVF_OK, cf.conv_fused_last_error()
    assert bool((y[:, n:] == -7).all()) and bool((y[:before] == -7).all()) and bool((y[rows - after:] == -7).all())
    for i in range(e):
        a, b = int(off[i]), int(off[i + 1])
        if a < b:
            ref = rx[a:b] @ rw[i].T + bias[i].double()
            size = rx[a:b].abs() @ rw[i].abs().T + bias[i].abs().double()
            check(y[a:b, :n], ref.clamp(min=0), size, k, e4m3, out_bf16)
    y2 = torch.full_like(y, -7.0)
    lin(x16, doff, xs, y=y2[:, :n])
    assert torch.equal(y, y2)


@pytest.mark.parametrize("act,clip,lo,hi", [(cf.CONVF_ACT_RELU6, (0, 0), 0.0, 6.0), (cf.CONVF_ACT_CLIP, (-2.5, 3.0), -2.5, 3.0)])
def test_activation_clamps(act, clip, lo, hi):
    g = gen(4)
    x, w, xs, ws = layer_inputs(g, 40, 1, 70, 256, True)
    rx, rw = real64(x, w, xs, ws)
    lin = cf.BlockLinear(w[0], ws[0], act=act, clip=clip)
    check(lin(x, xs), (rx @ rw[0].T).clamp(lo, hi), rx.abs() @ rw[0].abs().T, 256, True, False)


@pytest.mark.parametrize("rows", [9, 300, 700])
def test_scale_strides_and_a_nan_stay_in_their_row(rows):
    g = gen(rows)
    n, k = 300, 1000
    x, w, xs, ws = layer_inputs(g, rows, 1, n, k, True)
    lin = cf.BlockLinear(rows16(w)[0], ws[0], act=cf.CONVF_ACT_RELU)
    y = lin(rows16(x), xs)
    turned = xs.t().contiguous().t()           # block by block
    wide = torch.full((rows, 2 * xs.shape[1]), float("nan"), device="cuda")[:, ::2]
    wide.copy_(xs)
    assert torch.equal(lin(rows16(x), turned), y) and torch.equal(lin(rows16(x), wide), y)
    xs2 = xs.clone()
    xs2[rows // 2, 3] = float("nan")
    z = lin(rows16(x), xs2)
    assert bool(z[rows // 2].isnan().all())
    z[rows // 2] = y[rows // 2]
    assert torch.equal(z, y)


def test_bad_offsets_are_reported_and_reach_nothing_else():
    g = gen(3)
    x, w, xs, ws = layer_inputs(g, 64, 4, 96, 256, True)
    lin = cf.ExpertLinear(w, ws)
    for off in ([0, 30, 20, 40, 64], [-5, 10, 20, 30, 64], [0, 10, 20, 30, 99], [2 ** 31 - 1, 0, -2 ** 31, 5, 64]):
        buf = torch.full((66, 96), -7.0, device="cuda")
        lin(x, torch.tensor(off, dtype=torch.int32, device="cuda"), xs, y=buf[1:65])
        torch.cuda.synchronize()
        assert lin.status() == cf.CONVF_ERR_INVALID_ARG and "offsets" in cf.conv_fused_last_error()
        assert bool((buf[0] == -7).all()) and bool((buf[65] == -7).all())
        lin.clear_status()
    y = lin(x, torch.tensor([0, 10, 20, 30, 64], dtype=torch.int32, device="cuda"), xs)
    torch.cuda.synchronize()
    assert lin.status() == cf.CONVF_OK and bool(y.isfinite().all())


def test_stream_0_is_the_default_stream(monkeypatch):
    x, w, xs, ws = layer_inputs(gen(3), 5, 1, 64, 256, True)
    lin = cf.BlockLinear(w[0], ws[0])
    names, seen = _binding._Torch, []
    run, quantize = names.run, names.quantize
    monkeypatch.setattr(names, "run", lambda layer, args, stream: seen.append(stream) or run(layer, args, stream))
    monkeypatch.setattr(names, "quantize", lambda args, stream: seen.append(stream) or quantize(args, stream))
    with torch.cuda.stream(torch.cuda.Stream()):
        y = lin(x, xs, stream=0)
        cf.quantize_blocks(y, stream=0)
    torch.cuda.synchronize()
    assert seen == [0, 0] and torch.equal(y, lin(x, xs))


def test_other_stream_and_graph():
    g = gen(8)
    x, w, xs, ws = layer_inputs(g, 70, 3, 260, 640, True)
    off = torch.tensor([0, 20, 20, 70], dtype=torch.int32, device="cuda")
    lin = cf.ExpertLinear(w, ws, out_bf16=True)
    want = lin(x, off, xs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = torch.zeros_like(want)
    with torch.cuda.stream(side):
        x2 = torch.zeros_like(x)
        x2.view(torch.uint8).copy_(x.view(torch.uint8))   # the producer, on this stream
        lin(x2, off, xs, y=y)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)
    for stream in (side, side.cuda_stream):   # given: it writes outputs of its own
        side.wait_stream(torch.cuda.current_stream())
        z = lin(x, off, xs, stream=stream)
        a, b = cf.quantize_blocks(z, stream=stream)
        torch.cuda.current_stream().wait_stream(side)
        c, d = cf.quantize_blocks(want)
        assert torch.equal(z, want) and torch.equal(a.view(torch.uint8), c.view(torch.uint8)) and torch.equal(b, d)
    src = torch.randn((70, 640), generator=g, device="cuda").to(torch.bfloat16)
    q = torch.empty((70, 640), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((70, 5), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cf.quantize_blocks(src, q=q, scale=s)
        lin(q, off, s, y=y)
    for k in range(3):
        src.normal_(generator=g)
        graph.replay()
        assert torch.equal(y, lin(*[(t[0], off, t[1]) for t in [cf.quantize_blocks(src)]][0]))


def test_rows_far_apart():
    """x, y and their offsets in bytes pass 2^31 (and the weights' 2^32)."""
    rows, n, k = 3, 144, 256
    g = gen(12)
    ld = (1 << 30) + 32
    big = torch.zeros((rows - 1) * ld + k, dtype=torch.bfloat16, device="cuda")
    x, w, _, _ = layer_inputs(g, rows, 3, n, k, False)
    xv = torch.as_strided(big, (rows, k), (ld, 1))
    xv.copy_(x)
    wbig = torch.zeros(2 * ((1 << 30) + 64) + n * k, dtype=torch.bfloat16, device="cuda")
    wv = torch.as_strided(wbig, (3, n, k), ((1 << 30) + 64, k, 1))
    wv.copy_(w)
    off = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    lin = cf.ExpertLinear(wv)
    want = cf.ExpertLinear(w)(x, off)
    assert torch.equal(lin(xv, off), want)
    ybig = torch.zeros((rows - 1) * (1 << 29) + n, device="cuda")
    lin(xv, off, y=torch.as_strided(ybig, (rows, n), (1 << 29, 1)))
    assert torch.equal(torch.as_strided(ybig, (rows, n), (1 << 29, 1)), want)
    q, s = cf.quantize_blocks(xv)
    q2, s2 = cf.quantize_blocks(x)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)


def test_refusals_on_tensors():
    w = torch.zeros((2, 32, 64), dtype=torch.bfloat16, device="cuda")
    x = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    lin = cf.ExpertLinear(w)
    with pytest.raises(ValueError):
        lin(x[:, :32], off)
    with pytest.raises(ValueError):
        lin(x.float(), off)
    with pytest.raises(ValueError):
        lin(x, off.long())
    with pytest.raises(ValueError):
        lin(x, off[:2])
    with pytest.raises(ValueError):
        lin(x, off, torch.zeros((8, 1), device="cuda"))
    with pytest.raises(ValueError):
        lin(x, off, y=torch.zeros((8, 32), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(cf.ConvFusedError) as e:
        lin(torch.zeros((8, 67), dtype=torch.bfloat16, device="cuda")[:, :64], off)
    assert e.value.status == cf.CONVF_ERR_UNSUPPORTED and "16 bytes" in str(e.value)
    with pytest.raises(cf.ConvFusedError) as e:
        lin(torch.zeros(8 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(8, 64), off)
    assert e.value.status == cf.CONVF_ERR_INVALID_ARG and "16-byte" in str(e.value)
    both = torch.zeros((8, 96), dtype=torch.float32, device="cuda")
    with pytest.raises(cf.ConvFusedError) as e:
        lin(both.view(torch.bfloat16)[:, :64], off, y=both[:, :32])
    assert "overlap" in str(e.value)
    with pytest.raises(ValueError):
        cf.ExpertLinear(w.float())
    with pytest.raises(ValueError):
        cf.ExpertLinear(w.to(torch.float8_e4m3fn))
    with pytest.raises(ValueError):
        cf.BlockLinear(w)
    with pytest.raises(ValueError):
        cf.quantize_blocks(x.half())
    with pytest.raises(ValueError):
        cf.quantize_blocks(x, index=off.long())
    with pytest.raises(cf.ConvFusedError):
        cf.quantize_blocks(x, index=off, block_rows=128)
    with pytest.raises(cf.ConvFusedError):
        cf.quantize_blocks(x, block_rows=64)


def test_create_reports_an_injected_device_allocation_failure():
    w = torch.zeros((32, 64), dtype=torch.bfloat16, device="cuda")
    cf.conv_fused_debug_fail_alloc(2)   # the layer, then its device words
    with pytest.raises(cf.ConvFusedError) as e:
        cf.BlockLinear(w)
    assert e.value.status == cf.CONVF_ERR_OOM and "(injected)" in str(e.value)
    x = torch.ones((3, 64), dtype=torch.bfloat16, device="cuda")
    assert torch.equal(cf.BlockLinear(w)(x), torch.zeros((3, 32), device="cuda"))


# ------------------------------------------------------------------------------ every kernel form

FORMS = ["few_rows tile=16x128 split=1", "few_rows tile=16x128 split=4", "few_rows tile=32x128 split=1",
         "few_rows tile=64x128 split=1", "many_rows tile=128x256", "many_rows tile=256x256"]
SEARCH = [(r, e, n, k) for e in (1, 3, 9, 33) for k in (1040, 2064, 130, 4112) for n in (1032, 2061, 4100)
          for r in (1, 9, 30, 61, 130, 300, 530, 1061, 2100, 4333)]


def layer_of_form(form, e4m3, dtype):
    """(layer, rows, experts, n, k) of the first size whose plan is `form`."""
    for r, e, n, k in SEARCH:
        w = torch.zeros((e, n, -(-k // 16) * 16), dtype=dtype, device="cuda")[:, :, :k]
        ws = torch.zeros((e, -(-n // 128), -(-k // 128)), device="cuda") if e4m3 else None
        for out_bf16 in (True, False):
            lin = cf.ExpertLinear(w, ws, out_bf16=out_bf16)
            if form in lin.describe(r):
                return lin, r, e, n, k
            lin.close()
    pytest.fail(f"no size of the search runs {form}")


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("e4m3", [True, False])
def test_every_form_is_exact_on_integers(form, e4m3):
    """Integers whose sums are exact: each form at ragged sizes, with its own bias, clamp and row stride."""
    dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    lin, rows, e, n, k = layer_of_form(form, e4m3, dtype)
    g = gen(rows + n)
    x = torch.randint(-4, 5, (rows, k), generator=g, device="cuda").float()
    w = torch.randint(-2, 3, (e, n, k), generator=g, device="cuda").float()
    kb = -(-k // 128)
    xs = 2.0 ** torch.randint(-1, 2, (rows, kb), generator=g, device="cuda").float() if e4m3 else None
    ws = 2.0 ** torch.randint(-1, 2, (e, -(-n // 128), kb), generator=g, device="cuda").float() if e4m3 else None
    bias = torch.randint(-3, 4, (e, n), generator=g, device="cuda").float()
    cuts = [rows * (i + 1) // e for i in range(e - 1)]
    off = torch.tensor([0] + cuts + [rows], dtype=torch.int32, device="cuda")
    rx, rw = real64(x, w, xs, ws)
    ref = torch.empty((rows, n), dtype=torch.float64, device="cuda")
    for i in range(e):
        a, b = int(off[i]), int(off[i + 1])
        ref[a:b] = rx[a:b] @ rw[i].T
    x16, w16 = rows16(x.to(dtype)), rows16(w.to(dtype))
    for out_bf16 in (False, True):
        out = torch.bfloat16 if out_bf16 else torch.float32
        for b, act, clip in ((None, cf.CONVF_ACT_NONE, (0, 0)), (bias, cf.CONVF_ACT_NONE, (0, 0)),
                             (None, cf.CONVF_ACT_CLIP, (-3.0, 5.5)), (bias, cf.CONVF_ACT_RELU, (0, 0))):
            want = ref.clone()
            if b is not None:
                for i in range(e):
                    want[int(off[i]):int(off[i + 1])] += b[i].double()
            if act == cf.CONVF_ACT_RELU:
                want = want.clamp(min=0)
            elif act == cf.CONVF_ACT_CLIP:
                want = want.clamp(*clip)
            layer = cf.ExpertLinear(w16, ws, bias=b, act=act, clip=clip, out_bf16=out_bf16)
            for pad, shift in ((0, 0), (8, 0), (1, 1)):   # rows of y side by side, 16-byte aligned apart, and unaligned
                buf = torch.full((rows * (n + pad) + 8,), -7.0, dtype=out, device="cuda")
                y = torch.as_strided(buf, (rows, n), (n + pad, 1), shift)
                layer(x16, off, xs, y=y)
                assert torch.equal(y.double(), want.to(out).double()), (out_bf16, b is not None, act, pad)
                y.fill_(-7.0)
                assert bool((buf == -7).all())   # nothing beside y
            assert layer.status() == cf.CONVF_OK, cf.conv_fused_last_error()
            layer.close()
    torch.cuda.synchronize()
    lin.close()
