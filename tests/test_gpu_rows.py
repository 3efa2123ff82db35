"""Rows to int8 with a scale each, and the root-mean-square norm in front of 8-bit values, on the GPU against the
definitions in 64 bits.

What is equal and what is near.  The 8-bit values follow from float32 operations that are each rounded to nearest
(sum, product, quotient), so they are equal to the definition's, element for element; a quotient of two float32
numbers in 64 bits, rounded to float32, is the float32 quotient.  The norm's factor is not so defined: its sum of
`cols` squares adds in an order of its own, with one rounding of 2^-24 for each step of a chain of at most
cols / 1024 * 16 + 64 additions (16 columns of a thread for every 16 * 512 columns, then the threads' sums); mean, eps,
root and two products add five more.  Gated values: expf is within 2 units in the last place (2^-22), the sum, the
quotient and the product round once each, 2^-20 in all with room for the quotient by the scale."""
import pytest
import torch

import convolution_onnx_conv_gb300 as cf
from test_gpu_linear import quantised_64

pytestmark = pytest.mark.gpu
BF16, F32, I8, E4M3 = torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(seed, *shape, dtype=F32):
    return torch.randn(shape, generator=gen(seed), device="cuda").to(dtype)


def int8_64(v):
    """(values, scales) of float32 rows `v`, given in 64 bits."""
    s = (v.abs().amax(1) / 127).float().double()
    q = torch.round((v / s[:, None]).float().double()).clamp(-127, 127)
    return torch.where(s[:, None] == 0, 0.0, q), s


def near_scale(got, s0, f, cols):
    ref = s0 * f
    assert bool(((got.double() - ref).abs() <= (cols / 64 + 80) * 2.0 ** -24 * ref).all())


def check_norm(x, w, eps, res, int8, out):
    """`out` of rms_norm_quantize against the definition."""
    h = x.float() if res is None else x.float() + res.float()
    t = (h if w is None else h * w.float()).double()
    h = h.double()
    f = 1 / torch.sqrt(h.pow(2).mean(1) + eps)
    if res is not None:
        assert out[2].dtype is res.dtype and torch.equal(out[2], h.to(res.dtype))
    if int8:
        q, s0 = int8_64(t)
    else:
        q, s0 = quantised_64(t)
        f = f[:, None]
    assert out[0].dtype is (I8 if int8 else E4M3) and torch.equal(out[0].double(), q)
    near_scale(out[1], s0, f, x.shape[1])


# ------------------------------------------------------------------------------ int8 rows

COLS = [1, 7, 128, 129, 512, 513, 2048, 2049, 4096, 4100, 8192, 8193, 20001]   # both sides of every width's kernel


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", COLS)
def test_rows(cols, dtype):
    for rows in (1, 5, 1300 if cols < 3000 else 700):
        x = randn(cols + rows, rows, cols, dtype=dtype) * 3
        x[rows // 2] = 0
        q, s = cf.quantize_rows(x)
        rq, rs = int8_64(x.double())
        assert q.stride(0) % 16 == 0 or rows == 1
        assert torch.equal(s.double(), rs) and torch.equal(q.double(), rq)


def test_rows_at_half_integers():
    """Quotients on and next to n + 1/2: scale 1 and powers of two, and scales of full length."""
    n = torch.arange(-127, 127, device="cuda").float() + 0.5
    for top in (127.0, 127.0 * 1024, 127 * 2.0 ** -30, 126.99999, 100.0, 3.3333333, 1e-3, 7e20, 3e-38):
        s = torch.tensor(top, device="cuda") / 127
        v = n * s
        x = torch.stack([v, torch.nextafter(v, torch.full_like(v, 1e30)), torch.nextafter(v, torch.full_like(v, -1e30))])
        x = torch.cat([x, torch.full((3, 1), top, device="cuda")], 1)
        q, s = cf.quantize_rows(x)
        rq, rs = int8_64(x.double())
        assert torch.equal(s.double(), rs) and torch.equal(q.double(), rq), top


def test_rows_of_every_scale():
    """Random significands: scales over float32's range, subnormal ones and those that underflow among them."""
    m = randn(1, 4000, 40).abs() + 0.5
    e = torch.randint(-149, 127, (4000, 1), generator=gen(2), device="cuda")
    x = torch.ldexp(m, e) * torch.sign(randn(3, 4000, 40))
    x = x.clamp(-3e38, 3e38)
    q, s = cf.quantize_rows(x)
    rq, rs = int8_64(x.double())
    assert torch.equal(s.double(), rs) and torch.equal(q.double(), rq)


def test_rows_that_are_no_numbers():
    x = randn(4, 6, 300)
    x[1, 7], x[2, 299], x[3, 0], x[4, 5] = float("nan"), float("inf"), -float("inf"), float("nan")
    x[4, 6] = float("inf")
    q, s = cf.quantize_rows(x)
    back = q.float() * s[:, None]
    assert bool(torch.isnan(back[1:5]).all()) and bool((q[1:5] == 0).all())
    rq, rs = int8_64(x[[0, 5]].double())
    assert torch.equal(q[[0, 5]].double(), rq) and torch.equal(s[[0, 5]].double(), rs)


@pytest.mark.parametrize("offset,ld", [(0, 300), (1, 300), (8, 304), (3, 301), (4, 320)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_any_alignment_and_stride(offset, ld, dtype):
    rows, cols = 37, 280
    x = torch.as_strided(randn(ld, rows * ld + 16, dtype=dtype), (rows, cols), (ld, 1), offset)
    qb = torch.full((rows * ld + 16,), 0x55, dtype=I8, device="cuda")
    q = torch.as_strided(qb, (rows, cols), (ld, 1), offset)
    sb = torch.full((rows + 2,), -1.0, device="cuda")
    cf.quantize_rows(x, q=q, scale=sb[1:-1])
    rq, rs = int8_64(x.double())
    assert torch.equal(sb[1:-1].double(), rs) and torch.equal(q.double(), rq)
    assert bool((sb[[0, -1]] == -1).all())
    keep = torch.ones_like(qb, dtype=torch.bool)
    torch.as_strided(keep, (rows, cols), (ld, 1), offset).fill_(False)
    assert bool((qb[keep] == 0x55).all())


@pytest.mark.parametrize("cols", [130, 1000, 2500, 5000, 9001])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_gathered_with_padding(cols, dtype):
    x = randn(cols, 50, cols, dtype=dtype)
    index = torch.randint(0, 50, (333,), generator=gen(5), device="cuda", dtype=torch.int32)
    index[3:6], index[330:] = -1, 50
    index[10:14] = 7   # the same row more than once
    q, s = cf.quantize_rows(x, index=index)
    ok = (index >= 0) & (index < 50)
    v = torch.where(ok[:, None], x.double()[index.long().clamp(0, 49)], 0.0)
    rq, rs = int8_64(v)
    assert torch.equal(s.double(), rs) and torch.equal(q.double(), rq)
    q, s = cf.quantize_rows(x[:0], index=index)   # no rows to take
    assert not q.any() and not s.any()


@pytest.mark.parametrize("cols", [1, 33, 512, 1000, 3001, 8192, 8200])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_gated(cols, dtype):
    x = (randn(cols, 200, 2 * cols) * 4).to(dtype)
    x[0, :cols] = -200   # gates that are shut
    x[1, :cols] = 200
    index = torch.randint(0, 200, (77,), generator=gen(6), device="cuda", dtype=torch.int32)
    for where in (None, index):
        q, s = cf.quantize_rows(x, index=where, gated=True)
        xs = (x if where is None else x[where.long()]).double()
        v = xs[:, :cols] * torch.sigmoid(xs[:, :cols]) * xs[:, cols:]
        m = v.abs().amax(1)
        live = m > 1e-30
        assert bool(((s.double() - m / 127).abs() <= 2.0 ** -20 * m / 127 + 1e-35).all())
        off = (q.double() - v / (m / 127)[:, None]).abs()[live]
        assert bool((off <= 0.5 + 127 * 2.0 ** -19).all())


# ------------------------------------------------------------------------------ norm

@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("res", [None, BF16, F32])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", COLS)
def test_norm(cols, dtype, res, int8):
    for rows in (1, 3, 1100 if cols < 3000 else 500):
        x = randn(cols + rows, rows, cols, dtype=dtype) * torch.exp(randn(rows, rows, 1)).to(dtype)
        r = None if res is None else randn(cols, rows, cols, dtype=res)
        w = (1 + randn(7, cols) / 4).to(BF16 if rows == 3 else F32)
        if rows == 3:
            x[1] = 0
            if r is not None:
                r[1] = 0
        check_norm(x, w, 1e-6, r, int8, cf.rms_norm_quantize(x, w, 1e-6, residual=r, int8=int8))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("cols", [100, 4096, 9000])
def test_norm_without_a_weight_and_with_other_eps(cols, int8):
    x = randn(8, 40, cols, dtype=BF16) * 1e-3
    for eps in (1e-6, 1.0, 1e-38):
        check_norm(x, None, eps, None, int8, cf.rms_norm_quantize(x, eps=eps, int8=int8))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("res", [BF16, F32])
@pytest.mark.parametrize("cols", [300, 2000, 3333, 8000, 8200])
def test_norm_in_place(cols, res, int8):
    """h over the residual, and over x."""
    x, r = randn(9, 300, cols, dtype=res), randn(10, 300, cols, dtype=res)
    w = randn(11, cols)
    a = r.clone()
    out = cf.rms_norm_quantize(x, w, residual=a, int8=int8, h=a)
    assert out[2] is a
    check_norm(x, w, 1e-6, r, int8, out)
    b = x.clone()
    check_norm(x, w, 1e-6, r, int8, cf.rms_norm_quantize(b, w, residual=r, int8=int8, h=b))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("res", [BF16, F32])
@pytest.mark.parametrize("cols", [512, 4096])
def test_norm_in_place_in_whole_rows(cols, res, int8):
    """As above, in rows that a kernel without checks takes, each CTA with several of them and the last asked for twice."""
    for rows in (1, 2900):
        x, r = randn(23, rows, cols, dtype=res), randn(24, rows, cols, dtype=res)
        w = randn(25, cols)
        a = r.clone()
        check_norm(x, w, 1e-6, r, int8, cf.rms_norm_quantize(x, w, residual=a, int8=int8, h=a))
        b = x.clone()
        check_norm(x, w, 1e-6, r, int8, cf.rms_norm_quantize(b, w, residual=r, int8=int8, h=b))


def test_one_row_gathered_many_times():
    x = randn(26, 9, 1000, dtype=BF16)
    index = torch.randint(0, 9, (700,), generator=gen(27), device="cuda", dtype=torch.int32)
    index[100:400] = 5
    q, s = cf.quantize_rows(x, index=index)
    rq, rs = cf.quantize_rows(x)
    assert torch.equal(q, rq[index.long()]) and torch.equal(s, rs[index.long()])


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("offset,ld", [(0, 300), (1, 300), (8, 304), (3, 301), (4, 320)])
@pytest.mark.parametrize("dtype,res", [(BF16, BF16), (BF16, F32), (F32, BF16)])
def test_norm_any_alignment_and_stride(offset, ld, dtype, res, int8):
    rows, cols = 29, 277

    def cut(seed, dtype):
        return torch.as_strided(randn(seed, rows * ld + 16, dtype=dtype), (rows, cols), (ld, 1), offset)

    x, r = cut(1, dtype), cut(2, res)
    w = randn(3, cols + 1)[1:]
    hb = torch.full((rows * ld + 16,), 3.0, dtype=res, device="cuda")
    qb = torch.full((rows * ld + 16,), 0x55, dtype=torch.uint8, device="cuda")
    keep = torch.ones_like(qb, dtype=torch.bool)
    torch.as_strided(keep, (rows, cols), (ld, 1), offset).fill_(False)
    q = torch.as_strided(qb, (rows, cols), (ld, 1), offset).view(I8 if int8 else E4M3)
    sb = torch.full((rows, 5), -1.0, device="cuda")
    scale = torch.empty(rows, device="cuda") if int8 else sb[:, :3]
    out = cf.rms_norm_quantize(x, w, 1e-5, residual=r, int8=int8, q=q, scale=scale, h=torch.as_strided(hb, (rows, cols), (ld, 1), offset))
    check_norm(x, w, 1e-5, r, int8, out)
    assert bool((qb[keep] == 0x55).all()) and bool((hb[keep] == 3).all()) and bool((sb[:, 3:] == -1).all())


def test_norm_of_rows_that_are_no_numbers():
    x = randn(12, 5, 700)
    x[1, 3], x[2, 699] = float("nan"), float("inf")
    for int8 in (False, True):
        q, s = cf.rms_norm_quantize(x, int8=int8)
        back = q.float() * (s[:, None] if int8 else s.repeat_interleave(128, 1)[:, :700])
        if int8:
            assert bool(torch.isnan(back[1]).all()) and bool(torch.isnan(back[2]).all())
        else:   # the infinity's block; the row's other values are finite, and 0 of infinitely much
            assert bool(torch.isnan(back[1]).all()) and bool(torch.isnan(back[2, 640:]).all()) and not back[2, :640].any()
        assert bool(torch.isfinite(back[[0, 3, 4]]).all())


def test_norm_repeats_bit_for_bit_and_rows_do_not_depend_on_their_neighbours():
    x, r, w = randn(13, 900, 5000, dtype=BF16), randn(14, 900, 5000, dtype=BF16), randn(15, 5000)
    a, b = (cf.rms_norm_quantize(x, w, residual=r, int8=True) for _ in range(2))
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    c = cf.rms_norm_quantize(x[123:124], w, residual=r[123:124], int8=True)
    assert all(torch.equal(u[123:124], v) for u, v in zip(a, c))


# ------------------------------------------------------------------------------ streams, graphs, no rows

def test_empty_calls():
    for x in (torch.empty((0, 40), device="cuda"), torch.empty((0, 40), dtype=BF16, device="cuda")):
        assert cf.quantize_rows(x)[0].shape == (0, 40)
        q, s, h = cf.rms_norm_quantize(x, residual=x)
        assert q.shape == (0, 40) and s.shape == (0, 1) and h.shape == (0, 40)


def test_on_another_stream_and_in_a_graph():
    x, r, w = randn(16, 64, 3000, dtype=BF16), randn(17, 64, 3000, dtype=BF16), randn(18, 3000)
    ref = (*cf.quantize_rows(x), *cf.rms_norm_quantize(x, w, residual=r), *cf.rms_norm_quantize(x, w, residual=r, int8=True))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = (*cf.quantize_rows(x, stream=stream), *cf.rms_norm_quantize(x, w, residual=r, stream=stream),
               *cf.rms_norm_quantize(x, w, residual=r, int8=True, stream=stream))
        side.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    xs = torch.zeros_like(x)
    with torch.cuda.graph(graph):
        got = (*cf.quantize_rows(xs), *cf.rms_norm_quantize(xs, w, residual=r), *cf.rms_norm_quantize(xs, w, residual=r, int8=True))
    for _ in range(2):
        xs.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(ref, got))


def test_one_call_behind_another_over_the_same_buffers():
    """Each call reads what the one before has written, many times: the residual in place through layers of rows."""
    x, w = randn(19, 200, 2000, dtype=BF16), 1 + randn(20, 2000) / 8
    r = randn(21, 200, 2000)
    ref = r.clone()
    for _ in range(20):
        ref = ref + x.float()
    for _ in range(20):
        out = cf.rms_norm_quantize(x, w, residual=r, int8=True, h=r)
    assert torch.equal(r, ref)
    check_norm(torch.zeros_like(ref), w, 1e-6, ref, True, (out[0], out[1], ref))


def test_rows_past_32_bits_of_offset():
    """The last rows of a buffer of more than 2^32 elements."""
    rows, ld = 6, 900_000_000
    buf = torch.empty(((rows - 1) * ld + 512,), dtype=BF16, device="cuda")
    x = torch.as_strided(buf, (rows, 512), (ld, 1))
    x.copy_(randn(22, rows, 512))
    q, s = cf.quantize_rows(x)
    rq, rs = int8_64(x.double())
    assert torch.equal(s.double(), rs) and torch.equal(q.double(), rq)
    check_norm(x, None, 1e-6, None, False, cf.rms_norm_quantize(x))
