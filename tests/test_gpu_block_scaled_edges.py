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


# ------------------------------------------------------------------------------ memory shared with the neighbours in the stream

@pytest.mark.parametrize("rows", [5, 40, 300])
def test_a_run_reads_what_the_runs_before_it_wrote(rows):
    """Quantiser and layer in turn over the same q, scales and index, without a wait between them: each begins
    while the one before still runs, and has to read what that one writes."""
    g, k, n = gen(rows), 640, 384
    src = [torch.randn((rows, k), generator=g, device="cuda").to(torch.bfloat16) * 4.0 ** i for i in range(4)]
    perm = [torch.randperm(rows, generator=g, device="cuda").to(torch.int32) for _ in range(4)]
    w = [torch.randn((n, k), generator=g, device="cuda") for _ in range(2)]
    wq, ws = cf.quantize_blocks(w[0], block_rows=128)
    lin = cf.BlockLinear(wq, ws, out_bf16=True)
    want = {}
    for j in range(2):
        cf.quantize_blocks(w[j], block_rows=128, q=wq, scale=ws)
        for i in range(4):
            torch.cuda.synchronize()
            a = cf.quantize_blocks(src[i], index=perm[i])
            torch.cuda.synchronize()
            want[i, j] = lin(*a)
            torch.cuda.synchronize()
    q, s = cf.quantize_blocks(src[0])
    where = torch.empty_like(perm[0])
    got = []
    for t in range(200):
        i, j = (t * 7 + t // 5) % 4, t // 3 % 2
        if t % 3 == 0:
            cf.quantize_blocks(w[j], block_rows=128, q=wq, scale=ws)   # the layer reads its weights in place
        where.copy_(perm[i])
        cf.quantize_blocks(src[i], index=where, q=q, scale=s)
        got.append((i, j, lin(q, s)))
    torch.cuda.synchronize()
    for t, (i, j, y) in enumerate(got):
        assert torch.equal(y, want[i, j]), t
    assert lin.status() == cf.CONVF_OK


# ------------------------------------------------------------------------------ offsets out of order

@pytest.mark.parametrize("rows", [64, 900])
@pytest.mark.parametrize("e4m3", [True, False])
def test_offsets_out_of_order_write_nothing(rows, e4m3):
    """The tiles of groups that overlap can be more than an int counts (every second one of 1024 experts taking
    2^27 rows), so that a run with such offsets has no tiles at all."""
    g, e, n, k = gen(rows), 5, 300, 256
    x = torch.randn((rows, k), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn((e, n, k), generator=g, device="cuda").to(torch.bfloat16)
    xs = ws = None
    if e4m3:
        x, xs = cf.quantize_blocks(x)
        parts = [cf.quantize_blocks(m, block_rows=128) for m in w]
        w = torch.stack([p[0].view(torch.uint8) for p in parts]).view(torch.float8_e4m3fn)
        ws = torch.stack([p[1] for p in parts])
    lin = cf.ExpertLinear(w, ws)
    y = torch.full((rows, n), -7.0, device="cuda")
    for off in ([0, rows, 0, rows, 0, rows], [0, 10, 20, 30, 40, rows + 1], [-1, 10, 20, 30, 40, rows], [0, 10, 9, 30, 40, rows],
                [0, 0, 0, 0, 2 ** 31 - 1, -2 ** 31]):
        lin(x, torch.tensor(off, dtype=torch.int32, device="cuda"), xs, y=y)
        torch.cuda.synchronize()
        assert lin.status() == cf.CONVF_ERR_INVALID_ARG and "offsets" in cf.conv_fused_last_error()
        lin.clear_status()
        assert bool((y == -7).all())
    lin(x, torch.tensor([0, 10, 20, 30, 40, rows], dtype=torch.int32, device="cuda"), xs, y=y)
    torch.cuda.synchronize()
    assert lin.status() == cf.CONVF_OK and bool((y != -7).all())


# ------------------------------------------------------------------------------ operands that overlap

def test_y_over_anything_that_the_run_reads_is_refused():
    e, n, k, rows = 2, 128, 256, 64
    buf = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")

    def at(byte, shape, dtype):
        size = torch.empty((), dtype=dtype).element_size()
        count = 1
        for s in shape:
            count *= s
        return buf[byte:byte + count * size].view(dtype).view(shape)

    w, ws, bias = at(0, (e, n, k), torch.float8_e4m3fn), at(65536, (e, 1, 2), torch.float32), at(66048, (e, n), torch.float32)
    x, xs, off = at(131072, (rows, k), torch.float8_e4m3fn), at(196608, (rows, 2), torch.float32), at(197632, (e + 1,), torch.int32)
    lin = cf.ExpertLinear(w, ws, bias=bias)
    size = rows * n * 4
    for name, first, length in (("weights", 0, e * n * k), ("w_scale", 65536, e * 8), ("bias", 66048, e * n * 4), ("x and", 131072, rows * k),
                                ("x_scale", 196608, rows * 8), ("offsets", 197632, (e + 1) * 4)):
        for byte in (first, first + length - 4, first - size + 4):
            if byte >= 0:
                with pytest.raises(cf.ConvFusedError) as err:
                    lin(x, off, xs, y=at(byte, (rows, n), torch.float32))
                assert err.value.status == cf.CONVF_ERR_INVALID_ARG and "overlap" in str(err.value), (name, byte)
    lin(x, off, xs, y=at(262144, (rows, n), torch.float32))


@pytest.mark.parametrize("rows", [3, 200])
def test_columns_of_one_buffer(rows):
    """x, y and a quantiser's operands as columns of the same rows, as a program that keeps its features side by
    side has them."""
    g, n, k = gen(rows), 96, 64
    w = torch.randn((n, k), generator=g, device="cuda").to(torch.bfloat16)
    lin = cf.BlockLinear(w, out_bf16=True)
    both = torch.randn((rows, k + n + 8), generator=g, device="cuda").to(torch.bfloat16)
    before = both.clone()
    want = lin(before[:, :k].contiguous())
    lin(both[:, :k], y=both[:, k:k + n])
    assert torch.equal(both[:, k:k + n], want)
    assert torch.equal(both[:, :k], before[:, :k]) and torch.equal(both[:, k + n:], before[:, k + n:])
    raw = both.view(torch.uint8)   # the quantised y in the bytes of x
    q, s = cf.quantize_blocks(want)
    out = raw[:, :n].view(torch.float8_e4m3fn)
    cf.quantize_blocks(both[:, k:k + n], q=out)
    assert torch.equal(out.view(torch.uint8), q.view(torch.uint8)) and torch.equal(both[:, k:k + n], want)
    with pytest.raises(cf.ConvFusedError):
        lin(both[:, :k], y=both[:, k - 8:k - 8 + n])


# ------------------------------------------------------------------------------ long reductions

def half_step(t):
    """Half the distance between bf16 numbers (8 significant bits) at t."""
    return torch.ldexp(torch.ones((), dtype=torch.float64), (torch.frexp(t.cpu().abs())[1] - 9)).cuda()


@pytest.mark.parametrize("rows,n,k,form", [(2100, 512, 1 << 17, "few_rows"), (2100, 2048, 1 << 16, "many_rows"), (3, 640, 1 << 19, "few_rows")])
def test_bf16_results_of_long_sums_of_one_sign(rows, n, k, form):
    """The tensor core adds 16 products at a time and truncates: 4096 / 16 = 256 additions, each off by at most
    2^-23 of the sum, then k / 4096 additions to nearest (2^-24 each), then the one rounding to bf16.  (Summed
    in its accumulator alone, 8 10^-4 at k = 2^17, every result is short by up to 1/2 of half a step.)"""
    g = gen(k)
    x = (1 + torch.rand((rows, k), generator=g, device="cuda")).to(torch.bfloat16)
    w = (1 + torch.rand((n, k), generator=g, device="cuda")).to(torch.bfloat16)
    lin = cf.BlockLinear(w, out_bf16=True)
    assert form in lin.describe(rows)
    y = lin(x).double()
    ref = torch.zeros((rows, n), dtype=torch.float64, device="cuda")
    for i in range(0, k, 1 << 14):
        ref += x[:, i:i + (1 << 14)].double() @ w[:, i:i + (1 << 14)].double().T
    off = ((y - ref).abs() - half_step(ref)) / ref
    assert float(off.max()) <= 256 * 2.0 ** -23 + k / 4096 * 2.0 ** -24, float(off.max())


# ------------------------------------------------------------------------------ one row has no stride

def test_one_row_out_of_a_buffer_of_odd_rows():
    g = gen(2)
    buf = torch.randn((4, 345), generator=g, device="cuda").to(torch.bfloat16)
    base = torch.cat([buf.flatten(), buf.flatten()])
    x = torch.as_strided(base, (1, 136), (345, 1), 8)
    w = torch.as_strided(base, (1, 136), (345, 1), 512)
    y = cf.BlockLinear(w)(x)
    ref = x.double() @ w.double().T
    assert float((y - ref).abs()) <= 140 * 2.0 ** -23 * float(x.double().abs() @ w.double().abs().T)
    q, s = cf.quantize_blocks(x)
    q2, s2 = cf.quantize_blocks(x.clone())
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)


@pytest.mark.parametrize("k", [1000, 4096])
@pytest.mark.parametrize("rows,n", [(5, 512), (300, 512), (2100, 2048)])
def test_fp32_results_of_bf16_operands_in_the_norm(rows, n, k):
    """256 products in the tensor core (16 additions, each off by at most 2^-23 of what is there: with signs at
    random and sizes that grow as the root, (1/2 + ... )^(1/2) of that in the mean square), the sums of 256
    added to nearest: 3e-7 of the result is seen, 6e-7 asked for.  Without the sums of 256: 1.2e-6."""
    g = gen(k + rows)
    wide = -(-k // 8) * 8
    x = torch.randn((rows, wide), generator=g, device="cuda").to(torch.bfloat16)[:, :k]
    w = torch.randn((n, wide), generator=g, device="cuda").to(torch.bfloat16)[:, :k]
    ref = x.double() @ w.double().T
    y = cf.BlockLinear(w)(x).double()
    assert float((y - ref).norm() / ref.norm()) < 6e-7


# ------------------------------------------------------------------------------ every split of the few-rows kernel

# a size (rows, experts, N, K) whose plan is each form that the plan can give
PLANS = {(True, 16, 1): (61, 1, 300, 520), (True, 16, 2): (300, 1, 136, 4112), (True, 16, 4): (9, 1, 72, 4112),
         (True, 16, 8): (5, 1, 72, 14352), (True, 32, 1): (530, 1, 2061, 130), (True, 32, 2): (1061, 8, 136, 8208),
         (True, 32, 4): (530, 1, 136, 14352), (True, 32, 8): (130, 1, 136, 30000), (True, 64, 1): (530, 1, 1032, 130),
         (True, 64, 2): (530, 1, 520, 8208), (True, 64, 4): (300, 1, 520, 8208), (True, 64, 8): (300, 1, 136, 14352),
         (False, 16, 1): (61, 1, 300, 264), (False, 16, 2): (300, 1, 136, 2064), (False, 16, 4): (9, 1, 72, 2064),
         (False, 16, 8): (5, 1, 72, 8208), (False, 32, 1): (530, 1, 520, 130), (False, 32, 2): (300, 1, 520, 4112),
         (False, 32, 4): (300, 1, 136, 8208), (False, 32, 8): (130, 1, 136, 14352), (False, 64, 1): (530, 1, 1032, 130),
         (False, 64, 2): (530, 1, 520, 8208), (False, 64, 4): (300, 1, 520, 8208), (False, 64, 8): (300, 1, 136, 16400)}


@pytest.mark.parametrize("e4m3,tile,split", PLANS)
def test_every_split_is_exact_on_integers(e4m3, tile, split):
    """Integers times powers of two, whose every sum is exact: 4 * 2 * 30000 * 4 below 2^20, in quarters."""
    rows, e, n, k = PLANS[e4m3, tile, split]
    g = gen(rows + k)
    dtype, kb = (torch.float8_e4m3fn if e4m3 else torch.bfloat16), -(-k // 128)
    x = torch.randint(-4, 5, (rows, k), generator=g, device="cuda").float()
    w = torch.randint(-2, 3, (e, n, k), generator=g, device="cuda").float()
    bias = torch.randint(-3, 4, (e, n), generator=g, device="cuda").float()
    rx, rw, xs, ws = x.double(), w.double(), None, None
    if e4m3:
        xs = 2.0 ** torch.randint(-1, 2, (rows, kb), generator=g, device="cuda").float()
        ws = 2.0 ** torch.randint(-1, 2, (e, -(-n // 128), kb), generator=g, device="cuda").float()
        rx = rx * xs.double().repeat_interleave(128, 1)[:, :k]
        rw = rw * ws.double().repeat_interleave(128, 2)[..., :k].repeat_interleave(128, 1)[:, :n]

    def aligned(t):
        wide = torch.zeros((*t.shape[:-1], -(-k // 16) * 16), device="cuda")
        wide[..., :k] = t
        return wide.to(dtype)[..., :k]

    off = torch.tensor([rows * i // e for i in range(e + 1)], dtype=torch.int32, device="cuda")
    ref = torch.cat([rx[int(off[i]):int(off[i + 1])] @ rw[i].T + bias[i].double() for i in range(e)])
    for out_bf16 in (False, True):
        lin = cf.ExpertLinear(aligned(w), ws, bias=bias, act=cf.CONVF_ACT_RELU, out_bf16=out_bf16)
        assert f"few_rows tile={tile}x128 split={split} " in lin.describe(rows)
        y = lin(aligned(x), off, xs)
        torch.cuda.synchronize()
        assert lin.status() == cf.CONVF_OK, cf.conv_fused_last_error()
        assert torch.equal(y.double(), ref.clamp(min=0).to(lin.out_dtype).double())


# ------------------------------------------------------------------------------ the experts' example

@pytest.mark.parametrize("tokens,experts,width,hidden,top", [(9, 3, 100, 75, 2), (200, 4, 1000, 333, 1)])
def test_expert_example_at_odd_sizes(tokens, experts, width, hidden, top):
    """Widths that are no multiple of 16: the weights' rows are padded.  (The bound is that of the quantising:
    four operands of 3 fraction bits, 2.6% each in the norm, 5.2% together; 10% is asked for.)"""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    from expert_feed_forward import example
    y, ref, layer, args = example(tokens, experts, width, hidden, top, seed=tokens)
    assert layer.up.status() == cf.CONVF_OK and layer.down.status() == cf.CONVF_OK
    assert float((y - ref).norm() / ref.norm()) < 0.10


# ------------------------------------------------------------------------------ layers in existence

def test_a_failed_create_leaves_no_layer_behind():
    w = torch.zeros((32, 64), dtype=torch.bfloat16, device="cuda")
    live = cf.conv_fused_debug_live_handles()
    lin = cf.BlockLinear(w)
    assert cf.conv_fused_debug_live_handles() == live + 1
    for n in (1, 2):   # the layer, its device words
        cf.conv_fused_debug_fail_alloc(n)
        with pytest.raises(cf.ConvFusedError) as e:
            cf.BlockLinear(w)
        assert e.value.status == cf.CONVF_ERR_OOM and "(injected)" in str(e.value)
        assert cf.conv_fused_debug_live_handles() == live + 1
    lin.close()
    assert cf.conv_fused_debug_live_handles() == live


# ------------------------------------------------------------------------------ behind a conv

def test_a_conv_feeds_the_quantiser_and_a_layer():
    """conv -> quantise -> linear over the same buffers without a wait between them: a conv's channels-last
    output is a matrix of rows, and each kernel begins while the one before still runs."""
    g = torch.Generator().manual_seed(9)
    N, C, H, K, n = 2, 32, 20, 64, 200
    wc = (torch.randn((K, C, 3, 3), generator=g) / 17).to(torch.bfloat16)
    xs = [torch.randn((N, C, H, H), generator=g).to(torch.bfloat16).contiguous(memory_format=torch.channels_last).cuda()
          for _ in range(3)]
    for out_bf16 in (False, True):
        conv = cf.FusedConv(N, C, H, H, K, 3, 3, wc, None, pads=(1, 1, 1, 1), act=cf.CONVF_ACT_RELU, out_bf16=out_bf16)
        wq, ws = cf.quantize_blocks(torch.randn((n, K), generator=g).cuda(), block_rows=128)
        lin = cf.BlockLinear(wq, ws, out_bf16=True)
        y = conv.new_output()
        rows = y.permute(0, 2, 3, 1).reshape(N * H * H, K)
        assert rows.data_ptr() == y.data_ptr()
        want = []
        for x in xs:
            conv(x, y)
            torch.cuda.synchronize()
            q, s = cf.quantize_blocks(rows)
            torch.cuda.synchronize()
            want.append(lin(q, s))
            torch.cuda.synchronize()
            ref = torch.nn.functional.conv2d(x.float(), wc.cuda().float(), padding=1).clamp(min=0)
            ref = ref.permute(0, 2, 3, 1).reshape(-1, K).double()
            back = q.double() * s.double().repeat_interleave(128, 1)[:, :K]
            # half a step of e4m3, of the value or of the smallest, and a bf16 rounding before
            assert bool(((back - ref).abs() <= ref * (2.0 ** -4 + 2.0 ** -7) + s.double() * 2.0 ** -9 + 1e-5).all())
        got = []
        for t in range(90):
            conv(xs[t % 3], y)
            cf.quantize_blocks(rows, q=q, scale=s)
            got.append(lin(q, s))
        torch.cuda.synchronize()
        assert all(torch.equal(got[t], want[t % 3]) for t in range(90))


# ------------------------------------------------------------------------------ what lies beside y's rows

@pytest.mark.parametrize("n", [1003, 2049, 2061, 2056])
@pytest.mark.parametrize("rows", [5, 70, 4100])
@pytest.mark.parametrize("out_bf16", [True, False])
@pytest.mark.parametrize("e4m3", [True, False])
def test_columns_beside_aligned_rows_of_y_are_kept(n, rows, out_bf16, e4m3):
    """Rows of y that begin on 16 bytes and end inside 16: whole tiles leave by TMA, whose stores are clipped by
    units of 16 bytes only."""
    g, k = gen(n + rows), 272
    x = torch.randint(-4, 5, (rows, k), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randint(-2, 3, (n, k), generator=g, device="cuda").to(torch.bfloat16)
    ref, xs, ws = x.double() @ w.double().T, None, None
    if e4m3:
        x, w = x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn)
        xs, ws = torch.ones((rows, 3), device="cuda"), torch.ones((-(-n // 128), 3), device="cuda")
    for bias in (None, torch.randint(-3, 4, (n,), generator=g, device="cuda").float()):
        lin = cf.BlockLinear(w, ws, bias=bias, out_bf16=out_bf16)
        wide = (n + 15) // 16 * 16 + 16
        buf = torch.full((rows + 2, wide), -7.0, dtype=lin.out_dtype, device="cuda")
        lin(x, xs, y=buf[1:rows + 1, :n])
        torch.cuda.synchronize()
        assert lin.status() == cf.CONVF_OK
        want = ref if bias is None else ref + bias.double()
        assert torch.equal(buf[1:rows + 1, :n].double(), want.to(lin.out_dtype).double())
        assert bool((buf[:, n:] == -7).all()) and bool((buf[0] == -7).all()) and bool((buf[-1] == -7).all())


@pytest.mark.parametrize("cols", [203, 209, 1000, 1017])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_columns_beside_aligned_rows_of_q_are_kept(cols, dtype, block_rows):
    rows, wide = 131, (cols + 31) // 32 * 32 + 32
    x = torch.randn((rows, wide), generator=gen(cols), device="cuda").to(dtype)[:, :cols]
    qb = torch.full((rows + 2, wide), 0x55, dtype=torch.uint8, device="cuda")
    sb = torch.full((rows + 2, -(-cols // 128) + 1), -7.0, device="cuda")
    srows, nb = -(-rows // block_rows), -(-cols // 128)
    cf.quantize_blocks(x, block_rows=block_rows, q=qb[1:rows + 1, :cols].view(torch.float8_e4m3fn), scale=sb[1:srows + 1, :nb])
    q, s = cf.quantize_blocks(x.contiguous(), block_rows=block_rows)
    assert torch.equal(qb[1:rows + 1, :cols], q.view(torch.uint8)) and torch.equal(sb[1:srows + 1, :nb], s)
    assert bool((qb[:, cols:] == 0x55).all()) and bool((qb[0] == 0x55).all()) and bool((qb[-1] == 0x55).all())
    assert bool((sb[:, nb:] == -7).all()) and bool((sb[0] == -7).all()) and bool((sb[srows + 1:] == -7).all())
