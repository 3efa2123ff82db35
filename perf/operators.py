"""Cases of the block-scaled 8-bit operators: quantising to e4m3 with a scale per block of 128,
the matrix product of such operands, and the products of row groups with an expert's weights each.

``run`` computes a case either in plain form (elementary torch operations in 32 bits, rounded
once at the end) or, where ``own`` is true, through the package's operators.  ``exact`` computes
the same outputs from the definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 128
TOP = 448.0   # the largest e4m3 value


def listed():
    return [
        # one token's activations before a quantised product: latency
        dict(name="quantise one token", op="quantise", mode="rows", rows=1, cols=2048, dtype="bf16"),
        # a 56x56 map of 256 channels, batch 32, as a conv of the ResNet-50 step writes it (fp32, channels last)
        dict(name="quantise conv map", op="quantise", mode="rows", rows=100352, cols=256, dtype="f32"),
        # tokens copied to the experts that take them (4 each), rows that end inside a block
        dict(name="quantise gathered rows", op="quantise", mode="gather", rows=16380, cols=2000, tokens=4095, dtype="bf16"),
        # between the two products of an expert's gated feed-forward layer
        dict(name="quantise gated", op="quantise", mode="gated", rows=8192, cols=2048, dtype="bf16"),
        # a weight matrix as it is converted, 128 x 128 blocks, ragged at both edges
        dict(name="quantise weights", op="quantise", mode="tiles", rows=5000, cols=4100, dtype="bf16"),
        # one token through a square layer: the weights' bytes
        dict(name="product one token", op="product", rows=1, n=4096, k=4096, bias=True, relu=False, out="bf16"),
        # a classifier head, 2048 features to 1000 classes, at an odd batch
        dict(name="product head", op="product", rows=1001, n=1000, k=2048, bias=True, relu=False, out="f32"),
        # a long prompt through a large layer
        dict(name="product prompt", op="product", rows=8192, n=8192, k=8192, bias=False, relu=True, out="bf16"),
        # a few tokens in flight, 32 rows over 24 of 64 experts: the weights' bytes
        dict(name="experts few tokens", op="experts", rows=32, experts=64, active=24, n=2048, k=2048, dtype="e4m3", out="bf16"),
        # a small batch over wide bf16 experts, odd sizes, experts without rows
        dict(name="experts small batch bf16", op="experts", rows=333, experts=16, active=13, n=1500, k=1000, dtype="bf16", out="f32"),
        # a prompt in bf16
        dict(name="experts prompt bf16", op="experts", rows=8190, experts=32, active=32, n=2048, k=1024, dtype="bf16", out="bf16"),
        # a batch of prompts in 8 bits
        dict(name="experts prompt", op="experts", rows=24576, experts=16, active=16, n=4096, k=2048, dtype="e4m3", out="bf16"),
    ]


def draw(rng: random.Random):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["quantise", "quantise", "product", "experts", "experts"])
    while True:
        if op == "quantise":
            mode = rng.choice(["rows", "gather", "gated", "tiles"])
            c = dict(op=op, mode=mode, rows=spread(1, 60000), cols=spread(64, 5000), dtype=rng.choice(["bf16", "bf16", "f32"]))
            if mode == "gather":
                c["tokens"] = max(1, c["rows"] // rng.choice([1, 2, 4, 8]))
            if c["rows"] * c["cols"] <= 30_000_000:
                break
        elif op == "product":
            c = dict(op=op, rows=spread(1, 8192), n=spread(64, 8192), k=spread(64, 8192), bias=rng.random() < 0.5, relu=rng.random() < 0.5,
                     out=rng.choice(["bf16", "f32"]))
            if c["rows"] * c["n"] * c["k"] <= 8192 ** 3 // 4:
                break
        else:
            e = spread(1, 64)
            c = dict(op=op, rows=spread(1, 24576), experts=e, active=0, n=spread(64, 4096), k=spread(64, 4096), dtype=rng.choice(["bf16", "e4m3"]),
                     out=rng.choice(["bf16", "f32"]))
            c["active"] = max(1, min(c["rows"], e - rng.randint(0, e // 3)))
            if c["rows"] * c["n"] * c["k"] <= 50_000_000_000 and e * c["n"] * c["k"] <= 270_000_000:
                break
    return c


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _activations(g, rows, cols, dtype):
    """Normal values of a different size for each row, with a few channels that stand out."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x *= torch.exp(torch.randn((rows, 1), generator=g, device="cuda"))
    x *= 1 + 15 * (torch.rand((1, cols), generator=g, device="cuda") < 0.01)
    return x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def _pad_rows(t):
    """`t` with its rows 16-byte aligned, as rows that a kernel's tile copies read have to be: a view of the wider buffer."""
    step = 16 // t.element_size()
    wide = -(-t.shape[-1] // step) * step
    if wide == t.shape[-1]:
        return t.contiguous()
    buf = torch.zeros((*t.shape[:-1], wide), dtype=torch.uint8 if t.element_size() == 1 else t.dtype, device=t.device)
    buf = buf.view(t.dtype)
    buf[..., : t.shape[-1]].view(torch.uint8 if t.element_size() == 1 else t.dtype).copy_(t.view(torch.uint8) if t.element_size() == 1 else t)
    return buf[..., : t.shape[-1]]


def _rows_to_e4m3(x):
    """(e4m3 values, scale per row and block of 128) of float rows."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    v = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - cols)).view(rows, nb, BLOCK)
    top = torch.full((), TOP, device=x.device)
    scale = v.abs().amax(-1) / top
    q = torch.where(scale[..., None] == 0, 0.0, v / scale[..., None]).clamp(-TOP, TOP)
    return q.view(rows, nb * BLOCK)[:, :cols].to(torch.float8_e4m3fn), scale


def _tiles_to_e4m3(x):
    """(e4m3 values, scale per block of 128 x 128) of a float matrix, or of several."""
    *lead, n, k = x.shape
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    v = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - k, 0, nb * BLOCK - n)).view(*lead, nb, BLOCK, kb, BLOCK)
    top = torch.full((), TOP, device=x.device)
    scale = v.abs().amax((-3, -1)) / top
    wide = scale[..., :, None, :, None]
    q = torch.where(wide == 0, 0.0, v / wide).clamp(-TOP, TOP)
    return q.reshape(*lead, nb * BLOCK, kb * BLOCK)[..., :n, :k].to(torch.float8_e4m3fn), scale


def _offsets(seed, case):
    """Rows by expert: `active` experts get at least one row, the others none, with popular experts among them."""
    r = np.random.RandomState(int(seed) % (1 << 31))
    e, a, t = case["experts"], case["active"], case["rows"]
    who = np.sort(r.permutation(e)[:a])
    p = np.exp(0.7 * r.randn(a))
    counts = np.zeros(e, np.int64)
    counts[who] = 1 + r.multinomial(t - a, p / p.sum())
    return np.concatenate([[0], np.cumsum(counts)])


def _inputs(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "quantise":
        mode = case["mode"]
        rows = case["tokens"] if mode == "gather" else case["rows"]
        wide = case["cols"] * (2 if mode == "gated" else 1)
        s["x"] = _activations(g, rows, wide, case["dtype"])
        if mode == "gated":
            s["x"] = s["x"] / 2   # gates of a few units, where the sigmoid is neither open nor shut
        if mode == "gather":
            s["index"] = torch.randint(0, rows, (case["rows"],), generator=g, device="cuda", dtype=torch.int32)
        return s
    rows, n, k = case["rows"], case["n"], case["k"]
    e = case.get("experts", 1)
    x = _activations(g, rows, k, "bf16")
    w = torch.randn((e, n, k), generator=g, device="cuda") / math.sqrt(k)
    if case.get("dtype", "e4m3") == "bf16":
        s["x"], s["w"] = _pad_rows(x), _pad_rows(w.to(torch.bfloat16))
        s["xs"] = s["ws"] = None
    else:
        x, s["xs"] = _rows_to_e4m3(x)
        w, s["ws"] = _tiles_to_e4m3(w)
        s["x"], s["w"] = _pad_rows(x), _pad_rows(w)
    s["b"] = torch.randn((n,), generator=g, device="cuda") if case.get("bias") else None
    if case["op"] == "experts":
        off = _offsets(seed, case)
        s["host_offsets"] = off
        s["offsets"] = torch.from_numpy(off.astype(np.int32)).cuda()
    else:
        s["w"] = s["w"][0]
        s["ws"] = s["ws"][0]
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    out = torch.bfloat16 if case.get("out") == "bf16" else torch.float32
    if op == "experts":   # the longest group, which a program that lays rows out by expert knows
        s["longest"] = int(np.diff(s["host_offsets"]).max())
    if own:
        import convolution_onnx_conv_gb300 as cf
        s["cf"] = cf
        act = cf.CONVF_ACT_RELU if case.get("relu") else cf.CONVF_ACT_NONE
        if op == "product":
            s["layer"] = cf.BlockLinear(s["w"], s["ws"], bias=s["b"], act=act, out_bf16=out == torch.bfloat16)
        elif op == "experts":
            s["layer"] = cf.ExpertLinear(s["w"], s["ws"], out_bf16=out == torch.bfloat16)
    s["out_dtype"] = out
    return s


# ------------------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "quantise":
        x = s["x"]
        if s["mode"] == "tiles":
            return _tiles_to_e4m3(x)
        if s["mode"] == "gather":
            x = x[s["index"]]
        if s["mode"] == "gated":
            gate, up = x.float().chunk(2, dim=1)
            x = gate / (1 + torch.exp(-gate)) * up
        return _rows_to_e4m3(x)
    x = s["x"].float()
    w = s["w"].float()
    n, k = w.shape[-2:]
    if s["xs"] is not None:
        x = x * s["xs"].repeat_interleave(BLOCK, 1)[:, :k]
        w = w * s["ws"].repeat_interleave(BLOCK, -1).repeat_interleave(BLOCK, -2)[..., :n, :k]
    if op == "product":
        y = x @ w.T
        if s["b"] is not None:
            y = y + s["b"]
        if s["relu"]:
            y = y.clamp(min=0)
        return y.to(s["out_dtype"])
    # the groups side by side, padded to the longest
    off = s["offsets"].long()
    at = off[:-1, None] + torch.arange(s["longest"], device=x.device)
    there = at < off[1:, None]
    y = torch.bmm(x[at.clamp(max=x.shape[0] - 1)], w.transpose(1, 2))
    return y[there].to(s["out_dtype"])


def _run_own(s):
    op = s["op"]
    if op == "quantise":
        mode = s["mode"]
        return s["cf"].quantize_blocks(s["x"], index=s["index"] if mode == "gather" else None, gated=mode == "gated",
                                       block_rows=BLOCK if mode == "tiles" else 1)
    if op == "product":
        return s["layer"](s["x"], s["xs"])
    return s["layer"](s["x"], s["offsets"], s["xs"])


# ------------------------------------------------------------------------------ 64 bits

def _e4m3_64(t):
    """The nearest e4m3 value of each double, ties to even: 3 fraction bits, exponents down to -6, at most 448."""
    t = t.clamp(-TOP, TOP)
    _, e = torch.frexp(t)   # |t| = m 2^e, m in [1/2, 1)
    step = torch.ldexp(torch.ones_like(t), (e - 1).clamp(min=-6) - 3)
    return torch.round(t / step) * step


def exact(case, seed):
    s = _inputs(case, seed)
    x = s["x"].double()
    if case["op"] == "quantise":
        if case["mode"] == "gather":
            x = x[s["index"].long()]
        if case["mode"] == "gated":
            half = case["cols"]
            x = x[:, :half] * torch.sigmoid(x[:, :half]) * x[:, half:]
        q, tall = torch.empty_like(x), BLOCK if case["mode"] == "tiles" else 1
        nb = -(-case["cols"] // BLOCK)
        scale = torch.empty((-(-case["rows"] // tall), nb), dtype=torch.float64, device="cuda")
        for b in range(nb):
            v = x[:, b * BLOCK:(b + 1) * BLOCK]
            m = v.abs().amax(1)
            if tall > 1:
                m = torch.nn.functional.pad(m, (0, -m.numel() % tall)).view(-1, tall).amax(1)
            m = (m / TOP).float().double()   # a scale is a 32-bit number
            scale[:, b] = m
            m = m.repeat_interleave(tall)[: v.shape[0], None]
            q[:, b * BLOCK:(b + 1) * BLOCK] = torch.where(m == 0, torch.zeros_like(v), _e4m3_64(v / m))
        return q, scale
    n, k = case["n"], case["k"]

    def real(w, ws):
        w = w.double()
        if ws is not None:
            w *= ws.double()[torch.arange(n, device="cuda") // BLOCK][:, torch.arange(k, device="cuda") // BLOCK]
        return w

    if s["xs"] is not None:
        x *= s["xs"].double()[:, torch.arange(k, device="cuda") // BLOCK]
    if case["op"] == "product":
        y = torch.mm(x, real(s["w"], s["ws"]).t())
        if s["b"] is not None:
            y += s["b"].double()
        return torch.relu(y) if case["relu"] else y
    y = torch.empty((case["rows"], n), dtype=torch.float64, device="cuda")
    off = s["host_offsets"]
    for e in range(case["experts"]):
        a, b = int(off[e]), int(off[e + 1])
        if b > a:
            y[a:b] = torch.mm(x[a:b], real(s["w"][e], None if s["ws"] is None else s["ws"][e]).t())
    return y


def work(case):
    """Each input read once, each output written once; two operations per product and sum."""
    if case["op"] == "quantise":
        size = 2 if case["dtype"] == "bf16" else 4
        rows, cols, mode = case["rows"], case["cols"], case["mode"]
        nb = -(-cols // BLOCK)
        read = min(rows, case.get("tokens", rows)) * cols * size * (2 if mode == "gated" else 1)
        scales = 4 * nb * (-(-rows // BLOCK) if mode == "tiles" else rows)
        return {"bytes": read + (4 * rows if mode == "gather" else 0) + rows * cols + scales, "flops": 3 * rows * cols}
    rows, n, k = case["rows"], case["n"], case["k"]
    e = case.get("active", 1)
    e4m3 = case.get("dtype", "e4m3") == "e4m3"
    kb = -(-k // BLOCK)
    size = 1 if e4m3 else 2
    scales = 4 * (rows * kb + e * -(-n // BLOCK) * kb) if e4m3 else 0
    out = rows * n * (2 if case["out"] == "bf16" else 4)
    extra = 4 * n if case.get("bias") else 0
    extra += 4 * (case["experts"] + 1) if case["op"] == "experts" else 0
    return {"bytes": (rows * k + e * n * k) * size + scales + out + extra, "flops": 2 * rows * n * k}
