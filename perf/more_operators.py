"""Cases of the 8-bit integer operators: quantising rows to int8 with a scale each, the root-mean-square
norm with the residual's addition and 8-bit output, the matrix product of int8 operands with scales per
row and channel, and the products of row groups with an expert's int8 weights each.

``run`` computes a case either in plain form (elementary torch operations in 32 bits, rounded once at the
end) or, where ``own`` is true, through the package's operators.  ``exact`` computes the same outputs from
the definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 128
TOP8 = 127.0    # the largest int8 value that is used (the range is symmetric)
TOPF = 448.0    # the largest e4m3 value
EPS = 1e-6


def listed():
    return [
        # one token's activations before an int8 product: latency
        dict(name="rows one token", op="rows", mode="rows", rows=1, cols=2048, dtype="bf16"),
        # between the two products of a gated feed-forward layer, a prompt
        dict(name="rows gated", op="rows", mode="gated", rows=8192, cols=2048, dtype="bf16"),
        # a weight matrix as it is converted, a scale per output channel, ragged
        dict(name="rows weights", op="rows", mode="rows", rows=5000, cols=4100, dtype="f32"),
        # one token between two layers, residual stream in bf16, for a block-scaled layer: latency
        dict(name="norm one token", op="norm", rows=1, cols=4096, dtype="bf16", res="bf16", out="e4m3"),
        # a prompt between two layers, for a block-scaled layer
        dict(name="norm prompt", op="norm", rows=8192, cols=4096, dtype="bf16", res="bf16", out="e4m3"),
        # a residual stream kept in fp32, odd sizes, for an int8 layer
        dict(name="norm ragged", op="norm", rows=4095, cols=2000, dtype="bf16", res="f32", out="int8"),
        # one token through a square layer: the weights' bytes
        dict(name="product one token", op="product", rows=1, n=4096, k=4096, bias=True, relu=False, out="bf16"),
        # a classifier head, 2048 features to 1000 classes, at an odd batch
        dict(name="product head", op="product", rows=1001, n=1000, k=2048, bias=True, relu=False, out="f32"),
        # a batch of tokens in flight through a wide layer
        dict(name="product batch", op="product", rows=96, n=8192, k=2048, bias=False, relu=True, out="bf16"),
        # a long prompt through a large layer
        dict(name="product prompt", op="product", rows=8192, n=8192, k=8192, bias=False, relu=False, out="bf16"),
        # a few tokens in flight, 32 rows over 24 of 64 experts: the weights' bytes
        dict(name="experts few tokens", op="experts", rows=32, experts=64, active=24, n=2048, k=2048, out="bf16"),
        # a prompt over experts, odd sizes, experts without rows
        dict(name="experts prompt", op="experts", rows=8190, experts=32, active=29, n=2000, k=1030, out="f32"),
    ]


def draw(rng: random.Random):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rows", "norm", "product", "product", "experts"])
    while True:
        if op == "rows":
            mode = rng.choice(["rows", "gather", "gated"])
            c = dict(op=op, mode=mode, rows=spread(1, 60000), cols=spread(64, 12000), dtype=rng.choice(["bf16", "bf16", "f32"]))
            if mode == "gather":
                c["tokens"] = max(1, c["rows"] // rng.choice([1, 2, 4, 8]))
            if c["rows"] * c["cols"] <= 30_000_000:
                break
        elif op == "norm":
            c = dict(op=op, rows=spread(1, 60000), cols=spread(64, 12000), dtype=rng.choice(["bf16", "bf16", "f32"]),
                     res=rng.choice(["none", "bf16", "bf16", "f32"]), out=rng.choice(["e4m3", "int8"]))
            if c["rows"] * c["cols"] <= 30_000_000:
                break
        elif op == "product":
            c = dict(op=op, rows=spread(1, 8192), n=spread(64, 8192), k=spread(64, 8192), bias=rng.random() < 0.5, relu=rng.random() < 0.5,
                     out=rng.choice(["bf16", "f32"]))
            if c["rows"] * c["n"] * c["k"] <= 8192 ** 3 // 4:
                break
        else:
            e = spread(1, 64)
            c = dict(op=op, rows=spread(1, 24576), experts=e, active=0, n=spread(64, 4096), k=spread(64, 4096), out=rng.choice(["bf16", "f32"]))
            c["active"] = max(1, min(c["rows"], e - rng.randint(0, e // 3)))
            if c["rows"] * c["n"] * c["k"] <= 50_000_000_000 and e * c["n"] * c["k"] <= 270_000_000:
                break
    return c


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 23)


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _activations(g, rows, cols, dtype):
    """Normal values of a different size for each row, with a few channels that stand out."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x *= torch.exp(torch.randn((rows, 1), generator=g, device="cuda"))
    x *= 1 + 15 * (torch.rand((1, cols), generator=g, device="cuda") < 0.01)
    return x.to(_type(dtype))


def _pad_rows(t):
    """`t` (int8) with its rows 16-byte aligned, as rows that a kernel's tile copies read have to be: a view of the wider buffer."""
    wide = -(-t.shape[-1] // 16) * 16
    if wide == t.shape[-1]:
        return t.contiguous()
    buf = torch.zeros((*t.shape[:-1], wide), dtype=t.dtype, device=t.device)
    buf[..., : t.shape[-1]] = t
    return buf[..., : t.shape[-1]]


def _rows_to_int8(v):
    """(int8 values, scale per row) of float rows."""
    scale = v.abs().amax(-1) / torch.full((), TOP8, device=v.device)
    wide = scale[..., None]
    q = torch.where(wide == 0, 0.0, torch.round(v / wide)).clamp(-TOP8, TOP8)
    return q.to(torch.int8), scale


def _rows_to_e4m3(v):
    """(e4m3 values, scale per row and block of 128) of float rows."""
    rows, cols = v.shape
    nb = -(-cols // BLOCK)
    v = torch.nn.functional.pad(v, (0, nb * BLOCK - cols)).view(rows, nb, BLOCK)
    scale = v.abs().amax(-1) / torch.full((), TOPF, device=v.device)
    q = torch.where(scale[..., None] == 0, 0.0, v / scale[..., None]).clamp(-TOPF, TOPF)
    return q.view(rows, nb * BLOCK)[:, :cols].to(torch.float8_e4m3fn), scale


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
    if case["op"] == "rows":
        mode = case["mode"]
        rows = case["tokens"] if mode == "gather" else case["rows"]
        s["x"] = _activations(g, rows, case["cols"] * (2 if mode == "gated" else 1), case["dtype"])
        if mode == "gated":
            s["x"] = s["x"] / 2   # gates of a few units, where the sigmoid is neither open nor shut
        if mode == "gather":
            s["index"] = torch.randint(0, rows, (case["rows"],), generator=g, device="cuda", dtype=torch.int32)
        return s
    if case["op"] == "norm":
        rows, cols = case["rows"], case["cols"]
        s["x"] = _activations(g, rows, cols, case["dtype"])
        s["r"] = None if case["res"] == "none" else _activations(g, rows, cols, case["res"])
        s["w"] = 1 + torch.randn((cols,), generator=g, device="cuda") / 8
        return s
    rows, n, k = case["rows"], case["n"], case["k"]
    e = case.get("experts", 1)
    x, s["xs"] = _rows_to_int8(_activations(g, rows, k, "bf16").float())
    w, s["ws"] = _rows_to_int8(torch.randn((e, n, k), generator=g, device="cuda") / math.sqrt(k))
    s["x"], s["w"] = _pad_rows(x), _pad_rows(w)
    s["b"] = torch.randn((n,), generator=g, device="cuda") if case.get("bias") else None
    if case["op"] == "experts":
        off = _offsets(seed, case)
        s["host_offsets"] = off
        s["offsets"] = torch.from_numpy(off.astype(np.int32)).cuda()
    else:
        s["w"], s["ws"] = s["w"][0], s["ws"][0]
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "experts":   # the longest group, which a program that lays rows out by expert knows
        s["longest"] = int(np.diff(s["host_offsets"]).max())
    if own:
        import convolution_onnx_conv_gb300 as cf
        s["cf"] = cf
        if op == "product":
            s["layer"] = cf.Int8Linear(s["w"], s["ws"], bias=s["b"], act=cf.CONVF_ACT_RELU if case["relu"] else cf.CONVF_ACT_NONE,
                                       out_bf16=case["out"] == "bf16")
        elif op == "experts":
            s["layer"] = cf.ExpertLinear(s["w"], s["ws"], out_bf16=case["out"] == "bf16")
    return s


# ------------------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "rows":
        x = s["x"]
        if s["mode"] == "gather":
            x = x[s["index"]]
        x = x.float()
        if s["mode"] == "gated":
            gate, up = x.chunk(2, dim=1)
            x = gate / (1 + torch.exp(-gate)) * up
        return _rows_to_int8(x)
    if op == "norm":
        # the row's factor is positive, so that it scales the quantised values' scales and nothing else
        h = s["x"].float()
        if s["r"] is not None:
            h = h + s["r"].float()
        factor = 1 / torch.sqrt((h * h).mean(1) + EPS)
        if s["out"] == "int8":
            q, scale = _rows_to_int8(h * s["w"])
            scale = scale * factor
        else:
            q, scale = _rows_to_e4m3(h * s["w"])
            scale = scale * factor[:, None]
        return (q, scale) if s["r"] is None else (q, scale, h.to(s["r"].dtype))
    x, w = s["x"].float(), s["w"].float()
    if op == "product":
        y = (x @ w.T) * (s["xs"][:, None] * s["ws"])
        if s["b"] is not None:
            y = y + s["b"]
        if s["relu"]:
            y = y.clamp(min=0)
        return y.to(_type(s["out"]))
    # the groups side by side, padded to the longest
    off = s["offsets"].long()
    at = off[:-1, None] + torch.arange(s["longest"], device=x.device)
    there = at < off[1:, None]
    at = at.clamp(max=x.shape[0] - 1)
    y = torch.bmm(x[at], w.transpose(1, 2)) * (s["xs"][at][:, :, None] * s["ws"][:, None, :])
    return y[there].to(_type(s["out"]))


def _run_own(s):
    op = s["op"]
    if op == "rows":
        return s["cf"].quantize_rows(s["x"], index=s.get("index"), gated=s["mode"] == "gated")
    if op == "norm":
        return s["cf"].rms_norm_quantize(s["x"], s["w"], EPS, residual=s["r"], int8=s["out"] == "int8")
    if op == "product":
        return s["layer"](s["x"], s["xs"])
    return s["layer"](s["x"], s["offsets"], s["xs"])


# ------------------------------------------------------------------------------ 64 bits

def _e4m3_64(t):
    """The nearest e4m3 value of each double, ties to even: 3 fraction bits, exponents down to -6, at most 448."""
    t = t.clamp(-TOPF, TOPF)
    _, e = torch.frexp(t)   # |t| = m 2^e, m in [1/2, 1)
    step = torch.ldexp(torch.ones_like(t), (e - 1).clamp(min=-6) - 3)
    return torch.round(t / step) * step


def exact(case, seed):
    s = _inputs(case, seed)
    x = s["x"].double()
    cols = case.get("cols")
    if case["op"] == "rows":
        if case["mode"] == "gather":
            x = x[s["index"].long()]
        if case["mode"] == "gated":
            x = x[:, :cols] * torch.sigmoid(x[:, :cols]) * x[:, cols:]
        return None, x.abs().amax(1) / TOP8   # (integers are compared with the plain form's)
    if case["op"] == "norm":
        if s["r"] is not None:
            x = x + s["r"].double()
        inv = torch.rsqrt(x.pow(2).sum(1) / cols + EPS)
        v = x * inv[:, None] * s["w"].double()
        if case["out"] == "int8":
            out = (None, v.abs().amax(1) / TOP8)
        else:
            nb = -(-cols // BLOCK)
            scale = torch.empty((case["rows"], nb), dtype=torch.float64, device="cuda")
            q = torch.empty_like(v)
            for b in range(nb):
                part = v[:, b * BLOCK:(b + 1) * BLOCK]
                m = part.abs().amax(1) / TOPF
                scale[:, b] = m
                q[:, b * BLOCK:(b + 1) * BLOCK] = torch.where(m[:, None] == 0, torch.zeros_like(part), _e4m3_64(part / m[:, None]))
            out = (q, scale)
        return out if s["r"] is None else (*out, x)
    n = case["n"]
    if case["op"] == "product":
        y = torch.mm(x * s["xs"].double()[:, None], (s["w"].double() * s["ws"].double()[:, None]).t())
        if s["b"] is not None:
            y += s["b"].double()
        return torch.relu(y) if case["relu"] else y
    y = torch.empty((case["rows"], n), dtype=torch.float64, device="cuda")
    off = s["host_offsets"]
    for e in range(case["experts"]):
        a, b = int(off[e]), int(off[e + 1])
        if b > a:
            y[a:b] = torch.mm(x[a:b] * s["xs"][a:b, None].double(), (s["w"][e].double() * s["ws"][e].double()[:, None]).t())
    return y


def work(case):
    """Each input read once, each output written once; two operations per product and sum."""
    rows = case["rows"]
    if case["op"] in ("rows", "norm"):
        cols = case["cols"]
        size = {"bf16": 2, "f32": 4, "none": 0}
        if case["op"] == "rows":
            gated = case["mode"] == "gated"
            read = min(rows, case.get("tokens", rows)) * cols * size[case["dtype"]] * (2 if gated else 1)
            read += 4 * rows if case["mode"] == "gather" else 0
            return {"bytes": read + rows * cols + 4 * rows, "flops": (8 if gated else 3) * rows * cols}
        scales = 4 * rows * (1 if case["out"] == "int8" else -(-cols // BLOCK))
        return {"bytes": rows * cols * (size[case["dtype"]] + 2 * size[case["res"]] + 1) + 4 * cols + scales, "flops": 7 * rows * cols}
    n, k, e = case["n"], case["k"], case.get("active", 1)
    out = rows * n * (2 if case["out"] == "bf16" else 4)
    extra = 4 * n if case.get("bias") else 0
    extra += 4 * (case["experts"] + 1) if case["op"] == "experts" else 0
    return {"bytes": rows * k + e * n * k + 4 * (rows + e * n) + out + extra, "flops": 2 * rows * n * k}
