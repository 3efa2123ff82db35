"""A feed-forward layer of experts in 8 bits, from tokens to tokens: each token goes to `top` of the
experts, through

    y = sum over its experts e of  p_e * down_e( silu(gate_e(x)) * up_e(x) )

in five launches: the tokens' rows are quantised as they are copied to their experts, the first product
gives gate and up side by side, the gated values are quantised in the pass that gates them, the second
product gives the experts' outputs, and these are added up per token.

    python examples/expert_feed_forward.py [tokens]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import convolution_onnx_conv_gb300 as cf  # noqa: E402


class ExpertFeedForward:
    """`w_gate_up` [experts][2 * hidden][width] (the gate's rows first) and `w_down` [experts][width][hidden],
    float CUDA tensors, quantised here to e4m3 with a scale per 128 x 128 block."""

    def __init__(self, w_gate_up, w_down):
        def layer(w):
            experts, n, k = w.shape
            wide = -(-k // 16) * 16   # rows of a layer's weights lie a multiple of 16 bytes apart
            q = torch.empty_strided((experts, n, k), (n * wide, wide, 1), dtype=torch.float8_e4m3fn, device=w.device)
            scale = torch.empty((experts, -(-n // 128), -(-k // 128)), device=w.device)
            for e in range(experts):
                cf.quantize_blocks(w[e], block_rows=128, q=q[e], scale=scale[e])
            return cf.ExpertLinear(q, scale, out_bf16=True)

        self.experts = w_gate_up.shape[0]
        self.up, self.down = layer(w_gate_up), layer(w_down)

    def route(self, logits, top):
        """(expert of each token's choices, their weights): the `top` largest, softmax over those."""
        value, expert = torch.topk(logits.float(), top, dim=1)
        return expert, torch.softmax(value, 1)

    def __call__(self, x, expert, weight):
        """y [tokens][width] for x (bf16 or fp32), `expert` and `weight` [tokens][top]."""
        tokens, top = expert.shape
        order = torch.argsort(expert.reshape(-1), stable=True)          # choices by expert
        counts = torch.bincount(expert.reshape(-1), minlength=self.experts)
        offsets = torch.zeros(self.experts + 1, dtype=torch.int32, device=x.device)
        offsets[1:] = counts.cumsum(0)
        q, s = cf.quantize_blocks(x, index=(order // top).to(torch.int32))
        h = self.up(q, offsets, s)                                      # [gate | up]
        q, s = cf.quantize_blocks(h, gated=True)
        out = self.down(q, offsets, s)
        place = torch.empty_like(order)
        place[order] = torch.arange(order.numel(), device=x.device)     # of each choice's row
        return (out[place.view(tokens, top)].float() * weight[..., None]).sum(1)


def reference(w_gate_up, w_down, x, expert, weight):
    """The same layer in 64 bits, without quantising."""
    y = torch.zeros(x.shape[0], w_down.shape[1], dtype=torch.float64, device=x.device)
    for e in range(w_gate_up.shape[0]):
        token, choice = torch.nonzero(expert == e, as_tuple=True)
        if token.numel():
            gate, up = (x[token].double() @ w_gate_up[e].double().T).chunk(2, 1)
            h = torch.nn.functional.silu(gate) * up
            y[token] += weight[token, choice, None].double() * (h @ w_down[e].double().T)
    return y


def example(tokens=512, experts=16, width=1024, hidden=768, top=2, seed=0):
    """(layer's output, its 64-bit reference, the layer, its arguments) for random weights and tokens."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w1 = torch.randn((experts, 2 * hidden, width), generator=g, device="cuda") / width ** 0.5
    w2 = torch.randn((experts, width, hidden), generator=g, device="cuda") / hidden ** 0.5
    x = torch.randn((tokens, width), generator=g, device="cuda").to(torch.bfloat16)
    layer = ExpertFeedForward(w1, w2)
    expert, weight = layer.route(torch.randn((tokens, experts), generator=g, device="cuda"), top)
    return layer(x, expert, weight), reference(w1, w2, x, expert, weight), layer, (x, expert, weight)


if __name__ == "__main__":
    y, ref, layer, args = example(int(sys.argv[1]) if len(sys.argv) > 1 else 512)
    for status in (layer.up.status(), layer.down.status()):
        assert status == cf.CONVF_OK, cf.conv_fused_last_error()
    print(layer.up.describe(args[1].numel()))
    print(layer.down.describe(args[1].numel()))
    print(f"error against 64 bits without quantising: {float((y - ref).norm() / ref.norm()):.3f} of the output")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(3):
        layer(*args)
    start.record()
    for _ in range(20):
        layer(*args)
    end.record()
    torch.cuda.synchronize()
    print(f"{start.elapsed_time(end) / 20 * 1e3:.0f} us a pass, routing by torch included")
