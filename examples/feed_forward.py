"""A gated feed-forward layer trained in FP8 and served in INT8.

    python examples/feed_forward.py [--tokens 4096 --hidden 7168 --ffn 2048]

Training: y = W_down (act(x W_gate^T) * (x W_up^T)) is fitted to a fixed layer
of the same shape.  Master weights are FP32; every product of the step runs on
E4M3 codes with fine-grained scales:

    forward    gemm_gated (keeps gate and up), quantize_act, gemm
    backward   gemm (dh), gated_backward (dY along features and along tokens),
               gemm_rowscaled twice (the weight gradients), gemm (dx)

Experts: the same block over routed rows, one call for all experts.
Serving: the trained weights quantized per output channel to int8, activations
per token; one token at a time and in a batch:

    quantize_token_i8, gemm_i8_gated, quantize_token_i8, gemm_i8
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fine_grained_block_fp8q_amd as fq   # noqa: E402

BF16 = torch.bfloat16


class Layer:
    """Gate, up and down projections with FP32 master weights."""

    def __init__(self, hidden, ffn, seed, act="silu"):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.act = act
        self.w1 = torch.randn((2 * ffn, hidden), generator=g, device="cuda") / hidden ** 0.5
        self.w2 = torch.randn((hidden, ffn), generator=g, device="cuda") / ffn ** 0.5

    def forward(self, x):
        """x: bf16 [M][hidden] -> bf16 [M][hidden]; keeps what backward needs."""
        w1, w2 = self.w1.to(BF16), self.w2.to(BF16)
        h, gate_up = fq.gemm_gated(*fq.quantize_act(x), *fq.quantize_weight(w1), act=self.act,
                                   save_gate_up=True)
        y = fq.gemm(*fq.quantize_act(h), *fq.quantize_weight(w2), out_dtype=BF16)
        self.saved = x, h, gate_up, w1, w2
        return y

    def backward(self, dy):
        """dy: bf16 [M][hidden], M a multiple of 128 -> (dx, dw1, dw2)."""
        x, h, gate_up, w1, w2 = self.saved
        dh = fq.gemm(*fq.quantize_act(dy), *fq.quantize_weight_t(w2), out_dtype=BF16)
        dw2 = fq.gemm_rowscaled(*fq.quantize_act_t(dy), *fq.quantize_act_t(h))
        q, s, qt, st = fq.gated_backward(dh, gate_up, act=self.act)
        dx = fq.gemm(q, s, *fq.quantize_weight_t(w1), out_dtype=BF16)
        dw1 = fq.gemm_rowscaled(qt, st, *fq.quantize_act_t(x))
        return dx, dw1, dw2


def train(layer, target, tokens, hidden, steps, lr):
    losses = []
    for k in range(steps):
        g = torch.Generator(device="cuda")
        g.manual_seed(1000 + k)
        x = torch.randn((tokens, hidden), generator=g, device="cuda").to(BF16)
        e = layer.forward(x).float() - target.forward(x).float()
        losses.append(float(e.square().mean()))
        dy = (e * (2.0 / hidden)).to(BF16)
        _, dw1, dw2 = layer.backward(dy)
        layer.w1 -= lr / tokens * dw1
        layer.w2 -= lr / tokens * dw2
    return losses


class Int8Layer:
    """The layer with int8 weights, one scale per output channel."""

    def __init__(self, layer):
        self.act = layer.act
        self.w1 = fq.quantize_token_i8(layer.w1.to(BF16))
        self.w2 = fq.quantize_token_i8(layer.w2.to(BF16))

    def __call__(self, x):
        h = fq.gemm_i8_gated(*fq.quantize_token_i8(x), *self.w1, act=self.act)
        return fq.gemm_i8(*fq.quantize_token_i8(h), *self.w2, out_dtype=BF16)


def experts(layers, x, counts):
    """Rows of x grouped by expert -> bf16 outputs, one call a projection."""
    off = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
    w1 = [fq.quantize_weight(l.w1.to(BF16)) for l in layers]
    w2 = [fq.quantize_weight(l.w2.to(BF16)) for l in layers]
    stack = lambda ws: (torch.stack([w[0] for w in ws]), torch.stack([w[1] for w in ws]))   # noqa: E731
    h = fq.grouped_gemm_gated(*fq.quantize_act(x), off, *stack(w1), act=layers[0].act)
    return fq.grouped_gemm(*fq.quantize_act(h), off, *stack(w2), out_dtype=BF16)


def timed(f, n=50):
    for _ in range(5):
        f()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(n):
        f()
    torch.cuda.synchronize()
    return (time.perf_counter() - t) / n * 1e6


def rel(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=4096, help="per training step, a multiple of 128")
    ap.add_argument("--hidden", type=int, default=7168, help="a multiple of 128")
    ap.add_argument("--ffn", type=int, default=2048, help="a multiple of 128")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=150.0)
    a = ap.parse_args(argv)
    target, layer = Layer(a.hidden, a.ffn, 1), Layer(a.hidden, a.ffn, 2)
    losses = train(layer, target, a.tokens, a.hidden, a.steps, a.lr)
    print(f"training in FP8: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")

    served = Int8Layer(layer)
    x = torch.randn((256, a.hidden), device="cuda").to(BF16)
    y = layer.forward(x)
    print(f"served in INT8: {rel(served(x), y):.4f} of the FP8 outputs' norm off them")
    for m in (1, 16, 256):
        print(f"  {m:4d} tokens: {timed(lambda: served(x[:m])):7.1f} us a call")

    layers = [Layer(a.hidden, a.ffn, 10 + e) for e in range(4)]
    counts = [100, 0, 29, 127]
    y = experts(layers, x, counts)
    lo, worst = 0, 0.0
    for l, n in zip(layers, counts):
        if n:
            worst = max(worst, rel(y[lo:lo + n], l.forward(x[lo:lo + n])))
        lo += n
    print(f"experts in one call: within {worst:.1e} of each expert's own call")
    return losses


if __name__ == "__main__":
    if not torch.cuda.is_available():
        sys.exit("needs an MI355X (gfx950) GPU")
    main()
