"""An inverted-bottleneck block with 4-bit products: depthwise 3x3 convolution, norm,
1x1 convolution that widens, gelu, 1x1 convolution that narrows, gate and residual.

The depthwise convolution runs in NCHW; from there on the channels are the rows'
values (NHWC), and the norm hands its output to the first product in MXFP4,
the first product its own to the second.  The block's gate, residual scale and the
next block's norm are one call, so a chain of blocks reads and writes the
residual stream once a block.  The feed-forward half of a transformer layer is the
same four calls without the convolution.

    python examples/mx_inverted_bottleneck.py [--n 32 --size 28 --channels 512 --expand 4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from cnn_convolution_fwd_amd import binding as cfwd  # noqa: E402


class InvertedBottleneck:
    """Weights as a checkpoint gives them (float32): depthwise [c, 1, 3, 3], norm weight and bias [c], widen [f, c] and
    narrow [c, f] with their biases, gate [c] (the layer's scale).  The two matrices are kept in 4 bits."""

    def __init__(self, weights, eps: float = 1e-6):
        self.depthwise = weights["depthwise"].bfloat16().contiguous()
        self.norm_w, self.norm_b = weights["norm_w"], weights["norm_b"]
        self.widen, self.widen_b = cfwd.mx_quantize(weights["widen"]), weights["widen_b"]
        self.narrow, self.narrow_b = cfwd.mx_quantize(weights["narrow"]), weights["narrow_b"]
        self.gate = weights["gate"].bfloat16()
        self.eps = eps

    def __call__(self, x):
        """x, and the result, NHWC bfloat16 [n, h, w, c]."""
        c = x.shape[-1]
        d = cfwd.conv2d_fwd(cfwd.convert_layout(x, "NHWC", "NCHW"), self.depthwise, padding=1, groups=c)
        d = cfwd.convert_layout(d, "NCHW", "NHWC")
        _, h = cfwd.gated_norm(None, residual=d, pre="layer", pre_weight=self.norm_w, pre_bias=self.norm_b,
                               eps=self.eps, out_dtype="mx", want_sum=False)
        u = cfwd.mx_matmul(h, self.widen, bias=self.widen_b, act="gelu", out_dtype="mx")
        o = cfwd.mx_matmul(u, self.narrow, bias=self.narrow_b, out_dtype="bf16")
        y, _ = cfwd.gated_norm(o, residual=x, gate=self.gate, pre="none")
        return y


def random_weights(c: int, f: int, seed: int = 0, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device=device)  # noqa: E731
    return {"depthwise": normal(c, 1, 3, 3) / 3, "norm_w": 1 + 0.1 * normal(c), "norm_b": 0.1 * normal(c),
            "widen": normal(f, c) * c ** -0.5, "widen_b": 0.1 * normal(f), "narrow": normal(c, f) * f ** -0.5,
            "narrow_b": 0.1 * normal(c), "gate": 0.5 * normal(c)}


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--n", type=int, default=32)
    ap.add_argument("--size", type=int, default=28)
    ap.add_argument("--channels", type=int, default=512)
    ap.add_argument("--expand", type=int, default=4)
    a = ap.parse_args(argv)
    block = InvertedBottleneck(random_weights(a.channels, a.channels * a.expand))
    x = torch.randn(a.n, a.size, a.size, a.channels, device="cuda").bfloat16()
    for _ in range(3):
        y = block(x)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(20):
        y = block(x)
    end.record()
    end.synchronize()
    us = start.elapsed_time(end) / 20 * 1e3
    flops = 4.0 * x.numel() * a.channels * a.expand
    print("%s block, %d -> %d channels: %.1f us, %.1f TFLOP/s in the products, output rms %.3f"
          % (tuple(x.shape), a.channels, a.channels * a.expand, us, flops / us / 1e6, float(y.float().square().mean().sqrt())))


if __name__ == "__main__":
    main()
