"""The inverted-bottleneck example end to end, against the same chain in 64 bits.

Each call is held to its own bound elsewhere; here the chain is: the reference
rounds where the block does (bf16 after the depthwise convolution and after the
second product, MXFP4 before each product).  What is left are the roundings of o and
y to bf16 (2^-9 each, of the larger of the two summands) and 4-bit values
that a difference in the last bits of their arguments rounds the other way (fewer than
1 in 10^4, each by at most a step of half its size: 2^-7 in the norm of y): 1e-2.
"""
import os
import sys

import numpy as np
import pytest

import oracle
from cnn_convolution_fwd_amd.workloads import bf16_bits, bf16_to_f32
from tests import mx_reference as R
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def bf16(x):
    return bf16_to_f32(bf16_bits(np.asarray(x, np.float32))).astype(np.float64)


@pytest.mark.parametrize("n,h,w,c,f", [(2, 7, 7, 64, 256), (1, 9, 5, 72, 200), (4, 14, 14, 128, 512)])
def test_block(n, h, w, c, f):
    torch = torch_cuda()
    from mx_inverted_bottleneck import InvertedBottleneck, random_weights
    weights = random_weights(c, f, seed=n)
    x = torch.randn(n, h, w, c, device="cuda").bfloat16()
    y = InvertedBottleneck(weights)(x).float().cpu().numpy().astype(np.float64).reshape(-1, c)
    k = {name: t.float().cpu().numpy() for name, t in weights.items()}
    xh = x.float().cpu().numpy()
    d, _ = oracle.conv2d(np.ascontiguousarray(xh.transpose(0, 3, 1, 2)), bf16(k["depthwise"]).astype(np.float32), 1, 1, 1, c)
    d = bf16(np.asarray(d).transpose(0, 2, 3, 1)).reshape(-1, c)
    hn, _ = R.norm(d, np.zeros_like(d), "layer", k["norm_w"], k["norm_b"], 1e-6)
    u, _ = R.matmul(R.rounded(hn), R.rounded(k["widen"]), k["widen_b"], "gelu")
    o, _ = R.matmul(R.rounded(u), R.rounded(k["narrow"]), k["narrow_b"])
    want = xh.reshape(-1, c).astype(np.float64) + bf16(k["gate"]) * bf16(o)
    assert np.linalg.norm(y - want) <= 1e-2 * np.linalg.norm(want)


def test_main_runs(capsys):
    from mx_inverted_bottleneck import main
    torch_cuda()
    main(["--n", "2", "--size", "8", "--channels", "64"])
    assert "TFLOP/s" in capsys.readouterr().out
