"""Codes of values all over a block's range, bit for bit against the 64-bit reference."""
import numpy as np
import pytest

from cnn_convolution_fwd_amd import binding as B
from tests import mx_reference as R
from tests.test_gpu_mx import host, say, torch_cuda

pytestmark = pytest.mark.gpu


def check(t):
    x = host(t)
    got = B.mx_quantize(t)
    codes, scales = R.pack(*R.quantize(x))
    assert np.array_equal(got.scales.cpu().numpy(), scales)
    assert np.array_equal(got.codes.cpu().numpy(), codes)
    assert np.array_equal(host(B.mx_dequantize(got)), R.values(codes, scales, x.shape[1]))
    return codes


@pytest.mark.parametrize("below", range(7))
def test_every_finite_bf16_value_below_its_blocks_largest(below):
    """31 values and, as the block's largest, a power of two up to six binades above them: every code from 0 to 6 is met."""
    torch = torch_cuda()
    bits = np.arange(65536)
    bits = bits[(bits & 0x7f80) != 0x7f80]
    bits = np.concatenate([bits, np.zeros(-len(bits) % 31, np.int64)]).reshape(-1, 31)
    exponent = np.minimum(((bits & 0x7f80) >> 7).max(1, keepdims=True) + below, 254)
    bits = np.concatenate([bits, exponent << 7], 1)
    say("every bf16 value", below)
    t = torch.from_numpy(bits.astype(np.uint16).view(np.int16)).cuda().view(torch.bfloat16)
    codes = check(t)
    nibbles = np.unique(np.concatenate([codes & 15, codes >> 4]) & 7)
    assert {0: {6, 7}, 1: {4, 5, 6}, 2: {2, 3, 4}, 3: {1, 2}, 4: {0, 1}, 5: {0}, 6: {0}}[below] <= set(nibbles.tolist())


def test_fp32_values_at_random_and_beside_ties():
    torch = torch_cuda()
    rng = np.random.default_rng(9)
    x = rng.uniform(1, 2, (1 << 15, 32)) * 2.0 ** rng.integers(-6, 1, (1 << 15, 32)) * rng.choice([-1, 1], (1 << 15, 32))
    say("random fp32")
    check(torch.from_numpy((x * 2.0 ** rng.integers(-120, 120, (1 << 15, 1))).astype(np.float32)).cuda())
    ties = np.concatenate([R.MIDDLES, [6.0, 7.0, 0.5, 1, 1.5, 2, 3, 4]]).astype(np.float32)
    near = np.concatenate([ties, np.nextafter(ties, np.float32(9)), np.nextafter(ties, np.float32(0))])
    block = np.zeros((2, 64), np.float32)
    block[:, :45], block[:, 45:] = near, 4.0
    block[1] = -block[1]
    say("beside ties")
    for e in (-126, -100, 0, 60, 124):
        check(torch.from_numpy(np.ldexp(block, e)).cuda())
