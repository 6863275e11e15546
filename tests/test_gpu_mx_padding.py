"""Bytes of a row's scales past its blocks do not count, whatever they hold, in every kernel of the product."""
import pytest

from cnn_convolution_fwd_amd import binding as B
from tests.test_gpu_mx import say, torch_cuda

pytestmark = pytest.mark.gpu


# 1, 2 and 3 blocks in the last word of scales: few rows (16, 32 and 64 of them), few tiles 64 and 128 rows high, a sum in
# parts, x resident for 256 and for 512 values, tiles of 128 in several rounds, tiles of 256
@pytest.mark.parametrize("m,n,k", [(4, 300, 1060), (30, 300, 140), (60, 500, 200), (500, 1000, 2100), (70, 300, 4000),
                                   (1500, 2500, 700), (130, 1500, 9000), (2100, 2200, 96), (2100, 2200, 140),
                                   (2100, 2200, 290), (2100, 2200, 420), (66000, 128, 700), (66000, 128, 730),
                                   (4000, 2600, 2049), (4000, 2600, 2140)])
def test_padding_of_scales_is_ignored(m, n, k):
    torch = torch_cuda()
    x, w = B.mx_quantize(torch.randn(m, k, device="cuda")), B.mx_quantize(torch.randn(n, k, device="cuda"))
    want = B.mx_matmul(x, w, out_dtype="f32")
    kb = -(-k // 32)
    assert kb % 4 and bool(want.isfinite().all())
    for t in (x, w):
        say("padding", m, n, k, "x" if t is x else "w")
        t.scales[:, kb:] = 255
        assert torch.equal(B.mx_matmul(x, w, out_dtype="f32"), want)
        t.scales[:, kb:] = 127
