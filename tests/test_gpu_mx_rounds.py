"""MXFP4 products whose workgroups walk several tiles, and products that quantise x on their way, in every form."""
import pytest

from cnn_convolution_fwd_amd import binding as B
from tests import mx_reference as R
from tests.test_gpu_mx import host, say, torch_cuda

pytestmark = pytest.mark.gpu


def draw(m, k, seed, spread):
    torch = torch_cuda()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(m, k, generator=g, device="cuda") * (spread * torch.randn(m, 1, generator=g, device="cuda")).exp()


def close(got, v, size, k, act, dtype_y):
    y = R.activate(v.cpu().numpy(), act)
    err = 1.2 * (k / 8 + 4) * R.U * size.cpu().numpy() + 2.0 ** -20 * abs(v.cpu().numpy())
    if dtype_y == "mx":
        R.assert_mx_close(got.codes.cpu().numpy(), got.scales.cpu().numpy(), y, err)
    else:
        R.assert_close(host(got), y, err, dtype_y == "bf16")


# Sums of more than 512 values over more 128 x 128 tiles than two for each CU, where few columns keep 256 x 256 tiles from
# being fewer: 516, 547 and 524 tiles (rows of y that are whole 16-byte runs in both types, in fp32 alone, in neither) by
# 512 workgroups, and 1056 of three columns, the third round of them partial.
@pytest.mark.parametrize("m,n,k", [(66000, 128, 640), (70000, 100, 700), (67000, 101, 520), (45000, 300, 600)])
def test_several_tiles_a_workgroup(m, n, k):
    x, w = B.mx_quantize(draw(m, k, m + k, 1.0)), B.mx_quantize(draw(n, k, n + k, 0.0))
    xv, wv = B.mx_dequantize(x).double(), B.mx_dequantize(w).double()
    bias = 3 * draw(1, n, k, 0.0)[0]
    v, size = xv @ wv.t() + bias.double(), xv.abs() @ wv.abs().t() + bias.double().abs()
    for act in ("none", "gelu"):
        for dtype_y in ("f32", "bf16", "mx"):
            say("matmul", m, n, k, act, dtype_y)
            close(B.mx_matmul(x, w, bias=bias, act=act, out_dtype=dtype_y), v, size, k, act, dtype_y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1000, 9000, 16400])
@pytest.mark.parametrize("m,k", [(1, 4096), (1, 130), (4, 5000), (16, 2048), (13, 1002)])
def test_x_is_quantised_on_the_way(m, n, k, dtype):
    """One, two and four sets of columns a workgroup, x of either type to each type of y: bit for bit the product of
    x's MXFP4 form, and within its bounds of the product in 64 bits."""
    torch = torch_cuda()
    x = draw(m, k, m + k, 1.0).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    w = B.mx_quantize(draw(n, k, n, 0.0))
    bias = 3 * draw(1, n, k, 0.0)[0]
    packed = B.mx_quantize(x)
    xv, wv = B.mx_dequantize(packed).double(), B.mx_dequantize(w).double()
    v, size = xv @ wv.t() + bias.double(), xv.abs() @ wv.abs().t() + bias.double().abs()
    for act in ("none", "silu"):
        for dtype_y in ("f32", "bf16", "mx"):
            say("raw x", m, n, k, dtype, act, dtype_y)
            got = B.mx_matmul(x, w, bias=bias, act=act, out_dtype=dtype_y)
            want = B.mx_matmul(packed, w, bias=bias, act=act, out_dtype=dtype_y)
            if dtype_y == "mx":
                assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
            else:
                assert torch.equal(got, want)
            close(got, v, size, k, act, dtype_y)
