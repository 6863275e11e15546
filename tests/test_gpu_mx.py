"""MXFP4 quantisation and product on the GPU against the 64-bit reference:
codes and scales bit for bit, products within the bounds of mx_reference."""
import sys

import numpy as np
import pytest

from cnn_convolution_fwd_amd import binding as B
from tests import mx_reference as R
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def draw(rng, rows, k, dtype):
    """Values over many binades, exact in dtype: (float64 array, device tensor)."""
    torch = torch_cuda()
    x = rng.normal(size=(rows, k)) * 2.0 ** rng.integers(-12, 12, (rows, 1)) * np.exp(0.8 * rng.normal(size=k))
    t = torch.from_numpy(x.astype(np.float32)).cuda()
    t = t.bfloat16() if dtype == "bf16" else t
    return t.float().cpu().numpy().astype(np.float64), t


def mx(x):
    """Reference MXFP4 of x: (values, MxTensor on the device)."""
    torch = torch_cuda()
    codes, scales = R.pack(*R.quantize(x))
    return R.values(codes, scales, x.shape[1]), B.MxTensor(torch.from_numpy(codes).cuda(),
                                                            torch.from_numpy(scales).cuda(), x.shape[1])


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------ quantisation

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 31), (3, 32), (2, 33), (5, 64), (7, 100), (1, 4096), (257, 129),
                                    (64, 1000), (3, 4097)])
def test_quantize_bits(rows, k, dtype):
    rng = np.random.default_rng(rows * 10007 + k)
    x, t = draw(rng, rows, k, dtype)
    say("quantize", rows, k, dtype)
    got = B.mx_quantize(t)
    codes, scales = R.pack(*R.quantize(x))
    assert np.array_equal(got.scales.cpu().numpy(), scales)
    assert np.array_equal(got.codes.cpu().numpy(), codes)
    back = B.mx_dequantize(got, dtype)
    assert np.array_equal(host(back), R.values(codes, scales, k))


def test_quantize_every_bf16():
    """Every bf16 value, 32 of one exponent a block, and every special value's block."""
    torch = torch_cuda()
    bits = np.arange(65536, dtype=np.uint16).reshape(-1, 32)
    t = torch.from_numpy(bits.view(np.int16).copy()).cuda().view(torch.bfloat16)
    x = host(t)
    got = B.mx_quantize(t)
    codes, scales = R.pack(*R.quantize(x))
    assert np.array_equal(got.codes.cpu().numpy(), codes) and np.array_equal(got.scales.cpu().numpy(), scales)


def test_quantize_ties_zeros_and_specials():
    torch = torch_cuda()
    x = np.zeros((9, 64), np.float32)
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.99, -0.25, -0.75, -5.0, -7.5, -0.0, 4.0]
    for i, e in enumerate((0, -100, 90, -126)):
        x[i, :16] = np.ldexp(np.array(ties, np.float32), e)
    x[4, 3], x[5, 40], x[6, 0] = np.nan, np.inf, -np.inf
    x[7, 5] = 2.0 ** -149
    got = B.mx_quantize(torch.from_numpy(x).cuda())
    codes, scales = R.pack(*R.quantize(x))
    assert np.array_equal(got.codes.cpu().numpy(), codes) and np.array_equal(got.scales.cpu().numpy(), scales)
    back = host(B.mx_dequantize(got))
    assert np.isnan(back[4, :32]).all() and (back[4, 32:] == 0).all() and np.isnan(back[5, 32:]).all()


def test_quantize_strided_and_unaligned_rows():
    torch = torch_cuda()
    for dtype in ("f32", "bf16"):
        x, t = draw(np.random.default_rng(5), 33, 203, dtype)
        for view, ref in ((t[:, 1:102], x[:, 1:102]), (t[1::2, 3:], x[1::2, 3:]), (t[5, 7:], x[5:6, 7:])):
            got = B.mx_quantize(view)
            codes, scales = R.pack(*R.quantize(ref))
            assert np.array_equal(got.codes.cpu().numpy().reshape(codes.shape), codes)
            assert np.array_equal(got.scales.cpu().numpy().reshape(scales.shape), scales)
    nhwc = torch.randn(2, 3, 5, 40, device="cuda")
    assert B.mx_quantize(nhwc).shape == (2, 3, 5, 40)
    assert B.mx_dequantize(B.mx_quantize(nhwc)).shape == (2, 3, 5, 40)
    assert B.mx_quantize(torch.empty(0, 40, device="cuda")).codes.shape == (0, 32)


def test_quantize_writes_nothing_else():
    torch = torch_cuda()
    rows, k = 3, 70
    cp, sp = B.mx_pitches(k)
    codes = torch.full((rows * cp + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows * sp + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    out = B.MxTensor(codes[:rows * cp].view(rows, cp), scales[:rows * sp].view(rows, sp), k)
    B.mx_quantize(torch.randn(rows, k, device="cuda"), out=out)
    assert (codes[rows * cp:] == 0xA5).all() and (scales[rows * sp:] == 0xA5).all()


# ------------------------------------------------------------ product

def check(x, xt, w, wt, dtype_y, bias=None, act="none"):
    torch = torch_cuda()
    bt = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
    y, err = R.matmul(x, w, None if bias is None else bias.astype(np.float32), act)
    got = B.mx_matmul(xt, wt, bias=bt, act=act, out_dtype=dtype_y)
    if dtype_y == "mx":
        R.assert_mx_close(got.codes.cpu().numpy(), got.scales.cpu().numpy(), y, err)
    else:
        R.assert_close(host(got), y, err, dtype_y == "bf16")
    return got


SIZES = [(1, 1, 1), (1, 8, 32), (1, 17, 33), (2, 130, 300), (3, 64, 256), (13, 1000, 2000), (16, 16, 4096),
         (17, 33, 100), (31, 32, 255), (32, 96, 257), (33, 129, 512), (64, 64, 64), (65, 1, 700), (100, 260, 31),
         (128, 128, 128), (129, 257, 600), (200, 384, 1024), (500, 72, 40), (257, 513, 289), (1, 4096, 512),
         (5, 40, 16384), (1000, 8, 96)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype_y", ["f32", "bf16", "mx"])
def test_matmul(m, n, k, dtype_y):
    rng = np.random.default_rng(m * 1000003 + n * 1009 + k)
    say("matmul", m, n, k, dtype_y)
    x, xt = mx(rng.normal(size=(m, k)) * np.exp(rng.normal(size=(m, 1))))
    w, wt = mx(rng.normal(size=(n, k)) * np.exp(0.5 * rng.normal(size=k)))
    check(x, xt, w, wt, dtype_y)
    check(x, xt, w, wt, dtype_y, bias=rng.normal(size=n) * 3, act=["relu", "silu", "gelu"][(m + n + k) % 3])


@pytest.mark.parametrize("m,n,k", [(2100, 2200, 96), (4100, 2300, 300), (8200, 1030, 70), (2561, 2817, 40),
                                   (2900, 2900, 3000), (2561, 2817, 2500), (4000, 2600, 2049)])
@pytest.mark.parametrize("dtype_y", ["f32", "bf16", "mx"])
def test_matmul_many_tiles(m, n, k, dtype_y):
    """More tiles than the device holds at once, ragged in both directions, short and long sums (64-bit products on the GPU)."""
    torch = torch_cuda()
    rng = np.random.default_rng(m + n + k)
    say("matmul", m, n, k, dtype_y)
    x, xt = mx(rng.normal(size=(m, k)) * np.exp(rng.normal(size=(m, 1))))
    w, wt = mx(rng.normal(size=(n, k)))
    bias = (rng.normal(size=n) * 3).astype(np.float32)
    xd, wd, bd = torch.from_numpy(x).cuda(), torch.from_numpy(w).cuda(), torch.from_numpy(bias).cuda()
    v = (xd @ wd.t() + bd.double()).cpu().numpy()
    size = (xd.abs() @ wd.abs().t() + bd.double().abs()).cpu().numpy()
    y, err = R.activate(v, "silu"), 1.2 * (k / 8 + 4) * R.U * size + 2.0 ** -20 * np.abs(v)
    got = B.mx_matmul(xt, wt, bias=bd, act="silu", out_dtype=dtype_y)
    if dtype_y == "mx":
        R.assert_mx_close(got.codes.cpu().numpy(), got.scales.cpu().numpy(), y, err)
    else:
        R.assert_close(host(got), y, err, dtype_y == "bf16")


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("m,n,k", [(4, 200, 640), (300, 200, 640)])
def test_matmul_activations_over_a_wide_range(act, m, n, k):
    rng = np.random.default_rng(7)
    x, xt = mx(rng.normal(size=(m, k)) * 2.0 ** rng.integers(-10, 6, (m, 1)))
    w, wt = mx(rng.normal(size=(n, k)))
    for dtype_y in ("f32", "mx"):
        check(x, xt, w, wt, dtype_y, act=act)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", [(1, 96, 500), (1, 1000, 4096), (4, 33, 129), (16, 256, 2048), (40, 70, 333),
                                   (200, 136, 640)])
def test_matmul_quantises_x_as_quantize_does(m, n, k, dtype):
    """x in 16 or 32 bits gives, bit for bit, what its MXFP4 form gives; rows may be strided."""
    torch = torch_cuda()
    rng = np.random.default_rng(m + n + k)
    _, t = draw(rng, m, k + 5, dtype)
    _, wt = mx(rng.normal(size=(n, k)))
    for view in (t[:, 5:], t[:, 2:k + 2], t[:, :k].contiguous()):
        say("raw x", m, n, k, dtype, view.stride())
        got = B.mx_matmul(view, wt, out_dtype="f32")
        assert torch.equal(got, B.mx_matmul(B.mx_quantize(view), wt, out_dtype="f32"))
        x = R.rounded(host(view))
        y, err = R.matmul(x, R.values(wt.codes.cpu().numpy(), wt.scales.cpu().numpy(), k))
        R.assert_close(host(got), y, err)


@pytest.mark.parametrize("m", [1, 8, 40, 70, 300])
def test_matmul_nan_rows_and_extreme_scales(m):
    """A NaN or infinite block makes its row of y NaN and no other; a NaN block of w its column; scales at the ends of their range."""
    torch = torch_cuda()
    rng = np.random.default_rng(11)
    k, n = 700, 150
    x = rng.normal(size=(m, k))
    x[m // 2, 100] = np.inf
    if m > 1:
        x[0] *= 2.0 ** -120
        x[m - 1, 650] = np.nan
    w = rng.normal(size=(n, k))
    w[3, 690] = np.nan
    w[5] = 0.0
    if m > 2:
        w[7] *= 2.0 ** 100
    xv, xt = mx(x)
    wv, wt = mx(w)
    for dtype_y in ("f32", "bf16", "mx"):
        check(xv, xt, wv, wt, dtype_y)
    got = host(B.mx_matmul(xt, wt, out_dtype="f32"))
    assert np.isnan(got[:, 3]).all() and np.isnan(got[m // 2]).all()
    assert np.isnan(host(B.mx_matmul(torch.from_numpy(x).float().cuda(), wt))[m // 2]).all()


@pytest.mark.parametrize("m,n,k", [(1, 130, 600), (3, 70, 2100), (50, 40, 100), (140, 300, 520)])
def test_matmul_writes_nothing_else(m, n, k):
    torch = torch_cuda()
    rng = np.random.default_rng(3)
    _, xt = mx(rng.normal(size=(m, k)))
    _, wt = mx(rng.normal(size=(n, k)))
    for dt in (torch.float32, torch.bfloat16):
        buf = torch.full((m * n + 64,), 7.0, dtype=dt, device="cuda")
        B.mx_matmul(xt, wt, out=buf[:m * n].view(m, n))
        assert (buf[m * n:] == 7).all()
        off = buf[3:3 + m * n].view(m, n)  # y at an address that is aligned to its elements alone
        assert torch.equal(B.mx_matmul(xt, wt, out=off), B.mx_matmul(xt, wt, out_dtype="f32").to(dt))
    cp, sp = B.mx_pitches(n)
    codes = torch.full((m * cp + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((m * sp + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    B.mx_matmul(xt, wt, out=B.MxTensor(codes[:m * cp].view(m, cp), scales[:m * sp].view(m, sp), n))
    assert (codes[m * cp:] == 0xA5).all() and (scales[m * sp:] == 0xA5).all()


@pytest.mark.parametrize("m,n,k", [(1, 512, 4096), (24, 1000, 4096), (130, 640, 8192), (600, 512, 512)])
def test_matmul_is_reproducible_and_takes_a_dirty_workspace(m, n, k):
    torch = torch_cuda()
    rng = np.random.default_rng(4)
    _, t = draw(rng, m, k, "bf16")
    _, wt = mx(rng.normal(size=(n, k)))
    first = B.mx_matmul(t, wt, out_dtype="f32")
    desc = B.MxMatmulDesc(m, n, k, B.BF16, B.F32, k, 0)
    ws = torch.full((max(1, B.mx_matmul_workspace_size(desc)),), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(B.mx_matmul(t, wt, out_dtype="f32", workspace=ws), first)


def test_matmul_on_another_stream_and_in_a_graph():
    torch = torch_cuda()
    rng = np.random.default_rng(6)
    _, t = draw(rng, 20, 1024, "bf16")
    _, wt = mx(rng.normal(size=(256, 1024)))
    want = B.mx_matmul(t, wt, act="gelu", out_dtype="f32")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = B.mx_matmul(t, wt, act="gelu", out_dtype="f32")
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    static = t.clone()
    with torch.cuda.graph(graph):
        y = B.mx_matmul(static, wt, act="gelu", out_dtype="f32")
    for i in range(4):
        static.copy_(t * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, B.mx_matmul(t * (i + 1), wt, act="gelu", out_dtype="f32"))


def test_matmul_of_nhwc_activations_is_a_pointwise_convolution():
    """The product over channels equals the 1x1 convolution of the same 4-bit values."""
    torch = torch_cuda()
    rng = np.random.default_rng(8)
    x = rng.normal(size=(2 * 7 * 9, 64))
    xv, xt = mx(x)
    wv, wt = mx(rng.normal(size=(96, 64)))
    x4 = B.MxTensor(xt.codes.view(2, 7, 9, -1), xt.scales.view(2, 7, 9, -1), 64)
    y = B.mx_matmul(x4, wt, out_dtype="f32")
    conv = B.conv2d_fwd(torch.from_numpy(xv.reshape(2, 7, 9, 64)).float().cuda(),
                        torch.from_numpy(wv.reshape(96, 64, 1, 1)).float().cuda(), layout="NHWC")
    assert y.shape == (2, 7, 9, 96)
    _, err = R.matmul(xv, wv)
    assert (np.abs(host(y) - host(conv)).reshape(-1, 96) <= 2 * err + 1e-5 * np.abs(xv) @ np.abs(wv).T).all()


def test_matmul_empty():
    torch = torch_cuda()
    _, wt = mx(np.ones((8, 40)))
    assert B.mx_matmul(torch.empty(0, 40, device="cuda"), wt).shape == (0, 8)
    assert B.mx_matmul(torch.empty(3, 0, 40, device="cuda"), wt).shape == (3, 0, 8)


@pytest.mark.parametrize("case", ["k", "w_type", "bias", "act", "out", "dtype", "rows", "device", "scales"])
def test_refusals(case):
    torch = torch_cuda()
    x = torch.randn(4, 64, device="cuda")
    w = B.mx_quantize(torch.randn(8, 64, device="cuda"))
    with pytest.raises((ValueError, TypeError)):
        if case == "k":
            B.mx_matmul(x[:, :32].contiguous(), w)
        elif case == "w_type":
            B.mx_matmul(x, x)
        elif case == "bias":
            B.mx_matmul(x, w, bias=torch.zeros(7, device="cuda"))
        elif case == "act":
            B.mx_matmul(x, w, act="tanh")
        elif case == "out":
            B.mx_matmul(x, w, out=torch.empty(4, 9, device="cuda"))
        elif case == "dtype":
            B.mx_quantize(x.half())
        elif case == "rows":
            B.mx_quantize(x.t())
        elif case == "device":
            B.mx_matmul(x.cpu(), w)
        else:
            B.mx_dequantize(B.MxTensor(w.codes, w.scales[:, :1], 64))
