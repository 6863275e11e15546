"""MXFP4 products at the sizes where one way of computing them gives way to another, against products in 64 bits."""
import numpy as np
import pytest

from cnn_convolution_fwd_amd import binding as B
from tests import mx_reference as R
from tests.test_gpu_mx import host, mx, say, torch_cuda

pytestmark = pytest.mark.gpu

SHAPES = [
    # short sums: one, two, three and four stages of 128; whole and ragged runs of y; one column of tiles; few rows left
    (2100, 2200, 128), (2100, 2200, 256), (2200, 2056, 512), (2305, 2049, 129), (33000, 100, 130), (34000, 64, 500),
    (2100, 2200, 513),
    # few tiles: 64 and 128 rows high, sums in parts
    (500, 1000, 2100), (70, 300, 4000), (1500, 2500, 700), (130, 1500, 9000), (65, 128, 16500), (64, 16400, 600),
    (60, 512, 16384), (64, 16384, 40),
    # few rows: 16, 32 and 64 by one, two and four sets of columns; several runs of K a wave
    (20, 16500, 300), (30, 9000, 1000), (64, 9000, 1000), (50, 1000, 8000), (9, 16400, 4500), (3, 40, 70000), (16, 8200, 2500),
    (1, 16384, 130), (32, 16384, 4096), (33, 16384, 1024),
]


def product(m, n, k, bias):
    torch = torch_cuda()
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    x, xt = mx(rng.normal(size=(m, k)) * np.exp(rng.normal(size=(m, 1))))
    w, wt = mx(rng.normal(size=(n, k)))
    xd, wd = torch.from_numpy(x).cuda(), torch.from_numpy(w).cuda()
    v, size = xd @ wd.t(), xd.abs() @ wd.abs().t()
    bd = None
    if bias:
        bd = torch.from_numpy((rng.normal(size=n) * 3).astype(np.float32)).cuda()
        v, size = v + bd.double(), size + bd.double().abs()
    return xt, wt, bd, v.cpu().numpy(), size.cpu().numpy()


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_products(m, n, k):
    for bias, act in ((False, "none"), (True, "gelu")):
        xt, wt, bd, v, size = product(m, n, k, bias)
        y, err = R.activate(v, act), 1.2 * (k / 8 + 4) * R.U * size + 2.0 ** -20 * np.abs(v)
        for dtype_y in ("f32", "bf16", "mx"):
            say("matmul", m, n, k, bias, act, dtype_y)
            got = B.mx_matmul(xt, wt, bias=bd, act=act, out_dtype=dtype_y)
            if dtype_y == "mx":
                R.assert_mx_close(got.codes.cpu().numpy(), got.scales.cpu().numpy(), y, err)
            else:
                R.assert_close(host(got), y, err, dtype_y == "bf16")


@pytest.mark.parametrize("m,n,k", [(2100, 2200, 200), (2200, 2056, 400), (500, 1000, 700), (1500, 2500, 700)])
def test_writes_nothing_else(m, n, k):
    torch = torch_cuda()
    xt, wt, _, _, _ = product(m, n, k, False)
    for dt in (torch.float32, torch.bfloat16):
        say("matmul", m, n, k, dt)
        buf = torch.full((m * n + 64,), 7.0, dtype=dt, device="cuda")
        B.mx_matmul(xt, wt, out=buf[:m * n].view(m, n))
        assert (buf[m * n:] == 7).all()
    cp, sp = B.mx_pitches(n)
    codes = torch.full((m * cp + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((m * sp + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    B.mx_matmul(xt, wt, out=B.MxTensor(codes[:m * cp].view(m, cp), scales[:m * sp].view(m, sp), n))
    assert (codes[m * cp:] == 0xA5).all() and (scales[m * sp:] == 0xA5).all()


@pytest.mark.parametrize("m,n,k", [(33000, 100, 250), (2100, 2200, 500), (70, 300, 700), (20, 9000, 300)])
def test_a_nan_stays_in_its_row_or_column(m, n, k):
    """A NaN block of x or w, last or first of a row, makes its row or column of y NaN and nothing else."""
    torch = torch_cuda()
    rng = np.random.default_rng(k)
    x, w = rng.normal(size=(m, k)), rng.normal(size=(n, k))
    x[m - 1, k - 1], x[m // 2, 0], w[n - 2, k - 1] = np.nan, np.inf, np.nan
    (_, xt), (_, wt) = mx(x), mx(w)
    bad = np.zeros((m, n), bool)
    bad[m - 1], bad[m // 2], bad[:, n - 2] = True, True, True
    for dtype_y in ("f32", "bf16"):
        say("matmul", m, n, k, dtype_y)
        assert np.array_equal(np.isnan(host(B.mx_matmul(xt, wt, out_dtype=dtype_y))), bad)
    back = host(B.mx_dequantize(B.mx_matmul(xt, wt, act="relu", out_dtype="mx")))
    blocks = np.repeat(np.add.reduceat(bad, np.arange(0, n, 32), axis=1) > 0, 32, axis=1)[:, :n]
    assert np.array_equal(np.isnan(back), blocks)
