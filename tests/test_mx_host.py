"""Argument checks of the MXFP4 and gated-norm entry points on the host: every
refusal names its reason and happens before anything is launched (no GPU here)."""
import ctypes

import pytest

from cnn_convolution_fwd_amd import binding as B

P = 1 << 20  # stands for a device pointer: no refused call looks behind it


def status(st):
    return st, B.library().cfwd_last_error().decode()


def matmul(m=70, n=8, k=64, x_dtype=B.BF16, y_dtype=B.F32, stride=64, act=0, x=P, xs=None, w=P * 2, ws=P * 3, bias=None,
           y=P * 4, ys=None, work=P * 5, work_bytes=1 << 20):
    d = B.MxMatmulDesc(m, n, k, x_dtype, y_dtype, stride, act)
    return status(B.library().cfwd_mx_matmul(ctypes.byref(d), x, xs, w, ws, bias, y, ys, work, work_bytes, None))


def norm(rows=4, c=64, per=0, eps=1e-6, post=1, pre=1, dtype=B.BF16, stream=B.BF16, out=B.BF16, b=P, r=P * 2, gate=None,
         pw=None, s=P * 3, h=P * 4, hs=None):
    d = B.GatedNormDesc(rows, c, per, 1.0, eps, post, pre, dtype, stream, out)
    return status(B.library().cfwd_gated_norm(ctypes.byref(d), b, r, gate, pw, None, None, None, s, h, hs, None))


def test_sizes():
    c, s = ctypes.c_size_t(), ctypes.c_size_t()
    f = B.library().cfwd_mx_size
    for rows, k, want in ((3, 33, (96, 12)), (0, 5, (0, 0)), (1, 128, (64, 4)), (2, 129, (160, 16)),
                          (1 << 33, 1 << 20, (1 << 52, 1 << 48))):
        assert f(rows, k, ctypes.byref(c), ctypes.byref(s)) == B.OK and (c.value, s.value) == want
        assert rows == 0 or (c.value // rows, s.value // rows) == B.mx_pitches(k)
    for rows, k in ((-1, 5), (1, 0), (1, (1 << 22) + 1)):
        assert f(rows, k, ctypes.byref(c), ctypes.byref(s)) == B.ERR_INVALID_ARG
    assert f(1, 1, None, None) == B.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(k=0), dict(dtype=B.I8), dict(dtype=B.MXFP4), dict(dtype=9),
                                dict(x=None), dict(x=P + 1), dict(codes=P * 2 + 8), dict(scales=P * 3 + 2), dict(stride=63),
                                dict(codes=P), dict(scales=P), dict(scales=P * 2)])
def test_quantize_refusals(kw):
    a = dict(rows=4, k=64, dtype=B.BF16, x=P, stride=64, codes=P * 2, scales=P * 3)
    a.update(kw)
    st, why = status(B.library().cfwd_mx_quantize(a["rows"], a["k"], a["dtype"], a["x"], a["stride"], a["codes"],
                                                  a["scales"], None))
    assert st == B.ERR_INVALID_ARG and why


@pytest.mark.parametrize("kw", [dict(y=P * 2), dict(y=P + 2), dict(y=None), dict(dtype=B.MXFP4)])
def test_dequantize_refusals(kw):
    a = dict(dtype=B.F32, y=P)
    a.update(kw)
    st, why = status(B.library().cfwd_mx_dequantize(4, 64, a["dtype"], P * 2, P * 3, a["y"], None))
    assert st == B.ERR_INVALID_ARG and why


@pytest.mark.parametrize("kw", [dict(m=-1), dict(n=0), dict(k=0), dict(k=(1 << 22) + 1), dict(x_dtype=B.I8),
                                dict(y_dtype=B.I8), dict(stride=10), dict(act=4), dict(act=-1), dict(x=None),
                                dict(w=None), dict(ws=None), dict(y=None), dict(xs=P * 6), dict(ys=P * 6),
                                dict(x_dtype=B.MXFP4), dict(y_dtype=B.MXFP4), dict(w=P * 2 + 8), dict(ws=P * 3 + 1),
                                dict(x=P + 1), dict(y=P * 4 + 2), dict(bias=P * 7 + 2), dict(y=P), dict(y=P * 2),
                                dict(y=P * 3), dict(bias=P * 4), dict(work=P * 2), dict(work=P * 4),
                                dict(work=P * 5 + 16)])
def test_matmul_refusals(kw):
    st, why = matmul(**kw)
    assert st == B.ERR_INVALID_ARG and why


def test_matmul_workspace_and_size_limits():
    assert matmul(work=None)[0] == B.ERR_WORKSPACE
    assert matmul(work_bytes=16)[0] == B.ERR_WORKSPACE
    d = B.MxMatmulDesc(1 << 36, 1 << 20, 64, B.BF16, B.F32, 64, 0)
    with pytest.raises(B.CfwdError) as e:
        B.mx_matmul_workspace_size(d)
    assert e.value.status == B.ERR_UNSUPPORTED
    assert B.mx_matmul_workspace_size(B.MxMatmulDesc(0, 8, 64, B.BF16, B.F32, 64, 0)) == 0
    assert B.mx_matmul_workspace_size(B.MxMatmulDesc(70, 8, 64, B.BF16, B.F32, 64, 0)) >= 70 * 32 + 70 * 4


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(c=0), dict(c=(1 << 22) + 1), dict(post=3), dict(pre=-1),
                                dict(dtype=B.I8), dict(stream=B.I8), dict(dtype=B.F32), dict(out=B.F32),
                                dict(out=B.MXFP4), dict(hs=P * 6), dict(eps=-1.0), dict(eps=float("nan")),
                                dict(eps=float("inf")), dict(per=-1), dict(b=None, r=None), dict(s=None, h=None),
                                dict(b=P + 1), dict(h=P * 4 + 1), dict(pw=P * 6 + 2), dict(h=P), dict(h=P * 2),
                                dict(s=P + 128), dict(s=P * 4), dict(gate=P * 3), dict(pw=P * 3)])
def test_gated_norm_refusals(kw):
    st, why = norm(**kw)
    assert st == B.ERR_INVALID_ARG and why


def test_nothing_to_do():
    assert matmul(m=0, x=None, y=None, w=None, ws=None, work=None)[0] == B.OK
    assert norm(rows=0, b=None, r=None)[0] == B.OK
    assert B.library().cfwd_mx_quantize(0, 5, B.F32, None, 5, None, None, None) == B.OK


def test_convolutions_refuse_the_new_names():
    """The types and activations that only the new calls take stay refused elsewhere."""
    d = B.make_desc(1, 4, 8, 8, 4, 3, 3, 1, 1)
    d.dtype = B.MXFP4
    with pytest.raises(B.CfwdError) as e:
        B.output_dims(d)
    assert e.value.status == B.ERR_INVALID_ARG
    d.dtype = B.F32
    ep = B.Epilogue(None, None, B.ACT_SILU)
    st = B.conv2d_fwd_ex_raw(d, B.algo("direct"), P, P * 2, 0, 0, ep, P * 3, P * 4, 1 << 20, 0)
    assert st == B.ERR_INVALID_ARG
