"""Sizes whose byte counts would pass 64 bits are refused, and the largest ones that are taken are counted right (no GPU here)."""
import ctypes

import pytest

from cnn_convolution_fwd_amd import binding as B
from tests.test_mx_host import P, matmul, norm, status


def quantize(rows, k, stride, codes=P * 2, scales=P * 3):
    return status(B.library().cfwd_mx_quantize(rows, k, B.F32, P, stride, codes, scales, None))


@pytest.mark.parametrize("rows,k,stride", [((1 << 32) + 1, 64, 1 << 32), (1 << 38, 64, 1 << 40), ((1 << 22) + 1, 64, 1 << 40),
                                           ((1 << 38) + 1, 64, 64), (1 << 40, 1 << 22, 1 << 22)])
def test_rows_and_strides_together(rows, k, stride):
    st, why = quantize(rows, k, stride)
    assert st == B.ERR_INVALID_ARG and ("x_stride" in why or "rows" in why)


def test_a_products_strides():
    st, why = matmul(m=1 << 24, stride=1 << 40)
    assert st == B.ERR_INVALID_ARG and "x_stride" in why


@pytest.mark.parametrize("kw", [dict(rows=1 << 40, c=1 << 22), dict(rows=(1 << 38) + 1)])
def test_rows_of_norms(kw):
    st, why = norm(dtype=B.F32, stream=B.F32, out=B.F32, **kw)
    assert st == B.ERR_INVALID_ARG and "rows" in why


def test_overlaps_of_the_largest_tensors_are_seen():
    top = 1 << 62
    st, why = norm(dtype=B.F32, stream=B.F32, out=B.F32, rows=1 << 38, c=1 << 22, h=P + top - 4, s=None)
    assert st == B.ERR_INVALID_ARG and "overlap" in why
    st, why = quantize(1 << 38, 1 << 22, 1 << 22, codes=P + top - 16)
    assert st == B.ERR_INVALID_ARG and "overlap" in why
    st, why = quantize(1 << 20, 64, 1 << 40, codes=P + top - (1 << 42))
    assert st == B.ERR_INVALID_ARG and "overlap" in why
    st, why = status(B.library().cfwd_mx_dequantize(1 << 38, 1 << 22, B.F32, P * 16, P + (1 << 61) + (1 << 60), P, None))
    assert st == B.ERR_INVALID_ARG and "overlap" in why
    d = ctypes.c_size_t()
    assert B.library().cfwd_mx_size(1 << 38, 1 << 22, ctypes.byref(d), ctypes.byref(ctypes.c_size_t())) == B.OK
    assert d.value == 1 << 59


def test_what_depends_on_the_device_is_kept_for_each(monkeypatch):
    """A workspace depends on the device's CUs: another device's is asked for anew."""
    asked = iter([100, 200])
    monkeypatch.setattr(B, "mx_matmul_workspace_size", lambda desc: next(asked))
    B._mx_matmul_desc.cache_clear()
    try:
        sizes = (70, 8, 64, B.BF16, B.F32, 64, 0)
        assert [B._mx_matmul_desc(dev, *sizes)[1] for dev in (0, 1, 0, 1)] == [100, 200, 100, 200]
    finally:
        B._mx_matmul_desc.cache_clear()
