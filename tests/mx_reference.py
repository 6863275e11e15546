"""64-bit numpy reference of the MXFP4 operators and the gated norms, written
from the formulas in include/cfwd.h (no code shared with the library), and the
error bounds that the GPU tests hold the kernels to.

Bounds.  fp32 has a rounding unit of u = 2^-24.
* Product: exact products, sums in some order with at most one rounding for
  every 8 products, then bias: |err| <= (k / 8 + 4) u (sum |x w| + |bias|).
* Activation: slopes are below 1.2; its own error stays below 2^-20 |v| (the
  exponent's argument is rounded to a relative u and is scaled by |v|).
* Row sums of the norms: at most 64 roundings on any path, so 64 u = 2^-18
  relative to the sum of magnitudes; the same again on what is computed from it.
* One rounding to bf16: 2^-8 of the result.
* A 4-bit result may be any code that a value within the bound rounds to.
"""
import numpy as np

U = 2.0 ** -24
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
MIDDLES = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])


def pad_blocks(x):
    rows, k = x.shape
    kb = -(-k // 32)
    v = np.zeros((rows, kb * 32))
    v[:, :k] = x
    return v.reshape(rows, kb, 32)


def exponent_bytes(amax):
    """Exponent byte of blocks with these largest magnitudes (NaN or inf: 255)."""
    fine = np.isfinite(amax)
    _, e = np.frexp(np.where(fine, amax, 1.0))  # amax = f 2^e, f in [0.5, 1)
    byte = np.clip(e - 1 - 2 + 127, 0, None)
    return np.where(fine, np.where(amax == 0, 0, byte), 255).astype(np.int64)


def magnitude_codes(a):
    """Code of the E2M1 magnitude nearest to a >= 0, ties to the even code."""
    c = np.searchsorted(MIDDLES, a)  # middles below a
    tie = (c < 7) & (MIDDLES[np.minimum(c, 6)] == a)
    return c + (tie & (c % 2 == 1))


def quantize(x):
    """(nibbles [rows][kb][32], bytes [rows][kb]) of float x [rows][k]."""
    v = pad_blocks(np.asarray(x, np.float64))
    with np.errstate(invalid="ignore"):
        amax = np.where(np.isnan(v).any(-1), np.nan, np.abs(v).max(-1))
    byte = exponent_bytes(amax)
    bad = (byte == 255)[..., None]
    a = np.abs(np.where(bad, 0.0, v)) * 2.0 ** (127.0 - np.where(bad, 127, byte[..., None]))
    nib = magnitude_codes(a) | (np.signbit(v).astype(np.int64) << 3)
    return np.where(bad, 0, nib), byte


def pack(nib, byte):
    """codes [rows][16 kb] and scales [rows][kb rounded up to 4] as uint8."""
    rows, kb, _ = nib.shape
    codes = (nib[..., 0::2] | (nib[..., 1::2] << 4)).reshape(rows, kb * 16).astype(np.uint8)
    scales = np.full((rows, -(-kb // 4) * 4), 127, np.uint8)
    scales[:, :kb] = byte
    return codes, scales


def values(codes, scales, k):
    """Values that codes and scales stand for, in 64 bits."""
    c = np.asarray(codes).astype(np.int64)
    rows, kb = c.shape[0], c.shape[1] // 16
    nib = np.stack([c & 15, c >> 4], -1).reshape(rows, kb, 32)
    s = np.asarray(scales)[:, :kb].astype(np.float64)
    unit = np.where(s == 255, np.nan, 2.0 ** (s - 127))
    v = np.where(nib > 7, -1.0, 1.0) * GRID[nib & 7] * unit[..., None]
    return v.reshape(rows, kb * 32)[:, :k]


def rounded(x):
    """x as MXFP4 holds it."""
    codes, scales = pack(*quantize(x))
    return values(codes, scales, np.asarray(x).shape[1])


def activate(v, act):
    with np.errstate(over="ignore", invalid="ignore"):
        if act == "relu":
            return np.where(v < 0, 0.0, v)
        if act == "silu":
            return v / (1 + np.exp(-v))
        if act == "gelu":
            return 0.5 * v * (1 + np.tanh(np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)))
    return v


def matmul(x, w, bias=None, act="none"):
    """(y, bound) of act(x w^T + bias) for MXFP4-exact x and w."""
    b = np.zeros(w.shape[0]) if bias is None else np.asarray(bias, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        v = x @ w.T + b
        err = (x.shape[1] / 8 + 4) * U * (np.abs(x) @ np.abs(w).T + np.abs(b))
    if act != "none":
        err = 1.2 * err + 2.0 ** -20 * np.abs(v)
    return activate(v, act), err


def norm(v, err, kind, weight, bias, eps):
    """(norm of v, bound) over the last axis, for v known to within err."""
    if kind == "none":
        return v, err
    w = 1.0 if weight is None else np.asarray(weight, np.float64)
    c = 0.0 if bias is None else np.asarray(bias, np.float64)
    mean = v.mean(-1, keepdims=True) if kind == "layer" else 0.0
    d = v - mean
    rstd = 1 / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    out = d * rstd * w + c
    err_rms = np.sqrt((err * err).mean(-1, keepdims=True))
    size = np.abs(v) + np.abs(mean) + (np.abs(v).mean(-1, keepdims=True) if kind == "layer" else 0.0)
    bound = np.abs(w) * rstd * (err + 2 * err_rms * (1 + np.abs(d) * rstd)) + 64 * U * (size * rstd * np.abs(w) + np.abs(c))
    return out, bound


def gated_norm(b, r, gate, per, alpha, post, post_w, post_b, pre, pre_w, pre_b, eps):
    """(s, bound of s, h, bound of h)."""
    rows = (b if b is not None else r).shape[0]
    zero = np.zeros_like(b if b is not None else r)
    v, err = norm(b if b is not None else zero, zero, post, post_w, post_b, eps)
    if gate is not None:
        g = gate[np.arange(rows) // per]
        v, err = v * g, np.abs(g) * err + 2 * U * np.abs(v * g)
    if r is not None:
        err = err + 2 * U * (np.abs(alpha * r) + np.abs(v))
        v = np.float64(np.float32(alpha)) * r + v
    h, err_h = norm(v, err, pre, pre_w, pre_b, eps)
    return v, err, h, err_h


def assert_close(got, want, bound, bf16=False):
    """got within bound of want (and one rounding to bf16); NaN and infinities in the same places."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    lim = np.broadcast_to(bound, want.shape)[fine] + (2.0 ** -8 * np.abs(want[fine]) if bf16 else U * np.abs(want[fine]))
    off = np.abs(got[fine] - want[fine])
    lim = lim + 2.0 ** -133  # results under the smallest normal number
    assert (off <= lim).all(), "off by %g times the bound" % float((off / lim).max())


def assert_mx_close(codes, scales, want, bound):
    """codes / scales are a quantisation of some values within bound of want; padding is 0 and 127."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    rows, n = want.shape
    kb = -(-n // 32)
    assert codes.shape == (rows, kb * 16) and scales.shape == (rows, -(-kb // 4) * 4)
    assert (scales[:, kb:] == 127).all()
    c = codes.astype(np.int64)
    nib = np.stack([c & 15, c >> 4], -1).reshape(rows, kb, 32)
    assert (nib.reshape(rows, -1)[:, n:] & 7 == 0).all()
    v, e = pad_blocks(want), pad_blocks(np.broadcast_to(bound, want.shape))
    bad = ~np.isfinite(v).all(-1)
    got = scales[:, :kb].astype(np.int64)
    assert ((got == 255) == bad).all()
    assert (nib[bad] == 0).all()
    v, e = np.where(bad[..., None], 0.0, v), np.where(bad[..., None], 0.0, e)
    a = np.abs(v)
    lo, hi = exponent_bytes(np.maximum(a - e, 0).max(-1)), exponent_bytes((a + e).max(-1))
    assert ((lo <= got) & (got <= hi) | bad).all(), "a block's scale is outside its bound"
    unit = 2.0 ** (127.0 - np.where(bad, 127, got))[..., None]
    signed = np.where(nib > 7, -1.0, 1.0) * GRID[nib & 7]

    def to_grid(t):
        return np.where(t < 0, -1.0, 1.0) * GRID[magnitude_codes(np.abs(t))]

    ok = (to_grid((v - e) * unit) <= signed) & (signed <= to_grid((v + e) * unit))
    assert ok[~bad].all(), "%d codes are outside their bounds" % int((~ok[~bad]).sum())
