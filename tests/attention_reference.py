"""64-bit numpy reference of rotary positions, the paged MXFP4 cache and attention, written from the formulas in
include/cfwd.h (no code shared with the library), and the error bounds that the GPU tests hold the kernels to.

Bounds.  fp32 has a rounding unit of u = 2^-24.
* Rotation: sine and cosine are within 2^-23, two products and a sum round by u each, relative to |a| + |b|:
  (2^-23 + 2 u) (|a| + |b|) = 2^-22 (|a| + |b|); then one rounding to the output's type.
* Scores: products of two bf16 (or of a bf16 and a value of the cache) are exact, the sum over dim in some order with one
  rounding a product: dim u sum |q k|; times scale, and the weight's exponent is rounded to u of its size twice (the
  product with scale log2(e), whose own rounding it is, and the difference from the maximum).  A weight's relative error
  is then at most d = scale dim u sum |q k| + 3 u (|s| + |m|) + 2^-21 (the power of two), plus its rounding to bf16, 2^-8.
  Over the cache a query enters in two 8-bit parts, exactly or within 2^-21 of its largest of 128 values, which adds
  scale 2^-21 max |q| sum |k| to a score's error.
* Output: o = sum w v / sum w with every w off by a relative r: off by sum w r (v - o) / sum w, and by a factor 1 + r
  (below 1.02) for what is of second order; the sums over n keys add n u of sum w |v| / sum w, joined parts 64 u; then
  one rounding to bf16, 2^-8 of the result.
"""
import numpy as np

U = 2.0 ** -24
HALF = {"f32": U, "bf16": 2.0 ** -8}


def axes_and_frequencies(rotary, sections, base, order):
    axes, freq, pairs = [], [], rotary // 2
    if order == "turns":
        left = list(sections)
        while sum(left):
            for a in range(len(left)):
                if left[a]:
                    left[a] -= 1
                    axes.append(a)
    else:
        axes = [a for a, n in enumerate(sections) for _ in range(n)]
    if order == "each":
        freq = [base ** (-i / n) for n in sections for i in range(n)]
    else:
        freq = [base ** (-i / pairs) for i in range(pairs)]
    return np.array(axes, np.int64), np.array(freq)


def rotate(x, positions, axes, freq, adjacent):
    """(result, |a| + |b| of every value's pair) of x [tokens, heads, dim]."""
    pairs = len(axes)
    angle = (positions.astype(np.float64)[:, axes] * freq)[:, None]
    first = np.arange(pairs) * (2 if adjacent else 1)
    second = first + (1 if adjacent else pairs)
    y, size = x.copy(), np.zeros_like(x)
    a, b = x[..., first], x[..., second]
    y[..., first] = a * np.cos(angle) - b * np.sin(angle)
    y[..., second] = a * np.sin(angle) + b * np.cos(angle)
    size[..., first] = size[..., second] = np.abs(a) + np.abs(b)
    return y, size


def attend(q, k, v, causal, scale, parts=False):
    """(output, bound before its own rounding) of one sequence: q [nq, heads, dim], k and v [nk, kv heads, dim]; parts:
    queries enter in two parts."""
    nq, heads, dim = q.shape
    nk, kv_heads, _ = k.shape
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for h in range(heads):
        g = h // (heads // kv_heads)
        for i in range(nq):
            n = nk - nq + 1 + i if causal else nk
            if n <= 0:
                continue
            keys, values = k[:n, g], v[:n, g]
            with np.errstate(invalid="ignore"):
                s = keys @ q[i, h] * scale
                m = s.max()
                w = np.exp(s - m)
                r = scale * dim * U * (np.abs(keys) @ np.abs(q[i, h])) + 3 * U * (np.abs(s) + abs(m)) + 2.0 ** -21 + 2.0 ** -8
                if parts:
                    for d in range(0, dim, 128):
                        r += scale * 2.0 ** -21 * np.abs(q[i, h, d:d + 128]).max() * np.abs(keys[:, d:d + 128]).sum(1)
                w /= w.sum()
                out[i, h] = w @ values
                bound[i, h] = 1.02 * ((w * r) @ np.abs(values - out[i, h])) + (n + 64) * U * (w @ np.abs(values))
    return out, bound


def check(got, want, bound, dtype="bf16"):
    """Every value within its bound and the one rounding to dtype; NaN where want is NaN."""
    got = np.asarray(got, np.float64)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), "NaN in %d places instead of %d" % (np.isnan(got).sum(), nan.sum())
    err = np.abs(got - want)
    most = bound + HALF[dtype] * (np.abs(want) + bound) + 1e-38
    bad = ~nan & ~(err <= most)
    assert not bad.any(), "%d of %d values off, worst %.3g of %.3g" % (
        bad.sum(), bad.size, err[bad].max(), most[bad][err[bad].argmax()])
