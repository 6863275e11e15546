"""Rotary positions, the paged MXFP4 cache, and attention over it and over packed prompts, against 64 bits."""
import numpy as np
import pytest

from cnn_convolution_fwd_amd import binding as B
from tests import attention_reference as A
from tests import mx_reference as M
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

DT = {"f32": "float32", "bf16": "bfloat16"}


def heads(torch, seed, tokens, n, dim, dtype="bf16", spread=1.0):
    g = torch.Generator()
    g.manual_seed(seed)
    x = torch.randn(tokens, n, dim, generator=g) * torch.randn(n, dim, generator=g).mul(0.4).exp() * spread
    return x.to(getattr(torch, DT[dtype])).cuda()


def np64(t):
    return t.double().cpu().numpy()


def ints(torch, values, dtype=None):
    return torch.tensor(values, dtype=dtype or torch.int32, device="cuda")


# ------------------------------------------------------------------ rotary positions

ROPE = [  # tokens, q heads, k heads, dim, rotary, sections, order
    (1, 32, 8, 128, 128, (64,), "runs"), (5, 3, 1, 64, 64, (10, 12, 10), "runs"), (7, 2, 2, 80, 40, (7, 13), "turns"),
    (3, 1, 0, 72, 72, (12, 24), "each"), (33, 4, 4, 96, 90, (45,), "each"), (2, 1, 1, 7, 6, (1, 0, 2), "runs"),
    (1, 1, 1, 1, 0, (0,), "runs"), (1000, 12, 3, 128, 64, (16, 16), "turns"), (4100, 2, 1, 32, 32, (16,), "runs"),
    (9, 2, 1, 1024, 1024, (512,), "runs"),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("tokens,h,kh,dim,rotary,sections,order", ROPE)
def test_rope(tokens, h, kh, dim, rotary, sections, order, adjacent, dtype):
    torch = torch_cuda()
    qkv = heads(torch, tokens, tokens, h + 2 * kh + 1, dim, dtype)  # parts of one tensor, one head of which is nobody's
    q, k = qkv[:, :h], qkv[:, h:h + kh] if kh else None
    rng = np.random.default_rng(dim)
    positions = rng.integers(-1000, 1 << 20, (tokens, len(sections)))
    table = B.rope_table(rotary, sections, base=10000.0, order=order)
    axes, freq = A.axes_and_frequencies(rotary, sections, 10000.0, order)
    before = qkv.clone()
    wide = ints(torch, positions, torch.int64)
    got_q, got_k = B.rope(q, k, wide, table, adjacent=adjacent)
    assert torch.equal(qkv, before) and (got_k is None) == (k is None)
    for x, y in ((q, got_q), (k, got_k)):
        if x is not None:
            want, size = A.rotate(np64(x), positions, axes, freq, adjacent)
            A.check(np64(y), want, size * 2.0 ** -22, dtype)
            if rotary < dim:
                assert torch.equal(y[..., rotary:], x[..., rotary:])
    # in place, from 32-bit positions: the same bits, and nothing else touched
    in_place = B.rope(q, k, wide.int(), table, adjacent=adjacent, q_out=q, k_out=k)
    assert in_place[0] is q and torch.equal(q, got_q) and (k is None or torch.equal(k, got_k))
    assert torch.equal(qkv[:, h + kh:], before[:, h + kh:])


def test_rope_far_positions():
    """Angles stay exact to 2^-32 of a turn where 32 bits, and even 64-bit products, would lose them."""
    torch = torch_cuda()
    positions = np.array([[0], [1], [-1], [2 ** 31 - 1], [-2 ** 31], [2 ** 24 + 1], [2 ** 40 + 12345]])
    freq = [1.0, 0.5, 2.0 ** -10, 2.0 ** -20]  # their products with positions are exact in 64 bits
    table = B.rope_table(8, frequencies=freq)
    x = torch.zeros(7, 1, 8, device="cuda")
    x[..., :4] = 1
    y = np64(B.rope(x, None, ints(torch, positions, torch.int64), table)[0])[:, 0]
    angle = positions * np.array(freq)
    assert np.abs(y[:, :4] - np.cos(angle)).max() <= 2.0 ** -22 and np.abs(y[:, 4:] - np.sin(angle)).max() <= 2.0 ** -22


def test_rope_axes_out_of_range_stay():
    torch = torch_cuda()
    table = B.rope_table(16, (4, 4))
    pairs = table.pairs.clone()
    pairs[1, 1], pairs[6, 1], pairs[3, 1] = 2, -1, 1 << 30
    x = heads(torch, 3, 5, 2, 16, "f32")
    y, _ = B.rope(x, None, ints(torch, np.full((5, 2), 7)), B.RopeTable(pairs, 2))
    still = [1, 6, 3, 9, 14, 11]
    assert torch.equal(y[..., still], x[..., still]) and not torch.equal(y[..., [0, 8]], x[..., [0, 8]])


def test_rope_unaligned_rows():
    torch = torch_cuda()
    for dtype in ("bf16", "f32"):
        flat = heads(torch, 5, 1, 1, 4000, dtype).view(-1)
        q = flat[1:].as_strided((6, 3, 20), (101, 33, 1))
        p = ints(torch, np.arange(6))
        want = B.rope(q.contiguous(), None, p, B.rope_table(20))[0]
        assert torch.equal(B.rope(q, None, p, B.rope_table(20))[0], want)
        out = torch.zeros(4000, dtype=q.dtype, device="cuda")
        view = out[3:].as_strided((6, 3, 20), (97, 31, 1))
        B.rope(q, None, p, B.rope_table(20), q_out=view)
        assert torch.equal(view, want)
        view.zero_()
        assert not out.any()


# ------------------------------------------------------------------ the cache

class Paged:
    """A cache whose pages belong to sequences of these lengths, in no order, with dirty pages between."""

    def __init__(self, torch, lengths, page, n_heads, dim, seed=0, fill=True):
        rng = np.random.default_rng(seed)
        counts = [-(-n // page) for n in lengths]
        total = sum(counts) + 2
        order = rng.permutation(total)
        self.lengths, self.page, self.dim, self.heads = lengths, page, dim, n_heads
        self.rows = np.full((len(lengths), max(counts + [1]) + 1), 1 << 30)  # entries that no token needs: nonsense
        at = 0
        for i, n in enumerate(counts):
            self.rows[i, :n] = order[at:at + n]
            at += n
        self.table = ints(torch, self.rows)
        self.cache = B.mx_cache(total, page, n_heads, dim)
        cp, sp = B.mx_pitches(dim)
        shape = (total, n_heads, page)
        for t in self.cache:
            codes = rng.integers(0, 256, (*shape, cp), dtype=np.uint8)
            scales = rng.integers(118, 126, (*shape, sp), dtype=np.uint8)
            # slots that no sequence owns hold NaN, and so do the bytes past a row's blocks
            owned = np.zeros((total, page), bool)
            for i, n in enumerate(lengths):
                for t0 in range(n):
                    owned[self.rows[i, t0 // page], t0 % page] = True
            scales.transpose(0, 2, 1, 3)[~owned] = 255
            scales[..., -(-dim // 32):] = 255
            if dim % 32:  # codes past the row's values are 0
                keep = np.arange(cp) < dim // 2
                codes = np.where(keep, codes, 0).astype(np.uint8)
            t.codes.copy_(torch.from_numpy(codes))
            t.scales.copy_(torch.from_numpy(scales))

    def slots(self, seq, first, count):
        t = np.arange(first, first + count)
        return self.rows[seq, t // self.page] * self.page + t % self.page

    def values(self, which, seq):
        """Tokens [n, heads, dim] of a sequence, from codes and scales."""
        t = self.cache[which]
        codes, scales = t.codes.cpu().numpy(), t.scales.cpu().numpy()
        n = self.lengths[seq]
        out = np.zeros((n, self.heads, self.dim))
        for i in range(n):
            p, o = self.rows[seq, i // self.page], i % self.page
            out[i] = M.values(codes[p, :, o], scales[p, :, o], self.dim)
        return out


CACHE = [  # lengths, page, heads, dim
    ([1], 16, 1, 32), ([5, 0, 33, 16], 16, 2, 64), ([100, 7], 48, 3, 80), ([64, 65, 63], 64, 8, 128), ([3, 9], 1, 1, 1),
    ([40, 40], 7, 2, 40), ([700], 256, 4, 256), ([2] * 70, 16, 1, 33),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,page,n,dim", CACHE)
def test_cache_write_and_read(lengths, page, n, dim, dtype):
    torch = torch_cuda()
    paged = Paged(torch, lengths, page, n, dim)
    before = [(t.codes.clone(), t.scales.clone()) for t in paged.cache]
    kept = [x // 3 for x in lengths]
    new = [x - y for x, y in zip(lengths, kept)]
    slots = np.concatenate([paged.slots(i, a, b) for i, (a, b) in enumerate(zip(kept, new))])
    slots = np.concatenate([slots[:1], [-1], slots[1:], [paged.cache.k.codes.shape[0] * page]])  # two of padding
    kv = heads(torch, dim, len(slots), 2 * n, dim, dtype)
    kv[1], kv[-1] = float("nan"), 7.0
    if len(slots) > 4:
        kv[2, 0, 0], kv[3, -1, -1] = float("inf"), float("nan")
    k, v = kv[:, :n], kv[:, n:]
    for idx in (torch.int32, torch.int64):
        for t, (c, s) in zip(paged.cache, before):
            t.codes.copy_(c)
            t.scales.copy_(s)
        B.mx_cache_write(k, v, paged.cache, ints(torch, slots, idx))
        for t, x, (c, s) in zip(paged.cache, (k, v), before):
            nib, byte = M.quantize(np64(x).reshape(-1, dim))
            codes, scales = M.pack(nib, byte)
            want_c, want_s = c.cpu().numpy(), s.cpu().numpy()
            for i, slot in enumerate(slots):
                if 0 <= slot < want_c.shape[0] * page:
                    want_c[slot // page, :, slot % page] = codes.reshape(len(slots), n, -1)[i]
                    want_s[slot // page, :, slot % page] = scales.reshape(len(slots), n, -1)[i]
            assert np.array_equal(t.codes.cpu().numpy(), want_c) and np.array_equal(t.scales.cpu().numpy(), want_s)
    total = sum(lengths)
    starts = ints(torch, np.concatenate([[0], np.cumsum(lengths)]))
    full = getattr(torch, DT[dtype])
    out = torch.full((2, total + 3, n, dim), 7.0, dtype=full, device="cuda")
    got = B.mx_cache_read(paged.cache, paged.table, starts, total + 3, k_out=out[0], v_out=out[1])
    for which in (0, 1):
        want = np.concatenate([paged.values(which, i) for i in range(len(lengths))])
        assert np.array_equal(np64(got[which])[:total], want, equal_nan=True) and bool((out[which, total:] == 7).all())
    fresh = B.mx_cache_read(paged.cache, paged.table, starts, total, dtype=dtype)
    assert all(torch.equal(a.view(torch.uint8), b[:total].contiguous().view(torch.uint8)) for a, b in zip(fresh, out))


def test_cache_read_with_bad_pages_and_starts():
    """Rows whose page is none of the cache's, or outside the table, are left as they were; so is all that starts misplace."""
    torch = torch_cuda()
    paged = Paged(torch, [40, 20], 16, 2, 64)
    table = paged.table.clone()
    table[0, 1], table[1, 0] = -1, 1 << 30
    out = torch.full((2, 80, 2, 64), 7.0, device="cuda")
    B.mx_cache_read(paged.cache, table[:, :2].contiguous(), ints(torch, [0, 40, 60]), 80, k_out=out[0], v_out=out[1])
    want = paged.values(0, 0)
    assert np.array_equal(np64(out[0])[:16], want[:16]) and bool((out[0, 16:40] == 7).all())
    assert bool((out[0, 40:56] == 7).all()) and bool((out[0, 60:] == 7).all())
    for starts in ([5, 3, 1], [-7, 1 << 30, 2], [70, 75, 1 << 30]):
        B.mx_cache_read(paged.cache, table, ints(torch, starts), 80)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ attention over the cache

DECODE = [  # lengths, tokens, page, heads, kv heads, dim
    ([1], 1, 16, 1, 1, 32), ([31, 32, 33, 0], 1, 16, 8, 2, 64), ([500], 1, 16, 32, 8, 128), ([129, 5, 1], 1, 64, 6, 2, 96),
    ([3, 0, 200, 2], 4, 32, 8, 2, 128), ([1000, 17], 1, 48, 7, 1, 256), ([300, 40], 7, 16, 8, 1, 128),
    ([64, 130], 5, 128, 16, 2, 256), ([5, 400], 9, 16, 16, 2, 64), ([70], 40, 16, 4, 2, 32), ([260, 3], 2, 64, 9, 3, 160),
    ([2500, 1, 900], 1, 256, 4, 4, 128), ([20] * 70, 1, 16, 2, 1, 64),
]


@pytest.mark.parametrize("lengths,tokens,page,h,kh,dim", DECODE)
def test_cache_attention(lengths, tokens, page, h, kh, dim):
    torch = torch_cuda()
    paged = Paged(torch, lengths, page, kh, dim, seed=dim)
    q = heads(torch, dim, len(lengths) * tokens, h, dim).view(len(lengths), tokens, h, dim)
    got = B.mx_cache_attention(q, paged.cache, paged.table, ints(torch, lengths))
    assert torch.equal(got, B.mx_cache_attention(q, paged.cache, paged.table, ints(torch, lengths)))
    for i in range(len(lengths)):
        k, v = paged.values(0, i), paged.values(1, i)
        want, bound = A.attend(np64(q[i]), k, v, True, dim ** -0.5, parts=True)
        A.check(np64(got[i]), want, bound)


def test_cache_attention_calls():
    """Strided queries, a scale, out and workspace of the caller's (dirty), another stream, no tokens, no sequences."""
    torch = torch_cuda()
    lengths = [300, 41]
    paged = Paged(torch, lengths, 32, 2, 64)
    qkv = heads(torch, 1, 2 * 3, 12, 64).view(2, 3, 12, 64)
    q = qkv[:, 1:, 2:10]
    n = ints(torch, lengths)
    want = B.mx_cache_attention(q.contiguous(), paged.cache, paged.table, n, scale=0.3)
    ws = torch.full((1 << 25,), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((3, 2, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    got = B.mx_cache_attention(q, paged.cache, paged.table, n, scale=0.3, out=out[:2], workspace=ws)
    assert torch.equal(got, want) and bool((out[2] == 7).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(B.mx_cache_attention(q, paged.cache, paged.table, n, scale=0.3), want)
    one = B.mx_cache_attention(q[:, -1], paged.cache, paged.table, n, scale=0.3)
    assert one.shape == (2, 8, 64) and torch.equal(one, want[:, -1])
    assert B.mx_cache_attention(q[:0], paged.cache, paged.table[:0], n[:0]).shape == (0, 2, 8, 64)
    assert B.mx_cache_attention(q[:, :0], paged.cache, paged.table, n).shape == (2, 0, 8, 64)


def test_cache_attention_bad_lengths_and_pages():
    """Lengths below 0 count as 0, past the table as its end; tokens on pages outside the cache are not seen."""
    torch = torch_cuda()
    paged = Paged(torch, [64, 64], 16, 1, 64)
    table = paged.table[:, :4].contiguous()
    q = heads(torch, 2, 2, 4, 64)
    got = B.mx_cache_attention(q, paged.cache, table, ints(torch, [-5, 1 << 30]))
    assert not got[0].any()
    assert torch.equal(got[1], B.mx_cache_attention(q, paged.cache, table, ints(torch, [64, 64]))[1])
    table[1, 1], table[1, 2], table[0] = -1, 1 << 30, 1 << 20
    got = B.mx_cache_attention(q, paged.cache, table, ints(torch, [64, 64]))
    assert not got[0].any()
    k, v = (np.concatenate([paged.values(w, 1)[:16], paged.values(w, 1)[48:]]) for w in (0, 1))
    want, bound = A.attend(np64(q[1:]), k, v, False, 64 ** -0.5, parts=True)
    A.check(np64(got[1:]), want, bound)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_cache_attention_nan_where_it_is_seen(dim):
    """A NaN key makes every query that sees it NaN, a NaN value the 32 columns of its block; the others stay as they are."""
    torch = torch_cuda()
    length, tokens = 200, 6
    paged = Paged(torch, [length], 16, 1, dim)
    q = heads(torch, 3, tokens, 2, dim).view(1, tokens, 2, dim)
    n = ints(torch, [length])
    clean = B.mx_cache_attention(q, paged.cache, paged.table, n)
    for at in (3, length - 3):
        seen = [i for i in range(tokens) if at < length - tokens + 1 + i]
        for which in (0, 1):
            t = paged.cache[which]
            codes, scales = t.codes.clone(), t.scales.clone()
            page, off = paged.rows[0, at // 16], at % 16
            t.codes[page, 0, off, 16:32], t.scales[page, 0, off, 1] = 0, 255
            got = B.mx_cache_attention(q, paged.cache, paged.table, n)
            t.codes.copy_(codes)
            t.scales.copy_(scales)
            nan = torch.zeros_like(got, dtype=torch.bool)
            for i in seen:
                nan[0, i, :, slice(None) if which == 0 else slice(32, 64)] = True
            assert torch.equal(torch.isnan(got), nan)
            assert torch.equal(got[~nan], clean[~nan])


# ------------------------------------------------------------------ packed prompts

PROMPT = [  # queries, keys, heads, kv heads, dim
    ([1], None, 1, 1, 8), ([77], None, 8, 2, 128), ([5, 0, 64, 130, 1], None, 4, 1, 64), ([33, 200], [70, 100], 6, 2, 72),
    ([300], None, 2, 2, 40), ([20, 3], [500, 0], 7, 1, 128), ([65, 9], [64, 1000], 3, 3, 256), ([128, 127, 129], None, 2, 1, 96),
    ([3] * 70, None, 2, 2, 64), ([1, 2], [2100, 2000], 16, 2, 128), ([140], [150], 24, 24, 80), ([200], None, 33, 1, 248),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,h,kh,dim", PROMPT)
def test_attention(nq, nk, h, kh, dim, causal):
    torch = torch_cuda()
    nk = nk or nq
    qa, ka = np.concatenate([[0], np.cumsum(nq)]), np.concatenate([[0], np.cumsum(nk)])
    # rows before the first sequence and behind the last are nobody's, and hold NaN
    q = heads(torch, dim, qa[-1] + 3, h, dim)
    kv = heads(torch, dim + 1, ka[-1] + 5, 2 * kh + 1, dim)
    q[0], q[-2:] = float("nan"), float("nan")
    kv[0], kv[-4:] = float("nan"), float("nan")
    kv[:, -1] = float("nan")
    k, v = kv[:, :kh], kv[:, kh:2 * kh]
    out = torch.full((qa[-1] + 3, h, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    got = B.attention(q, k, v, ints(torch, qa + 1), ints(torch, ka + 1), causal=causal, out=out)
    assert got is out and bool((out[0] == 7).all()) and bool((out[-2:] == 7).all())
    again = B.attention(q, k, v, ints(torch, qa + 1), ints(torch, ka + 1), causal=causal)
    assert torch.equal(again[1:-2], out[1:-2])
    for i in range(len(nq)):
        a, b = slice(qa[i] + 1, qa[i + 1] + 1), slice(ka[i] + 1, ka[i + 1] + 1)
        want, bound = A.attend(np64(q[a]), np64(k[b]), np64(v[b]), causal, dim ** -0.5)
        A.check(np64(got[a]), want, bound)


def test_attention_large_tiles():
    """Enough rows for every form of the kernel, against the same kernel's rows taken alone and a sample in 64 bits."""
    torch = torch_cuda()
    for dim, h, kh in ((64, 16, 16), (96, 16, 4), (128, 32, 8)):
        nq = [1500, 700, 1, 2600]
        qa = np.concatenate([[0], np.cumsum(nq)])
        qkv = heads(torch, dim, qa[-1], h + 2 * kh, dim)
        q, k, v = qkv[:, :h], qkv[:, h:h + kh], qkv[:, h + kh:]
        for causal in (True, False):
            got = B.attention(q, k, v, ints(torch, qa), causal=causal)
            for i in (0, 1, 2, 3):
                rows = sorted({0, nq[i] // 2, nq[i] - 1, min(255, nq[i] - 1)})
                b = slice(qa[i], qa[i + 1])
                for r in rows:
                    keys = slice(qa[i], qa[i] + r + 1) if causal else b
                    want, bound = A.attend(np64(q[qa[i] + r:qa[i] + r + 1]), np64(k[keys]), np64(v[keys]), False, dim ** -0.5)
                    A.check(np64(got[qa[i] + r:qa[i] + r + 1]), want, bound)


def test_attention_scores_of_any_size():
    """Scores from far below to far above fp32's exponent range for e^s, and rows whose maximum grows key by key."""
    torch = torch_cuda()
    n, dim = 400, 64
    q, k, v = (heads(torch, i, n, 2, dim) for i in (1, 2, 3))
    for spread in (1e-3, 30.0, 300.0):
        got = B.attention(q * spread, k, v, ints(torch, [0, n]))
        want, bound = A.attend(np64(q * spread), np64(k), np64(v), True, dim ** -0.5)
        A.check(np64(got), want, bound)
    k = k.abs() * torch.linspace(0.01, 4, n, device="cuda")[:, None, None].bfloat16()
    q = q.abs()
    got = B.attention(q, k, v, ints(torch, [0, n]), scale=1.0)
    want, bound = A.attend(np64(q), np64(k), np64(v), True, 1.0)
    A.check(np64(got), want, bound)


def test_attention_starts_out_of_range():
    torch = torch_cuda()
    q, k = heads(torch, 1, 50, 2, 64), heads(torch, 2, 60, 1, 64)
    want = B.attention(q, k, k, ints(torch, [0, 50]), ints(torch, [0, 60]))
    got = B.attention(q, k, k, ints(torch, [-9, 1 << 30]), ints(torch, [-1 << 30, 1 << 30]))
    assert torch.equal(got, want)
    for starts in ([40, 10, 30], [1 << 30, 0, 50]):
        B.attention(q, k, k, ints(torch, starts), ints(torch, starts))
    torch.cuda.synchronize()
    assert B.attention(q[:0], k, k, ints(torch, [0, 0]), ints(torch, [0, 60])).shape == (0, 2, 64)
    assert not B.attention(q, k[:0], k[:0], ints(torch, [0, 50]), ints(torch, [0, 0])).any()


@pytest.mark.parametrize("dim", [64, 80, 128, 256])
def test_attention_values_that_are_not_finite(dim):
    """NaN and infinities reach the queries that see them, all of those and no others; keys that are NaN as well."""
    torch = torch_cuda()
    n, h, kh = 150, 4, 2
    q, k, v = heads(torch, 1, n, h, dim), heads(torch, 2, n, kh, dim), heads(torch, 3, n, kh, dim)
    starts = ints(torch, [0, n])
    clean = B.attention(q, k, v, starts)
    for at in (0, 31, 32, 70, 100, n - 1):
        for value in (float("nan"), float("inf"), -float("inf")):
            bad = v.clone()
            bad[at, 1, dim - 3] = value
            got = B.attention(q, k, bad, starts)
            want = clean.clone()
            want[at:, 2:, dim - 3] = value
            assert torch.equal(torch.isnan(got), torch.isnan(want))
            assert torch.equal(got[~torch.isnan(got)], want[~torch.isnan(want)])
        bad = k.clone()
        bad[at, 0, 5] = float("nan")
        got = B.attention(q, bad, v, starts)
        assert bool(torch.isnan(got[at:, :2]).all())
        rest = torch.isnan(got)
        rest[at:, :2] = False
        assert not rest.any() and torch.equal(got[:at], clean[:at]) and torch.equal(got[:, 2:], clean[:, 2:])
    bad = v.clone()
    bad[40, 0, 1], bad[60, 0, 1] = float("inf"), -float("inf")
    got = B.attention(q, k, bad, starts)[:, :2, 1]
    assert bool(got[:40].isfinite().all()) and bool((got[40:60] == float("inf")).all()) and bool(torch.isnan(got[60:]).all())
