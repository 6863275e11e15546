"""Rotary positions, the paged cache and attention as programs call them: one after the other through a layer, in graphs,
on several streams, from shared pages, with far strides and large tensors."""
import numpy as np
import pytest

from cnn_convolution_fwd_amd import binding as B
from tests import attention_reference as A
from tests.gpu_util import torch_cuda
from tests.test_gpu_attention import Paged, heads, ints, np64

pytestmark = pytest.mark.gpu


def starts_of(torch, lengths):
    return ints(torch, np.concatenate([[0], np.cumsum(lengths)]))


def read(torch, paged, lengths=None):
    """Keys and values [n, heads, dim] of every sequence, in 64 bits."""
    lengths = paged.lengths if lengths is None else lengths
    a = np.concatenate([[0], np.cumsum(lengths)])
    k, v = B.mx_cache_read(paged.cache, paged.table, ints(torch, a), int(a[-1]), dtype="f32")
    return [(np64(k[x:y]), np64(v[x:y])) for x, y in zip(a, a[1:])]


def test_layer_from_prompts_to_single_tokens():
    """Two prompts, a second chunk of each, then two steps of one token: products, positions, cache, attention and norm."""
    torch = torch_cuda()
    h, kh, dim, c = 8, 2, 64, 256
    w_in = B.mx_quantize(heads(torch, 1, (h + 2 * kh) * dim, 1, c, "f32").view(-1, c) / 16)
    w_out = B.mx_quantize(heads(torch, 2, c, 1, h * dim, "f32").view(c, -1) / 16)
    table = B.rope_table(dim, (8, 12, 12), base=1000.0)
    chunks = [(37, 90), (5, 12), (1, 1), (1, 1)]
    total = [sum(x) for x in zip(*chunks)]
    paged = Paged(torch, total, 16, kh, dim)
    done = [0, 0]
    for step, new in enumerate(chunks):
        tokens = sum(new)
        x = heads(torch, 10 + step, tokens, 1, c).view(tokens, c)
        qkv = B.mx_matmul(x, w_in, out_dtype="bf16").view(tokens, h + 2 * kh, dim)
        at = np.concatenate([np.arange(a, a + n) for a, n in zip(done, new)])
        positions = np.stack([at // 25, at // 5 % 5, at % 5], 1)
        q, k = B.rope(qkv[:, :h], qkv[:, h:h + kh], ints(torch, positions), table)
        v = qkv[:, h + kh:]
        axes, freq = A.axes_and_frequencies(dim, (8, 12, 12), 1000.0, "runs")
        for before, after in ((qkv[:, :h], q), (qkv[:, h:h + kh], k)):
            want, size = A.rotate(np64(before), positions, axes, freq, False)
            A.check(np64(after), want, size * 2.0 ** -22)
        slots = np.concatenate([paged.slots(i, a, n) for i, (a, n) in enumerate(zip(done, new))])
        B.mx_cache_write(k, v, paged.cache, ints(torch, slots))
        done = [a + n for a, n in zip(done, new)]
        cached = read(torch, paged, done)
        if step == 0:  # from the projection itself
            o = B.attention(q, k, v, starts_of(torch, new))
            pairs = [(np64(k[:37]), np64(v[:37])), (np64(k[37:]), np64(v[37:]))]
        elif step == 1:  # what lies in the cache first
            a = starts_of(torch, done)
            back = B.mx_cache_read(paged.cache, paged.table, a, sum(done))
            o, pairs = B.attention(q, *back, starts_of(torch, new), a), cached
        else:
            o, pairs = B.mx_cache_attention(q, paged.cache, paged.table, ints(torch, done)), cached
        first = 0
        for n, (keys, values) in zip(new, pairs):
            want, bound = A.attend(np64(q[first:first + n]), keys, values, True, dim ** -0.5, parts=step > 1)
            A.check(np64(o[first:first + n]), want, bound)
            first += n
        y = B.mx_matmul(o.view(tokens, h * dim), w_out, out_dtype="bf16")
        s = B.gated_norm(y, residual=x, post="rms")[0]
        assert s.shape == (tokens, c) and bool(s.isfinite().all())
    # the second chunk of both, now as several new tokens over the cache
    for i, n in enumerate(chunks[1]):
        q = heads(torch, i, n, h, dim)
        got = B.mx_cache_attention(q[None], paged.cache, paged.table[i:i + 1], ints(torch, total[i:i + 1]))
        want, bound = A.attend(np64(q), *read(torch, paged)[i], True, dim ** -0.5, parts=True)
        A.check(np64(got[0]), want, bound)


@pytest.mark.parametrize("page", [16, 48, 64])
def test_steps_in_graphs(page):
    """A step and a prompt captured once and replayed with other positions, slots, pages and lengths, in one workspace."""
    torch = torch_cuda()
    h, kh, dim, n = 8, 2, 128, 5
    paged = Paged(torch, [700, 3, 150, 64, 0], page, kh, dim)
    other = Paged(torch, [700, 3, 150, 64, 0], page, kh, dim)  # the same
    table, workspace = B.rope_table(dim), torch.full((1 << 26,), 255, dtype=torch.uint8, device="cuda")
    x, positions = heads(torch, 0, n, h + 2 * kh, dim), ints(torch, [[0]] * n)
    slots, lengths, pages = ints(torch, [-1] * n), ints(torch, [0] * n), paged.table.clone()
    prompt, starts = heads(torch, 1, 40, h, dim), ints(torch, [0, 40])
    keys, k_starts = heads(torch, 2, 3000, 2 * kh, dim), ints(torch, [0, 3000])

    def step(cache, ws):
        q, k = B.rope(x[:, :h], x[:, h:h + kh], positions, table)
        B.mx_cache_write(k, x[:, h + kh:], cache, slots)
        return B.mx_cache_attention(q, cache, pages, lengths, workspace=ws)

    def chunk(ws):
        return B.attention(prompt, keys[:, :kh], keys[:, kh:], starts, k_starts, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(paged.cache, workspace)
        chunk(workspace)
    torch.cuda.current_stream().wait_stream(side)
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        got = step(paged.cache, workspace)
    with torch.cuda.graph(second):
        got_chunk = chunk(workspace)
    rng = np.random.default_rng(page)
    for replay in range(5):
        x.copy_(heads(torch, 20 + replay, n, h + 2 * kh, dim))
        prompt.copy_(heads(torch, 30 + replay, 40, h, dim))
        at = [int(rng.integers(0, m)) if m else -1 for m in paged.lengths]
        positions.copy_(ints(torch, [[max(a, 0)] for a in at]))
        slots.copy_(ints(torch, [int(paged.slots(i, a, 1)[0]) if a >= 0 else -1 for i, a in enumerate(at)]))
        lengths.copy_(ints(torch, [a + 1 for a in at]))
        starts.copy_(ints(torch, [0, 40 - 7 * replay]))
        k_starts.copy_(ints(torch, [0, 3000 - 500 * replay]))
        first.replay()
        second.replay()
        want = step(other.cache, None)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and not got[4].any()
        assert torch.equal(got_chunk[:40 - 7 * replay], chunk(None)[:40 - 7 * replay])
        for a, b in zip(paged.cache, other.cache):
            assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


def test_two_streams_at_once():
    """Calls on two streams, each with what it allocates itself, give what they give alone."""
    torch = torch_cuda()
    sides = []
    for i, (lengths, dim) in enumerate((([5000, 700, 1], 128), ([9000], 64))):
        cache = B.mx_cache(200, 64, 2, dim)
        kv = heads(torch, i, 200 * 64, 4, dim)
        B.mx_cache_write(kv[:, :2], kv[:, 2:], cache, torch.arange(200 * 64, device="cuda"))
        table = torch.arange(200, device="cuda", dtype=torch.int32).flip(0).repeat(len(lengths), 1).contiguous()
        q = heads(torch, 9 + i, len(lengths), 16, dim)
        n, starts = ints(torch, lengths), ints(torch, [0, 3])

        def run(q=q, cache=cache, table=table, n=n, kv=kv, starts=starts):
            return (B.mx_cache_attention(q, cache, table, n),
                    B.attention(q[:3], kv[:4000, :2], kv[:4000, 2:], ints(torch, [0, len(q)]), ints(torch, [0, 4000])),
                    *B.mx_cache_read(cache, table[:1], starts, 3))
        sides.append((torch.cuda.Stream(), run, run()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (stream, run, _) in enumerate(sides):
            with torch.cuda.stream(stream):
                got[i].append(run())
    torch.cuda.synchronize()
    for results, (_, _, want) in zip(got, sides):
        for r in results:
            assert all(torch.equal(a, b) for a, b in zip(r, want))


@pytest.mark.parametrize("page", [16, 32, 48])
@pytest.mark.parametrize("rows", [4, 24, 56, 100])  # tokens times heads of a group: each form of the kernel
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 192, 256])
def test_every_form_over_the_cache(dim, rows, page):
    torch = torch_cuda()
    lengths, tokens = [210, 0, rows // 4 + 17], rows // 4
    paged = Paged(torch, lengths, page, 1, dim, seed=rows)
    q = heads(torch, rows, 3 * tokens, 4, dim).view(3, tokens, 4, dim)
    got = B.mx_cache_attention(q, paged.cache, paged.table, ints(torch, lengths))
    for i, (k, v) in enumerate(read(torch, paged)):
        want, bound = A.attend(np64(q[i]), k, v, True, dim ** -0.5, parts=True)
        A.check(np64(got[i]), want, bound)


@pytest.mark.parametrize("dim,tokens", [(64, 1), (128, 3), (256, 1)])
def test_long_cache_in_many_parts(dim, tokens):
    torch = torch_cuda()
    lengths = [20000, 63, 7001]
    paged = Paged(torch, [1], 64, 2, dim)
    cache = B.mx_cache(500, 64, 2, dim)
    kv = heads(torch, dim, 500 * 64, 4, dim, "f32")
    B.mx_cache_write(kv[:, :2], kv[:, 2:], cache, torch.randperm(500 * 64, device="cuda", dtype=torch.int32))
    paged.cache, paged.table = cache, torch.arange(3 * 166, device="cuda", dtype=torch.int32).view(3, 166)
    paged.table = torch.cat([paged.table, paged.table + 2], 1).contiguous()  # pages of several sequences
    q = heads(torch, 3, 3 * tokens, 6, dim).view(3, tokens, 6, dim)
    got = B.mx_cache_attention(q, cache, paged.table, ints(torch, lengths))
    for i, (k, v) in enumerate(read(torch, paged, lengths)):
        want, bound = A.attend(np64(q[i]), k, v, True, dim ** -0.5, parts=True)
        A.check(np64(got[i]), want, bound)


def test_many_sequences():
    """More than the 64 that one look takes in, empty ones among them, over the cache, out of it and packed."""
    torch = torch_cuda()
    rng = np.random.default_rng(5)
    lengths = [int(n) for n in rng.integers(0, 40, 200)]
    lengths[63:66], lengths[127:129], lengths[199] = [0, 0, 0], [150, 0], 0
    paged = Paged(torch, lengths, 16, 1, 32)
    q = heads(torch, 1, 200, 2, 32)
    got = B.mx_cache_attention(q, paged.cache, paged.table, ints(torch, lengths))
    flat = heads(torch, 2, sum(lengths), 4, 32)
    a = np.concatenate([[0], np.cumsum(lengths)])
    packed = B.attention(flat[:, :2], flat[:, 2:3], flat[:, 3:], ints(torch, a))
    for i, (k, v) in enumerate(read(torch, paged)):
        want = [paged.values(w, i) for w in (0, 1)]
        assert np.array_equal(k, want[0]) and np.array_equal(v, want[1])
        want, bound = A.attend(np64(q[i:i + 1]), k, v, True, 32 ** -0.5, parts=True)
        A.check(np64(got[i:i + 1]), want, bound)
        x = np64(flat[a[i]:a[i + 1]])
        want, bound = A.attend(x[:, :2], x[:, 2:3], x[:, 3:], True, 32 ** -0.5)
        A.check(np64(packed[a[i]:a[i + 1]]), want, bound)


@pytest.mark.parametrize("n,most", [(65, 300), (128, 200), (1000, 5), (5000, 3), (4097, 2)])
@pytest.mark.parametrize("h", [1, 6])
def test_very_many_packed_sequences(n, most, h):
    """Every sequence's rows as they are alone; many empty ones, at both ends as well."""
    torch = torch_cuda()
    rng = np.random.default_rng(n)
    lengths = rng.integers(0, most + 1, n) * (rng.random(n) < 0.7)
    if n != 128:
        lengths[:3], lengths[-70:] = 0, lengths[-70:] * (n != 1000)
    else:
        lengths[:] = 128  # whole tiles
    a = np.concatenate([[0], np.cumsum(lengths)]) + 2
    total = int(a[-1]) + 3
    qkv = heads(torch, n, total, h + 2, 32)
    out = torch.full((total, h, 32), 7.0, dtype=torch.bfloat16, device="cuda")
    B.attention(qkv[:, :h], qkv[:, h:h + 1], qkv[:, h + 1:], ints(torch, a), causal=n % 2 == 0, out=out)
    assert bool((out[:2] == 7).all()) and bool((out[-3:] == 7).all())
    few = [int(i) for i in rng.choice(np.flatnonzero(lengths), 40)] + [int(np.flatnonzero(lengths)[i]) for i in (0, -1)]
    for i in few:
        s = slice(int(a[i]), int(a[i + 1]))
        x = np64(qkv[s])
        want, bound = A.attend(x[:, :h], x[:, h:h + 1], x[:, h + 1:], n % 2 == 0, 32 ** -0.5)
        A.check(np64(out[s]), want, bound)
    # all of them, by parts of 64 sequences
    for i in range(0, n, 64):
        j = min(n, i + 64)
        s = slice(int(a[i]), int(a[j]))
        part = B.attention(qkv[s, :h], qkv[s, h:h + 1], qkv[s, h + 1:], ints(torch, a[i:j + 1] - a[i]), causal=n % 2 == 0)
        assert torch.equal(part, out[s])


@pytest.mark.parametrize("n", [64, 65, 1000, 4097])
def test_very_many_sequences_read(n):
    torch = torch_cuda()
    rng = np.random.default_rng(n)
    lengths = rng.integers(0, 4, n) * (rng.random(n) < 0.7)
    lengths[0], lengths[-1] = 0, 2 * (n % 2)
    cache = B.mx_cache(n, 3, 1, 32)
    kv = heads(torch, n, 3 * n, 2, 32, "f32")
    B.mx_cache_write(kv[:, :1], kv[:, 1:], cache, torch.arange(3 * n, device="cuda"))
    pages = rng.permutation(n)
    a = np.concatenate([[0], np.cumsum(lengths)])
    rows = np.concatenate([pages[i] * 3 + np.arange(m) for i, m in enumerate(lengths)])
    got = B.mx_cache_read(cache, ints(torch, pages[:, None]), ints(torch, a), int(a[-1]), dtype="f32")
    for t, out in zip(cache, got):
        want = B.mx_dequantize(t, dtype="f32").view(3 * n, 1, 32)[torch.as_tensor(rows, device="cuda")]
        assert torch.equal(out, want)


def test_shared_pages():
    """Sequences that begin with the same pages, and one page twice in a row."""
    torch = torch_cuda()
    paged = Paged(torch, [64, 64], 16, 2, 64)
    table = torch.stack([paged.table[0, :4], paged.table[0, [0, 1, 3, 2]], paged.table[0, [0, 0, 0, 0]]])
    table[1, 2:] = paged.table[1, 2:4]
    paged.table, n = table.contiguous(), [64, 50, 40]
    q = heads(torch, 4, 3, 4, 64)
    got = B.mx_cache_attention(q, paged.cache, paged.table, ints(torch, n))
    for i, (k, v) in enumerate(read(torch, paged, n)):
        want, bound = A.attend(np64(q[i:i + 1]), k, v, True, 0.125, parts=True)
        A.check(np64(got[i:i + 1]), want, bound)


def test_queries_of_any_size_over_the_cache():
    """A power of two passes from the queries to the scale without a bit's change; values of all sizes in one query keep to
    the bound; a query that is NaN or infinite spoils no other."""
    torch = torch_cuda()
    for dim in (32, 128, 256):
        paged = Paged(torch, [90, 300], 32, 1, dim)
        n = ints(torch, paged.lengths)
        q = heads(torch, dim, 2, 6, dim)
        want = B.mx_cache_attention(q, paged.cache, paged.table, n, scale=0.25)
        for power in (-40, -7, 9, 40):
            got = B.mx_cache_attention(q * 2.0 ** power, paged.cache, paged.table, n, scale=0.25 * 2.0 ** -power)
            assert torch.equal(got, want)
        mixed = q.clone()
        mixed[:, :3] *= 2.0 ** -torch.arange(dim, device="cuda").remainder(31)
        mixed[:, 4] = 0
        got = B.mx_cache_attention(mixed, paged.cache, paged.table, n)
        for i, (k, v) in enumerate(read(torch, paged)):
            out, bound = A.attend(np64(mixed[i:i + 1]), k, v, True, dim ** -0.5, parts=True)
            A.check(np64(got[i:i + 1]), out, bound)
        bad = q.clone()
        bad[0, 1, 3], bad[1, 5, -1], bad[1, 0, 0] = float("nan"), float("inf"), -float("inf")
        got = B.mx_cache_attention(bad, paged.cache, paged.table, n, scale=0.25)
        rest = torch.ones(2, 6, dtype=torch.bool, device="cuda")
        rest[0, 1] = rest[1, 5] = rest[1, 0] = False
        assert torch.equal(got[rest], want[rest]) and bool(torch.isnan(got[0, 1]).all())


def test_few_queries_over_many_keys_that_are_not_finite():
    """The keys in parts: NaN and infinities in any part, seen by some queries only at the end."""
    torch = torch_cuda()
    nq, nk, dim = 3, 4000, 64
    q, k, v = heads(torch, 1, nq, 2, dim), heads(torch, 2, nk, 1, dim), heads(torch, 3, nk, 1, dim)
    a, b = ints(torch, [0, nq]), ints(torch, [0, nk])
    clean = B.attention(q, k, v, a, b)
    for at in (0, 1999, nk - 3, nk - 2, nk - 1):
        sees = [at < nk - nq + 1 + i for i in range(nq)]
        bad = v.clone()
        bad[at, 0, 7] = float("nan")
        got = B.attention(q, k, bad, a, b)
        want = clean.clone()
        want[torch.tensor(sees, device="cuda"), :, 7] = float("nan")
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got[~torch.isnan(want)], want[~torch.isnan(want)])
        bad = k.clone()
        bad[at, 0, 7] = float("nan")
        got = B.attention(q, bad, v, a, b)
        assert [bool(torch.isnan(g).all()) for g in got] == sees
        assert all(torch.equal(g, c) for g, c, s in zip(got, clean, sees) if not s)


@pytest.mark.parametrize("nq,nk,h,kh,dim", [(1, 60000, 2, 1, 64), (3, 40000, 1, 1, 80), (2, 20000, 4, 2, 256), (1, 130000, 1, 1, 8)])
def test_few_queries_over_very_many_keys(nq, nk, h, kh, dim):
    """Hundreds of parts for a row, joined by several threads."""
    torch = torch_cuda()
    q, k, v = heads(torch, 1, nq + 2, h, dim), heads(torch, 2, nk, kh, dim), heads(torch, 3, nk, kh, dim)
    out = torch.full_like(q, 7.0)
    B.attention(q, k, v, ints(torch, [1, nq + 1]), ints(torch, [0, nk]), out=out)
    want, bound = A.attend(np64(q[1:-1]), np64(k), np64(v), True, dim ** -0.5)
    A.check(np64(out[1:-1]), want, bound)
    assert bool((out[0] == 7).all()) and bool((out[-1] == 7).all())


@pytest.mark.parametrize("dtype,tokens", [("bf16", 13000), ("f32", 6500)])
def test_large_tensors_pass_the_caches_by(dtype, tokens):
    """Above the size from which loads pass the caches by, the same bits as from parts below it."""
    torch = torch_cuda()
    qkv = heads(torch, 1, tokens, 48, 128, dtype)
    positions, table = torch.arange(tokens, device="cuda", dtype=torch.int32).view(-1, 1), B.rope_table(128)
    for adjacent in (False, True):
        q, k = B.rope(qkv[:, :32], qkv[:, 32:40], positions, table, adjacent=adjacent)
        for at in range(0, tokens, 2500 if dtype == "bf16" else 1250):
            s = slice(at, min(tokens, at + (2500 if dtype == "bf16" else 1250)))
            part = B.rope(qkv[s, :32], qkv[s, 32:40], positions[s], table, adjacent=adjacent)
            assert torch.equal(q[s], part[0]) and torch.equal(k[s], part[1])
    whole = qkv.view(-1, 16, 128)  # three times the tokens
    slots = torch.randperm(whole.shape[0], device="cuda")
    one, parts = (B.mx_cache(-(-whole.shape[0] // 64), 64, 8, 128) for _ in (0, 1))
    B.mx_cache_write(whole[:, :8], whole[:, 8:], one, slots)
    for at in range(0, whole.shape[0], 5000):
        s = slice(at, at + 5000)
        B.mx_cache_write(whole[s, :8], whole[s, 8:], parts, slots[s])
    for a, b in zip(one, parts):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


@pytest.mark.parametrize("tokens", [9000, 40000])
def test_large_padded_writes(tokens):
    """Tokens that are left out among many, with loads that pass the caches by and without, as in small calls."""
    torch = torch_cuda()
    kv = heads(torch, 1, tokens, 16, 128)
    slots = torch.randperm(tokens, device="cuda")
    slots[::7], slots[3::64], slots[-5:] = -1, tokens + 64, -(1 << 40)
    one, parts = (B.mx_cache(-(-tokens // 64), 64, 8, 128) for _ in (0, 1))
    B.mx_cache_write(kv[:, :8], kv[:, 8:], one, slots)
    for at in range(0, tokens, 1500):
        s = slice(at, at + 1500)
        B.mx_cache_write(kv[s, :8], kv[s, 8:], parts, slots[s])
    for a, b in zip(one, parts):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    left = torch.ones(tokens, dtype=torch.bool, device="cuda")
    left[slots[(slots >= 0) & (slots < tokens)]] = False
    empty = one.k.codes.transpose(1, 2).reshape(-1, 8 * 64)[:tokens][left]
    assert left.any() and not empty.any()


def test_far_pages():
    """A cache of more than 2^32 bytes: its last pages as a small cache's."""
    torch = torch_cuda()
    page, n_heads, dim, used = 64, 8, 128, 6
    far = B.mx_cache((1 << 23) // page + used, page, n_heads, dim)
    near = B.mx_cache(used, page, n_heads, dim)
    assert far.k.codes.numel() > 1 << 32
    kv = heads(torch, 1, used * page, 2 * n_heads, dim)
    slots = torch.randperm(used * page, device="cuda")
    base = far.k.codes.shape[0] - used
    B.mx_cache_write(kv[:, :8], kv[:, 8:], near, slots)
    B.mx_cache_write(kv[:, :8], kv[:, 8:], far, slots + base * page)
    table = ints(torch, [[5, 0, 3, 1], [2, 4, 0, 0]])
    starts, lengths = ints(torch, [0, 250, 370]), ints(torch, [250, 120])
    q = heads(torch, 2, 2, 16, dim)
    for a, b in zip(B.mx_cache_read(near, table, starts, 370), B.mx_cache_read(far, table + base, starts, 370)):
        assert torch.equal(a, b)
    assert torch.equal(B.mx_cache_attention(q, near, table, lengths), B.mx_cache_attention(q, far, table + base, lengths))


def test_far_strides():
    """Rows further apart than 32 bits count."""
    torch = torch_cuda()
    flat = torch.empty(300 << 24, dtype=torch.bfloat16, device="cuda")
    k = flat.as_strided((298, 2, 64), (1 << 24, 64, 1))
    v = flat[128:].as_strided((298, 2, 64), (1 << 24, 64, 1))
    q = flat[256:].as_strided((4, 4, 64), (1 << 30, 64, 1))
    for i, t in enumerate((k, v, q)):
        t.copy_(heads(torch, i, *t.shape))
    a, b = ints(torch, [0, 4]), ints(torch, [0, 298])
    assert torch.equal(B.attention(q, k, v, a, b), B.attention(q.contiguous(), k.contiguous(), v.contiguous(), a, b))
    positions, table = ints(torch, [[3], [9], [5], [700]]), B.rope_table(64)
    want = B.rope(q.contiguous(), None, positions, table)[0]
    assert torch.equal(B.rope(q, None, positions, table)[0], want)
    slots = torch.arange(298, device="cuda")
    near, far = (B.mx_cache(10, 32, 2, 64) for _ in (0, 1))
    B.mx_cache_write(k, v, far, slots)
    B.mx_cache_write(k.contiguous(), v.contiguous(), near, slots)
    assert all(torch.equal(x.codes, y.codes) and torch.equal(x.scales, y.scales) for x, y in zip(near, far))
    pages = torch.arange(10, device="cuda", dtype=torch.int32).view(1, 10)
    n = ints(torch, [298])
    for x in (q[None], q[3:, None]):  # the stride of an axis of one does not count
        got = B.mx_cache_attention(x, near, pages, n)
        assert got.any() and torch.equal(got, B.mx_cache_attention(x.contiguous(), near, pages, n))
