"""Argument checks of the rotary, cache and attention entry points on the host (every refusal names its reason and happens
before anything is launched: no GPU here), and the tests' own 64-bit reference against torch's on the CPU."""
import ctypes
import math

import numpy as np
import pytest

from cnn_convolution_fwd_amd import binding as B
from tests import attention_reference as A

P = 1 << 32  # stands for a device pointer: no refused call looks behind it


def status(st):
    return st, B.library().cfwd_last_error().decode()


def call(name, d, *args):
    return status(getattr(B.library(), name)(ctypes.byref(d) if d is not None else None, *args))


def refused(result, want=B.ERR_INVALID_ARG):
    st, why = result
    assert st == want and why, (st, why)


# ------------------------------------------------------------------ rotary positions

def rope(tokens=4, qh=2, kh=1, dim=64, pairs=32, axes=1, adjacent=0, wide=0, dtype=B.BF16, qs=256, qhs=64, ks=256, khs=64,
         qos=128, qohs=64, kos=64, kohs=64, q=P, k=P + 256, positions=P * 2, table=P * 3, qo=P * 4, ko=P * 5):
    d = B.RopeDesc(tokens, qh, kh, dim, pairs, axes, adjacent, wide, dtype, qs, qhs, ks, khs, qos, qohs, kos, kohs)
    return call("cfwd_rope", d, q, k, positions, table, qo, ko, None)


@pytest.mark.parametrize("kw", [
    dict(tokens=-1), dict(tokens=(1 << 38) + 1), dict(qh=-1), dict(kh=-1), dict(qh=0, kh=0), dict(qh=(1 << 16) + 1), dict(dim=0),
    dict(dim=1025, pairs=0), dict(pairs=-1), dict(pairs=33), dict(axes=0), dict(axes=1025), dict(dtype=B.I8),
    dict(dtype=B.MXFP4), dict(qs=-1), dict(khs=-64), dict(qs=1 << 60), dict(qos=64), dict(qohs=63), dict(kos=63), dict(kohs=-1),
    dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(positions=None), dict(table=None), dict(q=P + 1),
    dict(ko=P * 5 + 1), dict(positions=P * 2 + 2), dict(positions=P * 2 + 4, wide=1), dict(table=P * 3 + 8), dict(dtype=B.F32, q=P + 2),
    dict(qo=P), dict(qo=P + 256), dict(qo=P, qos=256, qohs=128), dict(ko=P * 4), dict(qo=P * 2), dict(ko=P * 3 - 8),
    dict(qo=P + 128, qos=256)])
def test_rope_refusals(kw):
    refused(rope(**kw))


def test_rope_calls_with_nothing_to_do():
    assert rope(tokens=0, q=None, positions=None)[0] == B.OK
    # in place there is nothing to turn without pairs, and nothing to copy
    assert rope(pairs=0, positions=None, table=None, qo=P, qos=256, ko=P + 256, kos=256)[0] == B.OK
    refused(call("cfwd_rope", None, P, P, P, P, P, P, None))


def test_rope_turns():
    f = B.library().cfwd_rope_turns
    assert f(0.0) == 0 and f(float("inf")) == 0 and f(float("nan")) == 0
    # frequency / (2 pi) in 2^-64: against exact whole-number arithmetic with 80 digits of pi
    pi = 31415926535897932384626433832795028841971693993751058209749445923078164062862090
    scale = 10 ** (len(str(pi)) - 1)
    for freq in (1.0, 0.5, 10000.0 ** -0.3, 2.0 ** -40, 1e-9, 7.25, -1.0, 1e5):
        num, den = freq.as_integer_ratio()
        exact = (num << 64) * scale // (2 * pi * den) % (1 << 64)
        off = (f(freq) - exact) % (1 << 64)
        off = min(off, (1 << 64) - off)
        assert off <= max(2, abs(freq) / (2 * math.pi) * 2), (freq, off)  # long double's 64 bits: half a unit of the quotient


# ------------------------------------------------------------------ the cache

def parts(pages=8, page=16, heads=2, dim=64, kc=P, ks=P * 2, vc=P * 3, vs=P * 4):
    return B.MxCacheParts(pages, page, heads, dim, kc, ks, vc, vs)


CACHE = [dict(pages=0), dict(page=0), dict(heads=0), dict(heads=(1 << 16) + 1), dict(dim=0), dict(dim=1025),
         dict(pages=1 << 20, page=1 << 11)]
BUFFERS = [dict(kc=None), dict(ks=None), dict(vc=None), dict(vs=None), dict(kc=P + 8), dict(vc=P * 3 + 4), dict(ks=P * 2 + 2),
           dict(vs=P * 4 + 1)]


def write(tokens=4, dtype=B.BF16, wide=0, k_row=128, k_head=64, v_row=128, v_head=64, k=P * 5, v=P * 6, slots=P * 7, **cache):
    d = B.MxCacheWriteDesc(tokens, dtype, wide, k_row, k_head, v_row, v_head)
    return call("cfwd_mx_cache_write", d, ctypes.byref(parts(**cache)), k, v, slots, None)


@pytest.mark.parametrize("kw", CACHE + BUFFERS + [
    dict(tokens=-1), dict(tokens=(1 << 38) + 1), dict(dtype=B.I8), dict(dtype=B.MXFP4), dict(k_row=-1), dict(v_head=-1), dict(k=None),
    dict(v=None), dict(slots=None), dict(k=P * 5 + 1), dict(dtype=B.F32, v=P * 6 + 2), dict(slots=P * 7 + 2),
    dict(slots=P * 7 + 4, wide=1), dict(vc=P), dict(ks=P + 16), dict(vs=P * 2), dict(k=P), dict(v=P * 4), dict(slots=P * 3),
    dict(k=P * 2 - 256)])
def test_cache_write_refusals(kw):
    refused(write(**kw))


def read(tokens=4, sequences=2, pitch=3, dtype=B.BF16, table=P * 5, starts=P * 6, k=P * 7, v=P * 8, **cache):
    d = B.MxCacheReadDesc(tokens, sequences, pitch, dtype)
    return call("cfwd_mx_cache_read", d, ctypes.byref(parts(**cache)), table, starts, k, v, None)


@pytest.mark.parametrize("kw", CACHE + BUFFERS + [
    dict(tokens=-1), dict(tokens=1 << 31), dict(sequences=-1), dict(pitch=0), dict(dtype=B.I8), dict(dtype=B.MXFP4),
    dict(table=None), dict(starts=None), dict(k=None), dict(v=None), dict(table=P * 5 + 2), dict(starts=P * 6 + 1),
    dict(k=P * 7 + 1), dict(dtype=B.F32, v=P * 8 + 2), dict(v=P * 7), dict(k=P), dict(v=P * 4), dict(k=P * 5),
    dict(v=P * 6 - 4)])
def test_cache_read_refusals(kw):
    refused(read(**kw))


def test_cache_calls_with_nothing_to_do():
    assert write(tokens=0, k=None)[0] == B.OK and read(tokens=0, k=None)[0] == B.OK and read(sequences=0, k=None)[0] == B.OK
    refused(call("cfwd_mx_cache_write", None, ctypes.byref(parts()), P, P, P, None))
    refused(call("cfwd_mx_cache_write", B.MxCacheWriteDesc(1, B.BF16, 0, 1, 1, 1, 1), None, P, P, P, None))
    refused(call("cfwd_mx_cache_read", B.MxCacheReadDesc(1, 1, 1, B.BF16), None, P, P, P, P, None))


# ------------------------------------------------------------------ attention over the cache

def over_cache(sequences=2, tokens=1, heads=4, pitch=40, scale=0.1, dtype=B.BF16, qss=512, qs=256, qhs=64, q=P * 5, table=P * 6,
               lengths=P * 7, o=P * 8, ws=P * 9, ws_bytes=1 << 30, kv=2, **cache):
    d = B.MxCacheAttentionDesc(sequences, tokens, heads, pitch, scale, dtype, qss, qs, qhs)
    return call("cfwd_mx_cache_attention", d, ctypes.byref(parts(heads=kv, **cache)), q, table, lengths, o, ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [k for k in CACHE if "heads" not in k] + BUFFERS + [
    dict(kv=0), dict(sequences=-1), dict(tokens=-1), dict(pitch=0), dict(pitch=1 << 27), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(heads=0), dict(heads=3), dict(heads=1 << 17), dict(qs=-8),
    dict(qhs=4), dict(qss=100), dict(qss=-512), dict(qs=1 << 60, tokens=2), dict(q=None), dict(table=None), dict(lengths=None),
    dict(o=None), dict(q=P * 5 + 8), dict(o=P * 8 + 2), dict(table=P * 6 + 1), dict(lengths=P * 7 + 2), dict(ws=P * 9 + 16),
    dict(o=P * 5), dict(o=P), dict(o=P * 6), dict(o=P * 7), dict(ws=P * 3), dict(ws=P * 5), dict(ws=P * 8)])
def test_cache_attention_refusals(kw):
    refused(over_cache(**kw))


@pytest.mark.parametrize("kw", [dict(dtype=B.F32), dict(dim=48), dict(dim=288), dict(page=8), dict(page=24), dict(tokens=1025),
                                dict(sequences=1 << 20, tokens=64), dict(pages=2, page=1 << 24, kv=4, pitch=1, dim=256),
                                dict(sequences=1 << 22, pitch=1 << 16)])
def test_cache_attention_unsupported(kw):
    refused(over_cache(**kw), B.ERR_UNSUPPORTED)


def test_cache_attention_workspace():
    refused(over_cache(ws=None), B.ERR_WORKSPACE)
    refused(over_cache(ws_bytes=256), B.ERR_WORKSPACE)
    assert over_cache(sequences=0, q=None)[0] == B.OK and over_cache(tokens=0, q=None)[0] == B.OK
    f, b = B.library().cfwd_mx_cache_attention_workspace_size, ctypes.c_size_t()
    c = parts(heads=2)
    d = B.MxCacheAttentionDesc(2, 1, 4, 40, 0.1, B.BF16, 512, 256, 64)
    assert f(ctypes.byref(d), ctypes.byref(c), ctypes.byref(b)) == B.OK and b.value > 0
    assert f(ctypes.byref(d), ctypes.byref(c), None) == B.ERR_INVALID_ARG
    assert f(None, ctypes.byref(c), ctypes.byref(b)) == B.ERR_INVALID_ARG
    assert f(ctypes.byref(d), None, ctypes.byref(b)) == B.ERR_INVALID_ARG


# ------------------------------------------------------------------ packed prompts

def attention(nq=200, nk=200, sequences=2, heads=4, kv=2, dim=64, causal=1, scale=0.1, dtype=B.BF16, qs=512, qhs=64, ks=512,
              khs=64, vs=512, vhs=64, q=P, k=P + 512, v=P + 768, a=P * 2, b=P * 3, o=P * 4, ws=P * 5, ws_bytes=1 << 30):
    d = B.AttentionDesc(nq, nk, sequences, heads, kv, dim, causal, scale, dtype, qs, qhs, ks, khs, vs, vhs)
    return call("cfwd_attention", d, q, k, v, a, b, o, ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(nq=-1), dict(nk=-1), dict(sequences=-1), dict(heads=0), dict(kv=0), dict(heads=3), dict(heads=1 << 17), dict(dim=0),
    dict(scale=0.0), dict(scale=-0.5), dict(scale=float("nan")), dict(scale=float("inf")), dict(qs=-8), dict(khs=-8), dict(qs=513),
    dict(khs=68), dict(vs=516), dict(q=None), dict(k=None), dict(v=None), dict(a=None), dict(b=None), dict(o=None),
    dict(q=P + 8), dict(k=P + 520), dict(v=P + 770), dict(o=P * 4 + 8), dict(a=P * 2 + 1), dict(b=P * 3 + 2), dict(o=P),
    dict(o=P + 512), dict(o=P * 2), dict(o=P * 3)])
def test_attention_refusals(kw):
    refused(attention(**kw))


@pytest.mark.parametrize("kw", [dict(dtype=B.F32), dict(dim=60), dict(dim=264), dict(nq=1 << 30), dict(nk=(1 << 31) - 4096),
                                dict(ks=56), dict(vs=(1 << 24) + 8)])
def test_attention_unsupported(kw):
    refused(attention(**kw), B.ERR_UNSUPPORTED)


def test_attention_workspace():
    few = dict(nq=5, nk=9000, sequences=1, k=P * 6, v=P * 7, ks=128, vs=128)  # few rows, many keys: split
    refused(attention(ws=None, **few), B.ERR_WORKSPACE)
    refused(attention(ws_bytes=1, **few), B.ERR_WORKSPACE)
    refused(attention(**{**few, "ws": P * 5 + 8}))
    for ws in (P, P * 2, P * 3, P * 4, P * 6, P * 7):
        refused(attention(**{**few, "ws": ws}))
    assert attention(nq=0, q=None)[0] == B.OK and attention(sequences=0, q=None)[0] == B.OK
    refused(call("cfwd_attention", None, P, P, P, P, P, P, P, 0, None))
    f, b = B.library().cfwd_attention_workspace_size, ctypes.c_size_t()
    for nq, nk, some in ((5, 9000, True), (5, 100, False), (100000, 100000, False)):
        d = B.AttentionDesc(nq, nk, 1, 4, 2, 64, 1, 0.1, B.BF16, 512, 64, 512, 64, 512, 64)
        assert f(ctypes.byref(d), ctypes.byref(b)) == B.OK and (b.value > 0) == some
    assert f(ctypes.byref(d), None) == B.ERR_INVALID_ARG and f(None, ctypes.byref(b)) == B.ERR_INVALID_ARG


# ------------------------------------------------------------------ the Python calls

def test_binding_refusals():
    torch = pytest.importorskip("torch")
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    table, positions = B.rope_table(64, device="cpu"), torch.zeros(3, 1, dtype=torch.int32)
    starts = torch.zeros(2, dtype=torch.int32)
    cache = B.mx_cache(4, 16, 2, 64, device="cpu")
    pages, lengths, slots = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    bad = [
        lambda: B.rope(q, k, positions, table), lambda: B.rope(q[0], k, positions, table), lambda: B.rope(q, k[:2], positions, table),
        lambda: B.rope(q, k.float(), positions, table), lambda: B.rope(q, None, positions, table, k_out=k),
        lambda: B.rope(q, k, positions[:2], table), lambda: B.rope(q, k, positions.float(), table),
        lambda: B.rope(q.half(), None, positions, table), lambda: B.rope(q, k, positions, table, q_out=k),
        lambda: B.rope(q.transpose(1, 2), None, positions, table),
        lambda: B.rope(q, k, positions, B.RopeTable(table.pairs.int(), 1)),
        lambda: B.mx_cache_write(k, k, cache, slots), lambda: B.mx_cache_write(q, q, cache, slots),
        lambda: B.mx_cache_write(k, k, cache.k, slots), lambda: B.mx_cache_write(k, k, B.MxCache(cache.k, cache.v._replace(cols=60)), slots),
        lambda: B.mx_cache_read(cache, pages, starts, 3), lambda: B.mx_cache_attention(q, cache, pages, lengths),
        lambda: B.mx_cache_attention(q[..., :32], cache, pages, lengths), lambda: B.attention(q, k, k, starts),
        lambda: B.attention(q, k, k[:2], starts), lambda: B.attention(q, k, k.float(), starts),
        lambda: B.rope_table(7), lambda: B.rope_table(8, (1, 2)), lambda: B.rope_table(8, (5, -1)), lambda: B.rope_table(8, order="no"),
        lambda: B.rope_table(8, frequencies=(1.0,)), lambda: B.rope_table(8, ()),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)) as e:
            f()
        assert str(e.value), i


def test_rope_table():
    pytest.importorskip("torch")
    turns = lambda freq: round(freq / (2 * math.pi) * 2 ** 64) % 2 ** 64  # noqa: E731
    for sections, order in (((2, 3, 3), "runs"), ((2, 3, 3), "turns"), ((2, 0, 6), "each"), ((8,), "runs")):
        t = B.rope_table(16, sections, base=100.0, order=order, device="cpu")
        axes, freq = A.axes_and_frequencies(16, sections, 100.0, order)
        assert t.axes == len(sections) and t.pairs.shape == (8, 2) and t.pairs[:, 1].tolist() == axes.tolist()
        for got, f in zip(t.pairs[:, 0].tolist(), freq):
            assert abs(got % 2 ** 64 - turns(f)) <= 2 ** 12  # a double's 53 bits of 64
    assert B.rope_table(0, device="cpu").pairs.shape == (0, 2)


# ------------------------------------------------------------------ the tests' reference

def test_reference_attention():
    torch = pytest.importorskip("torch")
    g = torch.Generator()
    g.manual_seed(1)
    q, k, v = (torch.randn(n, h, 24, generator=g, dtype=torch.float64) for n, h in ((7, 6), (12, 2), (12, 2)))
    wide = lambda t: t.repeat_interleave(3, 1).transpose(0, 1)  # noqa: E731
    for causal in (False, True):
        mask = torch.ones(7, 12, dtype=torch.bool).tril(5) if causal else torch.ones(7, 12, dtype=torch.bool)
        want = torch.nn.functional.scaled_dot_product_attention(q.transpose(0, 1), wide(k), wide(v), attn_mask=mask, scale=0.2)
        got, bound = A.attend(q.numpy(), k.numpy(), v.numpy(), causal, 0.2)
        assert np.abs(got - want.transpose(0, 1).numpy()).max() < 1e-14 and (bound >= 0).all()
    out, bound = A.attend(q.numpy(), k[:3].numpy(), v[:3].numpy(), True, 0.2)
    assert not out[:4].any() and not bound[:4].any() and np.array_equal(out[4, :3], np.repeat(v[:1, :1].numpy(), 3, 1)[0])


def test_reference_rotation():
    rng = np.random.default_rng(0)
    x, positions = rng.standard_normal((5, 2, 10)), rng.integers(-50, 50, (5, 2))
    axes, freq = np.array([0, 1, 1, 0]), np.array([1.0, 0.5, 0.25, 2.0])
    turn = np.exp(1j * positions[:, axes] * freq)[:, None]
    for adjacent in (False, True):
        a, b = (x[..., 0:8:2], x[..., 1:8:2]) if adjacent else (x[..., :4], x[..., 4:8])
        z = (a + 1j * b) * turn
        y, _ = A.rotate(x, positions, axes, freq, adjacent)
        ya, yb = (y[..., 0:8:2], y[..., 1:8:2]) if adjacent else (y[..., :4], y[..., 4:8])
        assert np.abs(ya - z.real).max() < 1e-14 and np.abs(yb - z.imag).max() < 1e-14 and np.array_equal(y[..., 8:], x[..., 8:])
