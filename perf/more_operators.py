"""Cases and plain forms of the operators around attention with a 4-bit cache.

Four operators of large language models, which image and video networks with
attention over patches use in the same places; with the 4-bit products and the
gated norms they make a whole layer:

* rope: rotary positions with several axes (time, height, width) of queries and
  keys: pair i of a head turns by position[axis(i)] * frequency(i);
* cache: keys and values quantised to MXFP4 as they are written to a paged cache,
  and read back, a row of pages for each sequence;
* decode: attention of one or a few new tokens of every sequence over that cache;
* prompt: attention of whole prompts, packed one after the other, causal or not,
  with fewer heads of keys and values than of queries, and keys that were there
  before the queries.

A query with no key to see has an output of 0.

The cache of keys, and the one of values, is an MXFP4 tensor [pages, heads, page,
dim]: codes uint8 [..., 16 * ceil(dim / 32)] (two values a byte, the even one in
the low four bits), scales uint8 [..., ceil(dim / 32) rounded up to 4].
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One token of one sequence, far into its text: latency alone.
        dict(name="rope_one_token", op="rope", tokens=1, heads=32, kv_heads=8, dim=128, rotary=128, sections="64",
             order="runs", base=500000.0, adjacent=False, far=100000, dtype="bf16"),
        # A clip of 16 frames of 28 x 28 patches, three axes, queries and keys out of one projection: bandwidth.
        dict(name="rope_video", op="rope", tokens=12544, heads=32, kv_heads=8, dim=128, rotary=128,
             sections="16 24 24", order="runs", base=1000000.0, adjacent=False, far=1000, dtype="bf16"),
        # A decoding step of 64 sequences: one new token each, and the short sequences read back: latency.
        dict(name="cache_step", op="cache", sequences=64, kept=16, new=1, spread="ragged", kv_heads=8, dim=128, page=64,
             dtype="bf16"),
        # Four long prompts into an empty cache, and back for the next chunk's attention: bandwidth.
        dict(name="cache_prompts", op="cache", sequences=4, kept=0, new=8192, spread="even", kv_heads=8, dim=128, page=64,
             dtype="bf16"),
        # One sequence of a few hundred tokens: latency, the long axis split to have any work for the device.
        dict(name="decode_one", op="decode", sequences=1, longest=500, spread="even", tokens=1, heads=32, kv_heads=8,
             dim=128, page=16),
        # A batch of sequences of all lengths: the cache's bytes.
        dict(name="decode_batch", op="decode", sequences=64, longest=8192, spread="uniform", tokens=1, heads=32,
             kv_heads=8, dim=128, page=64),
        # One very long sequence, four tokens at once (three guesses checked with the token before them).
        dict(name="decode_long", op="decode", sequences=1, longest=131072, spread="even", tokens=4, heads=64, kv_heads=8,
             dim=128, page=64),
        # A short question alone: latency.
        dict(name="prompt_short", op="prompt", sequences=1, longest=77, prefix=0, spread="even", heads=32, kv_heads=8,
             dim=128, causal=True),
        # 32 images of 28 x 28 patches, every patch sees its whole image.
        dict(name="prompt_images", op="prompt", sequences=32, longest=784, prefix=0, spread="even", heads=16, kv_heads=16,
             dim=64, causal=False),
        # Prompts of all lengths, packed.
        dict(name="prompt_packed", op="prompt", sequences=16, longest=4096, prefix=0, spread="ragged", heads=32,
             kv_heads=8, dim=128, causal=True),
        # The next chunk of a long prompt: few queries, many keys.
        dict(name="prompt_chunk", op="prompt", sequences=1, longest=256, prefix=16384, spread="even", heads=32, kv_heads=8,
             dim=128, causal=True),
        # One long prompt: the matrix cores.
        dict(name="prompt_long", op="prompt", sequences=1, longest=16384, prefix=0, spread="even", heads=32, kv_heads=8,
             dim=128, causal=True),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["rope", "cache", "decode", "decode", "prompt", "prompt"])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 16])
    heads = kv_heads * rng.choice([1, 1, 2, 3, 4, 7, 8])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "rope":
        dim = rng.choice([32, 64, 72, 80, 96, 128, 256])
        pairs = dim // 2 if rng.random() < 0.7 else dim // 4
        axes = rng.choice([1, 2, 3])
        cut = sorted(rng.randint(0, pairs) for _ in range(axes - 1))
        sections = " ".join(str(b - a) for a, b in zip([0] + cut, cut + [pairs]))
        tokens = _log(rng, 1, min(32768, 12544 * 40 * 128 // ((heads + kv_heads) * dim)))
        return dict(op=op, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, rotary=2 * pairs, sections=sections,
                    order=rng.choice(["runs", "turns", "each"]), base=rng.choice([10000.0, 1000000.0]),
                    adjacent=rng.random() < 0.4, far=rng.choice([100, 10000, 1000000]), dtype=dtype)
    page = rng.choice([16, 32, 48, 64, 128, 256])
    spread = rng.choice(["even", "ragged", "uniform"])
    if op == "cache":
        dim = rng.choice([32, 64, 80, 96, 128, 256])
        sequences = _log(rng, 1, 64)
        most = max(1, 4 * 8192 * 8 * 128 // (sequences * kv_heads * dim * _ES[dtype] // 2))
        longest = _log(rng, 1, min(8192, most))
        kept = rng.choice([0, longest // 3, longest - 1])
        return dict(op=op, sequences=sequences, kept=kept, new=longest - kept, spread=spread, kv_heads=kv_heads, dim=dim,
                    page=page, dtype=dtype)
    sequences = _log(rng, 1, 64)
    if op == "decode":
        dim = rng.choice([32, 64, 96, 128, 128, 256])
        tokens = rng.choice([1, 1, 1, 2, 4, 7])
        longest = _log(rng, tokens, min(131072, 64 * 4096 * 8 * 128 // (sequences * kv_heads * dim)))
        return dict(op=op, sequences=sequences, longest=longest, spread=spread, tokens=tokens, heads=heads,
                    kv_heads=kv_heads, dim=dim, page=page)
    dim = rng.choice([40, 64, 72, 80, 96, 128, 128, 256])
    longest = _log(rng, 1, 4096)
    prefix = rng.choice([0, 0, 0, _log(rng, 1, 8192)])
    sequences = max(1, min(sequences, int(16384 * 16384 * 32 * 128 // 2 // (longest * (longest + prefix) * heads * dim)),
                           65536 * 32 * 128 // (longest * heads * dim)))
    return dict(op=op, sequences=sequences, longest=longest, prefix=prefix, spread=spread, heads=heads, kv_heads=kv_heads,
                dim=dim, causal=rng.random() < 0.7)


def _sections(case):
    """Pairs of every axis."""
    return [int(n) for n in case["sections"].split()]


def _lengths(n, longest, spread, least=1):
    """Lengths of n sequences, one of them the longest; of several ragged ones one has no more than the least."""
    if spread == "even" or n == 1:
        return [longest] * n
    rng = random.Random(n * 1000003 + longest)
    if spread == "uniform":
        some = [rng.randint(least, longest) for _ in range(n - 1)]
    else:
        some = [_log(rng, max(least, 1), max(longest, 1)) for _ in range(n - 1)]
        if n > 3:
            some[1] = least
    some.insert(rng.randrange(n), longest)
    return some


def _decode_lengths(case):
    """Tokens in the cache, the new ones among them; one of several ragged sequences has none at all."""
    lengths = _lengths(case["sequences"], case["longest"], case["spread"], case["tokens"])
    if case["spread"] == "ragged" and case["sequences"] > 3:
        lengths[lengths.index(min(lengths))] = 0
    return lengths


def _prompt_lengths(case):
    """(queries, keys) of every sequence; one of several ragged ones has no queries, one fewer keys than queries."""
    q = _lengths(case["sequences"], case["longest"], case["spread"])
    rng = random.Random(case["prefix"])
    k = [n + (case["prefix"] if case["spread"] == "even" else rng.randint(0, case["prefix"])) for n in q]
    if case["spread"] == "ragged" and case["sequences"] > 5:
        q[2], k[4] = 0, k[4] // 2
    return q, k


def _cache_lengths(case):
    """(tokens there before, new tokens) of every sequence."""
    n, spread = case["sequences"], case["spread"]
    return _lengths(n, case["kept"], spread, 0) if case["kept"] else [0] * n, _lengths(n, case["new"], spread)


def _starts(lengths):
    starts = [0]
    for n in lengths:
        starts.append(starts[-1] + n)
    return starts


# ------------------------------------------------------------------ what a pass cannot do without

def _row_bytes(dim):
    kb = -(-dim // 32)
    return 16 * kb + -(-kb // 4) * 4


def work(case):
    op, dim = case["op"], case["dim"]
    if op == "rope":
        n = case["tokens"] * (case["heads"] + case["kv_heads"])
        return {"bytes": 2 * n * dim * _ES[case["dtype"]] + 4 * case["tokens"] * len(_sections(case)),
                "flops": 3 * n * case["rotary"]}
    if op == "cache":
        kept, new = _cache_lengths(case)
        rows = case["kv_heads"] * 2
        es = _ES[case["dtype"]]
        # new tokens read and written in 4 bits; all tokens read in 4 bits and written
        return {"bytes": rows * (sum(new) * (dim * es + _row_bytes(dim)) + sum(kept + new) * (dim * es + _row_bytes(dim))),
                "flops": 2 * rows * dim * (sum(new) + sum(kept + new))}
    if op == "decode":
        lengths, tokens = _decode_lengths(case), case["tokens"]
        seen = sum(max(0, n - i) for n in lengths for i in range(tokens))
        return {"bytes": 2 * case["kv_heads"] * sum(lengths) * _row_bytes(dim)
                + 4 * case["sequences"] * tokens * case["heads"] * dim,
                "flops": 4 * seen * case["heads"] * dim}
    q, k = _prompt_lengths(case)
    seen = 0
    for nq, nk in zip(q, k):
        if not case["causal"]:
            seen += nq * nk
        else:  # the last query sees all nk keys, the one before it one fewer
            seen += nq * nk - nq * (nq - 1) // 2 if nk >= nq else nk * (nk + 1) // 2
    return {"bytes": 2 * dim * (2 * case["heads"] * sum(q) + 2 * case["kv_heads"] * sum(k)),
            "flops": 4 * seen * case["heads"] * dim}


# ------------------------------------------------------------------ the inputs

def _heads(g, tokens, heads, dim, dtype):
    """Normal values whose channels differ in size, as a projection's do."""
    x = torch.randn(tokens, heads, dim, generator=g, device="cuda")
    return x.mul_(torch.randn(heads, dim, generator=g, device="cuda").mul_(0.4).exp_()).to(_DT[dtype])


def _pages(g, lengths, page):
    """(table of pages [sequences, most], number of pages): pages in no order, and a few that no sequence owns."""
    counts = [-(-n // page) for n in lengths]
    total = sum(counts) + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lengths), max(1, max(counts)), dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(counts):
        table[i, :n] = order[at:at + n]
        at += n
    return table, total


def _filled(g, pages, heads, page, dim):
    """A cache's codes and scales as earlier writes left them."""
    codes, scales = [], []
    size = torch.randn(heads, 1, dim, generator=g, device="cuda").mul_(0.4).exp_()
    step = max(1, (1 << 25) // (heads * page * dim))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        x = torch.randn(n, heads, page, dim, generator=g, device="cuda").mul_(size)
        c, s = _pack(x.view(-1, dim))
        codes.append(c.view(n, heads, page, -1))
        scales.append(s.view(n, heads, page, -1))
    return torch.cat(codes), torch.cat(scales)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": case}
    op, dim = case["op"], case["dim"]
    if op == "rope":
        h, kh = case["heads"], case["kv_heads"]
        qkv = _heads(g, case["tokens"], h + 2 * kh, dim, case["dtype"])
        s["q"], s["k"] = qkv[:, :h], qkv[:, h:h + kh]
        axes = len(_sections(case))
        if axes == 3 and case["tokens"] % 784 == 0:  # frames of 28 x 28 patches
            i = torch.arange(case["tokens"], device="cuda")
            at = int(torch.randint(case["far"], (1,), generator=g, device="cuda"))
            s["positions"] = torch.stack((i // 784 + at, i // 28 % 28 + at, i % 28 + at), 1).to(torch.int32)
        else:
            s["positions"] = torch.randint(case["far"], (case["tokens"], axes), generator=g, device="cuda").to(torch.int32)
        if own:
            from cnn_convolution_fwd_amd import binding as cfwd
            s["table"] = cfwd.rope_table(case["rotary"], _sections(case), base=case["base"], order=case["order"])
        else:
            s["table"] = _rope_table(case)
    elif op == "cache":
        kept, new = _cache_lengths(case)
        total = [a + b for a, b in zip(kept, new)]
        s["table"], pages = _pages(g, total, case["page"])
        s["k_cache"] = _filled(g, pages, case["kv_heads"], case["page"], dim)
        s["v_cache"] = _filled(g, pages, case["kv_heads"], case["page"], dim)
        kv = _heads(g, sum(new), 2 * case["kv_heads"], dim, case["dtype"])
        s["k"], s["v"] = kv[:, :case["kv_heads"]], kv[:, case["kv_heads"]:]
        s["slots"] = torch.cat([_slots(s["table"][i], torch.arange(a, a + b, device="cuda"), case["page"])
                                for i, (a, b) in enumerate(zip(kept, new))]).to(torch.int32)
        s["starts"], s["tokens"] = _ints(_starts(total)), sum(total)
    elif op == "decode":
        s["host_lengths"] = _decode_lengths(case)
        s["table"], pages = _pages(g, s["host_lengths"], case["page"])
        s["k_cache"] = _filled(g, pages, case["kv_heads"], case["page"], dim)
        s["v_cache"] = _filled(g, pages, case["kv_heads"], case["page"], dim)
        s["lengths"] = _ints(s["host_lengths"])
        s["q"] = _heads(g, case["sequences"] * case["tokens"], case["heads"], dim, "bf16").view(
            case["sequences"], case["tokens"], case["heads"], dim)
    else:
        q, k = _prompt_lengths(case)
        s["host_lengths"] = (q, k)
        h, kh = case["heads"], case["kv_heads"]
        if q == k:  # one projection gave all three
            qkv = _heads(g, sum(q), h + 2 * kh, dim, "bf16")
            s["q"], s["k"], s["v"] = qkv[:, :h], qkv[:, h:h + kh], qkv[:, h + kh:]
        else:
            s["q"] = _heads(g, sum(q), h, dim, "bf16")
            s["k"], s["v"] = _heads(g, sum(k), kh, dim, "bf16"), _heads(g, sum(k), kh, dim, "bf16")
        s["q_starts"], s["k_starts"] = _ints(_starts(q)), _ints(_starts(k))
    return s


# ------------------------------------------------------------------ plain forms

def _rope_table(case):
    """Axis and frequency (radians a position, 64 bits) of every pair."""
    pairs, sections = case["rotary"] // 2, _sections(case)
    axes = []
    if case["order"] == "turns":  # the axes take turns until their sections are used up
        left = list(sections)
        while any(left):
            for a in range(len(left)):
                if left[a]:
                    axes.append(a)
                    left[a] -= 1
    else:
        for a, n in enumerate(sections):
            axes += [a] * n
    if case["order"] == "each":  # every axis has frequencies of its own
        freq = [case["base"] ** (-i / n) for n in sections for i in range(n)]
    else:
        freq = [case["base"] ** (-p / pairs) for p in range(pairs)]
    return (torch.tensor(axes, device="cuda", dtype=torch.int64),
            torch.tensor(freq, device="cuda", dtype=torch.float64))


def _rotate(x, cos, sin, pairs, adjacent):
    x = x.to(cos.dtype)
    turned, rest = x[..., :2 * pairs], x[..., 2 * pairs:]
    if adjacent:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = turned[..., :pairs], turned[..., pairs:]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, rest), -1)


def _to_mx(x):
    """Blocks of x [rows][k] (32 bits): E2M1 values [rows][kb][32], and the blocks' exponent bytes [rows][kb]."""
    rows, k = x.shape
    kb = -(-k // 32)
    v = torch.nn.functional.pad(x, (0, kb * 32 - k)).view(rows, kb, 32)
    field = (v.abs().amax(-1).view(torch.int32) >> 23) & 255  # the largest value's exponent, biased
    byte = torch.where(field == 255, field, (field - 2).clamp(min=0))  # E2M1's largest exponent is 2
    v = v * ((254 - byte.clamp(max=253)) << 23).view(torch.float32).unsqueeze(-1)
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.copysign(((a / step).round() * step).clamp(max=6), v)
    return torch.where((byte == 255).unsqueeze(-1), torch.zeros_like(q), q), byte


def _pack(x):
    """(codes, scales) of x [rows][k]."""
    q, byte = _to_mx(x)
    a = q.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.int32)
    code = (code | (torch.signbit(q).to(torch.int32) << 3)).view(x.shape[0], -1, 2)
    codes = (code[..., 0] | (code[..., 1] << 4)).to(torch.uint8)
    scales = torch.nn.functional.pad(byte, (0, -byte.shape[1] % 4), value=127).to(torch.uint8)
    return codes.contiguous(), scales.contiguous()


def _unpack(codes, scales, k):
    """The values, in 32 bits, of rows of codes and scales [..., bytes]."""
    lead = codes.shape[:-1]
    c = codes.to(torch.int32)
    kb = codes.shape[-1] // 16
    c = torch.stack((c & 15, c >> 4), -1).view(*lead, kb, 32)
    mag = c & 7
    low = mag.to(torch.float32) * 0.5
    a = torch.where(mag < 4, low, torch.where(mag < 6, low * 2 - 2, low * 4 - 8))
    byte = scales.to(torch.int32)[..., :kb, None]
    unit = torch.where(byte == 0, 0x00400000, byte << 23).view(torch.float32)
    unit = torch.where(byte == 255, float("nan"), unit)
    return (torch.where(c > 7, -a, a) * unit).view(*lead, 32 * kb)[..., :k]


def _slots(pages, at, page):
    """Places in the cache of a sequence's tokens `at`."""
    return pages[at // page].long() * page + at % page


def _gather(cache, pages, n, dim):
    """The first n tokens' values [heads][n][dim], in 32 bits, of the sequence that owns these pages."""
    codes, scales = cache
    page = codes.shape[2]
    pages = pages[:-(-n // page)].long()
    c = codes[pages].transpose(0, 1).flatten(1, 2)[:, :n]
    s = scales[pages].transpose(0, 1).flatten(1, 2)[:, :n]
    return _unpack(c, s, dim)


def _attend(q, k, v, causal):
    """q [heads][nq][dim], k and v [kv heads][nk][dim], all in 32 bits: [heads][nq][dim]."""
    heads, nq, dim = q.shape
    kv_heads, nk, _ = k.shape
    group = heads // kv_heads
    out = torch.zeros_like(q)
    if nk == 0 or nq == 0:
        return out
    step = max(1, (1 << 28) // (nk * group))
    keys = torch.arange(nk, device=q.device)
    for j in range(kv_heads):
        for at in range(0, nq, step):
            rows = q[j * group:(j + 1) * group, at:at + step]
            score = torch.matmul(rows, k[j].t()) * dim ** -0.5
            if causal:
                last = torch.arange(at, at + rows.shape[1], device=q.device) + (nk - nq)
                score = score.masked_fill(keys > last[:, None], -math.inf)
            top = score.amax(-1, keepdim=True).clamp(min=-1e38)  # of a row with no key as well
            p = (score - top).exp()
            out[j * group:(j + 1) * group, at:at + step] = torch.matmul(p, v[j]) / p.sum(-1, keepdim=True).clamp(min=1e-38)
    return out


def _plain(s):
    case = s["case"]
    op, dim = case["op"], case["dim"]
    if op == "rope":
        axes, freq = s["table"]
        angle = s["positions"].double()[:, axes] * freq
        cos, sin = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)
        return {n: _rotate(s[n], cos, sin, case["rotary"] // 2, case["adjacent"]).to(s[n].dtype) for n in ("q", "k")}
    if op == "cache":
        slots = s["slots"].long()
        where, offset = slots // case["page"], slots % case["page"]
        out = {}
        for n in ("k", "v"):
            codes, scales = s[n + "_cache"]
            x = s[n].float()
            c, b = _pack(x.reshape(-1, dim))
            codes[where, :, offset] = c.view(*x.shape[:2], -1)
            scales[where, :, offset] = b.view(*x.shape[:2], -1)
        kept, new = _cache_lengths(case)
        for n in ("k", "v"):
            rows = [_gather(s[n + "_cache"], s["table"][i], a + b, dim) for i, (a, b) in enumerate(zip(kept, new))]
            out[n] = torch.cat(rows, 1).transpose(0, 1).to(s[n].dtype).contiguous()
        return out
    if op == "decode":
        out = torch.zeros_like(s["q"])
        for i, n in enumerate(s["host_lengths"]):
            k, v = (_gather(s[c], s["table"][i], n, dim) for c in ("k_cache", "v_cache"))
            out[i] = _attend(s["q"][i].float().transpose(0, 1), k, v, True).transpose(0, 1).to(out.dtype)
        return out
    out = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    (q, k), qa, ka = s["host_lengths"], 0, 0
    for nq, nk in zip(q, k):
        rows = _attend(s["q"][qa:qa + nq].float().transpose(0, 1), s["k"][ka:ka + nk].float().transpose(0, 1),
                       s["v"][ka:ka + nk].float().transpose(0, 1), case["causal"])
        out[qa:qa + nq] = rows.transpose(0, 1).to(out.dtype)
        qa, ka = qa + nq, ka + nk
    return out


# ------------------------------------------------------------------ this framework

def _own(s):
    from cnn_convolution_fwd_amd import binding as cfwd
    case = s["case"]
    op = case["op"]
    if op == "rope":
        q, k = cfwd.rope(s["q"], s["k"], s["positions"], s["table"], adjacent=case["adjacent"])
        return {"q": q, "k": k}
    if op == "prompt":
        return cfwd.attention(s["q"], s["k"], s["v"], s["q_starts"], s["k_starts"], causal=case["causal"])
    cache = cfwd.MxCache(cfwd.MxTensor(*s["k_cache"], case["dim"]), cfwd.MxTensor(*s["v_cache"], case["dim"]))
    if op == "cache":
        cfwd.mx_cache_write(s["k"], s["v"], cache, s["slots"])
        k, v = cfwd.mx_cache_read(cache, s["table"], s["starts"], s["tokens"], dtype=case["dtype"])
        return {"k": k, "v": v}
    return cfwd.mx_cache_attention(s["q"], cache, s["table"], s["lengths"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits

def _mx64(x):
    """x rounded to MXFP4 by the definition, in 64 bits: the nearest of the eight magnitudes, a tie to the even code."""
    rows, k = x.shape
    v = torch.zeros(rows, -(-k // 32) * 32, dtype=torch.float64, device=x.device)
    v[:, :k] = x
    v = v.view(rows, -1, 32)
    top = v.abs().amax(-1, keepdim=True)
    exponent = (torch.frexp(top).exponent - 1 - 2).clamp(-127, 125)  # floor(log2) less that of 4
    exponent = torch.where(top == 0, -127, exponent)
    unit = torch.ldexp(torch.ones_like(top), exponent)
    a = v.abs() / unit
    middles = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=x.device)
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    code = torch.searchsorted(middles, a)
    tie = (code < 7) & (middles[code.clamp(max=6)] == a)
    code = code + (tie & (code % 2 == 1))
    return (v.sign() * values[code] * unit).view(rows, -1)[:, :k]


def _cached64(cache, table, lengths, dim):
    """Values [tokens][heads][dim] of all sequences, one after the other."""
    codes, scales = cache
    magnitudes = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                              device="cuda")
    page = codes.shape[2]
    parts = [torch.zeros(0, codes.shape[1], dim, dtype=torch.float64, device="cuda")]
    for row, n in zip(table.tolist(), lengths):
        for at in range(0, n, page):
            rows = min(page, n - at)
            c, b = codes[row[at // page], :, :rows], scales[row[at // page], :, :rows]
            v = torch.empty(*c.shape[:2], 2 * c.shape[2], dtype=torch.float64, device="cuda")
            v[..., 0::2], v[..., 1::2] = magnitudes[(c & 15).long()], magnitudes[(c >> 4).long()]
            v *= torch.exp2(b.double() - 127)[..., :c.shape[2] // 16].repeat_interleave(32, -1)
            parts.append(v[..., :dim].transpose(0, 1))
    return torch.cat(parts)


def _softmax64(q, k, v, causal):
    """q [nq][heads][dim], k and v [nk][kv heads][dim] in 64 bits."""
    nq, heads, dim = q.shape
    nk, kv_heads = k.shape[:2]
    out = torch.zeros(nq, heads, dim, dtype=torch.float64, device=q.device)
    if nk == 0:
        return out
    step = max(1, (1 << 27) // nk)
    for h in range(heads):
        keys, values = k[:, h * kv_heads // heads], v[:, h * kv_heads // heads]
        for a in range(0, nq, step):
            rows = q[a:a + step, h]
            weight = rows @ keys.t() / math.sqrt(dim)
            if causal:
                seen = torch.ones_like(weight, dtype=torch.bool).tril(nk - nq + a)
                weight = torch.where(seen, weight, torch.full_like(weight, -math.inf))
                some = seen.any(1)
                out[a:a + step, h][some] = torch.softmax(weight[some], 1) @ values
            else:
                out[a:a + step, h] = torch.softmax(weight, 1) @ values
    return out


def exact(case, seed):
    if case["op"] == "rope":
        s = prepare(case, seed)
        axes, freq = _rope_table(case)
        angle = (s["positions"].to(torch.float64)[:, axes] * freq)[:, None]
        pairs = case["rotary"] // 2
        first = torch.arange(pairs, device="cuda") * (2 if case["adjacent"] else 1)
        second = first + (1 if case["adjacent"] else pairs)
        out = {}
        for n in ("q", "k"):
            x = s[n].double()
            y = x.clone()
            turned = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(angle), angle)
            y[..., first], y[..., second] = turned.real, turned.imag
            out[n] = y
        return out
    s = prepare(case, seed)
    dim = case["dim"]
    if case["op"] == "cache":
        kept, new = _cache_lengths(case)
        out = {}
        for n in ("k", "v"):
            rows = _mx64(s[n].double().reshape(-1, dim)).view(s[n].shape)
            old, parts, at = _cached64(s[n + "_cache"], s["table"], kept, dim), [], 0
            for first, a, b in zip(_starts(kept), kept, new):
                parts += [old[first:first + a], rows[at:at + b]]
                at += b
            out[n] = torch.cat(parts)
        return out
    if case["op"] == "decode":
        lengths = s["host_lengths"]
        k, v = (_cached64(s[c], s["table"], lengths, dim) for c in ("k_cache", "v_cache"))
        at = _starts(lengths)
        return torch.stack([_softmax64(s["q"][i].double(), k[at[i]:at[i + 1]], v[at[i]:at[i + 1]], True)
                            for i in range(len(lengths))])
    (q, k), parts = s["host_lengths"], []
    qa, ka = _starts(q), _starts(k)
    for i in range(len(q)):
        rows, keys = slice(qa[i], qa[i + 1]), slice(ka[i], ka[i + 1])
        parts.append(_softmax64(s["q"][rows].double(), s["k"][keys].double(), s["v"][keys].double(), case["causal"]))
    return torch.cat(parts)
