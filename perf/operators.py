"""Cases and plain forms of the 4-bit feed-forward operators.

Three operators of large language models, which a network of 1x1
convolutions over channel-last activations uses in the same places:

* quantisation to microscaled 4-bit floating point (MXFP4) and back: blocks of
  32 consecutive values along a row share a power-of-two scale of 8 bits, the
  values are E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives);
* the product of two MXFP4 matrices, y = act(x w^T + bias), whose x may also be
  given in 16 or 32 bits and is then quantised by the call;
* the norms before and after a block, fused with its gate and its residual
  scale: s = residual_scale * r + gate * post(b), h = pre(s).

A case's "op" says which one it times; "block" runs them together as the
feed-forward step of a network does.

MXFP4 tensors are stored as a matrix of codes, uint8 [rows][16 * ceil(cols / 32)]
(two values a byte, the even one in the low four bits), and one of scales,
uint8 [rows][ceil(cols / 32) rounded up to 4] (2^(byte - 127), 255 = NaN).
"""
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}
EPS = 1e-6


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One token's activations before a 4-bit layer: latency alone.
        dict(name="quantize_one_token", op="quantize", rows=1, k=4096, dtype="bf16"),
        # A batch of 32 images, 56 x 56 pixels, 256 channels, channel-last: bandwidth.
        dict(name="quantize_pixels", op="quantize", rows=100352, k=256, dtype="bf16"),
        # Serving one token: after attention, before the feed-forward layer.
        dict(name="norm_one_token", op="norm", rows=1, c=4096, groups=1, post="rms", pre="rms", gate=True,
             dtype="bf16", stream="bf16"),
        # 64 images of 7 x 7 pixels and 512 channels, a gate for each image, residual stream in 32 bits.
        dict(name="norm_pixels", op="norm", rows=3136, c=512, groups=64, post="none", pre="layer", gate=True,
             dtype="bf16", stream="f32"),
        # A long prompt: bandwidth.
        dict(name="norm_prompt", op="norm", rows=16384, c=8192, groups=1, post="rms", pre="rms", gate=True,
             dtype="bf16", stream="bf16"),
        # One token through a wide 4-bit layer: the weights are read once.
        dict(name="matmul_one_token", op="matmul", m=1, n=16384, k=4096, x="bf16", y="bf16", act="silu", bias=False),
        # A classifier head over a few rows; neither size is a multiple of a tile.
        dict(name="matmul_few_rows", op="matmul", m=13, n=1000, k=2000, x="f32", y="f32", act="none", bias=True),
        # A short prompt: too few tiles to fill the device without splitting the sum.
        dict(name="matmul_short_prompt", op="matmul", m=500, n=4096, k=4096, x="bf16", y="bf16", act="none",
             bias=False),
        # The widening 1x1 convolution of an inverted bottleneck, 32 images of 56 x 56 pixels: mostly the output's bytes.
        dict(name="matmul_pixels", op="matmul", m=100352, n=1024, k=256, x="bf16", y="bf16", act="gelu", bias=True),
        # Large and square, both sides in 4 bits already: the matrix cores.
        dict(name="matmul_large", op="matmul", m=8192, n=8192, k=8192, x="mx", y="bf16", act="none", bias=False),
        # A decoding step of four sequences through a whole feed-forward block.
        dict(name="block_decode", op="block", rows=4, c=4096, hidden=16384, groups=1, post="rms", pre="rms",
             act="silu", bias=False),
        # The same for 32 images of 28 x 28 pixels and 512 channels, a gate for each image.
        dict(name="block_pixels", op="block", rows=25088, c=512, hidden=2048, groups=32, post="none", pre="layer",
             act="gelu", bias=True),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["quantize", "norm", "matmul", "matmul", "block"])
    if op == "quantize":
        rows = _log(rng, 1, 100352)
        return dict(op=op, rows=rows, k=_log(rng, 1, min(16384, max(1, 100352 * 256 // rows))),
                    dtype=rng.choice(["bf16", "f32"]))
    if op == "norm":
        rows = _log(rng, 1, 100352)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, rows=rows, c=_log(rng, 8, min(16384, 16384 * 4096 // rows)),
                    groups=rng.choice([1, 1, min(rows, 7)]), post=rng.choice(["none", "rms", "layer"]),
                    pre=rng.choice(["rms", "layer"]), gate=rng.random() < 0.7, dtype=dtype,
                    stream="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]))
    if op == "matmul":
        m = rng.choice([_log(rng, 1, 64), _log(rng, 64, 100352)])
        n = _log(rng, 8, min(16384, 100352 * 1024 // m))
        k = _log(rng, 16, min(16384, 8192 ** 3 // (m * n), 8192 * 8192 // max(m, n)))
        return dict(op=op, m=m, n=n, k=k, x=rng.choice(["bf16", "f32", "mx"]), y=rng.choice(["bf16", "bf16", "f32"]),
                    act=rng.choice(["none", "relu", "silu", "gelu"]), bias=rng.random() < 0.5)
    rows = _log(rng, 1, 25088)
    c = _log(rng, 32, min(8192, 25088 * 512 // rows))
    return dict(op=op, rows=rows, c=c, hidden=_log(rng, 32, min(16384, 25088 * 512 * 2048 // (rows * c), 4 * c)),
                groups=rng.choice([1, min(rows, 3)]), post=rng.choice(["none", "rms"]),
                pre=rng.choice(["rms", "layer"]), act=rng.choice(["silu", "gelu"]), bias=rng.random() < 0.5)


# ------------------------------------------------------------------ the inputs

def _mx_bytes(rows, k):
    kb = -(-k // 32)
    return rows * (16 * kb + -(-kb // 4) * 4)


def work(case):
    op = case["op"]
    if op == "quantize":
        r, k, es = case["rows"], case["k"], _ES[case["dtype"]]
        # x read, codes and scales written, the values they stand for written
        return {"bytes": 2 * r * k * es + _mx_bytes(r, k), "flops": 2 * r * k}
    if op == "norm":
        r, c = case["rows"], case["c"]
        es, ss = _ES[case["dtype"]], _ES[case["stream"]]
        params = 4 * c * ((case["post"] != "none") + (case["post"] == "layer") + 1 + (case["pre"] == "layer"))
        gate = case["groups"] * c * es if case["gate"] else 0
        return {"bytes": 2 * r * c * (es + ss) + params + gate, "flops": 12 * r * c}
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        x = _mx_bytes(m, k) if case["x"] == "mx" else m * k * _ES[case["x"]]
        return {"bytes": x + _mx_bytes(n, k) + m * n * _ES[case["y"]] + (4 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    r, c, f = case["rows"], case["c"], case["hidden"]
    # b and r read, s and o written; the weights of both products
    return {"bytes": 4 * r * c * 2 + _mx_bytes(f, c) + _mx_bytes(c, f), "flops": 4 * r * c * f}


def _activations(g, rows, k, dtype):
    """Normal values whose channels differ in size, as activations' do: a few channels are many times the others."""
    x = torch.randn(rows, k, generator=g, device="cuda")
    return x.mul_(torch.randn(k, generator=g, device="cuda").mul_(0.8).exp_()).to(_DT[dtype])


def _weights(g, n, k):
    """A 4-bit weight matrix as a checkpoint holds it."""
    return _pack(torch.randn(n, k, generator=g, device="cuda") * k ** -0.5)


def _norm_inputs(g, case, dtype, stream):
    rows, c = case["rows"], case["c"]
    near_one = lambda: 1 + 0.1 * torch.randn(c, generator=g, device="cuda")  # noqa: E731
    near_zero = lambda: 0.1 * torch.randn(c, generator=g, device="cuda")  # noqa: E731
    s = {"b": _activations(g, rows, c, dtype), "r": _activations(g, rows, c, stream)}
    s["post_w"] = near_one() if case["post"] != "none" else None
    s["post_b"] = near_zero() if case["post"] == "layer" else None
    s["pre_w"] = near_one()
    s["pre_b"] = near_zero() if case["pre"] == "layer" else None
    s["gate"] = torch.randn(case["groups"], c, generator=g, device="cuda").to(_DT[dtype]) if case.get("gate", True) else None
    s["residual_scale"] = 0.75
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "quantize":
        s["x"] = _activations(g, case["rows"], case["k"], case["dtype"])
    elif case["op"] == "norm":
        s.update(_norm_inputs(g, case, case["dtype"], case["stream"]))
    elif case["op"] == "matmul":
        x = _activations(g, case["m"], case["k"], "f32" if case["x"] == "mx" else case["x"])
        s["x"] = _pack(x) if case["x"] == "mx" else x
        s["w"] = _weights(g, case["n"], case["k"])
        s["bias"] = torch.randn(case["n"], generator=g, device="cuda") if case["bias"] else None
    else:
        s.update(_norm_inputs(g, case, "bf16", "bf16"))
        c, f = case["c"], case["hidden"]
        s["w1"], s["w2"] = _weights(g, f, c), _weights(g, c, f)
        s["bias1"] = torch.randn(f, generator=g, device="cuda") if case["bias"] else None
        s["bias2"] = torch.randn(c, generator=g, device="cuda") if case["bias"] else None
    return s


# ------------------------------------------------------------------ plain forms

def _to_mx(x):
    """Blocks of x [rows][k] (32 bits): E2M1 values [rows][kb][32], and the blocks' exponent bytes [rows][kb]."""
    rows, k = x.shape
    kb = -(-k // 32)
    v = torch.nn.functional.pad(x, (0, kb * 32 - k)).view(rows, kb, 32)
    amax = v.abs().amax(-1)
    field = (amax.view(torch.int32) >> 23) & 255  # the largest value's exponent, biased
    byte = torch.where(field == 255, field, (field - 2).clamp(min=0))  # E2M1's largest exponent is 2
    inverse = ((254 - byte.clamp(max=253)) << 23).view(torch.float32)
    v = v * inverse.unsqueeze(-1)
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.copysign(((a / step).round() * step).clamp(max=6), v)
    return torch.where((byte == 255).unsqueeze(-1), torch.zeros_like(q), q), byte


def _scale(byte):
    """2^(byte - 127) in 32 bits; 255 stands for NaN."""
    s = torch.where(byte == 0, 0x00400000, byte << 23).view(torch.float32)
    return torch.where(byte == 255, float("nan"), s)


def _mx_values(x):
    """x [rows][k] (32 bits) rounded to MXFP4, in 32 bits."""
    q, byte = _to_mx(x)
    return (q * _scale(byte).unsqueeze(-1)).view(x.shape[0], -1)[:, :x.shape[1]]


def _pack(x):
    """(codes, scales, k) of x [rows][k]."""
    q, byte = _to_mx(x)
    a = q.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.int32)
    code = (code | (torch.signbit(q).to(torch.int32) << 3)).view(x.shape[0], -1, 2)
    codes = (code[..., 0] | (code[..., 1] << 4)).to(torch.uint8)
    kb = byte.shape[1]
    scales = torch.nn.functional.pad(byte, (0, -kb % 4), value=127).to(torch.uint8)
    return codes.contiguous(), scales.contiguous(), x.shape[1]


def _unpack(t):
    """The values, in 32 bits, that (codes, scales, k) stand for."""
    codes, scales, k = t
    c = codes.to(torch.int32)
    c = torch.stack((c & 15, c >> 4), -1).view(codes.shape[0], -1, 32)
    mag = c & 7
    low = mag.to(torch.float32) * 0.5
    a = torch.where(mag < 4, low, torch.where(mag < 6, low * 2 - 2, low * 4 - 8))
    v = torch.where(c > 7, -a, a) * _scale(scales.to(torch.int32))[:, :c.shape[1], None]
    return v.view(codes.shape[0], -1)[:, :k]


def _act(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "silu":
        return v / (1 + (-v).exp())
    if act == "gelu":  # the form with tanh
        return 0.5 * v * (1 + (0.7978845608028654 * (v + 0.044715 * v * v * v)).tanh())
    return v


def _norm(v, kind, w, b):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v / (v.square().mean(-1, keepdim=True) + EPS).sqrt() * w.to(v.dtype)
    return v if b is None else v + b.to(v.dtype)


def _gated_norm(s, to):
    """s and h of the fused norms, computed in the type `to`."""
    case = s["case"]
    b = _norm(s["b"].to(to), case["post"], s["post_w"], s["post_b"])
    if s["gate"] is not None:
        per = -(-case["rows"] // case["groups"])
        b = b * s["gate"].to(to).repeat_interleave(per, 0)[:case["rows"]]
    t = s["residual_scale"] * s["r"].to(to) + b
    return t, _norm(t, case["pre"], s["pre_w"], s["pre_b"])


def _linear(x, w, bias, act):
    y = x @ w.t()
    return _act(y if bias is None else y + bias.to(y.dtype), act)


def _plain(s):
    case = s["case"]
    if case["op"] == "quantize":
        return _mx_values(s["x"].float()).to(s["x"].dtype)
    if case["op"] == "norm":
        t, h = _gated_norm(s, torch.float32)
        return {"s": t.to(s["r"].dtype), "h": h.to(s["b"].dtype)}
    if case["op"] == "matmul":
        x = _unpack(s["x"]) if case["x"] == "mx" else _mx_values(s["x"].float())
        return _linear(x, _unpack(s["w"]), s["bias"], case["act"]).to(_DT[case["y"]])
    t, h = _gated_norm(s, torch.float32)
    u = _linear(_mx_values(h), _unpack(s["w1"]), s["bias1"], case["act"])
    o = _linear(_mx_values(u), _unpack(s["w2"]), s["bias2"], "none")
    return {"s": t.to(torch.bfloat16), "o": o.to(torch.bfloat16)}


# ------------------------------------------------------------------ this framework

def _own(s):
    from cnn_convolution_fwd_amd import binding as cfwd
    case = s["case"]
    if case["op"] == "quantize":
        return cfwd.mx_dequantize(cfwd.mx_quantize(s["x"]), dtype=case["dtype"])
    if case["op"] == "matmul":
        x = cfwd.MxTensor(*s["x"]) if case["x"] == "mx" else s["x"]
        return cfwd.mx_matmul(x, cfwd.MxTensor(*s["w"]), bias=s["bias"], act=case["act"], out_dtype=case["y"])
    t, h = cfwd.gated_norm(s["b"], residual=s["r"], gate=s["gate"], residual_scale=s["residual_scale"],
                           post=case["post"], post_weight=s["post_w"], post_bias=s["post_b"], pre=case["pre"],
                           pre_weight=s["pre_w"], pre_bias=s["pre_b"], eps=EPS,
                           out_dtype="mx" if case["op"] == "block" else case["dtype"])
    if case["op"] == "norm":
        return {"s": t, "h": h}
    u = cfwd.mx_matmul(h, cfwd.MxTensor(*s["w1"]), bias=s["bias1"], act=case["act"], out_dtype="mx")
    return {"s": t, "o": cfwd.mx_matmul(u, cfwd.MxTensor(*s["w2"]), bias=s["bias2"], out_dtype="bf16")}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits

def _mx64(x):
    """x rounded to MXFP4 by the definition, in 64 bits: the nearest of the eight magnitudes, a tie to the even code."""
    rows, k = x.shape
    kb = -(-k // 32)
    v = torch.zeros(rows, kb * 32, dtype=torch.float64, device=x.device)
    v[:, :k] = x
    v = v.view(rows, kb, 32)
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
    return (v.sign() * values[code] * unit).view(rows, kb * 32)[:, :k]


def _values64(t):
    codes, scales, k = t
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                         device=codes.device)
    v = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    v[:, 0::2] = table[(codes & 15).long()]
    v[:, 1::2] = table[(codes >> 4).long()]
    unit = torch.exp2(scales.double() - 127)[:, :codes.shape[1] // 16]
    return (v * unit.repeat_interleave(32, 1))[:, :k]


def _act64(v, act):
    if act == "gelu":
        return v * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (v + 0.044715 * v ** 3))
    return {"none": v, "relu": torch.relu(v), "silu": v * torch.sigmoid(v)}[act]


def _norm64(v, kind, w, b):
    if kind == "none":
        return v
    centre = v.mean(1, keepdim=True) if kind == "layer" else 0.0
    v = (v - centre) * torch.rsqrt((v - centre).pow(2).mean(1, keepdim=True) + EPS) * w.double()
    return v + (0.0 if b is None else b.double())


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _mx64(s["x"].double())
    if case["op"] == "matmul":
        x = _values64(s["x"]) if case["x"] == "mx" else _mx64(s["x"].double())
        y = torch.matmul(x, _values64(s["w"]).t())
        return _act64(y if s["bias"] is None else y + s["bias"].double(), case["act"])
    b = _norm64(s["b"].double(), case["post"], s["post_w"], s["post_b"])
    if s["gate"] is not None:
        rows = torch.arange(case["rows"], device="cuda") // -(-case["rows"] // case["groups"])
        b = b * s["gate"].double()[rows]
    t = b + s["residual_scale"] * s["r"].double()
    h = _norm64(t, case["pre"], s["pre_w"], s["pre_b"])
    if case["op"] == "norm":
        return {"s": t, "h": h}
    zero1 = 0.0 if s["bias1"] is None else s["bias1"].double()
    zero2 = 0.0 if s["bias2"] is None else s["bias2"].double()
    u = _act64(torch.matmul(_mx64(h), _values64(s["w1"]).t()) + zero1, case["act"])
    return {"s": t, "o": torch.matmul(_mx64(u), _values64(s["w2"]).t()) + zero2}
