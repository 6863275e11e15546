"""The fused norms, gate and residual scale on the GPU against the 64-bit reference."""
import sys

import numpy as np
import pytest

from cnn_convolution_fwd_amd import binding as B
from tests import mx_reference as R
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

EPS = 1e-5


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def tensor(x, dtype):
    torch = torch_cuda()
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()
    return t.bfloat16() if dtype == "bf16" else t


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def run(rng, rows, c, dtype="bf16", stream="bf16", post="rms", pre="rms", gate_rows=1, use_b=True, use_r=True,
        affine=True, out="same", spread=1.0, **more):
    """One call and the check of both its outputs; returns (s, h)."""
    b = tensor(rng.normal(size=(rows, c)) * np.exp(spread * rng.normal(size=(rows, 1))), dtype) if use_b else None
    r = tensor(rng.normal(size=(rows, c)) + 0.3, stream) if use_r else None
    gate = tensor(rng.normal(size=(gate_rows, c)), dtype) if gate_rows else None
    vec = lambda at: tensor(at + 0.3 * rng.normal(size=c), "f32") if affine else None  # noqa: E731
    args = dict(post_weight=vec(1), post_bias=vec(0), pre_weight=vec(1), pre_bias=vec(0))
    s, h = B.gated_norm(b, residual=r, gate=gate, residual_scale=0.7, post=post, pre=pre, eps=EPS,
                        out_dtype="mx" if out == "mx" else None, **args, **more)
    at = lambda t: None if t is None else host(t)  # noqa: E731
    per = -(-rows // gate_rows) if gate_rows else 1
    ws, es, wh, eh = R.gated_norm(at(b), at(r), at(gate), per, 0.7, post, at(args["post_weight"]),
                                  at(args["post_bias"]), pre, at(args["pre_weight"]), at(args["pre_bias"]),
                                  float(np.float32(EPS)))
    if s is not None:
        R.assert_close(host(s), ws, es, s.dtype == torch_cuda().bfloat16)
    if pre == "none":
        assert h is None
    elif out == "mx":
        R.assert_mx_close(h.codes.cpu().numpy(), h.scales.cpu().numpy(), wh, eh)
    else:
        R.assert_close(host(h), wh, eh, h.dtype == torch_cuda().bfloat16)
    return s, h


LENGTHS = [1, 2, 7, 8, 9, 31, 32, 33, 63, 64, 65, 100, 128, 129, 250, 256, 257, 511, 512, 513, 777, 1000, 1024, 1025,
           2048, 2049, 4000, 4096, 4097, 8191, 8192, 8193, 16384, 16385, 20001]


@pytest.mark.parametrize("c", LENGTHS)
@pytest.mark.parametrize("dtype,stream", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_lengths(c, dtype, stream):
    rng = np.random.default_rng(c)
    for out in ("same", "mx"):
        say("gated norm", c, dtype, stream, out)
        run(rng, 5, c, dtype, stream, out=out)
        run(rng, 3, c, dtype, stream, post="layer", pre="layer", out=out)


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("c", [40, 520, 4096, 17000])
def test_norms_and_missing_parts(post, pre, c):
    rng = np.random.default_rng(c)
    for rows, gate_rows in ((1, 1), (10, 3), (9, 0), (7, 7)):
        run(rng, rows, c, post=post, pre=pre, gate_rows=gate_rows)
        run(rng, rows, c, post=post, pre=pre, gate_rows=gate_rows, use_r=False, affine=False)
    run(rng, 4, c, post=post, pre=pre, use_b=False, gate_rows=0)
    if pre != "none":
        s, _ = run(rng, 4, c, post=post, pre=pre, want_sum=False)
        assert s is None


@pytest.mark.parametrize("rows,c", [(1, 4096), (3, 64), (1000, 96), (4099, 16), (700, 1536), (3136, 512), (2500, 2048),
                                    (600, 8192)])
def test_many_rows(rows, c):
    rng = np.random.default_rng(rows)
    run(rng, rows, c, gate_rows=min(rows, 64))
    run(rng, rows, c, "bf16", "f32", post="none", pre="layer", out="mx")


@pytest.mark.parametrize("c", [96, 4096, 17000])
def test_sum_in_place(c):
    """s written over the residual, and over b, equals s written apart."""
    torch = torch_cuda()
    rng = np.random.default_rng(1)
    b, r = tensor(rng.normal(size=(6, c)), "bf16"), tensor(rng.normal(size=(6, c)), "bf16")
    for post, pre in (("rms", "rms"), ("none", "layer"), ("layer", "none")):
        s, h = B.gated_norm(b, r, post=post, pre=pre)
        for target in ("r", "b"):
            b2, r2 = b.clone(), r.clone()
            s2, h2 = B.gated_norm(b2, r2, post=post, pre=pre, sum_out=r2 if target == "r" else b2)
            assert torch.equal(s, s2) and (h is None or torch.equal(h, h2))


@pytest.mark.parametrize("c", [33, 1000, 17000])
def test_special_rows(c):
    """A row of zeros, of one value, with a NaN, with an infinity: each row stands alone."""
    torch = torch_cuda()
    rng = np.random.default_rng(2)
    x = rng.normal(size=(6, c))
    x[1] = 0.0
    x[2] = 5.0
    x[3, c // 2] = np.nan
    x[4, 0] = np.inf
    t = tensor(x, "f32")
    for pre in ("rms", "layer"):
        s, h = B.gated_norm(None, t, pre=pre, eps=EPS)
        assert torch.equal(torch.nan_to_num(s), torch.nan_to_num(t))
        got = host(h)
        for i in (0, 1, 2, 5):
            want, err = R.norm(host(t)[i:i + 1], np.zeros((1, c)), pre, None, None, float(np.float32(EPS)))
            R.assert_close(got[i:i + 1], want, err + 1e-30)
        assert np.isnan(got[3]).all() and np.isnan(got[4, 0])
        q = B.gated_norm(None, t, pre=pre, eps=EPS, out_dtype="mx")[1]
        byte = q.scales.cpu().numpy()[:, :-(-c // 32)]
        assert (byte[3] == 255).all() and (byte[[0, 1, 2, 5]] != 255).all() and byte[4, 0] == 255


def test_writes_nothing_else():
    torch = torch_cuda()
    for rows, c in ((3, 45), (2, 1000), (1, 17001)):
        b, r = torch.randn(rows, c, device="cuda"), torch.randn(rows, c, device="cuda")
        s = torch.full((rows * c + 64,), 7.0, device="cuda")
        h = torch.full((rows * c + 64,), 7.0, device="cuda")
        B.gated_norm(b, r, sum_out=s[:rows * c].view(rows, c), out=h[:rows * c].view(rows, c))
        assert (s[rows * c:] == 7).all() and (h[rows * c:] == 7).all()
        cp, sp = B.mx_pitches(c)
        codes = torch.full((rows * cp + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        scales = torch.full((rows * sp + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        B.gated_norm(b, r, out=B.MxTensor(codes[:rows * cp].view(rows, cp), scales[:rows * sp].view(rows, sp), c))
        assert (codes[rows * cp:] == 0xA5).all() and (scales[rows * sp:] == 0xA5).all()


def test_unaligned_tensors_and_batches():
    """Rows at addresses aligned to their elements alone; leading axes."""
    torch = torch_cuda()
    buf = torch.randn(2, 5 * 203 + 1, device="cuda").bfloat16()
    b, r = buf[0, 1:].view(5, 203), buf[1, 1:].view(5, 203)
    s, h = B.gated_norm(b, r, post="rms", pre="layer")
    s2, h2 = B.gated_norm(b.clone(), r.clone(), post="rms", pre="layer")
    assert torch.equal(s, s2) and torch.equal(h, h2)
    s, h = B.gated_norm(torch.randn(2, 3, 4, 64, device="cuda"), out_dtype="mx")
    assert s.shape == (2, 3, 4, 64) and h.shape == (2, 3, 4, 64)
    s, h = B.gated_norm(torch.empty(0, 64, device="cuda"))
    assert s.shape == h.shape == (0, 64)
    f = torch.randn(4, 64, device="cuda")
    assert B.gated_norm(None, f, out_dtype="bf16")[1].dtype == torch.bfloat16


def test_in_a_graph():
    torch = torch_cuda()
    b, r = torch.randn(7, 1024, device="cuda"), torch.randn(7, 1024, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s, h = B.gated_norm(b, r, post="rms", pre="layer")
    for _ in range(4):
        b.normal_()
        graph.replay()
        torch.cuda.synchronize()
        s2, h2 = B.gated_norm(b, r, post="rms", pre="layer")
        assert torch.equal(s, s2) and torch.equal(h, h2)


@pytest.mark.parametrize("case", ["none", "shape", "gate", "weight", "norm", "dtype", "strides", "stream", "overlap", "eps"])
def test_refusals(case):
    torch = torch_cuda()
    b, r = torch.randn(4, 64, device="cuda"), torch.randn(4, 64, device="cuda")
    with pytest.raises((ValueError, TypeError, B.CfwdError)):
        if case == "none":
            B.gated_norm(None)
        elif case == "shape":
            B.gated_norm(b, r[:3])
        elif case == "gate":
            B.gated_norm(b, r, gate=torch.ones(4, 63, device="cuda"))
        elif case == "weight":
            B.gated_norm(b, r, pre_weight=torch.ones(64, device="cuda").bfloat16())
        elif case == "norm":
            B.gated_norm(b, r, pre="batch")
        elif case == "dtype":
            B.gated_norm(b.half(), r.half())
        elif case == "strides":
            B.gated_norm(b[:, ::2], r[:, ::2])
        elif case == "stream":
            B.gated_norm(b, r.bfloat16())
        elif case == "overlap":
            B.gated_norm(b, r, out=b)
        else:
            B.gated_norm(b, r, eps=-1.0)
