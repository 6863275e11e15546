"""Calls of the gated norm beside the ordinary ones: what its arguments may be and what they then mean."""
import pytest

from cnn_convolution_fwd_amd import binding as B
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


def test_scalars_given_as_tensors_count_with_their_values_at_the_call():
    torch = torch_cuda()
    b, r = torch.randn(4, 64, device="cuda"), torch.randn(4, 64, device="cuda")
    for device in ("cpu", "cuda"):
        scale, eps = torch.tensor(0.5, device=device), torch.tensor(1e-6, device=device)
        for value in (0.5, 2.0, -3.0):
            scale.fill_(value)
            eps.fill_(abs(value))
            got = B.gated_norm(b, r, residual_scale=scale, eps=eps)
            want = B.gated_norm(b, r, residual_scale=value, eps=float(eps))
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("c", [7, 64, 1000, 12000, 17000])
@pytest.mark.parametrize("post", ["rms", "layer"])
def test_an_absent_block_counts_as_its_posts_bias(c, post):
    """Also with eps = 0, where the norm of a row of zeros would be 0 / 0."""
    torch = torch_cuda()
    r, gate, w, bias = (torch.randn(*s, device="cuda") for s in ((5, c), (c,), (c,), (c,)))
    for pre in ("rms", "layer", "none"):
        for more in (dict(), dict(post_weight=w), dict(post_weight=w, post_bias=bias), dict(post_bias=bias, gate=gate)):
            s, h = B.gated_norm(None, r, residual_scale=0.5, post=post, pre=pre, eps=0.0, **more)
            add = torch.zeros(c, device="cuda") if "post_bias" not in more else bias * gate if "gate" in more else bias
            # 0.5 r is exact; the sum, or the sum and the product before it, is rounded to 2^-24
            assert bool(((s.double() - 0.5 * r.double() - add.double()).abs() <= 2.0 ** -23 * (r.abs() + add.abs())).all())
            want = B.gated_norm(None, s, pre=pre, eps=0.0)[1]
            assert (h is None and want is None) or torch.equal(h, want)


@pytest.mark.parametrize("c", [7, 40, 100, 512, 1001, 4096, 8192, 9000, 17000])
def test_the_norm_of_a_stream_alone_has_either_type(c):
    """Without b and gate h is float32 or bfloat16 as out_dtype or out says, from a stream of either type."""
    torch = torch_cuda()
    full = {"f32": torch.float32, "bf16": torch.bfloat16}
    r = torch.randn(5, c, device="cuda").bfloat16()
    for pre in ("rms", "layer"):
        kw = dict(residual_scale=0.5, pre=pre, pre_weight=torch.randn(c, device="cuda"))
        for stream in ("f32", "bf16"):
            _, want = B.gated_norm(None, r.float(), out_dtype="f32", **kw)  # 0.5 r is the same number in all of them
            for to in ("f32", "bf16"):
                s, h = B.gated_norm(None, r.to(full[stream]), out_dtype=to, **kw)
                assert s.dtype == full[stream] and h.dtype == full[to]
                assert torch.equal(s.float(), 0.5 * r.float()) and torch.equal(h, want.to(full[to]))
                out = torch.full((5 * c + 64,), 7.0, dtype=full[to], device="cuda")
                s, h = B.gated_norm(None, r.to(full[stream]), out=out[:5 * c].view(5, c), want_sum=False, **kw)
                assert s is None and torch.equal(h, want.to(full[to])) and bool((out[5 * c:] == 7).all())
    with pytest.raises(B.CfwdError):
        B.gated_norm(r.float(), r)
    with pytest.raises(B.CfwdError):
        B.gated_norm(None, r, gate=torch.randn(c, device="cuda"))


def test_no_h_for_out():
    """pre none has no h: an out is refused, not left unwritten."""
    torch = torch_cuda()
    r = torch.randn(4, 64, device="cuda")
    for out in (torch.empty_like(r), B.mx_quantize(r)):
        with pytest.raises(ValueError):
            B.gated_norm(r, r, pre="none", out=out)
    assert B.gated_norm(r, r, pre="none")[1] is None
