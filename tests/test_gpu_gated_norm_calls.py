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
