"""The training operators called for another stream than the current one, on the GPU."""
import pytest
import torch

import swiglu_activation_cast_amd as mx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("as_handle", [False, True])
def test_handover_to_the_default_stream(as_handle):
    """Called from a side stream for the default one: the default stream waits
    for the side stream's work on the inputs, and what the call allocated is not
    handed out again on the side stream before the default stream is done."""
    x = torch.randn((4000, 768), device="cuda").to(torch.bfloat16)
    dy, w = torch.randn_like(x), torch.randn(768, device="cuda")
    y, mean, rstd = mx.mxtrain_layer_norm_fwd(x, w)
    want = mx.mxtrain_layer_norm_bwd(dy, x, mean, rstd, w)
    torch.cuda.synchronize()
    default = torch.cuda.default_stream()
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            late = torch.zeros_like(dy)
            late.copy_(dy)
            got = mx.mxtrain_layer_norm_bwd(late, x, mean, rstd, w, stream=0 if as_handle else default)
            junk = torch.full((1 << 22,), float("nan"), device="cuda")  # would land in a workspace reused too early
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del junk, late
