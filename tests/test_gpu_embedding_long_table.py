"""The embedding gradient's zeros past 2^31 pieces, where their numbers need 64
bits and the clearing workgroups go round: rows shorter than a piece, cleared by
element."""
import pytest
import torch

import swiglu_activation_cast_amd as mx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [5, 3000])
def test_zeros_go_round(tokens):
    """Without a sort, where the marks of one round are cleared for the next, and
    with one."""
    V, H = 310_000_000, 7
    # by element: fewer columns than the 8 of a bf16 piece; a round is INT32_MAX / 512 workgroups of 256 elements
    assert H < 8 and V * H > 2**31 and V * H > 2 * (2**31 // 512 * 256)
    words = torch.arange(tokens, device="cuda") * (V // tokens) + 3
    dw = mx.mxtrain_embedding_bwd(torch.ones((tokens, H), device="cuda"), words, V,
                                  out=torch.full((V, H), 9.0, dtype=torch.bfloat16, device="cuda"))
    assert bool((dw[words] == 1).all())
    dw[words] = 0
    for lo in range(0, V, 1 << 26):
        assert not dw[lo:lo + (1 << 26)].any()
