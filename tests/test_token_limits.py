"""The embedding gradient's limit of tokens and columns, without a GPU: every call
below is refused."""
import pytest

import swiglu_activation_cast_amd as mx

NULL, OVERFLOW = 1, 6
BF16, F32 = 0, 1
A = 1 << 20  # a fake, aligned "device address" (never dereferenced)


def embed_bwd(T, H, tt, wt, V=100):
    """Without the workspace that so many tokens need: what is within the limit is
    refused for that."""
    return mx.train_lib().mxtrain_embedding_bwd(A, H, tt, A, 1, 1, T, 0, 1.0, V, H, A, H, wt, 0, None, 0, None)


# ceil(T / 64) times the strips of a row, 512 columns or 256 of fp32 into fp32, at most 2^23 - 1
@pytest.mark.parametrize("tt,wt,strip", [(BF16, BF16, 512), (BF16, F32, 512), (F32, BF16, 512), (F32, F32, 256)])
def test_border(tt, wt, strip):
    ws = mx.train_lib().mxtrain_embedding_bwd_workspace
    for T, strips in ((2**29, 1), (2**29 - 63, 1), (2**28, 2), (65, 2**22), (511, 2**20)):
        for H in ({strips * strip, (strips - 1) * strip + 1} - {2**31}):
            assert embed_bwd(T, H, tt, wt) == OVERFLOW and ws(T, 100, H, tt, wt) == 0
    for T, strips in ((2**29 - 64, 1), (2**28 - 64, 2), (65, 2**22 - 1), (448, 2**20)):
        assert embed_bwd(T, strips * strip, tt, wt) == NULL and ws(T, 100, strips * strip, tt, wt) > 0
