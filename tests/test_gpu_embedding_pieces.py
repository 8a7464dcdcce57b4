"""The embedding's kernels at sizes where their numbering of pieces changes: from
1048576 pieces of rows a lookup takes two of them a thread."""
import pytest
import torch

import swiglu_activation_cast_amd as mx

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float32]


# the last workgroup of 512 pieces has a few first pieces (4098 tokens) or all of them and
# some second ones (4480; with whole fp32 pieces no second one)
@pytest.mark.parametrize("wt", TYPES)
@pytest.mark.parametrize("yt", TYPES)
@pytest.mark.parametrize("H", [2050, 2056])
@pytest.mark.parametrize("T", [4098, 4480])
def test_lookup_of_two_pieces_a_thread(T, H, wt, yt):
    """To the bit where the scale is one (a bf16 result is then one rounding, as
    torch's); with another one product and its rounding, u = 2^-24 of the value and
    as much for the scale's own, half a step, 2^-8, of a bf16 result."""
    V, first = 3000, 40
    per = -(-H // (4 if wt == yt == torch.float32 else 8))
    assert T * per >= 2 * 256 * 2048 and T * per % 512 != 0
    g = torch.Generator(device="cuda")
    g.manual_seed(T + H)
    w = torch.randn((V, H), generator=g, device="cuda").to(wt)
    for dtype in (torch.int64, torch.int32):
        print(f"case: lookup {T} of {V}x{H} {wt} {yt} {dtype}", flush=True)
        ids = torch.randint(first - 50, first + V + 50, (T,), generator=g, device="cuda").to(dtype)
        key = ids.long() - first
        inside = ((key >= 0) & (key < V))[:, None]
        rows = torch.where(inside, w[key.clamp(0, V - 1)], 0)
        wide = torch.full((T, H + 5), 9.0, dtype=yt, device="cuda")
        y = mx.mxtrain_embedding_fwd(w, ids, first=first, out=wide[:, 3:3 + H])
        assert torch.equal(y, rows.to(yt))
        assert bool((wide[:, :3] == 9).all()) and bool((wide[:, 3 + H:] == 9).all())
        y = mx.mxtrain_embedding_fwd(w, ids, first=first, scale=1.7, out_dtype=yt)
        ref = rows.double() * 1.7
        assert bool(((y.double() - ref).abs() <= ref.abs() * (2 * U + (2.0 ** -8 if yt == torch.bfloat16 else 0.0))).all())
        assert not y[~inside[:, 0]].any()
