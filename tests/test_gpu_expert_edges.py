"""The experts' products at their smallest operands (no K, a single row) and with
far more experts than rows."""
import pytest
import torch

import swiglu_activation_cast_amd as mx

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def whole(shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-4, 5, shape, generator=g, device="cuda").to(BF16)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,N", [(16, 32), (5, 33), (300, 1030)])
def test_no_depth_gives_zeros(T, N, dtype):
    ends = torch.tensor([T // 2, T], dtype=torch.int32, device="cuda")
    for b, transpose_b in ((whole((2, N, 0), 1), True), (whole((2, 0, N), 1), False)):
        out = torch.full((T, N), 7.0, dtype=dtype, device="cuda")
        mx.mxtrain_grouped_gemm(whole((T, 0), 1), b, ends, transpose_b=transpose_b, out=out)
        assert not out.any()
    empty = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert not mx.mxtrain_grouped_gemm_k(whole((0, T), 1), whole((0, N), 1), empty, out_dtype=dtype).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("K", [1, 4, 12, 70, 257])
def test_a_single_contiguous_row_of_any_length(K, dtype):
    """Sums of fewer than 2^18 products of numbers up to 4 are exact."""
    N, one = 40, torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    pad = -K % 8
    x, w = whole((1, K), K), whole((2, N, K + pad), K + 1)[..., :K]
    y = mx.mxtrain_grouped_gemm(x, w, one, out_dtype=dtype)
    assert torch.equal(y, (x.double() @ w[1].double().T).to(dtype))
    # one row of weights, and a depth of one
    xs, w1 = whole((9, K + pad), K + 2)[:, :K], whole((1, 1, K), K + 3)
    nine = torch.tensor([9], dtype=torch.int32, device="cuda")
    assert torch.equal(mx.mxtrain_grouped_gemm(xs, w1, nine, out_dtype=dtype), (xs.double() @ w1[0].double().T).to(dtype))
    d, wd = whole((9, 8), K + 4)[:, :1], whole((1, 1, K), K + 5)
    got = mx.mxtrain_grouped_gemm(d, wd, nine, transpose_b=False, out_dtype=dtype)
    assert torch.equal(got, (d.double() @ wd[0].double()).to(dtype))
    # one token's weight gradient
    dy = whole((1, 33), K + 6)
    got = mx.mxtrain_grouped_gemm_k(dy, x, one, out_dtype=dtype)
    assert not got[0].any() and torch.equal(got[1], (dy.double().T @ x.double()).to(dtype))


def test_far_more_experts_than_rows():
    """As many tiles as rows can fill are launched, not as many as experts
    (65535 experts of 16392 columns would be more than a launch holds)."""
    G, T, N, K = 65535, 70, 16392, 8
    print(f"case: {T} rows over {G} experts", flush=True)
    g = torch.Generator()
    g.manual_seed(11)
    owner = torch.sort(torch.randint(0, G, (T,), generator=g)).values
    owner[-1] = G - 1
    ends = torch.bincount(owner, minlength=G).cumsum(0).to(torch.int32).cuda()
    owner = owner.cuda()
    x, used = whole((T, K), 10), whole((T, N, K), 9)
    w = torch.full((G, N, K), float("nan"), dtype=BF16, device="cuda")  # 17 GB
    w[owner] = used
    y = mx.mxtrain_grouped_gemm(x, w, ends, out_dtype=F32)
    assert torch.equal(y, (w[owner].float() * x.float()[:, None, :]).sum(2))
