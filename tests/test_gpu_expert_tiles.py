"""The experts' products in 256 x 256 tiles: whole rounds, the cut-down last
round (halves, quarters), short tiles of a group's last rows, on whole numbers
up to 4 (every sum below 2^24 and so exact in fp32 whatever its order).

A launch runs in rounds of 256 tiles, one per compute unit.  Each case says
which last round it is made for, and the test checks that by counting its tiles.
"""
import pytest
import torch

import swiglu_activation_cast_amd as mx
from test_gpu_expert_products import bounds, padded, ref_k, ref_m, whole

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
CUS = 256


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def last_round(tiles):
    tail = tiles % CUS
    return "none" if tail == 0 else "quarters" if tail <= CUS // 4 else "halves" if tail <= CUS // 2 else "whole"


# ends with an empty group, last tiles of up to 64 and up to 128 rows, an end
# below the one before it and one past the last row; N across and off the cuts
# of a tile (64, 128); K off the stages (64) and their chunks (8)
ENDS = [1000, 1000, 1060, 700, 1188, 2500, 4300]
GROUPED = [(4300, ENDS, 3684, 72, "quarters"), (4300, ENDS, 4200, 129, "halves"), (4300, ENDS, 5007, 200, "whole"),
           (4300, ENDS, 3000, 328, "whole"), (4200, ENDS, 3584 + 64, 100, "quarters"), (4400, ENDS, 4140, 65, "halves"),
           (4096, [4096], 4096, 136, "none"), (2049, [2049], 2048 * 4 + 1, 96, "quarters")]


@pytest.mark.parametrize("transpose_b", [True, False])
@pytest.mark.parametrize("T,ends,N,K,last", GROUPED)
def test_grouped_products(T, ends, N, K, last, transpose_b):
    print(f"case: grouped {T}x{N}x{K} transpose_b {transpose_b}, last round {last}", flush=True)
    G, cols = len(ends), (N + 255) // 256
    rows = sum((hi - lo + 255) // 256 for lo, hi in bounds(ends, T))
    # what the choice of tile looks at: groups of even size
    assert K > 64 and G * ((-(-T // G) + 255) // 256) * cols >= CUS * 2 // 3 and T // G > 128
    assert last_round(rows * cols) == last
    g = gen(T + N + K)
    a = padded(whole((T, K), g), -K % 8 + 8, float("nan"))
    b = padded(whole((G, N, K) if transpose_b else (G, K, N), g), (-K if transpose_b else -N) % 8 + 8, float("nan"))
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    want = ref_m(a, b, ends, transpose_b)
    for dtype, pad in ((F32, 0), (BF16, 3), (BF16, 0), (F32, 4)):
        base = torch.full((T, N + pad), 77.0, dtype=dtype, device="cuda")
        mx.mxtrain_grouped_gemm(a, b, e, transpose_b=transpose_b, out=base[:, :N])
        n = want.shape[0]
        assert torch.equal(base[:n, :N], want.to(dtype))
        assert bool((base[n:] == 77.0).all()) and bool((base[:, N:] == 77.0).all())


# tokens, ends, M, N of the weight gradient
OVER_TOKENS = [(520, [300, 300, 520], 2100, 2600, "quarters"), (700, [90, 91, 40, 699], 1900, 2700, "halves"),
               (333, [100, 400], 3400, 3600, "whole"), (300, [0, 300], 4000, 2000, "none"), (130, [130], 4097, 4100, "quarters"),
               (600, [64, 200, 600], 1921, 2369, "whole")]


@pytest.mark.parametrize("T,ends,M,N,last", OVER_TOKENS)
def test_weight_gradients(T, ends, M, N, last):
    print(f"case: grouped over tokens {T}x{M}x{N}, last round {last}", flush=True)
    G = len(ends)
    tiles = G * ((M + 255) // 256) * ((N + 255) // 256)
    assert T // G > 64 and tiles >= CUS * 2 // 3 and last_round(tiles) == last
    g = gen(T * 3 + M + N)
    a, b = (padded(whole((T, w), g), -w % 8 + 8, float("nan")) for w in (M, N))
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    want = ref_k(a, b, ends)
    for dtype in (F32, BF16):
        assert torch.equal(mx.mxtrain_grouped_gemm_k(a, b, e, out_dtype=dtype), want.to(dtype))
        base = torch.full((G, M + 1, N + 5), 77.0, dtype=dtype, device="cuda")
        mx.mxtrain_grouped_gemm_k(a, b, e, out=base[:, :M, :N])
        assert torch.equal(base[:, :M, :N], want.to(dtype))
        assert bool((base[:, M:] == 77.0).all()) and bool((base[:, :, N:] == 77.0).all())
