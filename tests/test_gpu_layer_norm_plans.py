"""Layer norm on the row plans that the shapes of test_gpu_layer_norm.py do not
reach, at that file's tolerances: the forward with 32 elements a thread (many
rows of 8193 .. 16384 columns moved as vectors), by element with 16 (as wide),
the backward by element with 16 (4097 .. 8192 columns), with its columns in
workgroups of their own and joined, 64 threads of 16 elements by element (many
odd rows of 513 .. 1024), 16 threads a row by element (many odd rows up to 128)."""
import pytest
import torch

from test_gpu_layer_norm import test_forward_and_backward as forward_and_backward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N", [(1030, 12296), (5, 9001), (1027, 9001), (5, 5001), (300, 5001), (1100, 5001), (1027, 777),
                                 (1030, 99), (1029, 513), (1025, 16384), (257, 8191)])
def test_other_row_plans(M, N, dtype):
    forward_and_backward(M, N, dtype)
