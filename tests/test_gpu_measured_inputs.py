"""The measured cases' inputs (perf/more_operators.py): one seed means one input,
whichever preparation it is, since results of one are set against those of
another."""
import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def cases():
    spec = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("V,T", [(65536, 16640), (131071, 65537), (64, 1), (4099, 65537)])
def test_words_are_those_of_exact_sums(V, T):
    """Against running sums of the host, in whole numbers.  (2^40 / (i + 2.7) rounds
    alike in every IEEE division.)"""
    case = {"op": "embed", "tokens": T, "vocab": V, "width": 8, "dtype": "f32", "out": "f32", "ids": "i64"}
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    sums = np.cumsum((2.0 ** 40 / (np.arange(V) + 2.7)).astype(np.int64))
    draws = torch.randint(int(sums[-1]), (T,), generator=g, device="cuda").cpu().numpy()
    spread = torch.randperm(V, generator=g, device="cuda").cpu().numpy()
    want = spread[np.searchsorted(sums, draws, side="right")]
    assert np.array_equal(cases().prepare(case, 5)["t"].cpu().numpy(), want)


def test_two_preparations_are_equal():
    m = cases()
    for case in m.listed():
        print(f"case: {case['name']}", flush=True)
        a, b, c = (m.prepare(case, seed) for seed in (3, 3, 4))
        tensors = [k for k, v in a.items() if isinstance(v, torch.Tensor) and k != "order"]
        assert tensors and all(torch.equal(a[k], b[k]) for k in tensors)
        drawn = next(k for k in ("t", "e", "x") if k in tensors)
        assert not torch.equal(a[drawn], c[drawn])
