"""moe_adapter_matmul where its sums leave the ordinary range, against 64 bits."""
import math

import pytest
import torch

from moe_refs import DTYPES
from symmetric_memory_moe_gb300.torch_heap import TorchSymmHeap
from test_gpu_moe_adapter import make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def heap():
    h = TorchSymmHeap(1, 0)
    yield h
    h.close()


@pytest.mark.parametrize("T,r,dt", [(1, 8, "bf16"), (20, 16, "f16"), (300, 72, "bf16")])
def test_an_infinite_sum_keeps_its_sign(heap, T, r, dt):
    """With x, scale and B above 0, an infinity in A (or x) is one in every output, as in the
    formula: the other terms are finite and no factor is 0."""
    i = make(T, 64, 136, 2, r, dt, 5, "one")
    i.update(x=i["x"].abs() + 0.5, b=i["b"].abs() + 0.5, scale=i["scale"].abs() + 0.5)
    for sign in (1, -1):
        a = i["a"].clone()
        a[1, 3, r - 1] = sign * math.inf
        y = run(heap, dict(i, a=a), dt)
        assert (y == sign * math.inf).all()
    # in x: W and the sums over A are of one sign too
    j = dict(i, x=i["x"].clone(), w=i["w"].abs() + 0.5, a=i["a"].abs() + 0.5)
    j["x"][0, 5] = math.inf
    y = run(heap, j, dt)
    assert (y[0] == math.inf).all() and torch.isfinite(y[1:]).all()
    assert y.dtype == DTYPES[dt]
