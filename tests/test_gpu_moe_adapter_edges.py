"""moe_adapter_matmul where its sums leave the ordinary range, against 64 bits."""
import math

import pytest
import torch

from moe_refs import DTYPES
from symmetric_memory_moe_gb300 import abi
from symmetric_memory_moe_gb300.torch_heap import TorchSymmHeap
from test_gpu_moe_adapter import check, make, run

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


@pytest.mark.parametrize("r", [8, 16, 32, 40, 128])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_the_rank_sums_keep_24_bits(heap, T, r, dt):
    """What is left of scale x A after W has taken away its first two values of the type.
    x picks one row of A, B is the identity and scale a power of two times a float of 24
    bits, so h = scale A[0] is one rounded product; every further product and partial
    sum is a multiple of h's last bit below 2 |h|, exact in 32 bits in any order.  h is
    about 2^8, so that its last bit (2^-16) is well within fp16."""
    k, n = 64, 136
    g = torch.Generator(device="cuda").manual_seed(r + T)
    x = torch.zeros(T, k, device="cuda")
    x[:, :3] = 1
    a = torch.zeros(2, k, r, device="cuda")
    a[:, 0] = 1 + torch.randint(0, 128, (2, r), generator=g, device="cuda") / 128
    scale = 128 + 64 * torch.rand(2, generator=g, device="cuda")
    h = a[1, 0] * scale[1]                                  # in 32 bits
    h1 = h.to(DTYPES[dt]).float()
    h2 = (h - h1).to(DTYPES[dt]).float()
    w = torch.zeros(k, n, device="cuda")
    w[1, :r], w[2, :r] = -h1, -h2
    b = torch.zeros(2, r, n, device="cuda")
    b[:, :, :r] = torch.eye(r, device="cuda")
    i = dict(x=x, w=w, a=a, b=b)
    i = {m: v.to(DTYPES[dt]) for m, v in i.items()}
    i.update(scale=scale, ids=torch.ones(T, dtype=torch.int32, device="cuda"))
    y = run(heap, i, dt).float()
    want = h - h1 - h2
    assert (want != 0).sum() > r // 3 or dt == "f16"
    assert (y[:, :r] == want).all() and not y[:, r:].any()


@pytest.mark.parametrize("r", [8, 16, 64])
@pytest.mark.parametrize("down", [6, 10, 14, 18])
def test_small_rank_sums_in_half_precision(heap, r, down):
    """A far below 1 and B above it: half precision has no bits there, the sums do."""
    i = make(70, 256, 264, 3, r, "f16", 9, "mixed")
    i["a"] = (i["a"].float() * 2.0 ** -down / 16).half()
    i["b"] = (i["b"].float() * 2.0 ** min(10, down)).half()
    i["w"] = (i["w"].float() * 2.0 ** -6).half()
    check(i, run(heap, i, "f16"), "f16")


def test_large_rank_sums_in_half_precision(heap):
    """scale x A beyond 65504, which B brings back."""
    i = make(70, 256, 264, 3, 16, "f16", 9, "mixed")
    i["a"] = (i["a"].float() * 2.0 ** 12).half()
    i["b"] = (i["b"].float() * 2.0 ** -14).half()
    i["scale"] = i["scale"].abs() + 2
    assert (i["x"].double() @ i["a"][1].double() * 2).abs().max() > 2e5
    check(i, run(heap, i, "f16"), "f16")


@pytest.mark.parametrize("T,k,n,r", [(1, 4096, 4096, 16), (70, 1024, 264, 72),
                                     (600, 512, 2048, 32)])
def test_a_budget_of_a_nanosecond(heap, T, k, n, r):
    """Every wait that is not over at once may give up: the call ends, writes nothing but y,
    and says so or is right; the next one, with time again, is right."""
    i = make(T, k, n, 3, r, "bf16", 2, "mixed")
    x, w = i["x"], i["w"]
    y = torch.full((T + 1, n), 7.0, dtype=x.dtype, device="cuda")
    ws = torch.empty(abi.moe_adapter_workspace(T, k, n, r), dtype=torch.uint8, device="cuda")
    abi.symm_set_spin_budget(heap.handle, 1)
    try:
        abi.moe_adapter_matmul(heap.handle, x.data_ptr(), k, w.data_ptr(), n, i["a"].data_ptr(),
                               i["b"].data_ptr(), i["scale"].data_ptr(), i["ids"].data_ptr(),
                               abi.SYMM_DTYPE_BF16, T, k, n, 3, r, y.data_ptr(), n, ws.data_ptr())
        code = abi.symm_check_error(heap.handle)[0]
    finally:
        abi.symm_set_spin_budget(heap.handle, 2_000_000_000)
    assert code in (abi.SYMM_OK, abi.SYMM_ETIMEDOUT) and (y[T] == 7).all()
    if code == abi.SYMM_OK:
        check(i, y[:T], "bf16")
    check(i, run(heap, i, "bf16"), "bf16")
