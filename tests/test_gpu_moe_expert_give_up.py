"""The bounded waits of the experts' operators with a budget of a nanosecond.  Every wait that is
not over soon may give up, and whichever it is, all roles of both CTAs of its pair must leave: the
call ends, writes nothing outside its outputs, and says so or is right; until the error is read,
later calls may give up as well; then the next one, with time again, is right.  Long
contractions keep the epilogue waiting, many tiles a pair keep the others waiting for it."""
import pytest
import torch

import expert_refs as ref
from moe_refs import CODES, TINY, U_OUT
from symmetric_memory_moe_gb300 import abi
from symmetric_memory_moe_gb300.torch_heap import TorchSymmHeap
from test_gpu_moe_expert import ACTS, POISON, backward, forward, make, near, ptr
from test_gpu_moe_fp4 import FMTS, operands, product

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def heap():
    h = TorchSymmHeap(1, 0)
    yield h
    h.close()


class ShortBudget:
    def __init__(self, heap):
        self.heap = heap

    def __enter__(self):
        abi.symm_set_spin_budget(self.heap.handle, 1)

    def __exit__(self, *_):
        abi.symm_set_spin_budget(self.heap.handle, 2_000_000_000)


def read(heap):
    code = abi.symm_check_error(heap.handle)[0]
    assert code in (abi.SYMM_OK, abi.SYMM_ETIMEDOUT)
    return code


@pytest.mark.parametrize("n,E,D,F", [(40, 2, 64, 32), (300, 1, 1 << 17, 64), (64, 8, 7168, 256),
                                     (20000, 2, 2048, 512)])
def test_forward(heap, n, E, D, F):
    i = make(n, E, D, F, "bf16", "even")
    y = torch.full((n + 1, D), POISON, dtype=BF16, device="cuda")
    gu = torch.full((n + 1, 2 * F), POISON, dtype=BF16, device="cuda")
    ws = torch.empty(abi.moe_expert_workspace(n, E, D, F), dtype=torch.uint8, device="cuda")
    for calls in (1, 2):
        with ShortBudget(heap):
            for _ in range(calls):
                abi.moe_expert_ffn(heap.handle, ptr(i["x"]), D, ptr(i["counts"]), ptr(i["w_gu"]),
                                   ptr(i["w_d"]), ACTS["silu"], CODES["bf16"], n, E, D, F, ptr(gu),
                                   ptr(y), D, ptr(ws))
            code = read(heap)
        assert (y[n] == POISON).all() and (gu[n] == POISON).all()
        again, saved = forward(heap, i, "bf16", "silu")
        r = ref.ffn(i["x"], i["counts"], i["w_gu"], i["w_d"], "silu", U_OUT["bf16"], TINY["bf16"])
        near(saved, r["gu"], r["egu"], "gu")
        near(again, r["y"], r["ey"], "y")
        if code == abi.SYMM_OK:
            assert torch.equal(y[:n], again) and torch.equal(gu[:n], saved)


@pytest.mark.parametrize("n,E,D,F", [(40, 2, 64, 32), (300, 1, 1 << 17, 64), (1 << 17, 1, 64, 64),
                                     (20000, 2, 2048, 512)])
def test_backward(heap, n, E, D, F):
    i = make(n, E, D, F, "bf16", "even")
    gu = torch.randn(n, 2 * F, generator=torch.Generator().manual_seed(n)).bfloat16().cuda()
    dx = torch.full((n + 1, D), POISON, dtype=BF16, device="cuda")
    g1 = torch.full((E + 1, D, 2 * F), POISON, dtype=BF16, device="cuda")
    g2 = torch.full((E + 1, F, D), POISON, dtype=BF16, device="cuda")
    ws = torch.empty(abi.moe_expert_workspace(n, E, D, F, True), dtype=torch.uint8, device="cuda")
    for calls in (1, 2):
        with ShortBudget(heap):
            for _ in range(calls):
                abi.moe_expert_ffn_backward(
                    heap.handle, ptr(i["dy"]), D, ptr(i["x"]), D, ptr(gu), ptr(i["counts"]),
                    ptr(i["w_gu"]), ptr(i["w_d"]), ACTS["silu"], CODES["bf16"], n, E, D, F, ptr(dx),
                    D, ptr(g1), ptr(g2), ptr(ws))
            code = read(heap)
        assert all((t[-1] == POISON).all() for t in (dx, g1, g2))
        again = backward(heap, i, gu, "bf16", "silu")
        r = ref.ffn_grad(i["dy"], i["x"], gu, i["counts"], i["w_gu"], i["w_d"], "silu",
                         U_OUT["bf16"], TINY["bf16"])
        for k, t in (("dx", dx), ("dw_gu", g1), ("dw_d", g2)):
            near(again[k], r[k], r["e" + k], k)
            if code == abi.SYMM_OK:
                assert torch.equal(t[:-1], again[k]), k


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("n,E,k,m", [(40, 2, 64, 40), (300, 1, 1 << 17, 256), (64, 8, 7168, 512),
                                     (20000, 2, 1024, 2048)])
def test_product(heap, n, E, k, m, fmt):
    (xc, xs, x), (wc, ws, w), c = operands(n, E, k, m, fmt, "even")
    c = c.cuda()
    y = torch.full((n + 1, m), POISON, dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    for calls in (1, 2):
        with ShortBudget(heap):
            for _ in range(calls):
                abi.moe_fp4_expert_matmul(
                    heap.handle, ptr(xc), xc.stride(0), ptr(xs), xs.stride(0), ptr(wc),
                    wc.stride(1), ptr(ws), ws.stride(1), ptr(c), None, None, FMTS[fmt],
                    CODES["bf16"], n, E, k, m, ptr(y), m)
            code = read(heap)
        assert (y[n] == POISON).all()
        again = product(heap, xc, xs, wc, ws, c, None, None, fmt, "bf16", k, m)
        for e, a, b in ref.runs(c):
            want, mag = x[a:b] @ w[e].t(), x[a:b].abs() @ w[e].abs().t()
            bound = U_OUT["bf16"] * want.abs() + (k + 8) * 2.0 ** -23 * mag + TINY["bf16"]
            near(again[a:b], want, bound * (1 + 2.0 ** -8), e)
        if code == abi.SYMM_OK:
            assert torch.equal(y[:n], again)
