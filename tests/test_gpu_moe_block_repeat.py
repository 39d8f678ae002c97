"""backward of the MoE block example called again after one forward pass: it reads what forward
left and changes none of it, so other gradients can follow and the same ones come out the same."""
import pytest
import torch

from symmetric_memory_moe_gb300 import abi
from symmetric_memory_moe_gb300.moe_block import MoeBlock
from test_gpu_moe_block_experts import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("F", [None, 40])
def test_backward_twice(F):
    W, T, D, E, k = 4, 24, 64, 8, 2
    b = MoeBlock(W, T, D, E, k, R=3, r=16, seed=W, F=F)
    g, x, mask, ids, gate = inputs(W, T, D)
    b.forward(x, mask, ids, gate)
    back = b._rows(b.back, b.back_rows).clone()

    def grads():
        return [torch.randn(W, T, D, generator=g).bfloat16().cuda() for _ in range(2)] + \
            [torch.rand(W, 2, generator=g).cuda()]

    first, other = grads(), grads()
    want = {n: t.clone() for n, t in b.backward(*first).items()}
    n = b.o["counts"].sum(1).tolist()  # the rows that came back, then the shared ones
    for w in range(W):
        now = b._rows(b.back, b.back_rows)[w]
        assert torch.equal(now[:n[w]], back[w, :n[w]]) and torch.equal(now[T * k:], back[w, T * k:])
    b.backward(*other)
    again = b.backward(*first)
    assert abi.symm_check_error(b.heap.handle)[0] == abi.SYMM_OK
    assert want.keys() == again.keys() and ("dw_gu" in want) == (F is not None)
    for name in want:
        assert torch.equal(again[name], want[name]), name
    b.close()
