"""The MoE block example with inputs that are not laid out, or not typed, as the library's."""
import pytest
import torch

from symmetric_memory_moe_gb300.moe_block import MoeBlock

pytestmark = pytest.mark.gpu


def test_strided_inputs_and_wrong_ones():
    W, T, D = 2, 20, 64
    b = MoeBlock(W, T, D, 4, 2, R=3, r=16)
    g = torch.Generator().manual_seed(1)
    x, dxo, dn = (torch.randn(W, T, D, generator=g).bfloat16().cuda() for _ in range(3))
    mask = (torch.rand(W, T, generator=g) < 0.8).to(torch.uint8).cuda()
    ids = torch.randint(-1, 3, (W, T), generator=g, dtype=torch.int32).cuda()
    gate, dl = torch.rand(W, T, generator=g).cuda(), torch.rand(W, 2, generator=g).cuda()

    def strided(t):  # the same values, dimensions in another order in memory
        return t.transpose(0, -1).contiguous().transpose(0, -1)

    want = [*b.forward(x, mask, ids, gate), *b.backward(dxo, dn, dl).values()]
    got = [*b.forward(*map(strided, (x, mask, ids, gate))),
           *b.backward(*map(strided, (dxo, dn, dl))).values()]
    for w, v in zip(want, got):
        assert torch.equal(w, v)
    for w, v in zip(want, b.forward(x, mask.bool(), ids, gate)):
        assert torch.equal(w, v)
    for bad in ((x.float(), mask, ids, gate), (x, mask.long(), ids, gate),
                (x, mask, ids.long(), gate), (x, mask, ids, gate.double()),
                (x[:1], mask, ids, gate), (x.cpu(), mask, ids, gate)):
        with pytest.raises(ValueError):
            b.forward(*bad)
    with pytest.raises(ValueError):
        b.backward(dxo, dn, dl.double())
    b.close()
