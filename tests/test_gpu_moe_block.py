"""The MoE block example: the operators together, against a dense 64-bit block.

The reference takes the block's own logits (the choice of experts follows
them exactly) and recomputes everything else in 64 bits.  Along the way to
xo and the next input a value is rounded to bf16 in h, in the expert's or the
shared row, and in the output, and the expert's product of bf16 values by the
library of PyTorch once more: four roundings of 2^-9 relatively at most, to which
the norms add no gain beyond 2 -- within 4 * 2 * 2^-9 = 2^-6 of the outputs' 2-norm."""
import pytest
import torch

import moe_refs as ref
from symmetric_memory_moe_gb300 import abi
from symmetric_memory_moe_gb300.moe_block import MoeBlock

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("W,T,D,E,k", [(4, 24, 64, 8, 2), (2, 61, 136, 6, 3), (3, 1, 64, 3, 1)])
def test_block(W, T, D, E, k):
    b = MoeBlock(W, T, D, E, k, R=3, r=16, seed=W)
    g = torch.Generator().manual_seed(T)
    x = torch.randn(W, T, D, generator=g).bfloat16().cuda()
    mask = (torch.rand(W, T, generator=g) < 0.8).to(torch.uint8).cuda()
    ids = torch.randint(-1, 3, (W, T), generator=g, dtype=torch.int32).cuda()
    gate = torch.rand(W, T, generator=g).cuda()
    xo, nxt = b.forward(x, mask, ids, gate)
    assert abi.symm_check_error(b.heap.handle)[0] == abi.SYMM_OK
    r = ref.route(b.logits, mask, k, 1, 1.0)
    assert torch.equal(b.o["experts"], r["experts"]) and torch.equal(b.o["counts"], r["counts"])

    xd = x.double()
    h = xd / torch.sqrt((xd * xd).mean(-1, keepdim=True) + b.eps) * b.w_in.double()
    every = torch.einsum("wtd,edf->wtef", h, b.experts.double())
    e = r["experts"].clamp(min=0).long()
    rows = torch.gather(every, 2, e[..., None].expand(-1, -1, -1, D))
    y = (r["weights"][..., None] * rows).sum(2) + h @ b.shared.double()
    for a in range(3):
        t = ids == a
        y[t] += b.scale[a].double() * (h[t] @ b.a[a].double()) @ b.b[a].double()
    u = y / torch.sqrt((y * y).mean(-1, keepdim=True) + b.eps) * b.w_post.double()
    want = b.res.double() * xd + gate.double()[..., None] * u
    wnext = want / torch.sqrt((want * want).mean(-1, keepdim=True) + b.eps) * b.w_next.double()
    for got, w in ((xo, want), (nxt, wnext)):
        assert (got.double() - w).norm() <= 2.0 ** -6 * w.norm()

    dxo, dn = (torch.randn(W, T, D, generator=g).bfloat16().cuda() for _ in range(2))
    dl = torch.rand(W, 2, generator=g).cuda()
    d = b.backward(dxo, dn, dl)
    back = b._rows(b.back, b.back_rows)
    for w in range(W):  # each stage's gradient, from the inputs it had
        i = dict(x=x[w], y=back[w], rows=b.rows[w], weights=b.weights[w], gate=gate[w], res=b.res,
                 w_post=b.w_post, w_pre=b.w_next, k=k + 1)
        o = ref.norm_grad(i, b.xo[w], b.rstd[w], dxo[w], dn[w])
        for n, m in (("dx", "dx"), ("dweights", "dweights"), ("dgate", "dgate")):
            err = 400 * ref.U32 * o[m + "_mag"] + (2.0 ** -8 * o[m].abs() if n == "dx" else 0)
            assert ((d[n][w].double() - o[m]).abs() <= err + 1e-37).all(), n
        named = ~torch.isnan(o["dy"][:, 0])
        assert ((d["drows"][w].double() - o["dy"])[named].abs() <=
                (400 * ref.U32 * o["dy_mag"] + 2.0 ** -8 * o["dy"].abs())[named] + 1e-37).all()
        assert not d["drows"][w][~named].any()
    dz, mag = ref.route_grad(b.logits.double(), r["experts"], r["counts"], r["tokens"], r["valid"],
                             k, 1, 1.0, d["dweights"][..., :k], dl)
    assert ((d["dlogits"].double() - dz).abs() <=
            2 * 220 * ref.U32 * mag + 2.0 ** -23 * dz.abs() + 1e-37).all()
    b.close()
