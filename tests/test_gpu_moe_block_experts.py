"""The MoE block example with feed-forward experts: router, AllToAll, experts and the way back,
forward and backward, against a dense 64-bit block; and with experts in 4 bits.

Forward, as in test_gpu_moe_block.py: to the outputs a value is rounded to bf16 in h, in the
feed-forward's product act(g) u and in its row, and in the output, four roundings of 2^-9 relatively
at most, to which the experts and norms add no gain beyond 2: within 4 * 2 * 2^-9 = 2^-6 of the
outputs' 2-norm.  Backward: the experts' gradients are taken from the stage's own inputs and carry
the bounds of tests/expert_refs.py."""
import pytest
import torch

import expert_refs as refs
import moe_refs as ref
from symmetric_memory_moe_gb300 import abi
from symmetric_memory_moe_gb300.moe_block import MoeBlock, main

pytestmark = pytest.mark.gpu


def inputs(W, T, D, masked=0.2):
    g = torch.Generator().manual_seed(T)
    x = torch.randn(W, T, D, generator=g).bfloat16().cuda()
    mask = (torch.rand(W, T, generator=g) >= masked).to(torch.uint8).cuda()
    ids = torch.randint(-1, 3, (W, T), generator=g, dtype=torch.int32).cuda()
    return g, x, mask, ids, torch.rand(W, T, generator=g).cuda()


def dense(b, x, r, ids, experts):
    """The block in 64 bits; experts(h, e): the rows h [.., D] through expert e."""
    xd = x.double()
    h = xd / torch.sqrt((xd * xd).mean(-1, keepdim=True) + b.eps) * b.w_in.double()
    y = h @ b.shared.double()
    for a in range(3):
        t = ids == a
        y[t] += b.scale[a].double() * (h[t] @ b.a[a].double()) @ b.b[a].double()
    for e in range(b.E):
        w = torch.where(r["experts"] == e, r["weights"], 0.0).sum(-1)
        y += w[..., None] * experts(h, e)
    return h, y


@pytest.mark.parametrize("W,T,D,E,k,F", [(4, 24, 64, 8, 2, 40), (2, 61, 136, 6, 3, 72),
                                         (3, 1, 64, 3, 1, 64), (2, 300, 256, 4, 2, 192)])
def test_feed_forward(W, T, D, E, k, F):
    b = MoeBlock(W, T, D, E, k, R=3, r=16, seed=W, F=F)
    g, x, mask, ids, gate = inputs(W, T, D)
    xo, nxt = b.forward(x, mask, ids, gate)
    assert abi.symm_check_error(b.heap.handle)[0] == abi.SYMM_OK
    r = ref.route(b.logits, mask, k, 1, 1.0)
    assert torch.equal(b.o["experts"], r["experts"])

    def expert(h, e):
        gu = h @ b.w_gu[e].double()
        return (refs.act("silu", gu[..., :F])[0] * gu[..., F:]) @ b.w_d[e].double()

    _, y = dense(b, x, r, ids, expert)
    u = y / torch.sqrt((y * y).mean(-1, keepdim=True) + b.eps) * b.w_post.double()
    want = b.res.double() * x.double() + gate.double()[..., None] * u
    wnext = want / torch.sqrt((want * want).mean(-1, keepdim=True) + b.eps) * b.w_next.double()
    for got, w in ((xo, want), (nxt, wnext)):
        assert (got.double() - w).norm() <= 2.0 ** -6 * w.norm()

    dxo, dn = (torch.randn(W, T, D, generator=g).bfloat16().cuda() for _ in range(2))
    d = b.backward(dxo, dn, torch.rand(W, 2, generator=g).cuda())
    assert abi.symm_check_error(b.heap.handle)[0] == abi.SYMM_OK
    # each expert's rows (token by token, PE by PE as they arrive) and their gradients
    dh, edh = torch.zeros(2, W, T, D, dtype=torch.float64, device="cuda")
    per = E // W
    for e in range(E):
        at = (r["experts"] == e).nonzero()  # PE, token, choice: in the order of arrival
        rows = b.rows[at[:, 0], at[:, 1], at[:, 2]].long()
        dy, xe = d["drows"][at[:, 0], rows], b.h[at[:, 0], at[:, 1]]
        _, gu, counts, _ = b.kept[e // per]
        start = int(counts[:e % per].sum())
        gu = gu[start:start + len(at)]
        c = torch.tensor([len(at)])
        o = refs.ffn_grad(dy, xe, gu, c, b.w_gu[e:e + 1], b.w_d[e:e + 1], "silu", 2.0 ** -8, 1e-38)
        for n in ("dw_gu", "dw_d"):
            assert ((d[n][e].double() - o[n][0]).abs() <= o["e" + n][0]).all(), n
        for i, (p, t, _) in enumerate(at.tolist()):
            dh[p, t] += o["dx"][i]
            edh[p, t] += o["edx"][i] + 2.0 ** -23 * k * o["dx"][i].abs()
    assert ((d["dh_experts"].double() - dh).abs() <= edh).all()
    b.close()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("W,T,D,E,k,F", [(2, 33, 64, 4, 2, 96), (1, 260, 288, 2, 1, 160)])
def test_fp4(W, T, D, E, k, F, fmt):
    """The 4-bit experts' rows against the same steps in 64 bits: quantised rows, their product
    rounded to bf16, the gated product quantised, its product.  What may differ is a bf16
    rounding on the way (2^-8 of an element) and a code beside a border that it moves: within
    2^-5 of the rows' 2-norm."""
    b = MoeBlock(W, T, D, E, k, R=3, r=16, seed=W, F=F, fp4=fmt)
    _, x, mask, ids, gate = inputs(W, T, D, masked=0)
    xo, _ = b.forward(x, mask, ids, gate)
    assert abi.symm_check_error(b.heap.handle)[0] == abi.SYMM_OK and torch.isfinite(xo).all()

    def weights(q, e):
        wc, ws, g = q
        kk = 2 * wc.shape[2]
        v = refs.values(refs.unpack(wc[e]), ws[e][:, :kk // refs.BLOCK[fmt]], fmt, None)
        return v * g[e].double()

    def rows(v):
        return refs.values(*refs.quantize(v, fmt, None), fmt, None)

    experts = b.o["experts"]
    back = b._rows(b.back, b.back_rows)
    for e in range(E):
        at = (experts == e).nonzero()
        got = back[at[:, 0], b.rows[at[:, 0], at[:, 1], at[:, 2]].long()].double()
        gu = (rows(b.h[at[:, 0], at[:, 1]]) @ weights(b.q_gu, e).t()).bfloat16().double()
        h = refs.act("silu", gu[:, :F])[0] * gu[:, F:]
        want = rows(h.float()) @ weights(b.q_d, e).t()
        assert (got - want).norm() <= 2.0 ** -5 * want.norm()
    with pytest.raises(ValueError):
        b.backward(x, x, torch.zeros(W, 2, device="cuda"))
    b.close()


@pytest.mark.parametrize("more", [["--F", "64"], ["--F", "64", "--fp4", "mx"],
                                  ["--F", "64", "--fp4", "nv"]])
def test_command(more, capsys):
    main(["--W", "2", "--tokens", "32", "--D", "64", "--experts", "4", "--topk", "2"] + more)
    assert '"code": 0' in capsys.readouterr().out
