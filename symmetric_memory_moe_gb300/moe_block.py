"""One mixture-of-experts block on the emulated PEs, with the library's operators.

  python -m symmetric_memory_moe_gb300.moe_block --W 8 --tokens 512 --D 1024

Per PE: the norm before the block; the router, whose per-expert counts are the
row counts of the AllToAll that takes every (token, choice) row to its expert's
PE and back; the experts; beside them the shared projection with one low-rank
adapter per request, written straight behind the returned rows; and one pass
from all those rows to the residual stream and the next block's input.
``backward`` returns the gradients from there to the rows, the router's logits
and the residual stream.  PyTorch supplies what the library has no operator for
(the router's and experts' own products, sorting rows by expert).
"""
from __future__ import annotations

import argparse
import json

import torch

from . import abi
from .torch_heap import TorchSymmHeap

BF16 = torch.bfloat16


def _p(t):
    return None if t is None else t.data_ptr()


def _plain(t, dtype, *shape):
    """t as the library takes it: dense rows of the type, on the GPU."""
    if t.dtype != dtype or tuple(t.shape) != shape or not t.is_cuda:
        raise ValueError(f"expected a CUDA tensor of {dtype}, {shape}, got {t.dtype}, "
                         f"{tuple(t.shape)} on {t.device}")
    return t.contiguous()


class MoeBlock:
    """W PEs of T tokens, width D, E experts (E / W per PE), k choices, R adapters of rank r."""

    def __init__(self, W, T, D, E, k, R=4, r=16, seed=0, eps=1e-6):
        assert E % W == 0 and D % 8 == 0
        self.W, self.T, self.D, self.E, self.k, self.R, self.r, self.eps = W, T, D, E, k, R, r, eps
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rnd(*s, scale=1.0):
            return torch.randn(*s, generator=g, device="cuda") * scale

        self.router = rnd(D, E, scale=D ** -0.5)
        self.experts = rnd(E, D, D, scale=D ** -0.5).to(BF16)
        self.shared = rnd(D, D, scale=D ** -0.5).to(BF16)
        self.a, self.b = rnd(R, D, r, scale=D ** -0.5).to(BF16), rnd(R, r, D, scale=r ** -0.5).to(BF16)
        self.scale = torch.rand(R, generator=g, device="cuda")
        self.w_in, self.w_post, self.w_next, self.res = (1 + rnd(D, scale=0.1) for _ in range(4))
        n = T * k                                     # rows a PE sends, at most
        self.back_rows = n + T                        # what returns, then the shared rows
        row, cap = 2 * D, W * n                       # a PE may receive every row there is
        self.heap = TorchSymmHeap(W, (n + 2 * cap + self.back_rows) * row + (4 << 20))
        self.send, self.recv, self.sent, self.back, self.signals = (
            self.heap.malloc(x) for x in (n * row, cap * row, cap * row, self.back_rows * row, 64))
        self.cap = cap
        f32, i32 = dict(device="cuda"), dict(device="cuda", dtype=torch.int32)
        self.o = dict(experts=torch.empty(W, T, k, **i32), weights=torch.empty(W, T, k, **f32),
                      counts=torch.empty(W, E, **i32), tokens=torch.empty(W, **i32),
                      stats=torch.empty(W, T, 2, **f32), loss=torch.empty(W, 2, **f32))
        size = max(abi.moe_route_workspace(W, T, E), abi.moe_block_norm_workspace(T, D),
                   abi.moe_adapter_workspace(T, D, D, r), abi.shmem_collective_workspace(W))
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def _rows(self, ptr, n):
        """[W, n, D] view of the symmetric object at ptr."""
        return self.heap.views(ptr, n * 2 * self.D).view(BF16).view(self.W, n, self.D)

    def forward(self, x, mask, ids, gate):
        """x [W, T, D] bf16, mask [W, T] uint8 (0: padding), ids [W, T] int32 adapters
        (-1: none), gate [W, T]: (residual stream, next input), [W, T, D] each."""
        W, T, D, E, k, o = self.W, self.T, self.D, self.E, self.k, self.o
        x = _plain(x, BF16, W, T, D)
        mask = _plain(mask.byte() if mask.dtype == torch.bool else mask, torch.uint8, W, T)
        ids, gate = _plain(ids, torch.int32, W, T), _plain(gate, torch.float32, W, T)
        self.x, self.gate = x, gate
        h = torch.empty_like(x)
        for w in range(W):
            abi.moe_block_norm(_p(x[w]), D, None, 0, None, 0, None, None, None, None, _p(self.w_in),
                               self.eps, abi.SYMM_DTYPE_BF16, T, D, 0, None, _p(h[w]), None)
        self.h = h
        self.logits = (h.float() @ self.router).contiguous()
        abi.moe_route(_p(self.logits), E, _p(mask), abi.SYMM_DTYPE_F32, W, T, E, k, 1, 1.0,
                      *[_p(o[n]) for n in ("experts", "weights", "counts", "tokens", "stats",
                                           "loss")], _p(self.ws))
        # rows in the order of their experts, and so of their PEs; rows without one last
        e = o["experts"].view(W, T * k).long()
        order = torch.argsort(torch.where(e < 0, E, e), dim=1, stable=True)
        place = torch.empty_like(order).scatter_(1, order, torch.arange(T * k, device=x.device)
                                                 .expand(W, -1).contiguous())
        self._rows(self.send, T * k).copy_(
            torch.gather(h, 1, (order // k)[..., None].expand(-1, -1, D)))
        pairs = o["counts"].view(W, W, E // W).sum(-1).long().contiguous()  # [from][to]
        abi.shmem_alltoall(self.heap.handle, self.send, self.recv, _p(pairs), W, 2 * D, T * k,
                           self.cap, _p(self.ws), self.signals)
        self._experts(o["counts"].long())
        returned = pairs.t().contiguous()
        abi.shmem_alltoall(self.heap.handle, self.sent, self.back, _p(returned), W, 2 * D, self.cap,
                           self.back_rows, _p(self.ws), self.signals)
        # the shared projection of every token, behind the rows that came back
        back = self._rows(self.back, self.back_rows)
        for w in range(W):
            abi.moe_adapter_matmul(self.heap.handle, _p(h[w]), D, _p(self.shared), D, _p(self.a),
                                   _p(self.b), _p(self.scale), _p(ids[w]), abi.SYMM_DTYPE_BF16, T,
                                   D, D, self.R, self.r, _p(back[w, T * k:]), D, _p(self.ws))
        mine = torch.arange(T, device=x.device).expand(W, T) + T * k
        self.rows = torch.cat([torch.where(o["experts"] < 0, -1, place.view(W, T, k)),
                               mine[..., None]], -1).to(torch.int32).contiguous()
        self.weights = torch.cat([o["weights"], torch.ones_like(o["weights"][..., :1])], -1)
        self.weights = self.weights.contiguous()
        self.xo, nxt = torch.empty_like(x), torch.empty_like(x)
        self.rstd = torch.empty(W, T, 2, device=x.device)
        for w in range(W):
            abi.moe_block_norm(_p(x[w]), D, _p(back[w]), D, _p(self.rows[w]), self.back_rows,
                               _p(self.weights[w]), _p(gate[w]), _p(self.res), _p(self.w_post),
                               _p(self.w_next), self.eps, abi.SYMM_DTYPE_BF16, T, D, k + 1,
                               _p(self.xo[w]), _p(nxt[w]), _p(self.rstd[w]))
        return self.xo, nxt

    def _experts(self, counts):
        """Each PE's received rows (by sender, then expert) times their experts."""
        per = self.E // self.W
        recv, sent = self._rows(self.recv, self.cap), self._rows(self.sent, self.cap)
        for d in range(self.W):
            mine = counts[:, d * per:(d + 1) * per]
            n = int(mine.sum())
            of = torch.repeat_interleave(torch.arange(per, device=counts.device).repeat(self.W),
                                         mine.reshape(-1))
            for e in range(per):
                at = (of == e).nonzero().flatten()
                sent[d, :n][at] = recv[d, :n][at] @ self.experts[d * per + e]

    def backward(self, dxo, dnext, dloss):
        """Gradients of what ``forward`` left: dx (through the residual stream), drows (of the
        rows that came back and the shared rows), dlogits, and the vectors' gradients."""
        W, T, D, E, k, o = self.W, self.T, self.D, self.E, self.k, self.o
        dxo, dnext = _plain(dxo, BF16, W, T, D), _plain(dnext, BF16, W, T, D)
        dloss = _plain(dloss, torch.float32, W, 2)
        back = self._rows(self.back, self.back_rows)
        dx, drows = torch.empty_like(dxo), torch.zeros_like(back)
        dweights, dgate = torch.empty_like(self.weights), torch.empty_like(self.gate)
        dvec = torch.empty(W, 3, D, device=dx.device)
        for w in range(W):
            abi.moe_block_norm_backward(
                _p(dxo[w]), _p(dnext[w]), _p(self.x[w]), _p(self.xo[w]), D, _p(back[w]), D,
                _p(self.rows[w]), self.back_rows, _p(self.weights[w]), _p(self.gate[w]),
                _p(self.res), _p(self.w_post), _p(self.w_next), _p(self.rstd[w]),
                abi.SYMM_DTYPE_BF16, T, D, k + 1, _p(dx[w]), _p(drows[w]), _p(dweights[w]),
                _p(dgate[w]), *[_p(v) for v in dvec[w]], _p(self.ws))
        dlogits = torch.empty_like(self.logits)
        dchoice = dweights[..., :k].contiguous()
        abi.moe_route_backward(_p(self.logits), E, abi.SYMM_DTYPE_F32, W, T, E, k, 1, 1.0,
                               *[_p(o[n]) for n in ("experts", "counts", "tokens", "stats")],
                               _p(dchoice), _p(dloss), _p(dlogits), E)
        dres, dw_post, dw_next = dvec.sum(0)
        return dict(dx=dx, drows=drows, dweights=dweights, dgate=dgate, dlogits=dlogits, dres=dres,
                    dw_post=dw_post, dw_next=dw_next)

    def close(self):
        torch.cuda.synchronize()
        self.heap.close()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("W", 8), ("tokens", 512), ("D", 1024), ("experts", 32), ("topk", 4)):
        ap.add_argument(f"--{name}", type=int, default=default)
    a = ap.parse_args(argv)
    block = MoeBlock(a.W, a.tokens, a.D, a.experts, a.topk)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.W, a.tokens, a.D, generator=g, device="cuda").to(BF16)
    mask = torch.ones(a.W, a.tokens, dtype=torch.uint8, device="cuda")
    ids = torch.randint(-1, 4, (a.W, a.tokens), generator=g, device="cuda", dtype=torch.int32)
    gate = torch.sigmoid(torch.randn(a.W, a.tokens, generator=g, device="cuda"))
    xo, nxt = block.forward(x, mask, ids, gate)
    d = block.backward(torch.randn_like(xo), torch.randn_like(nxt),
                       torch.full((a.W, 2), 0.01, device="cuda"))
    code, _ = abi.symm_check_error(block.heap.handle)
    print(json.dumps({"balance_loss": round(float(block.o["loss"][:, 0].mean()), 4),
                      "z_loss": round(float(block.o["loss"][:, 1].mean()), 4),
                      "rows_per_expert_max": int(block.o["counts"].sum(0).max()),
                      "grad_norm_logits": round(float(d["dlogits"].norm()), 4), "code": code}))
    block.close()


if __name__ == "__main__":
    main()
