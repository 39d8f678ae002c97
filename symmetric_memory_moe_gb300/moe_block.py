"""One mixture-of-experts block on the emulated PEs, with the library's operators.

  python -m symmetric_memory_moe_gb300.moe_block --W 8 --tokens 512 --D 1024

Per PE: the norm before the block; the router, whose per-expert counts are the
row counts of the AllToAll that takes every (token, choice) row to its expert's
PE and back; the experts; beside them the shared projection with one low-rank
adapter per request, written straight behind the returned rows; and one pass
from all those rows to the residual stream and the next block's input.
``backward`` returns the gradients from there to the rows, the router's logits
and the residual stream.  The experts are a matrix each (by PyTorch), or, given
the feed-forward's width F, gated feed-forwards with their gradients, or given
``fp4`` as well, served from 4-bit weights and rows:

  python -m symmetric_memory_moe_gb300.moe_block --F 512 [--fp4 nv]

PyTorch supplies what the library has no operator for (the router's product,
sorting rows by expert).
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
    """W PEs of T tokens, width D, E experts (E / W per PE), k choices, R adapters of rank r;
    F: width of the experts' gated feed-forward (None: a D x D matrix each); fp4: "mx" or "nv",
    experts in 4 bits (no gradients)."""

    def __init__(self, W, T, D, E, k, R=4, r=16, seed=0, eps=1e-6, F=None, fp4=None):
        assert E % W == 0 and D % 8 == 0 and (F is None or F % 8 == 0)
        assert fp4 is None or (F is not None and D % 32 == 0 and F % 32 == 0)
        self.W, self.T, self.D, self.E, self.k, self.R, self.r, self.eps = W, T, D, E, k, R, r, eps
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rnd(*s, scale=1.0):
            return torch.randn(*s, generator=g, device="cuda") * scale

        self.router = rnd(D, E, scale=D ** -0.5)
        self.F, self.fp4 = F, fp4
        if F is None:
            self.experts = rnd(E, D, D, scale=D ** -0.5).to(BF16)
        else:
            self.w_gu = rnd(E, D, 2 * F, scale=D ** -0.5).to(BF16)
            self.w_d = rnd(E, F, D, scale=F ** -0.5).to(BF16)
        self.shared = rnd(D, D, scale=D ** -0.5).to(BF16)
        self.a, self.b = rnd(R, D, r, scale=D ** -0.5).to(BF16), rnd(R, r, D, scale=r ** -0.5).to(BF16)
        self.scale = torch.rand(R, generator=g, device="cuda")
        self.w_in, self.w_post, self.w_next, self.res = (1 + rnd(D, scale=0.1) for _ in range(4))
        n = T * k                                     # rows a PE sends, at most
        self.back_rows = n + T                        # what returns, then the shared rows
        row, cap = 2 * D, W * n                       # a PE may receive every row there is
        grads = n if F is not None and not fp4 else 0  # the experts' gradients on their way back
        self.heap = TorchSymmHeap(W, (n + 2 * cap + self.back_rows + grads) * row + (4 << 20))
        self.send, self.recv, self.sent, self.back, self.signals = (
            self.heap.malloc(x) for x in (n * row, cap * row, cap * row, self.back_rows * row, 64))
        self.grads = self.heap.malloc(grads * row) if grads else None
        self.cap = cap
        f32, i32 = dict(device="cuda"), dict(device="cuda", dtype=torch.int32)
        self.o = dict(experts=torch.empty(W, T, k, **i32), weights=torch.empty(W, T, k, **f32),
                      counts=torch.empty(W, E, **i32), tokens=torch.empty(W, **i32),
                      stats=torch.empty(W, T, 2, **f32), loss=torch.empty(W, 2, **f32))
        size = max(abi.moe_route_workspace(W, T, E), abi.moe_block_norm_workspace(T, D),
                   abi.moe_adapter_workspace(T, D, D, r), abi.shmem_collective_workspace(W))
        if F is not None:
            size = max(size, abi.moe_expert_workspace(cap, E // W, D, F, True))
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        if fp4:  # the weights transposed: blocks lie along what is summed over
            self.q_gu = self._pack_weights(self.w_gu)
            self.q_d = self._pack_weights(self.w_d)

    def _pack(self, x, k, act, gscale=None):
        """Codes and scales of the rows of x: k values each, or act of 2k."""
        n, block = x.shape[0], 32 if self.fp4 == "mx" else 16
        fmt = abi.SYMM_FP4_MX if self.fp4 == "mx" else abi.SYMM_FP4_NV
        codes = torch.empty(n, k // 2, dtype=torch.uint8, device=x.device)
        scales = torch.empty(n, -(-k // block // 16) * 16, dtype=torch.uint8, device=x.device)
        abi.moe_fp4_quantize(_p(x), x.shape[1], act, abi.SYMM_DTYPE_BF16, fmt, _p(gscale), n, k,
                             _p(codes), codes.shape[1], _p(scales), scales.shape[1])
        return codes, scales

    def _pack_weights(self, w):
        """(codes, scales, each expert's own scale) of w [E][k][m], as rows [E * m][k]."""
        E, k, m = w.shape
        g = None
        if self.fp4 == "nv":
            g = torch.exp2(torch.ceil(torch.log2(w.float().abs().amax((1, 2)) / 2688)))
        packed = [self._pack(w[e].t().contiguous(), k, abi.SYMM_ACT_NONE,
                             None if g is None else g[e:e + 1]) for e in range(E)]
        codes, scales = (torch.stack(p) for p in zip(*packed))
        return codes, scales, torch.ones(E, device=w.device) if g is None else g

    def _project(self, packed, weights, first, counts, m):
        """Packed rows, grouped by expert, times the packed weights of experts first .. ."""
        (xc, xs), (wc, ws, g) = packed, weights
        fmt = abi.SYMM_FP4_MX if self.fp4 == "mx" else abi.SYMM_FP4_NV
        n, E, k = xc.shape[0], counts.shape[0], 2 * xc.shape[1]
        y = torch.empty(n, m, dtype=BF16, device=xc.device)
        abi.moe_fp4_expert_matmul(self.heap.handle, _p(xc), xc.shape[1], _p(xs), xs.shape[1],
                                  _p(wc[first]), wc.shape[2], _p(ws[first]), ws.shape[2],
                                  _p(counts), None, _p(g[first:]), fmt, abi.SYMM_DTYPE_BF16, n, E,
                                  k, m, _p(y), m)
        return y

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
        self.pairs = pairs
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
        """Each PE's received rows (by sender, then expert) through their experts."""
        per = self.E // self.W
        recv, sent = self._rows(self.recv, self.cap), self._rows(self.sent, self.cap)
        self.kept = []
        for d in range(self.W):
            mine = counts[:, d * per:(d + 1) * per]
            n = int(mine.sum())
            of = torch.repeat_interleave(torch.arange(per, device=counts.device).repeat(self.W),
                                         mine.reshape(-1))
            if self.F is not None:
                order = torch.argsort(of, stable=True)
                rows = mine.sum(0).to(torch.int32)
                sent[d, :n][order] = self._feed_forward(d, recv[d, :n][order], rows, order)
                continue
            for e in range(per):
                at = (of == e).nonzero().flatten()
                sent[d, :n][at] = recv[d, :n][at] @ self.experts[d * per + e]

    def _feed_forward(self, d, x, rows, order):
        """PE d's rows x, grouped by expert (`rows` of each), through their feed-forwards."""
        n, D, F, per = x.shape[0], self.D, self.F, self.E // self.W
        if self.fp4:
            gu = self._project(self._pack(x, D, abi.SYMM_ACT_NONE), self.q_gu, d * per, rows, 2 * F)
            return self._project(self._pack(gu, F, abi.SYMM_ACT_SILU), self.q_d, d * per, rows, D)
        gu = torch.empty(n, 2 * F, dtype=BF16, device=x.device)
        y = torch.empty_like(x)
        abi.moe_expert_ffn(self.heap.handle, _p(x), D, _p(rows), _p(self.w_gu[d * per]),
                           _p(self.w_d[d * per]), abi.SYMM_ACT_SILU, abi.SYMM_DTYPE_BF16, n, per, D,
                           F, _p(gu), _p(y), D, _p(self.ws))
        self.kept.append((x, gu, rows, order))
        return y

    def _experts_backward(self, drows):
        """Gradients of the feed-forwards' inputs, [W, T, D] summed over a token's choices, and
        of their weights, from those of the rows that came back."""
        W, T, D, F, k, per = self.W, self.T, self.D, self.F, self.k, self.E // self.W
        pairs = self.pairs
        self._rows(self.send, T * k).copy_(drows[:, :T * k])
        abi.shmem_alltoall(self.heap.handle, self.send, self.recv, _p(pairs), W, 2 * D, T * k,
                           self.cap, _p(self.ws), self.signals)
        recv, sent = self._rows(self.recv, self.cap), self._rows(self.sent, self.cap)
        dw_gu, dw_d = torch.empty_like(self.w_gu), torch.empty_like(self.w_d)
        for d, (x, gu, rows, order) in enumerate(self.kept):
            n = x.shape[0]
            dy, dx = recv[d, :n][order], torch.empty_like(x)
            abi.moe_expert_ffn_backward(
                self.heap.handle, _p(dy), D, _p(x), D, _p(gu), _p(rows), _p(self.w_gu[d * per]),
                _p(self.w_d[d * per]), abi.SYMM_ACT_SILU, abi.SYMM_DTYPE_BF16, n, per, D, F, _p(dx),
                D, _p(dw_gu[d * per]), _p(dw_d[d * per]), _p(self.ws))
            sent[d, :n][order] = dx
        returned = pairs.t().contiguous()
        # beside the rows that came back, which a second backward pass reads again
        abi.shmem_alltoall(self.heap.handle, self.sent, self.grads, _p(returned), W, 2 * D,
                           self.cap, T * k, _p(self.ws), self.signals)
        # row `rows` of what came back is that choice's; an absent choice's row was not sent
        at, back = self.rows[..., :k].long(), self._rows(self.grads, T * k).float()
        picked = torch.gather(back, 1, at.clamp(min=0).view(W, T * k, 1).expand(-1, -1, D))
        picked = torch.where((at >= 0).view(W, T * k, 1), picked, 0.0)
        return picked.view(W, T, k, D).sum(2), dw_gu, dw_d

    def backward(self, dxo, dnext, dloss):
        """Gradients of what ``forward`` left: dx (through the residual stream), drows (of the
        rows that came back and the shared rows), dlogits, and the vectors' gradients.  With
        feed-forward experts also theirs: dh_experts (of the norm's output, [W, T, D] in 32
        bits), dw_gu, dw_d.  What ``forward`` left stays: further calls may follow."""
        if self.fp4:
            raise ValueError("experts in 4 bits have no gradients")
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
        more = {}
        if self.F is not None:
            more = dict(zip(("dh_experts", "dw_gu", "dw_d"), self._experts_backward(drows)))
        return dict(more, dx=dx, drows=drows, dweights=dweights, dgate=dgate, dlogits=dlogits, dres=dres,
                    dw_post=dw_post, dw_next=dw_next)

    def close(self):
        torch.cuda.synchronize()
        self.heap.close()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("W", 8), ("tokens", 512), ("D", 1024), ("experts", 32), ("topk", 4)):
        ap.add_argument(f"--{name}", type=int, default=default)
    ap.add_argument("--F", type=int, help="gated feed-forward experts of this width")
    ap.add_argument("--fp4", choices=("mx", "nv"), help="those experts in 4 bits, forward only")
    a = ap.parse_args(argv)
    block = MoeBlock(a.W, a.tokens, a.D, a.experts, a.topk, F=a.F, fp4=a.fp4)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.W, a.tokens, a.D, generator=g, device="cuda").to(BF16)
    mask = torch.ones(a.W, a.tokens, dtype=torch.uint8, device="cuda")
    ids = torch.randint(-1, 4, (a.W, a.tokens), generator=g, device="cuda", dtype=torch.int32)
    gate = torch.sigmoid(torch.randn(a.W, a.tokens, generator=g, device="cuda"))
    xo, nxt = block.forward(x, mask, ids, gate)
    out = {"balance_loss": round(float(block.o["loss"][:, 0].mean()), 4),
           "z_loss": round(float(block.o["loss"][:, 1].mean()), 4),
           "rows_per_expert_max": int(block.o["counts"].sum(0).max())}
    if not a.fp4:
        d = block.backward(torch.randn_like(xo), torch.randn_like(nxt),
                           torch.full((a.W, 2), 0.01, device="cuda"))
        out["grad_norm_logits"] = round(float(d["dlogits"].norm()), 4)
    if a.F and not a.fp4:
        out["grad_norm_experts"] = round(float(d["dw_gu"].float().norm()), 4)
    out["code"], _ = abi.symm_check_error(block.heap.handle)
    print(json.dumps(out))
    block.close()


if __name__ == "__main__":
    main()
