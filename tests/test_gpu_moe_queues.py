"""The block's operators in turn in one queue with nothing that waits in between: norm, router,
projection with adapters, packing, products and feed-forwards, forward and backward."""
import pytest
import torch

from moe_refs import CODES
from symmetric_memory_moe_gb300 import abi
from symmetric_memory_moe_gb300.torch_heap import TorchSymmHeap
from test_gpu_moe_expert import ptr
from test_gpu_moe_expert_queues import BF16, Chain, Feed, queue, rnd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def heap():
    h = TorchSymmHeap(1, 0)
    yield h
    h.close()


class Norm:
    """The norm after a block and before the next, of one row a token, and its gradients."""

    def __init__(self, T, D, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dims = T, D
        self.x, self.y, self.dxo, self.dh = (rnd(g, T, D) for _ in range(4))
        self.w = [torch.rand(D, generator=g, device="cuda") + 0.5 for _ in range(3)]
        self.rows = torch.arange(T, dtype=torch.int32, device="cuda")[:, None].contiguous()
        self.weights = torch.rand(T, 1, generator=g, device="cuda")
        f32 = dict(device="cuda")
        self.o = [torch.zeros_like(self.x) for _ in range(4)] + [
            torch.zeros(T, 2, **f32), torch.zeros(T, 1, **f32), torch.zeros(3, D, **f32)]
        self.ws = torch.empty(abi.moe_block_norm_workspace(T, D), dtype=torch.uint8, device="cuda")

    def call(self):
        (T, D), dt = self.dims, CODES["bf16"]
        xo, h, dx, dy, rstd, dweights, dvec = self.o
        res, post, pre = (ptr(w) for w in self.w)
        abi.moe_block_norm(ptr(self.x), D, ptr(self.y), D, ptr(self.rows), T, ptr(self.weights),
                           None, res, post, pre, 1e-6, dt, T, D, 1, ptr(xo), ptr(h), ptr(rstd))
        abi.moe_block_norm_backward(
            ptr(self.dxo), ptr(self.dh), ptr(self.x), ptr(xo), D, ptr(self.y), D, ptr(self.rows), T,
            ptr(self.weights), None, res, post, pre, ptr(rstd), dt, T, D, 1, ptr(dx), ptr(dy),
            ptr(dweights), None, *[ptr(v) for v in dvec], ptr(self.ws))

    def out(self):
        return self.o


class Route:
    def __init__(self, G, T, E, k, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dims = G, T, E, k
        self.logits = torch.randn(G, T, E, generator=g, device="cuda")
        self.dweights = torch.randn(G, T, k, generator=g, device="cuda")
        self.dloss = torch.rand(G, 2, generator=g, device="cuda")
        f32, i32 = dict(device="cuda"), dict(device="cuda", dtype=torch.int32)
        self.o = [torch.zeros(G, T, k, **i32), torch.zeros(G, T, k, **f32),
                  torch.zeros(G, E, **i32), torch.zeros(G, **i32), torch.zeros(G, T, 2, **f32),
                  torch.zeros(G, 2, **f32), torch.zeros_like(self.logits)]
        self.ws = torch.empty(abi.moe_route_workspace(G, T, E), dtype=torch.uint8, device="cuda")

    def call(self):
        G, T, E, k = self.dims
        p = [ptr(t) for t in self.o]
        abi.moe_route(ptr(self.logits), E, None, abi.SYMM_DTYPE_F32, G, T, E, k, 1, 1.0, *p[:6],
                      ptr(self.ws))
        abi.moe_route_backward(ptr(self.logits), E, abi.SYMM_DTYPE_F32, G, T, E, k, 1, 1.0, p[0],
                               p[2], p[3], p[4], ptr(self.dweights), ptr(self.dloss), p[6], E)

    def out(self):
        return self.o


class Adapters:
    def __init__(self, heap, T, k, n, R, r, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heap, self.dims = heap, (T, k, n, R, r)
        self.x, self.w = rnd(g, T, k), rnd(g, k, n)
        self.a, self.b = rnd(g, R, k, r), rnd(g, R, r, n)
        self.scale = torch.rand(R, generator=g, device="cuda")
        self.ids = torch.randint(-1, R, (T,), generator=g, device="cuda", dtype=torch.int32)
        self.y = torch.zeros(T, n, dtype=BF16, device="cuda")
        self.ws = torch.empty(abi.moe_adapter_workspace(T, k, n, r), dtype=torch.uint8,
                              device="cuda")

    def call(self):
        T, k, n, R, r = self.dims
        abi.moe_adapter_matmul(self.heap.handle, ptr(self.x), k, ptr(self.w), n, ptr(self.a),
                               ptr(self.b), ptr(self.scale), ptr(self.ids), CODES["bf16"], T, k, n,
                               R, r, ptr(self.y), n, ptr(self.ws))

    def out(self):
        return [self.y]


@pytest.mark.parametrize("T", [8, 600, 9000])
def test_in_turn(heap, T):
    packs = [Chain(heap, T + i, 2, 736, 16, "mx", "gelu", i, i) for i in range(2)]
    small, wide = Feed(heap, T, 8, 256, 128, "silu", 2), Feed(heap, 70, 2, 1000, 328, "gelu", 3)
    norm, route = Norm(T, 1024, 4), Route(2, T, 64, 4, 5)
    shared = Adapters(heap, T, 512, 512, 3, 16, 6)
    for rounds in (1, 3, 60):
        queue(heap, [norm, route, shared, packs[0], small, norm, packs[1], shared, packs[0], wide,
                     route, packs[1], norm, shared], rounds)
        queue(heap, [packs[0], norm, packs[1], norm], rounds)
        queue(heap, [packs[0], shared, packs[1], shared], rounds)
        queue(heap, [small, norm, small, route, small, packs[0]], rounds)
