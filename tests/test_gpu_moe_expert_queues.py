"""Many of the experts' calls queued on one stream with nothing that waits in between, as a loop
over layers queues them: packing beside products and feed-forwards that are short, long, of one
tile and of more tiles than there are SMs.  (When each kernel let the next one start before it had
waited itself, a queue of eight packings and products never ended.)"""
import pytest
import torch

import expert_refs as ref
from moe_refs import CODES
from symmetric_memory_moe_gb300 import abi
from symmetric_memory_moe_gb300.torch_heap import TorchSymmHeap
from test_gpu_moe_expert import ACTS, ptr
from test_gpu_moe_fp4 import FMTS

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def heap():
    h = TorchSymmHeap(1, 0)
    yield h
    h.close()


def rnd(g, *s):
    return torch.randn(*s, generator=g, device="cuda").to(BF16)


class Chain:
    """act(g) u of gu [n][2k] packed, and its product with the packed weights of E experts."""

    def __init__(self, heap, n, E, k, m, fmt, name, last, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heap, self.dims, self.fmt, self.name = heap, (n, E, k, m), FMTS[fmt], name
        self.gu, w = rnd(g, n, 2 * k), rnd(g, E * m, k)
        lds = -(-k // ref.BLOCK[fmt] // 16) * 16
        byte = dict(dtype=torch.uint8, device="cuda")
        self.xc, self.xs = torch.zeros(n, k // 2, **byte), torch.zeros(n, lds, **byte)
        self.wc, self.ws = torch.zeros(E * m, k // 2, **byte), torch.zeros(E * m, lds, **byte)
        abi.moe_fp4_quantize(ptr(w), k, abi.SYMM_ACT_NONE, CODES["bf16"], self.fmt, None, E * m, k,
                             ptr(self.wc), k // 2, ptr(self.ws), lds)
        counts = [0] * E  # most rows are one expert's, the rest no one's
        counts[last % E] = n - n // 5
        self.counts = torch.tensor(counts, dtype=torch.int32, device="cuda")
        self.y = torch.zeros(n, m, dtype=BF16, device="cuda")

    def call(self):
        (n, E, k, m), lds = self.dims, self.xs.shape[1]
        abi.moe_fp4_quantize(ptr(self.gu), 2 * k, ACTS[self.name], CODES["bf16"], self.fmt, None, n,
                             k, ptr(self.xc), k // 2, ptr(self.xs), lds)
        abi.moe_fp4_expert_matmul(
            self.heap.handle, ptr(self.xc), k // 2, ptr(self.xs), lds, ptr(self.wc), k // 2,
            ptr(self.ws), lds, ptr(self.counts), None, None, self.fmt, CODES["bf16"], n, E, k, m,
            ptr(self.y), m)

    def out(self):
        return [self.y]


class Feed:
    """The feed-forward and its gradients."""

    def __init__(self, heap, n, E, D, F, name, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heap, self.dims, self.name = heap, (n, E, D, F), name
        self.x, self.dy = rnd(g, n, D), rnd(g, n, D)
        self.w1, self.w2 = rnd(g, E, D, 2 * F) * D ** -0.5, rnd(g, E, F, D) * F ** -0.5
        of = torch.randint(E, (n - n // 5,), generator=g, device="cuda")
        self.counts = torch.bincount(of, minlength=E).to(torch.int32)
        self.ws = torch.empty(abi.moe_expert_workspace(n, E, D, F, True), dtype=torch.uint8,
                              device="cuda")
        self.gu = torch.zeros(n, 2 * F, dtype=BF16, device="cuda")
        self.o = [torch.zeros_like(t) for t in (self.x, self.x, self.w1, self.w2)]

    def call(self):
        (n, E, D, F), act, dt = self.dims, ACTS[self.name], CODES["bf16"]
        y, dx, g1, g2 = self.o
        abi.moe_expert_ffn(self.heap.handle, ptr(self.x), D, ptr(self.counts), ptr(self.w1),
                           ptr(self.w2), act, dt, n, E, D, F, ptr(self.gu), ptr(y), D, ptr(self.ws))
        abi.moe_expert_ffn_backward(
            self.heap.handle, ptr(self.dy), D, ptr(self.x), D, ptr(self.gu), ptr(self.counts),
            ptr(self.w1), ptr(self.w2), act, dt, n, E, D, F, ptr(dx), D, ptr(g1), ptr(g2),
            ptr(self.ws))

    def out(self):
        return [self.gu] + self.o


def queue(heap, jobs, rounds):
    """Each job's outputs alone, then of `rounds` turns of all of them in one queue."""
    want = []
    for j in jobs:
        j.call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in j.out()])
    for j in jobs:
        for t in j.out():
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(rounds):
        for j in jobs:
            j.call()
    torch.cuda.synchronize()
    assert abi.symm_check_error(heap.handle)[0] == abi.SYMM_OK
    for j, w in zip(jobs, want):
        for got, t in zip(j.out(), w):
            assert torch.equal(got, t), j.dims


@pytest.mark.parametrize("fmt,name", [("mx", "gelu"), ("nv", "silu"), ("mx", "silu"),
                                      ("nv", "gelu")])
@pytest.mark.parametrize("n,E,k,m", [(31382, 2, 736, 16), (31382, 2, 736, 300), (9000, 3, 96, 8),
                                     (20000, 1, 32, 600), (500, 4, 1056, 1000), (3, 2, 64, 40)])
def test_packing_and_products(heap, n, E, k, m, fmt, name):
    jobs = [Chain(heap, n, E, k, m, fmt, name, i, i) for i in range(3)]
    for rounds in (1, 2, 3, 100):
        queue(heap, jobs, rounds)


@pytest.mark.parametrize("n,E,D,F", [(32, 32, 1024, 512), (3, 8, 64, 32), (1531, 5, 1000, 328),
                                     (20000, 4, 64, 64)])
def test_feed_forwards(heap, n, E, D, F):
    jobs = [Feed(heap, n, E, D, F, "silu", i) for i in range(3)]
    for rounds in (1, 3, 100):
        queue(heap, jobs, rounds)


def test_all_in_turn(heap):
    jobs = [Chain(heap, 31382, 2, 736, 16, "mx", "gelu", 0, 0),
            Feed(heap, 32, 32, 1024, 512, "silu", 1),
            Chain(heap, 64, 8, 2048, 1024, "nv", "silu", 1, 2),
            Feed(heap, 1531, 5, 1000, 328, "gelu", 3),
            Chain(heap, 9000, 3, 96, 8, "nv", "gelu", 2, 4),
            Feed(heap, 20000, 4, 64, 64, "silu", 5)]
    for rounds in (1, 3, 100):
        queue(heap, jobs, rounds)
