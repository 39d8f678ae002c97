"""All of the experts' calls on several streams at once, and from several host threads, each with
a stream, a heap and a workspace of its own: the feed-forward, its gradients, packing, unpacking
and the 4-bit product.  Results are those of the same calls one after another."""
import threading

import pytest
import torch

import expert_refs as ref
from moe_refs import CODES
from symmetric_memory_moe_gb300 import abi
from symmetric_memory_moe_gb300.torch_heap import TorchSymmHeap
from test_gpu_moe_expert import ACTS, POISON, make, ptr
from test_gpu_moe_fp4 import FMTS, operands

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
SIZES = [(900, 5, 512, 256, "nv"), (64, 8, 1024, 512, "mx"), (300, 2, 288, 160, "nv"),
         (1500, 3, 320, 192, "mx")]


class Job:
    """Inputs, outputs and workspace of one user; call() enqueues everything on its stream."""

    def __init__(self, seed, n, E, D, F, fmt):
        self.size, self.fmt = (n, E, D, F), fmt
        self.heap, self.stream = TorchSymmHeap(1, 0), torch.cuda.Stream()
        self.i = make(n, E, D, F, "bf16", "even", seed=seed)
        _, (self.wc, self.ws4, _), _ = operands(n, E, D, F, fmt, "even", seed=seed)
        self.ws = torch.empty(abi.moe_expert_workspace(n, E, D, F, True), dtype=torch.uint8,
                              device="cuda")
        new = dict(dtype=BF16, device="cuda")
        byte = dict(dtype=torch.uint8, device="cuda")
        self.o = dict(y=torch.empty(n, D, **new), gu=torch.empty(n, 2 * F, **new),
                      dx=torch.empty(n, D, **new), dw_gu=torch.empty_like(self.i["w_gu"]),
                      dw_d=torch.empty_like(self.i["w_d"]), codes=torch.empty(n, D // 2, **byte),
                      scales=torch.zeros(n, -(-D // ref.BLOCK[fmt] // 16) * 16, **byte),
                      values=torch.empty(n, D, **new), y4=torch.empty(n, F, **new))

    def call(self):
        (n, E, D, F), i, o, s = self.size, self.i, self.o, self.stream
        h, act, dt, fmt = self.heap.handle, ACTS["silu"], CODES["bf16"], FMTS[self.fmt]
        abi.moe_expert_ffn(h, ptr(i["x"]), D, ptr(i["counts"]), ptr(i["w_gu"]), ptr(i["w_d"]), act,
                           dt, n, E, D, F, ptr(o["gu"]), ptr(o["y"]), D, ptr(self.ws), stream=s)
        abi.moe_expert_ffn_backward(
            h, ptr(i["dy"]), D, ptr(i["x"]), D, ptr(o["gu"]), ptr(i["counts"]), ptr(i["w_gu"]),
            ptr(i["w_d"]), act, dt, n, E, D, F, ptr(o["dx"]), D, ptr(o["dw_gu"]), ptr(o["dw_d"]),
            ptr(self.ws), stream=s)
        c, b = o["codes"], o["scales"]
        abi.moe_fp4_quantize(ptr(i["x"]), D, abi.SYMM_ACT_NONE, dt, fmt, None, n, D, ptr(c),
                             c.shape[1], ptr(b), b.shape[1], stream=s)
        abi.moe_fp4_dequantize(ptr(c), c.shape[1], ptr(b), b.shape[1], fmt, None, n, D, dt,
                               ptr(o["values"]), D, stream=s)
        abi.moe_fp4_expert_matmul(
            h, ptr(c), c.shape[1], ptr(b), b.shape[1], ptr(self.wc), self.wc.stride(1),
            ptr(self.ws4), self.ws4.stride(1), ptr(i["counts"]), None, None, fmt, dt, n, E, D, F,
            ptr(o["y4"]), F, stream=s)

    def spoil(self):
        for t in self.o.values():
            t.fill_(POISON)
        torch.cuda.synchronize()

    def alone(self):
        """The outputs of one call with nothing beside it; the outputs are then spoilt."""
        self.spoil()
        self.call()
        torch.cuda.synchronize()
        want = {k: t.clone() for k, t in self.o.items()}
        self.spoil()
        return want

    def check(self, want):
        assert abi.symm_check_error(self.heap.handle, self.stream)[0] == abi.SYMM_OK
        for k, t in self.o.items():
            assert torch.equal(t, want[k]), (self.size, k)


@pytest.fixture
def jobs():
    js = [Job(j, *s) for j, s in enumerate(SIZES)]
    yield js
    torch.cuda.synchronize()
    for j in js:
        j.heap.close()


def test_streams(jobs):
    want = [j.alone() for j in jobs]
    for _ in range(20):
        for j in jobs:
            j.call()
    torch.cuda.synchronize()
    for j, w in zip(jobs, want):
        j.check(w)


def test_host_threads(jobs):
    want, start, bad = [j.alone() for j in jobs], threading.Barrier(len(jobs)), []

    def work(j):
        try:
            start.wait()
            for _ in range(50):
                j.call()
            j.stream.synchronize()
        except Exception as e:  # a thread's own failure does not fail the test
            bad.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad
    for j, w in zip(jobs, want):
        j.check(w)


def test_graphs_at_once(jobs):
    """A captured graph of each job, replayed on streams of their own at once."""
    want, graphs = [j.alone() for j in jobs], []
    for j in jobs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=j.stream):
            j.call()
        graphs.append(g)
    for _ in range(10):
        for j, g in zip(jobs, graphs):
            with torch.cuda.stream(j.stream):
                g.replay()
    torch.cuda.synchronize()
    for j, w in zip(jobs, want):
        j.check(w)
