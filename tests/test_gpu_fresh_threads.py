"""Calls that are the first thing a host thread does with CUDA, on tensors that another thread
made: the thread has no current context yet, which encoding a tensor map wants."""
import threading

import pytest
import torch

from moe_refs import CODES
from symmetric_memory_moe_gb300 import abi
from symmetric_memory_moe_gb300.torch_heap import TorchSymmHeap
from test_gpu_moe_adapter import make, ptr
from test_gpu_moe_expert_concurrent import SIZES, Job

pytestmark = pytest.mark.gpu


def in_a_new_thread(call):
    failed = []

    def work():
        try:
            call()
        except Exception as e:
            failed.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not failed, failed
    torch.cuda.synchronize()


@pytest.mark.parametrize("size", SIZES)
def test_experts(size):
    j = Job(1, *size)
    want = j.alone()
    in_a_new_thread(j.call)
    j.check(want)
    j.heap.close()


@pytest.mark.parametrize("T", [1, 70, 600])
def test_adapters(T):
    k, n, r, R = 512, 264, 16, 3
    heap, i, stream = TorchSymmHeap(1, 0), make(T, k, n, R, r, "bf16", 1), torch.cuda.Stream()
    y = torch.zeros(T, n, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(abi.moe_adapter_workspace(T, k, n, r), dtype=torch.uint8, device="cuda")

    def call():
        abi.moe_adapter_matmul(heap.handle, ptr(i["x"]), k, ptr(i["w"]), n, ptr(i["a"]),
                               ptr(i["b"]), ptr(i["scale"]), ptr(i["ids"]), CODES["bf16"], T, k, n,
                               R, r, ptr(y), n, ptr(ws), stream=stream)

    torch.cuda.synchronize()
    call()
    torch.cuda.synchronize()
    want = y.clone()
    y.zero_()
    torch.cuda.synchronize()
    in_a_new_thread(call)
    assert torch.equal(y, want) and want.any()
    assert abi.symm_check_error(heap.handle)[0] == abi.SYMM_OK
    heap.close()


def test_gather_and_product():
    W, m, k, n = 2, 128, 128, 128
    sig = abi.shmem_fused_ag_matmul_workspace(W, m, k, n)
    sizes = (2 * m * k, 2 * k * n, 2 * W * m * n, 2 * W * m * k, sig)
    heap, stream = TorchSymmHeap(W, sum(sizes) + (4 << 20)), torch.cuda.Stream()
    g = torch.Generator().manual_seed(0)
    a, b, c, gather, s = (heap.malloc(x) for x in sizes)
    heap.upload(a, torch.randn(W, m, k, generator=g).bfloat16())
    heap.upload(b, torch.randn(W, k, n, generator=g).bfloat16())

    def call():
        abi.shmem_fused_all_gather_matmul(heap.handle, a, b, c, gather, W, m, k, n,
                                          abi.SYMM_DTYPE_BF16, 128, s, stream=stream)

    torch.cuda.synchronize()
    call()
    torch.cuda.synchronize()
    want = heap.views(c, 2 * W * m * n).clone()
    heap.views(c, 2 * W * m * n).zero_()
    torch.cuda.synchronize()
    in_a_new_thread(call)
    assert torch.equal(heap.views(c, 2 * W * m * n), want) and want.any()
    assert abi.symm_check_error(heap.handle)[0] == abi.SYMM_OK
    heap.close()
