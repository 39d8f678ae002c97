"""The MoE block operators called by several host threads at once, and on several streams."""
import sys
import threading

import pytest
import torch

from symmetric_memory_moe_gb300 import abi
from symmetric_memory_moe_gb300.torch_heap import TorchSymmHeap
from test_gpu_moe_adapter import make, run

pytestmark = pytest.mark.gpu


def call_norm_backward(stream, D, k, keep):
    """The bound C call of a norm's backward pass of one token with k rows (0: none)."""
    t = dict(x=torch.ones(1, D, device="cuda", dtype=torch.bfloat16),
             y=torch.ones(max(k, 1), D, device="cuda", dtype=torch.bfloat16),
             w=torch.ones(D, device="cuda"), rstd=torch.ones(1, 2, device="cuda"),
             dx=torch.zeros(1, D, device="cuda", dtype=torch.bfloat16),
             dy=torch.zeros(max(k, 1), D, device="cuda", dtype=torch.bfloat16),
             ws=torch.zeros(abi.moe_block_norm_workspace(1, D), device="cuda", dtype=torch.uint8))
    keep.append(t)
    p = {n: v.data_ptr() for n, v in t.items()}
    y, dy, xo = (p["y"], p["dy"], p["x"]) if k else (None, None, None)
    args = (None, p["x"], p["x"], xo, D, y, D, None, k, None, None, None, None, p["w"], p["rstd"],
            abi.SYMM_DTYPE_BF16, 1, D, k, p["dx"], dy, None, None, None, None, None, p["ws"],
            stream.cuda_stream)
    fn = abi.lib().moe_block_norm_backward
    return lambda: fn(*args)


def call_norm(stream, D, keep):
    t = dict(x=torch.ones(1, D, device="cuda"), h=torch.zeros(1, D, device="cuda"),
             w=torch.ones(D, device="cuda"))
    keep.append(t)
    args = (t["x"].data_ptr(), D, None, 0, None, 0, None, None, None, None, t["w"].data_ptr(), 1e-6,
            abi.SYMM_DTYPE_F32, 1, D, 0, None, t["h"].data_ptr(), None, stream.cuda_stream)
    fn = abi.lib().moe_block_norm
    return lambda: fn(*args)


@pytest.mark.parametrize("what", ["backward", "forward"])
def test_norms_of_different_sizes_from_two_threads(what):
    """Calls that share a kernel but not its size of shared memory (172 against 57 KB, and
    112 against 42): none is refused, whatever the other thread does in between."""
    streams, keep, bad = [torch.cuda.Stream() for _ in range(4)], [], []
    if what == "backward":
        calls = [call_norm_backward(s, 7168, k, keep) for s, k in zip(streams, (8, 0, 8, 0))]
    else:
        calls = [call_norm(s, D, keep) for s, D in zip(streams, (4096, 1536, 4096, 1536))]
    torch.cuda.synchronize()
    start = threading.Barrier(len(calls))

    def work(call):
        start.wait()
        for _ in range(20000):
            rc = call()
            if rc or bad:
                bad.append((rc, abi.symm_last_error()))
                return

    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-5)
    try:
        threads = [threading.Thread(target=work, args=(c,)) for c in calls]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    torch.cuda.synchronize()
    assert not bad, bad[0]


def test_adapter_calls_in_flight_on_three_streams():
    """Each call's second launch holds tensor memory that another call's first one may be
    waiting for; all of them end, with the bits that each has alone."""
    heap = TorchSymmHeap(1, 0)
    cases = [(3000, 512, 1024, 6, 16, "bf16"), (64, 4096, 2048, 32, 16, "bf16"),
             (700, 264, 520, 5, 72, "f16")]
    inputs = [make(T, k, n, R, r, dt, T, "mixed") for T, k, n, R, r, dt in cases]
    want = [run(heap, i, c[-1]) for i, c in zip(inputs, cases)]
    streams = [torch.cuda.Stream() for _ in cases]
    out = [torch.empty_like(w) for w in want]
    ws = [torch.empty(abi.moe_adapter_workspace(c[0], c[1], c[2], c[4]), dtype=torch.uint8,
                      device="cuda") for c in cases]
    codes = {"f16": abi.SYMM_DTYPE_F16, "bf16": abi.SYMM_DTYPE_BF16}
    torch.cuda.synchronize()
    for _ in range(40):
        for (T, k, n, R, r, dt), i, y, w, s in zip(cases, inputs, out, ws, streams):
            abi.moe_adapter_matmul(heap.handle, i["x"].data_ptr(), k, i["w"].data_ptr(), n,
                                   i["a"].data_ptr(), i["b"].data_ptr(), i["scale"].data_ptr(),
                                   i["ids"].data_ptr(), codes[dt], T, k, n, R, r, y.data_ptr(), n,
                                   w.data_ptr(), stream=s)
    torch.cuda.synchronize()
    assert abi.symm_check_error(heap.handle)[0] == abi.SYMM_OK
    for y, w in zip(out, want):
        assert torch.equal(y, w)
    heap.close()
