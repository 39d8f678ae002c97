"""The MoE block operators called by several host threads at once, and on several streams."""
import sys
import threading

import pytest
import torch

from symmetric_memory_moe_gb300 import abi

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
