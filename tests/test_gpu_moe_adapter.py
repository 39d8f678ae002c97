"""GPU parity of moe_adapter_matmul against a 64-bit reference.

Products of two 16-bit values are exact in 32 bits.  Each of the k (or r)
additions of a sum errs by at most 2^-23 relatively -- what a truncating adder
can do -- so with M = sum_x |x| |W| + |scale| sum_i (sum_x |x| |A_i|) |B_i| the
32-bit value is within (k + r + 8) 2^-23 M of the exact one (the 8: the scale, the
join of partial sums, the sum of both parts), and the rounding to the output
type adds u_out of the result."""
import pytest
import torch

from moe_refs import CODES, DTYPES, TINY, U_OUT
from symmetric_memory_moe_gb300 import abi
from symmetric_memory_moe_gb300.torch_heap import TorchSymmHeap

pytestmark = pytest.mark.gpu

POISON = 7.0


@pytest.fixture(scope="module")
def heap():
    h = TorchSymmHeap(1, 0)
    yield h
    h.close()


def make(T, k, n, R, r, dt, seed, ids="mixed"):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda").to(DTYPES[dt])

    i = dict(x=rnd(T, k), w=rnd(k, n), a=None, b=None, scale=None, ids=None)
    if R:
        i.update(a=rnd(R, k, r), b=rnd(R, r, n),
                 scale=torch.randn(R, generator=g, device="cuda"))
        of = torch.randint(-1, R, (T,), generator=g, device="cuda")
        if ids == "runs":
            of = torch.sort(of)[0].flip(0)
        if ids == "none":
            of[:] = -1
        if ids == "one":
            of[:] = R - 1
        if ids == "wild":
            of[::3] = R
            of[1::3] = (1 << 31) - 1
            of[2::6] = -(1 << 31)
        i["ids"] = of.to(torch.int32)
    return i


def ptr(t):
    return None if t is None else t.data_ptr()


def spread(t, ld):
    buf = torch.full((t.shape[0], ld), POISON, dtype=t.dtype, device="cuda")
    buf[:, :t.shape[1]] = t
    return buf


def run(heap, i, dt, ldx=None, ldw=None, ldy=None, stream=None):
    T, k = i["x"].shape
    n = i["w"].shape[1]
    R, r = (0, 0) if i["a"] is None else (i["a"].shape[0], i["a"].shape[2])
    x, w = spread(i["x"], ldx or k), spread(i["w"], ldw or n)
    y = torch.full((T, ldy or n), POISON, dtype=x.dtype, device="cuda")
    ws = torch.empty(max(1, abi.moe_adapter_workspace(T, k, n, r)), dtype=torch.uint8,
                     device="cuda")
    ws.fill_(0xFF)  # needs no initialisation
    torch.cuda.synchronize()
    abi.moe_adapter_matmul(heap.handle, ptr(x), ldx or k, ptr(w), ldw or n, ptr(i["a"]),
                           ptr(i["b"]), ptr(i["scale"]), ptr(i["ids"]), CODES[dt], T, k, n, R, r,
                           ptr(y), ldy or n, ws.data_ptr(), stream=stream)
    torch.cuda.synchronize()
    assert abi.symm_check_error(heap.handle)[0] == abi.SYMM_OK
    assert (y[:, n:] == POISON).all()
    return y[:, :n].contiguous()


def check(i, y, dt, tokens=None):
    t = slice(None) if tokens is None else tokens
    x, w = i["x"][t].double(), i["w"].double()
    k, r = x.shape[1], 0
    want, mag = x @ w, x.abs() @ w.abs()
    if i["a"] is not None:
        R, r = i["a"].shape[0], i["a"].shape[2]
        ids = i["ids"][t].long()
        for a in set(ids.tolist()):
            if 0 <= a < R:
                m = ids == a
                A, B, s = i["a"][a].double(), i["b"][a].double(), i["scale"][a].double()
                want[m] += s * (x[m] @ A) @ B
                mag[m] += s.abs() * (x[m].abs() @ A.abs()) @ B.abs()
    tol = U_OUT[dt] * want.abs() + (k + r + 8) * 2.0 ** -23 * mag + TINY[dt]
    y = y[t].double()
    assert torch.isfinite(y).all()
    err = (y - want).abs()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("T,k,n,R,r,dt,ids", [
    (1, 8, 8, 1, 8, "bf16", "one"), (1, 64, 128, 2, 16, "f16", "one"),
    (1, 2048, 1000, 3, 16, "bf16", "one"), (2, 72, 136, 2, 8, "bf16", "mixed"),
    (15, 256, 264, 4, 24, "f16", "mixed"), (16, 1000, 2056, 5, 40, "bf16", "mixed"),
    (17, 520, 512, 17, 64, "f16", "mixed"), (33, 4096, 256, 3, 128, "bf16", "mixed"),
    (64, 1024, 1024, 64, 16, "bf16", "mixed"), (100, 136, 4104, 2, 8, "f16", "wild"),
    (128, 640, 384, 6, 32, "bf16", "none"), (200, 320, 640, 7, 8, "bf16", "runs"),
    (255, 192, 200, 3, 16, "f16", "runs"), (256, 256, 512, 4, 16, "bf16", "runs"),
    (257, 264, 520, 4, 16, "bf16", "mixed"), (600, 1032, 776, 9, 48, "f16", "runs"),
    (1000, 512, 2048, 2, 8, "bf16", "one"), (3000, 128, 1024, 40, 16, "bf16", "runs"),
    (2500, 64, 8, 3, 8, "f16", "mixed"), (77, 2048, 2048, 0, 0, "bf16", "none"),
    (5, 8, 16, 0, 0, "f16", "none"),
])
def test_values(heap, T, k, n, R, r, dt, ids):
    i = make(T, k, n, R, r, dt, T + k + n, ids)
    check(i, run(heap, i, dt), dt)


@pytest.mark.parametrize("T", [1, 40, 300, 2000])
def test_strides_streams_and_equal_bits(heap, T):
    k, n = 200, 328
    i = make(T, k, n, 5, 16, "bf16", T, "mixed")
    y = run(heap, i, "bf16")
    check(i, y, "bf16")
    st = torch.cuda.Stream()
    for ldx, ldw, ldy in ((208, 328, 328), (200, 336, 329), (256, 512, 333), (200, 328, 512)):
        assert torch.equal(run(heap, i, "bf16", ldx, ldw, ldy, stream=st), y)


def test_unused_adapters_may_hold_anything(heap):
    """NaN in adapters that no token names, and in tokens of their own."""
    i = make(50, 256, 300 // 4 * 4 + 4, 6, 16, "bf16", 3, "mixed")
    i["ids"][i["ids"] == 2] = -1
    i["ids"][i["ids"] == 4] = -1
    want = run(heap, i, "bf16")
    i["a"][2] = float("nan")
    i["b"][2] = float("inf")
    i["b"][4] = float("nan")
    i["scale"][4] = float("nan")
    assert torch.equal(run(heap, i, "bf16"), want)
    # a token's NaN stays in its own row
    i["x"][7] = float("nan")
    y = run(heap, i, "bf16")
    assert torch.isnan(y[7]).all()
    rest = torch.arange(50, device="cuda") != 7
    assert torch.equal(y[rest], want[rest])


@pytest.mark.parametrize("T,r,dt", [(50, 16, "bf16"), (50, 72, "f16"), (700, 32, "bf16")])
def test_a_request_with_a_broken_adapter_harms_no_other(heap, T, r, dt):
    """An infinity or NaN in one adapter stays with the tokens that use it."""
    i = make(T, 200, 520, 6, r, dt, 5, "mixed")
    want = run(heap, i, dt)
    for name, where, value in (("b", (2, r - 1, 519), float("inf")), ("b", (0, 0, 0), float("nan")),
                               ("b", (5, 3, 77), -float("inf")), ("a", (1, 199, 0), float("nan")),
                               ("a", (3, 0, r - 1), float("inf"))):
        j = dict(i, **{name: i[name].clone()})
        j[name][where] = value
        y = run(heap, j, dt)
        own = i["ids"] == where[0]
        assert own.any() and not own.all()
        assert torch.equal(y[~own], want[~own]), (name, where)
        assert not torch.isfinite(y[own]).all(1).any()
        if name == "b":  # the column that it enters, and at most its block of 128
            assert torch.isnan(y[own][:, where[2]]).all()
            far = torch.arange(520, device="cuda") // 128 != where[2] // 128
            assert torch.equal(y[own][:, far], want[own][:, far])


@pytest.mark.parametrize("T,k,n,R,r", [(1, 8192, 8192, 4, 16), (64, 7168, 2048, 32, 16),
                                       (8192, 4096, 4096, 8, 32)])
def test_large_sampled(heap, T, k, n, R, r):
    i = make(T, k, n, R, r, "bf16", 1, "runs")
    y = run(heap, i, "bf16")
    tokens = torch.unique(torch.linspace(0, T - 1, 64).long()).cuda()
    check(i, y, "bf16", tokens)


def test_offsets_past_32_bits(heap):
    """Rows of y 2^25 elements apart: 3.4e9 elements."""
    T, k, n, ldy = 100, 64, 128, 1 << 25
    i = make(T, k, n, 3, 8, "bf16", 4, "mixed")
    want = run(heap, i, "bf16")
    y = torch.empty(T, ldy, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(abi.moe_adapter_workspace(T, k, n, 8), dtype=torch.uint8, device="cuda")
    abi.moe_adapter_matmul(heap.handle, ptr(i["x"]), k, ptr(i["w"]), n, ptr(i["a"]), ptr(i["b"]),
                           ptr(i["scale"]), ptr(i["ids"]), 1, T, k, n, 3, 8, ptr(y), ldy,
                           ws.data_ptr())
    assert abi.symm_check_error(heap.handle)[0] == abi.SYMM_OK
    assert torch.equal(y[:, :n], want)


def test_graph_capture(heap):
    T, k, n, R, r = 20, 512, 1024, 4, 16
    i = make(T, k, n, R, r, "bf16", 6, "mixed")
    want = run(heap, i, "bf16")
    y = torch.zeros(T, n, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(abi.moe_adapter_workspace(T, k, n, r), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        abi.moe_adapter_matmul(heap.handle, ptr(i["x"]), k, ptr(i["w"]), n, ptr(i["a"]),
                               ptr(i["b"]), ptr(i["scale"]), ptr(i["ids"]), 1, T, k, n, R, r,
                               ptr(y), n, ws.data_ptr())
    for _ in range(2):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    assert abi.symm_check_error(heap.handle)[0] == abi.SYMM_OK


def test_no_tokens(heap):
    abi.moe_adapter_matmul(heap.handle, None, 8, None, 8, None, None, None, None, 1, 0, 8, 8, 0, 0,
                           None, 8, None)


@pytest.mark.parametrize("T,k,n", [(3, 4096, 4096), (300, 512, 1024)])
def test_inputs_written_just_before_on_the_stream(heap, T, k, n):
    """What an earlier kernel of the stream still writes is read after it: x, W,
    the adapters and the ids arrive by copies that take longer than a launch."""
    a, b = (make(T, k, n, 3, 16, "bf16", s, "mixed") for s in (1, 2))
    want = [run(heap, i, "bf16") for i in (a, b)]
    live = {m: v.clone() for m, v in a.items()}
    y = torch.empty(T, n, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(abi.moe_adapter_workspace(T, k, n, 16), dtype=torch.uint8, device="cuda")
    slow = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    got = []
    for j in range(6):
        slow.add_(1)
        for m in ("ids", "scale", "a", "b", "w", "x"):
            live[m].copy_((a, b)[j % 2][m])
        abi.moe_adapter_matmul(heap.handle, ptr(live["x"]), k, ptr(live["w"]), n, ptr(live["a"]),
                               ptr(live["b"]), ptr(live["scale"]), ptr(live["ids"]), 1, T, k, n, 3,
                               16, ptr(y), n, ws.data_ptr())
        got.append(y.clone())
    torch.cuda.synchronize()
    assert abi.symm_check_error(heap.handle)[0] == abi.SYMM_OK
    for j, g in enumerate(got):
        assert torch.equal(g, want[j % 2]), j
