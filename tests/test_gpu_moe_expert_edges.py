"""Calls of the experts' operators that the documentation allows and that are easily wrong:
counts that are no rows, rows that are not finite, captured and replayed calls, calls on several
streams at once, a single expert without counts, offsets past 32 bits."""
import pytest
import torch

import expert_refs as ref
from moe_refs import TINY, U_OUT
from symmetric_memory_moe_gb300 import abi
from symmetric_memory_moe_gb300.torch_heap import TorchSymmHeap
from test_gpu_moe_expert import POISON, backward, forward, make, near, ptr
from test_gpu_moe_fp4 import operands, product

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def heap():
    h = TorchSymmHeap(1, 0)
    yield h
    h.close()


def error(heap):
    """The recorded error (and the heap is clean again)."""
    return abi.symm_check_error(heap.handle)[0]


@pytest.mark.parametrize("counts", [[3, -1, 4], [5, 5, 7], [2 ** 31 - 1, 2 ** 31 - 1, 2],
                                    [0, 0, 17], [-2 ** 31, 8, 8]])
def test_counts_out_of_range(heap, counts):
    n, E, D, F = 16, 3, 64, 32
    i = make(n, E, D, F, "bf16", "even")
    i["counts"] = torch.tensor(counts, dtype=torch.int32, device="cuda")
    new = dict(dtype=BF16, device="cuda")
    y, gu = torch.full((n, D), POISON, **new), torch.full((n, 2 * F), POISON, **new)
    ws = torch.empty(abi.moe_expert_workspace(n, E, D, F, True), dtype=torch.uint8, device="cuda")
    abi.moe_expert_ffn(heap.handle, ptr(i["x"]), D, ptr(i["counts"]), ptr(i["w_gu"]),
                       ptr(i["w_d"]), 0, 1, n, E, D, F, ptr(gu), ptr(y), D, ptr(ws))
    assert error(heap) == abi.SYMM_ERANGE
    assert (y == POISON).all() and (gu == POISON).all()
    g1, g2 = torch.full_like(i["w_gu"], POISON), torch.full_like(i["w_d"], POISON)
    abi.moe_expert_ffn_backward(heap.handle, ptr(i["dy"]), D, ptr(i["x"]), D, ptr(gu),
                                ptr(i["counts"]), ptr(i["w_gu"]), ptr(i["w_d"]), 0, 1, n, E, D, F,
                                ptr(y), D, ptr(g1), ptr(g2), ptr(ws))
    assert error(heap) == abi.SYMM_ERANGE
    assert (y == POISON).all() and (g1 == POISON).all() and (g2 == POISON).all()
    (xc, xs, _), (wc, wsc, _), _ = operands(n, E, 64, 40, "nv", "even")
    y = torch.full((n, 40), POISON, **new)
    abi.moe_fp4_expert_matmul(heap.handle, ptr(xc), 32, ptr(xs), 16, ptr(wc), 32, ptr(wsc), 16,
                              ptr(i["counts"]), None, None, 1, 1, n, E, 64, 40, ptr(y), 40)
    assert error(heap) == abi.SYMM_ERANGE and (y == POISON).all()
    # and the heap's next call is as ever
    i = make(n, E, D, F, "bf16", "even")
    r = ref.ffn(i["x"], i["counts"], i["w_gu"], i["w_d"], "silu", U_OUT["bf16"], TINY["bf16"])
    near(forward(heap, i, "bf16", "silu")[0], r["y"], r["ey"], "y")


def test_no_rows_at_all(heap):
    i = make(40, 4, 64, 32, "bf16", "even")
    i["counts"].zero_()
    y, gu = forward(heap, i, "bf16", "silu")
    assert (y == POISON).all() and (gu == POISON).all()
    o = backward(heap, i, gu, "bf16", "silu")
    assert (o["dx"] == POISON).all() and not o["dw_gu"].any() and not o["dw_d"].any()


@pytest.mark.parametrize("n,kind", [(70, "even"), (600, "holes")])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_not_finite(heap, n, kind, bad):
    """A row that is not finite spoils itself and its own expert's weight gradients alone."""
    E, D, F = 3, 136, 72
    clean = make(n, E, D, F, "bf16", kind)
    e = int(clean["counts"].argmax())
    row = int(clean["counts"][:e].sum()) + 5
    i = {k: v.clone() for k, v in clean.items()}
    i["x"][row, 7] = bad
    i["dy"][row, 9] = bad
    y0, gu0 = forward(heap, clean, "bf16", "silu")
    y, gu = forward(heap, i, "bf16", "silu")
    rest = torch.arange(n, device="cuda") != row
    assert torch.equal(y[rest], y0[rest]) and torch.equal(gu[rest], gu0[rest])
    assert not torch.isfinite(gu[row]).all() and not torch.isfinite(y[row]).all()
    o0 = backward(heap, clean, gu0, "bf16", "silu")
    o = backward(heap, i, gu0, "bf16", "silu")
    assert torch.equal(o["dx"][rest], o0["dx"][rest]) and not torch.isfinite(o["dx"][row]).any()
    others = [x for x in range(E) if x != e]
    for k in ("dw_gu", "dw_d"):
        assert torch.equal(o[k][others], o0[k][others])
        assert not torch.isfinite(o[k][e]).all()


@pytest.mark.parametrize("fmt,nan", [("nv", 0x7f), ("mx", 0xff)])
def test_packed_not_finite(heap, fmt, nan):
    (xc, xs, _), (wc, ws, _), c = operands(300, 3, 288, 200, fmt, "even")
    c = c.cuda()
    y0 = product(heap, xc, xs, wc, ws, c, None, None, fmt, "bf16", 288, 200)
    xs[11, 2] = nan
    y = product(heap, xc, xs, wc, ws, c, None, None, fmt, "bf16", 288, 200)
    rest = torch.arange(300, device="cuda") != 11
    assert torch.equal(y[rest], y0[rest]) and torch.isnan(y[11]).all()
    ws[1, 150, 0] = nan
    y = product(heap, xc, xs, wc, ws, c, None, None, fmt, "bf16", 288, 200)
    a, b = int(c[0]), int(c[0] + c[1])
    rest[a:b] = False
    assert torch.equal(y[rest], y0[rest]) and torch.isnan(y[a:b, 150]).all()
    assert torch.equal(y[a:b, :150], y0[a:b, :150]) or a <= 11 < b


@pytest.mark.parametrize("n", [1, 50, 700])
def test_one_expert_without_counts(heap, n):
    i = make(n, 1, 200, 72, "bf16", "one")
    y, gu = forward(heap, i, "bf16", "gelu")
    y2, gu2 = forward(heap, i, "bf16", "gelu", counts=False)
    assert torch.equal(y, y2) and torch.equal(gu, gu2)
    o = backward(heap, i, gu, "bf16", "gelu")
    o2 = backward(heap, i, gu, "bf16", "gelu", counts=False)
    assert all(torch.equal(o[k], o2[k]) for k in o)
    (xc, xs, _), (wc, ws, _), c = operands(n, 1, 96, 72, "nv", "one")
    args = (None, None, "nv", "bf16", 96, 72)
    assert torch.equal(product(heap, xc, xs, wc, ws, c.cuda(), *args),
                       product(heap, xc, xs, wc, ws, None, *args))


def test_graph_replays_with_other_counts(heap):
    """Captured calls read the counts when they run; forward, backward and the 4-bit chain."""
    n, E, D, F = 400, 4, 256, 96
    i = make(n, E, D, F, "bf16", "even")
    (xc, xs, x4), (wc, ws4, w4), _ = operands(n, E, 256, 136, "nv", "even")
    new = dict(dtype=BF16, device="cuda")
    y, dx, gu = torch.zeros(n, D, **new), torch.zeros(n, D, **new), torch.zeros(n, 2 * F, **new)
    y4 = torch.zeros(n, 136, **new)
    g1, g2 = torch.empty_like(i["w_gu"]), torch.empty_like(i["w_d"])
    ws = torch.empty(abi.moe_expert_workspace(n, E, D, F, True), dtype=torch.uint8, device="cuda")
    p = {k: ptr(v) for k, v in i.items()}

    def calls(stream):
        abi.moe_expert_ffn(heap.handle, p["x"], D, p["counts"], p["w_gu"], p["w_d"], 0, 1, n, E, D,
                           F, ptr(gu), ptr(y), D, ptr(ws), stream=stream)
        abi.moe_expert_ffn_backward(heap.handle, p["dy"], D, p["x"], D, ptr(gu), p["counts"],
                                    p["w_gu"], p["w_d"], 0, 1, n, E, D, F, ptr(dx), D, ptr(g1),
                                    ptr(g2), ptr(ws), stream=stream)
        abi.moe_fp4_expert_matmul(heap.handle, ptr(xc), 128, ptr(xs), 16, ptr(wc), 128, ptr(ws4),
                                  16, p["counts"], None, None, 1, 1, n, E, 256, 136, ptr(y4), 136,
                                  stream=stream)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        calls(s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        calls(s)
    for counts in ([100] * 4, [0, 399, 1, 0], [17, 300, 3, 40], [0, 0, 0, 0], [1, 1, 1, 1]):
        i["counts"].copy_(torch.tensor(counts, dtype=torch.int32))
        for t in (y, dx, gu, y4):
            t.fill_(POISON)
        graph.replay()
        torch.cuda.synchronize()
        assert abi.symm_check_error(heap.handle)[0] == abi.SYMM_OK
        total = sum(counts)
        r = ref.ffn(i["x"], i["counts"], i["w_gu"], i["w_d"], "silu", U_OUT["bf16"], TINY["bf16"])
        near(y[:total], r["y"], r["ey"], "y")
        o = ref.ffn_grad(i["dy"], i["x"], gu, i["counts"], i["w_gu"], i["w_d"], "silu",
                         U_OUT["bf16"], TINY["bf16"])
        near(dx[:total], o["dx"], o["edx"], "dx")
        near(g1, o["dw_gu"], o["edw_gu"], "dw_gu")
        near(g2, o["dw_d"], o["edw_d"], "dw_d")
        for e, a, b in ref.runs(i["counts"]):
            want = x4[a:b] @ w4[e].t()
            mag = x4[a:b].abs() @ w4[e].abs().t()
            near(y4[a:b], want, 2.0 ** -8 * want.abs() + 264 * 2.0 ** -23 * mag + 1e-38, "fp4")
        for t in (y, dx, gu, y4):
            assert (t[total:] == POISON).all()


def test_streams_at_once(heap):
    """Calls on four streams at once, each with a workspace of its own; results as alone."""
    jobs = []
    for j, (n, E, D, F) in enumerate([(900, 5, 512, 256), (64, 8, 1024, 512), (300, 2, 264, 136),
                                      (1500, 3, 320, 192)]):
        i = make(n, E, D, F, "bf16", "even", seed=j)
        y, gu = forward(heap, i, "bf16", "silu")
        o = backward(heap, i, gu, "bf16", "silu")
        ws = torch.empty(abi.moe_expert_workspace(n, E, D, F, True), dtype=torch.uint8,
                         device="cuda")
        out = [torch.empty_like(t.contiguous()) for t in (y, gu, o["dx"], o["dw_gu"], o["dw_d"])]
        jobs.append((i, (n, E, D, F), ws, out, [y, gu, o["dx"], o["dw_gu"], o["dw_d"]],
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for i, (n, E, D, F), ws, (y, gu, dx, g1, g2), _, s in jobs:
            abi.moe_expert_ffn(heap.handle, ptr(i["x"]), D, ptr(i["counts"]), ptr(i["w_gu"]),
                               ptr(i["w_d"]), 0, 1, n, E, D, F, ptr(gu), ptr(y), D, ptr(ws),
                               stream=s)
            abi.moe_expert_ffn_backward(heap.handle, ptr(i["dy"]), D, ptr(i["x"]), D, ptr(gu),
                                        ptr(i["counts"]), ptr(i["w_gu"]), ptr(i["w_d"]), 0, 1, n,
                                        E, D, F, ptr(dx), D, ptr(g1), ptr(g2), ptr(ws), stream=s)
    torch.cuda.synchronize()
    assert abi.symm_check_error(heap.handle)[0] == abi.SYMM_OK
    for _, _, _, out, want, _ in jobs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_offsets_past_32_bits(heap):
    """Rows and outputs beyond 2^32 elements from their first."""
    n, ld, E, D, F = 1 << 20, 4104, 2, 64, 32
    i = make(300, E, D, F, "bf16", "one")
    x = torch.zeros(n, ld, dtype=BF16, device="cuda")
    y = torch.zeros(n, ld, dtype=BF16, device="cuda")
    x[n - 300:, :D] = i["x"]
    counts = torch.tensor([n - 300, 300], dtype=torch.int32, device="cuda")
    ws = torch.empty(abi.moe_expert_workspace(n, E, D, F), dtype=torch.uint8, device="cuda")
    abi.moe_expert_ffn(heap.handle, ptr(x), ld, ptr(counts), ptr(i["w_gu"]), ptr(i["w_d"]), 0, 1, n,
                       E, D, F, None, ptr(y), ld, ptr(ws))
    torch.cuda.synchronize()
    assert abi.symm_check_error(heap.handle)[0] == abi.SYMM_OK
    alone, _ = forward(heap, i, "bf16", "silu")
    assert torch.equal(y[n - 300:, :D], alone)
    assert not y[:n - 300, :D].any() and not y[:, D:].any()
    # codes of so many rows: the last ones' as of those alone
    c = torch.empty(n, 32, dtype=torch.uint8, device="cuda")
    s = torch.empty(n, 16, dtype=torch.uint8, device="cuda")
    abi.moe_fp4_quantize(ptr(x), ld, -1, 1, 1, None, n, D, ptr(c), 32, ptr(s), 16)
    c2, s2 = torch.empty_like(c[:300]), torch.empty_like(s[:300])
    abi.moe_fp4_quantize(ptr(i["x"]), D, -1, 1, 1, None, 300, D, ptr(c2), 32, ptr(s2), 16)
    v = torch.empty(n, ld, dtype=BF16, device="cuda")
    abi.moe_fp4_dequantize(ptr(c), 32, ptr(s), 16, 1, None, n, D, 1, ptr(v), ld)
    torch.cuda.synchronize()
    assert torch.equal(c[n - 300:], c2) and torch.equal(s[n - 300:, :4], s2[:, :4])
    code, scale = ref.quantize(i["x"], "nv", None)
    assert torch.equal(v[n - 300:, :D].double(), ref.values(code, scale, "nv", None))


def test_gradients_are_differences(heap):
    """Each gradient against central differences of the forward pass in 64 bits, along random
    directions: the formula's own check, with the kernel's bf16 rounding (2^-8 of each term)."""
    n, E, D, F = 60, 2, 64, 48
    i = make(n, E, D, F, "bf16", "even")
    _, gu = forward(heap, i, "bf16", "silu")
    o = backward(heap, i, gu, "bf16", "silu")
    g = torch.Generator(device="cuda").manual_seed(3)

    def loss(x, w_gu, w_d):
        total = 0.0
        for e, a, b in ref.runs(i["counts"]):
            h = x[a:b] @ w_gu[e]
            y = (ref.act("silu", h[:, :F])[0] * h[:, F:]) @ w_d[e]
            total = total + (y * i["dy"][a:b].double()).sum()
        return total

    base = [i[k].double() for k in ("x", "w_gu", "w_d")]
    for j, k in enumerate(("dx", "dw_gu", "dw_d")):
        v = torch.randn(base[j].shape, generator=g, device="cuda", dtype=torch.float64)
        step = 1e-4
        ends = [loss(*[t + s * step * v if m == j else t for m, t in enumerate(base)])
                for s in (1, -1)]
        want = (ends[0] - ends[1]) / (2 * step)
        terms = o[k].double() * v
        # independent roundings of gu, h, dg, du and the gradient: 2^-8 of a term each at most,
        # 8 standard deviations of their sum; differences err by step^2
        assert (terms.sum() - want).abs() <= 8 * 5 * 2.0 ** -8 * terms.norm() + 1e-3


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("name,dt", [(None, "f16"), ("silu", "bf16"), (None, "f32")])
def test_rows_of_a_wider_matrix(fmt, name, dt):
    """x with rows further apart than they are long, what lies between never read."""
    from test_gpu_moe_fp4 import CODES, FMTS, pack
    k = 96
    width = k if name is None else 2 * k
    g = torch.Generator(device="cuda").manual_seed(k)
    wide = torch.full((70, width + 40), float("nan"), device="cuda")
    wide[:, :width] = torch.randn(70, width, generator=g, device="cuda")
    wide = wide.to({"f16": torch.float16, "bf16": BF16, "f32": torch.float32}[dt])
    alone, scales = pack(wide[:, :width].contiguous(), fmt, None, name)
    c, s = torch.zeros_like(alone), torch.zeros_like(scales)
    abi.moe_fp4_quantize(ptr(wide), width + 40, -1 if name is None else 0, CODES[dt], FMTS[fmt],
                         None, 70, k, ptr(c), c.shape[1], ptr(s), s.shape[1])
    torch.cuda.synchronize()
    b = k // ref.BLOCK[fmt]
    assert torch.equal(c[:, :k // 2], alone[:, :k // 2]) and torch.equal(s[:, :b], scales[:, :b])


def test_host_threads_at_once():
    """Four host threads with a stream, a heap and a workspace each."""
    from concurrent.futures import ThreadPoolExecutor

    def job(j):
        n, E, D, F = 200 + 90 * j, 1 + j, 128 + 64 * j, 72
        h = TorchSymmHeap(1, 0)
        i = make(n, E, D, F, "bf16", "even", seed=j)
        y, gu = forward(h, i, "bf16", "silu", stream=torch.cuda.Stream())
        o = [backward(h, i, gu, "bf16", "silu") for _ in range(3)]
        h.close()
        return i, y, o

    with ThreadPoolExecutor(4) as ex:
        done = list(ex.map(job, range(4)))
    for i, y, o in done:
        r = ref.ffn(i["x"], i["counts"], i["w_gu"], i["w_d"], "silu", U_OUT["bf16"], TINY["bf16"])
        near(y, r["y"], r["ey"], "y")
        assert all(torch.equal(o[0][k], x[k]) for x in o[1:] for k in x)


def test_most_experts(heap):
    """As many experts as there may be, one row each and none."""
    i = make(512, 1024, 64, 32, "bf16", "even")
    i["counts"] = (torch.arange(1024) % 2 == 1).to(torch.int32).cuda()
    y, gu = forward(heap, i, "bf16", "silu")
    r = ref.ffn(i["x"], i["counts"], i["w_gu"], i["w_d"], "silu", U_OUT["bf16"], TINY["bf16"])
    near(y, r["y"], r["ey"], "y")
    o = backward(heap, i, gu, "bf16", "silu")
    g = ref.ffn_grad(i["dy"], i["x"], gu, i["counts"], i["w_gu"], i["w_d"], "silu", U_OUT["bf16"],
                     TINY["bf16"])
    for k in ("dx", "dw_gu", "dw_d"):
        near(o[k], g[k], g["e" + k], k)
