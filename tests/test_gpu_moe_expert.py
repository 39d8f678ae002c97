"""GPU parity of moe_expert_ffn and its gradients against a 64-bit reference.

Products of two 16-bit values are exact in 32 bits.  Each of the k additions of
a sum errs by at most 2^-23 relatively -- what a truncating adder can do -- so a
sum is within (k + 8) 2^-23 of the sum of its terms' magnitudes; values rounded
to the type on the way (h, dg, du) are off by u_out, half a step, and carry that
into the next sum (tests/expert_refs.py)."""
import pytest
import torch

import expert_refs as ref
from moe_refs import CODES, DTYPES, TINY, U_OUT
from symmetric_memory_moe_gb300 import abi
from symmetric_memory_moe_gb300.torch_heap import TorchSymmHeap

pytestmark = pytest.mark.gpu

ACTS = {"silu": abi.SYMM_ACT_SILU, "gelu": abi.SYMM_ACT_GELU}
POISON = 7.0


@pytest.fixture(scope="module")
def heap():
    h = TorchSymmHeap(1, 0)
    yield h
    h.close()


def counts_of(kind, n, E, g):
    """(rows per expert, rows of them in all)."""
    if kind == "one":  # all rows are the last expert's
        c = torch.zeros(E, dtype=torch.int32)
        c[-1] = n
        return c
    rows = n - max(1, n // 4) if kind == "tail" and n > 1 else n
    like = torch.rand(E, generator=g) + 0.1
    if kind == "holes":
        like[::2] = 0
        if not like.any():
            like[0] = 1
    return torch.bincount(torch.multinomial(like, rows, replacement=True, generator=g),
                          minlength=E).to(torch.int32)


def make(n, E, D, F, dt, kind, seed=0):
    g = torch.Generator().manual_seed(seed + n)

    def rnd(*s, scale=1.0):
        return (torch.randn(*s, generator=g) * scale).to(DTYPES[dt]).cuda()

    return dict(x=rnd(n, D), dy=rnd(n, D), w_gu=rnd(E, D, 2 * F, scale=D ** -0.5),
                w_d=rnd(E, F, D, scale=F ** -0.5), counts=counts_of(kind, n, E, g).cuda())


def spread(t, ld):
    buf = torch.full((t.shape[0], ld), POISON, dtype=t.dtype, device="cuda")
    buf[:, :t.shape[1]] = t
    return buf


def ptr(t):
    return None if t is None else t.data_ptr()


def forward(heap, i, dt, name, pad=0, gu=True, counts=True, stream=None):
    (n, D), (E, F, _) = i["x"].shape, i["w_d"].shape
    x = spread(i["x"], D + pad)
    y = torch.full((n, D + pad), POISON, dtype=x.dtype, device="cuda")
    gu = torch.full((n, 2 * F), POISON, dtype=x.dtype, device="cuda") if gu else None
    ws = torch.full((max(1, abi.moe_expert_workspace(n, E, D, F)),), 0xFF, dtype=torch.uint8,
                    device="cuda")  # NaN in every type: needs no initialisation
    torch.cuda.synchronize()
    abi.moe_expert_ffn(heap.handle, ptr(x), D + pad, ptr(i["counts"]) if counts else None,
                       ptr(i["w_gu"]), ptr(i["w_d"]), ACTS[name], CODES[dt], n, E, D, F, ptr(gu),
                       ptr(y), D + pad, ptr(ws), stream=stream)
    torch.cuda.synchronize()
    assert abi.symm_check_error(heap.handle)[0] == abi.SYMM_OK
    assert (y[:, D:] == POISON).all()
    return y[:, :D], gu


def backward(heap, i, gu, dt, name, pad=0, want=("dx", "dw_gu", "dw_d"), counts=True):
    (n, D), (E, F, _) = i["x"].shape, i["w_d"].shape
    x, dy = spread(i["x"], D + pad), spread(i["dy"], D + pad)
    o = dict(dx=torch.full((n, D + pad), POISON, dtype=x.dtype, device="cuda"),
             dw_gu=torch.full_like(i["w_gu"], float("nan")),
             dw_d=torch.full_like(i["w_d"], float("nan")))
    o = {k: v if k in want else None for k, v in o.items()}
    ws = torch.full((max(1, abi.moe_expert_workspace(n, E, D, F, True)),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    torch.cuda.synchronize()
    abi.moe_expert_ffn_backward(
        heap.handle, ptr(dy), D + pad, ptr(x), D + pad, ptr(gu), ptr(i["counts"]) if counts else None,
        ptr(i["w_gu"]), ptr(i["w_d"]), ACTS[name], CODES[dt], n, E, D, F, ptr(o["dx"]), D + pad,
        ptr(o["dw_gu"]), ptr(o["dw_d"]), ptr(ws))
    torch.cuda.synchronize()
    assert abi.symm_check_error(heap.handle)[0] == abi.SYMM_OK
    if o["dx"] is not None:
        assert (o["dx"][:, D:] == POISON).all()
        o["dx"] = o["dx"][:, :D]
    return o


def near(got, want, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    off = (got - want).abs()
    assert (off <= bound).all(), (what, float((off / bound).max()))


SHAPES = [
    (1, 1, 8, 8, "bf16", "silu", "even"), (1, 3, 64, 64, "f16", "gelu", "even"),
    (2, 2, 72, 40, "bf16", "gelu", "one"), (7, 4, 128, 64, "bf16", "silu", "holes"),
    (16, 1, 64, 128, "f16", "silu", "even"), (17, 5, 136, 72, "bf16", "silu", "tail"),
    (48, 1, 256, 192, "bf16", "silu", "even"), (49, 1, 200, 136, "f16", "silu", "even"),
    (64, 2, 1024, 64, "bf16", "gelu", "one"), (65, 1, 64, 1032, "bf16", "silu", "even"),
    (128, 33, 72, 264, "f16", "gelu", "holes"), (200, 3, 520, 328, "bf16", "silu", "tail"),
    (256, 1, 128, 128, "bf16", "silu", "one"), (257, 1, 136, 200, "bf16", "gelu", "one"),
    (300, 200, 64, 64, "bf16", "silu", "even"), (500, 1000, 40, 24, "f16", "silu", "even"),
    (1025, 2, 320, 192, "bf16", "silu", "holes"), (2500, 3, 192, 320, "f16", "silu", "tail"),
    (4200, 2, 264, 72, "bf16", "gelu", "even"), (600, 5, 2048, 1408, "bf16", "silu", "tail"),
]


@pytest.mark.parametrize("n,E,D,F,dt,name,kind", SHAPES)
def test_forward(heap, n, E, D, F, dt, name, kind):
    i = make(n, E, D, F, dt, kind)
    rows = int(i["counts"].sum())
    i["x"][rows:] = float("nan")  # what is behind the last expert's rows does not matter
    y, gu = forward(heap, i, dt, name, pad=8 * (n % 3))
    r = ref.ffn(i["x"], i["counts"], i["w_gu"], i["w_d"], name, U_OUT[dt], TINY[dt])
    near(gu[:rows], r["gu"], r["egu"], "gu")
    near(y[:rows], r["y"], r["ey"], "y")
    assert (y[rows:] == POISON).all() and (gu[rows:] == POISON).all()
    again, _ = forward(heap, i, dt, name, gu=False)
    assert torch.equal(again[:rows], y[:rows])  # the same bits without gu, and twice


@pytest.mark.parametrize("n,E,D,F,dt,name,kind", SHAPES)
def test_backward(heap, n, E, D, F, dt, name, kind):
    i = make(n, E, D, F, dt, kind, seed=1)
    rows = int(i["counts"].sum())
    g = torch.Generator().manual_seed(n)
    gu = torch.randn(n, 2 * F, generator=g).to(DTYPES[dt]).cuda()
    for t in (i["x"], i["dy"], gu):
        t[rows:] = float("inf")
    o = backward(heap, i, gu, dt, name, pad=8 * (n % 3))
    r = ref.ffn_grad(i["dy"], i["x"], gu, i["counts"], i["w_gu"], i["w_d"], name, U_OUT[dt],
                     TINY[dt])
    near(o["dx"][:rows], r["dx"], r["edx"], "dx")
    assert (o["dx"][rows:] == POISON).all()
    near(o["dw_gu"], r["dw_gu"], r["edw_gu"], "dw_gu")
    near(o["dw_d"], r["dw_d"], r["edw_d"], "dw_d")
    none = i["counts"] == 0
    assert not o["dw_gu"][none].any() and not o["dw_d"][none].any()
    for k in o:  # each alone: the same bits
        one = backward(heap, i, gu, dt, name, want=(k,))[k]
        assert torch.equal(one[:rows] if k == "dx" else one, o[k][:rows] if k == "dx" else o[k]), k
