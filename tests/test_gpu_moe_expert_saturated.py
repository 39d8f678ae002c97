"""The experts' activations where they saturate: gates from -1e4 to 1e4, among them those where
1 + exp(-g) leaves the range of a float.

Every tensor but the gates is made of zeros and ones so that each sum has one term and what comes
out is act(g), act'(g) or act(g) u itself, rounded to the type.  The bounds are relative to those
values, not to the gates.  With 2^-23 for an ulp: an exponential of x errs by 2 + 1.2 |x| ulp
where it neither overflows nor vanishes (|x| < 104), the approximate quotient by 2 ulp, Phi by 5,
each of at most 6 further operations by a half; a quotient by more than 2^126 may be 0, and what
is below the smallest normal float may be, too."""
import math

import pytest
import torch

import expert_refs as ref
from moe_refs import DTYPES, TINY, U_OUT
from symmetric_memory_moe_gb300.torch_heap import TorchSymmHeap
from test_gpu_moe_expert import backward, forward, near
from test_gpu_moe_fp4 import gscale, pack

pytestmark = pytest.mark.gpu

GATES = [0.0, -0.0, 1.0, -1.0, 5.0, -5.0, 10.0, -10.0, 13.0, -13.0, 20.0, -20.0, 50.0, -50.0, 80.0,
         -80.0, 86.5, -86.5, 87.0, -87.0, 87.5, -87.5, 88.0, -88.0, 88.5, -88.5, 89.0, -89.0, 100.0,
         -100.0, 1e4, -1e4]  # 1e4 is rounded to the type
U23 = 2.0 ** -23


@pytest.fixture(scope="module")
def heap():
    h = TorchSymmHeap(1, 0)
    yield h
    h.close()


def exact(name, g):
    """act(g), act'(g) in 64 bits and the bounds of their 32-bit evaluation."""
    tiny = 2.0 ** -126
    if name == "silu":
        p = 1 / (1 + torch.exp(-g))
        # of 1 + exp(-g) the exponential is 1 - p
        ep = U23 * (6 + (2 + 1.2 * g.abs().clamp(max=104)) * (1 - p))
        f, df = g * p, p * (1 + g * (1 - p))
        return (f, df, (ep + 2 * U23) * f.abs() + tiny * (1 + g.abs()),
                2 * p * (ep + 4 * U23) * (1 + g.abs()) + tiny * (1 + g.abs()))
    # the lower tail by erfc: what adds 1 to erf has nothing left of it below -9
    p, pdf = 0.5 * torch.erfc(-g / math.sqrt(2)), torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    f, df = g * p, p + g * pdf
    ed = U23 * (8 + 1.2 * (g * g / 2).clamp(max=104))
    return (f, df, 8 * U23 * f.abs() + tiny * (1 + g.abs()),
            8 * U23 * p + ed * (g * pdf).abs() + 2 * U23 * df.abs() + tiny * (1 + g.abs()))


def operands(dt):
    """One expert, 32 rows that each pick a row of the weights: gates as listed, values of one."""
    t = DTYPES[dt]
    D = F = len(GATES)
    x = torch.eye(D, device="cuda").to(t)
    w_gu = torch.ones(1, D, 2 * F, device="cuda").to(t)
    gates = torch.tensor(GATES, device="cuda")
    for i in range(D):  # every gate in every column once
        w_gu[0, i, :F] = gates.roll(i).to(t)
    w_d = torch.eye(F, device="cuda").to(t)[None].contiguous()
    return dict(x=x, dy=torch.ones_like(x), w_gu=w_gu, w_d=w_d,
                counts=torch.tensor([D], dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_forward(heap, name, dt):
    i = operands(dt)
    F = len(GATES)
    y, gu = forward(heap, i, dt, name)
    assert torch.equal(gu, i["w_gu"][0])
    f, _, ef, _ = exact(name, i["w_gu"][0, :, :F].double())
    near(y, f, ef * (1 + U_OUT[dt]) + U_OUT[dt] * f.abs() + TINY[dt], "y")


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_backward(heap, name, dt):
    i = operands(dt)
    F = len(GATES)
    gu = i["w_gu"][0].contiguous()
    o = backward(heap, i, gu, dt, name)
    f, df, ef, edf = exact(name, gu[:, :F].double())
    u, tiny = U_OUT[dt], TINY[dt]
    # rows of x are unit vectors: dw_gu is [dg | du] = [act'(g) | act(g)]; dw_d is act(g)^T 1
    near(o["dw_gu"][0, :, :F], df, edf * (1 + u) + u * df.abs() + tiny, "dg")
    near(o["dw_gu"][0, :, F:], f, ef * (1 + u) + u * f.abs() + tiny, "du")
    eh = ef * (1 + u) + u * f.abs() + tiny  # h is rounded, then summed over the rows
    want, off = f.sum(0)[:, None], (eh + (F + 8) * U23 * f.abs()).sum(0)[:, None]
    near(o["dw_d"][0], want.expand(F, F), (off * (1 + u) + u * want.abs() + tiny).expand(F, F),
         "dw_d")


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("name", ["silu", "gelu"])
@pytest.mark.parametrize("fmt,g", [("mx", None), ("nv", None), ("nv", 2.0 ** -40),
                                   ("nv", 2.0 ** -70)])
def test_quantize(fmt, g, name, dt):
    """A block for each gate, with values u of several sizes."""
    b = ref.BLOCK[fmt]
    k = len(GATES) * b
    gen = torch.Generator().manual_seed(b)
    u = torch.randn(9, k, generator=gen)
    gates = torch.tensor(GATES).repeat_interleave(b).expand(9, k)
    x = torch.cat([gates, u], 1).to(DTYPES[dt]).cuda()
    g = gscale(g)
    codes, scales = pack(x, fmt, g, name)
    gate, up = x[:, :k].double(), x[:, k:].double()
    f, _, ef, _ = exact(name, gate)
    h, off = f * up, ef * up.abs() + U23 * (f * up).abs()
    _, least = ref.quantize(torch.sign(h) * (h.abs() - off).clamp(min=0), fmt, g)
    _, most = ref.quantize(torch.sign(h) * (h.abs() + off), fmt, g)
    scale = scales[:, :k // b]
    assert (scale >= least).all() and (scale <= most).all()
    unit = ref.unit_of(scale, fmt, g).repeat_interleave(b, 1)
    code = ref.unpack(codes[:, :k // 2])
    size, grid = (code & 7).long(), torch.cat([ref.GRID, torch.tensor([1e300]).double()]).cuda()
    above = (grid[size] + grid[size + 1]) / 2 * unit
    below = torch.where(size > 0, (grid[size] + grid[(size - 1).clamp(min=0)]) / 2 * unit, -1.0)
    slack = off + U23 * h.abs()
    some = unit > 0
    assert (h.abs() <= above + slack)[some].all() and (h.abs() >= below - slack)[some].all()
    assert ((code > 7) == (h < 0))[(size > 0) & (h.abs() > off)].all()
