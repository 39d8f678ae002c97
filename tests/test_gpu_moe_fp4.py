"""4-bit rows and the experts' product of them against 64-bit references.

Packing is exact: codes and scales are compared bit for bit.  With an
activation the packed value h carries the error of a 32-bit evaluation
(expert_refs.act_error), so a code is right when it is a nearest one of some
value that near h, and likewise a scale.  In the product, codes times scales have
at most 12 bits and their products 24: exact in 32 bits; each of the k additions
errs by at most 2^-23 relatively, and 8 more roundings stand for the tensors' own
scales and the joins of partial sums."""
import pytest
import torch

import expert_refs as ref
from moe_refs import DTYPES, TINY, U_OUT
from symmetric_memory_moe_gb300 import abi
from symmetric_memory_moe_gb300.torch_heap import TorchSymmHeap
from test_gpu_moe_expert import ACTS, POISON, counts_of, near, ptr

pytestmark = pytest.mark.gpu

FMTS = {"mx": abi.SYMM_FP4_MX, "nv": abi.SYMM_FP4_NV}
CODES = {"f16": 0, "bf16": 1, "f32": 2}


@pytest.fixture(scope="module")
def heap():
    h = TorchSymmHeap(1, 0)
    yield h
    h.close()


def widths(k, fmt, more=0):
    return -(-k // 2 // 16) * 16 + more, -(-k // ref.BLOCK[fmt] // 16) * 16 + more


def pack(x, fmt, g=None, name=None, more=0):
    """The library's (codes, scales), rows `more` bytes further apart than needed."""
    n, k = x.shape
    k = k if name is None else k // 2
    wc, ws = widths(k, fmt, more)
    codes = torch.full((n, wc), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((n, ws), 0xA5, dtype=torch.uint8, device="cuda")
    dt = {v: c for c, v in DTYPES.items()}[x.dtype]
    torch.cuda.synchronize()
    abi.moe_fp4_quantize(ptr(x), x.stride(0), -1 if name is None else ACTS[name], CODES[dt],
                         FMTS[fmt], ptr(g), n, k, ptr(codes), wc, ptr(scales), ws)
    torch.cuda.synchronize()
    b = k // ref.BLOCK[fmt]
    assert (codes[:, k // 2:] == 0xA5).all() and (scales[:, b:] == 0xA5).all()
    return codes, scales


def gscale(v):
    return torch.tensor([v], device="cuda") if v else None


def rows(n, k, dt, seed=0, spread=True):
    g = torch.Generator(device="cuda").manual_seed(seed + k)
    x = torch.randn(n, k, generator=g, device="cuda")
    if spread:  # blocks of all sizes, from nothing to what the type holds
        x *= 2.0 ** torch.randint(-16, 9, (n, k // 16), generator=g,
                                  device="cuda").repeat_interleave(16, 1)
        x[:, :16][torch.rand(n, generator=g, device="cuda") < 0.2] = 0
        x[torch.rand(n, k, generator=g, device="cuda") < 0.05] = -0.0
    return x.to(DTYPES[dt])


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt,g", [("mx", None), ("nv", None), ("nv", 0.25), ("nv", 0.0371)])
@pytest.mark.parametrize("n,k,more", [(1, 32, 0), (3, 64, 16), (17, 96, 0), (5, 1056, 32),
                                      (64, 7168, 0), (1000, 480, 16)])
def test_quantize(n, k, more, fmt, g, dt):
    x, g = rows(n, k, dt), gscale(g)
    codes, scales = pack(x, fmt, g, more=more)
    code, scale = ref.quantize(x, fmt, g)
    assert torch.equal(scales[:, :scale.shape[1]], scale)
    assert torch.equal(codes[:, :k // 2], ref.pack(code))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_quantize_borders(fmt):
    """Values on, just below and just above every border of two codes."""
    mid = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7, 0])
    v = torch.cat([mid, mid * (1 - 2.0 ** -20), mid * (1 + 2.0 ** -20)])
    x = torch.zeros(64, 64)
    for i in range(64):
        for b in range(0, 64, 16):
            order = torch.randperm(30, generator=torch.Generator().manual_seed(i + b))
            x[i, b:b + 15] = v[order[:15]]
            x[i, b + 15] = 6
        x[i] *= (-1.0) ** i * 2.0 ** (i % 9 - 4)
    x = x.cuda()
    codes, scales = pack(x, fmt)
    code, scale = ref.quantize(x, fmt, None)
    assert torch.equal(scales[:, :scale.shape[1]], scale)
    assert torch.equal(codes, ref.pack(code))


@pytest.mark.parametrize("fmt,nan", [("mx", 0xff), ("nv", 0x7f)])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_quantize_not_finite(fmt, nan, dt):
    x = rows(6, 256, dt, spread=False)
    x[0, 3], x[1, 40], x[2, 255], x[3, 100] = float("inf"), -float("inf"), float("nan"), 0
    x[4], x[5] = torch.finfo(x.dtype).max, torch.finfo(x.dtype).tiny
    codes, scales = pack(x, fmt)
    code, scale = ref.quantize(x, fmt, None)
    b = ref.BLOCK[fmt]
    for r, at in ((0, 3), (1, 40), (2, 255)):
        assert scales[r, at // b] == nan
    assert torch.equal(scales[:, :scale.shape[1]], scale)
    assert torch.equal(codes[:, :128], ref.pack(code))


@pytest.mark.parametrize("dt,name", [("bf16", "silu"), ("f16", "gelu"), ("f32", "silu")])
@pytest.mark.parametrize("fmt,g", [("mx", None), ("nv", 0.5), ("nv", None)])
@pytest.mark.parametrize("n,k", [(3, 32), (70, 1408), (257, 224)])
def test_quantize_gated(n, k, fmt, g, dt, name):
    x, g = rows(n, 2 * k, dt, spread=False), gscale(g)
    codes, scales = pack(x, fmt, g, name)
    gate, up = x[:, :k].double(), x[:, k:].double()
    h = ref.act(name, gate)[0] * up
    off = (ref.act_error(gate)[0] * up.abs() + 2.0 ** -23 * h.abs())
    b = ref.BLOCK[fmt]
    _, least = ref.quantize(torch.sign(h) * (h.abs() - off).clamp(min=0), fmt, g)
    _, most = ref.quantize(torch.sign(h) * (h.abs() + off), fmt, g)
    scale = scales[:, :k // b]
    assert (scale >= least).all() and (scale <= most).all()
    unit = ref.unit_of(scale, fmt, g)
    code = ref.unpack(codes[:, :k // 2])
    v = ref.values(code, scale, fmt, g)
    # the values that round to a code: up to the middle of its gaps, at 6 all above
    code = (code & 7).long()
    grid = torch.cat([ref.GRID, torch.tensor([1e9], dtype=torch.float64)]).cuda()
    u = unit.repeat_interleave(b, 1)
    above = (grid[code] + grid[code + 1]) / 2 * u
    below = torch.where(code > 0, (grid[code] + grid[(code - 1).clamp(min=0)]) / 2 * u, -1.0)
    slack = off + 2.0 ** -23 * h.abs() + 1e-30
    assert ((h.abs() <= above + slack) | (u == 0)).all()
    assert ((h.abs() >= below - slack) | (u == 0)).all()
    assert ((torch.sign(v) == torch.sign(h)) | (v == 0)).all()


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt,g", [("mx", None), ("mx", 0.3), ("nv", None), ("nv", 0.0371)])
@pytest.mark.parametrize("n,k,more", [(1, 32, 0), (7, 96, 16), (300, 1056, 0)])
def test_dequantize(n, k, more, fmt, g, dt):
    gen = torch.Generator().manual_seed(n)
    wc, ws = widths(k, fmt, more)
    codes = torch.randint(0, 256, (n, wc), generator=gen, dtype=torch.uint8).cuda()
    lo, hi = (100, 150) if fmt == "mx" else (0, 127)
    scales = torch.randint(lo, hi, (n, ws), generator=gen, dtype=torch.uint8).cuda()
    scales[0, 0] = 0xff if fmt == "mx" else 0x7f  # NaN
    g = gscale(g)
    y = torch.full((n, k + 8), POISON, dtype=DTYPES[dt], device="cuda")
    torch.cuda.synchronize()
    abi.moe_fp4_dequantize(ptr(codes), wc, ptr(scales), ws, FMTS[fmt], ptr(g), n, k, CODES[dt],
                           ptr(y), k + 8)
    torch.cuda.synchronize()
    b = ref.BLOCK[fmt]
    want = ref.values(ref.unpack(codes[:, :k // 2]), scales[:, :k // b], fmt, g)
    assert (y[:, k:] == POISON).all() and torch.isnan(y[0, :b]).all()
    want[0, :b] = 0
    y[0, :b] = 0
    assert torch.equal(y[:, :k], want.float().to(DTYPES[dt]))


def product(heap, xc, xs, wc, ws, counts, gx, gw, fmt, dt, k, m, pad=0, stream=None):
    n, E = xc.shape[0], wc.shape[0]
    y = torch.full((n, m + pad), POISON, dtype=DTYPES[dt], device="cuda")
    torch.cuda.synchronize()
    abi.moe_fp4_expert_matmul(heap.handle, ptr(xc), xc.stride(0), ptr(xs), xs.stride(0), ptr(wc),
                              wc.stride(1), ptr(ws), ws.stride(1), ptr(counts), ptr(gx), ptr(gw),
                              FMTS[fmt], CODES[dt], n, E, k, m, ptr(y), m + pad, stream=stream)
    torch.cuda.synchronize()
    assert abi.symm_check_error(heap.handle)[0] == abi.SYMM_OK
    assert (y[:, m:] == POISON).all()
    return y[:, :m]


def operands(n, E, k, m, fmt, kind, seed=0, more=0):
    """Rows and weights packed by the reference, with the counts."""
    g = torch.Generator().manual_seed(seed + n)
    wc, ws = widths(k, fmt, more)

    def packed(*shape):
        x = torch.randn(*shape, k, generator=g)
        x *= 2.0 ** torch.randint(-3, 3, (*shape, k // 16), generator=g).repeat_interleave(16, -1)
        code, scale = ref.quantize(x.cuda(), fmt, None)
        c = torch.full((*shape, wc), 0xA5, dtype=torch.uint8, device="cuda")
        s = torch.full((*shape, ws), 0x70, dtype=torch.uint8, device="cuda")
        c[..., :k // 2], s[..., :scale.shape[-1]] = ref.pack(code), scale
        return c, s, ref.values(code, scale, fmt, None)

    return packed(n), packed(E, m), counts_of(kind, n, E, g)


@pytest.mark.parametrize("n,E,k,m,fmt,dt,kind", [
    (1, 1, 32, 1, "nv", "bf16", "even"), (1, 1, 32, 8, "mx", "f16", "even"),
    (2, 2, 64, 128, "nv", "f16", "one"), (5, 3, 256, 130, "mx", "bf16", "even"),
    (16, 1, 512, 64, "mx", "bf16", "even"), (17, 2, 288, 200, "nv", "bf16", "holes"),
    (48, 1, 1024, 256, "nv", "f16", "even"), (49, 1, 1056, 72, "mx", "bf16", "one"),
    (100, 7, 800, 333, "nv", "bf16", "tail"), (128, 1, 320, 128, "nv", "bf16", "one"),
    (129, 1, 352, 136, "mx", "f16", "one"), (192, 1, 2048, 128, "nv", "bf16", "one"),
    (193, 1, 96, 1000, "nv", "f16", "one"), (400, 300, 64, 40, "mx", "bf16", "even"),
    (1500, 4, 736, 520, "mx", "bf16", "tail"), (2500, 3, 1312, 264, "nv", "bf16", "holes"),
    (700, 5, 4096, 640, "nv", "bf16", "even"), (700, 5, 4096, 640, "mx", "f16", "tail")])
def test_product(heap, n, E, k, m, fmt, dt, kind):
    (xc, xs, x), (wc, ws, w), c = operands(n, E, k, m, fmt, kind, more=16 * (n % 2))
    g = torch.Generator().manual_seed(m)
    gx = (torch.rand(1, generator=g) + 0.5).cuda() if n % 3 else None
    gw = (torch.rand(E, generator=g) + 0.5).cuda() if n % 5 else None
    total = int(c.sum())
    xs[total:] = 0xff if fmt == "mx" else 0x7f  # NaN behind the last expert's rows
    y = product(heap, xc, xs, wc, ws, c.cuda(), gx, gw, fmt, dt, k, m, pad=n % 4)
    for e, a, b in ref.runs(c):
        s = (1.0 if gx is None else gx.double()) * (1.0 if gw is None else gw[e].double())
        want, mag = s * (x[a:b] @ w[e].t()), s * (x[a:b].abs() @ w[e].abs().t())
        bound = U_OUT[dt] * want.abs() + (k + 8) * 2.0 ** -23 * mag + TINY[dt]
        near(y[a:b], want, bound * (1 + 2.0 ** -8), e)
    assert (y[total:] == POISON).all()
