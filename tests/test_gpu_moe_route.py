"""GPU parity of moe_route and moe_route_backward against 64-bit references.

Experts, counts and token numbers are whole and must be equal.  With u =
2^-24 the unit of a float's rounding: a probability exp(l - m)/s errs by the
rounding of l - m (its size times u), the exponential (2 units in the last
place, 4u), the sum of E terms (at most 60 dependent additions) and the
quotient, so relatively by (|l - m| + 70) u; terms below exp(-40) are left
out of the relative check, being under 2^-57 of the largest.  Quotients of
two such, and products with the scale, stay within

    W = 2 (40 + 70) u = 220 u.

A sum over the T tokens of a group of positive terms adds at most T + 100
dependent additions: (W + (T + 100) u) relatively.  The z loss is such a sum of
lse^2 with lse = m + log s off by 70 u + 4 u |lse|.  A gradient element is a
sum of terms whose magnitudes the reference adds up (mag): its error is at
most 2 W mag, beside the rounding of the output."""
import math

import pytest
import torch

import moe_refs as ref
from moe_refs import CODES, DTYPES, U32
from symmetric_memory_moe_gb300 import abi

pytestmark = pytest.mark.gpu

W = 220 * U32


def make(G, T, E, dt, seed, kind="plain"):
    g = torch.Generator().manual_seed(seed)
    l = 2 * torch.randn(G, T, E, generator=g)
    mask = None
    if kind == "ties":
        l = torch.randint(-2, 3, (G, T, E), generator=g).float()
    if kind == "holes":
        l[torch.rand(G, T, E, generator=g) < 0.5] = -math.inf
        l[:, ::5] = -math.inf
        l[:, 1::5, 0] = math.nan
        l[:, 2::5] = torch.finfo(DTYPES[dt]).min
        mask = (torch.rand(G, T, generator=g) < 0.8).to(torch.uint8)
        l[mask == 0] = math.nan
    if kind == "infinite":
        l[:, ::2, E // 2] = math.inf
        l[:, ::4, E - 1] = math.inf
        l[:, 1::2] *= 1e4 if dt != "f16" else 1e3
    return l.to(DTYPES[dt]), mask


def forward(l, mask, k, dt, renorm, scale=1.0, ld=None, stream=None):
    G, T, E = l.shape
    ld = ld or E
    buf = torch.full((max(G * T * ld, 1),), 7.0, dtype=l.dtype, device="cuda")
    buf[:G * T * ld].view(G * T, ld)[:, :E] = l.reshape(-1, E).cuda()
    o = dict(experts=torch.full((G, T, k), 99, dtype=torch.int32), weights=torch.full((G, T, k), 9.),
             counts=torch.full((G, E), 99, dtype=torch.int32),
             tokens=torch.full((G,), 99, dtype=torch.int32),
             stats=torch.full((G, T, 2), 9.), loss=torch.full((G, 2), 9.))
    o = {n: v.cuda() for n, v in o.items()}
    m = None if mask is None else mask.cuda()
    ws = torch.empty(max(abi.moe_route_workspace(G, T, E), 16), dtype=torch.uint8, device="cuda")
    ws.fill_(0xA5)  # needs no initialisation
    torch.cuda.synchronize()
    abi.moe_route(buf.data_ptr(), ld, None if m is None else m.data_ptr(), CODES[dt], G, T, E, k,
                  renorm, scale, *[o[n].data_ptr() for n in ("experts", "weights", "counts",
                                                            "tokens", "stats", "loss")],
                  ws.data_ptr(), stream=stream)
    torch.cuda.synchronize()
    return buf, o


def check_forward(o, r, E, k, T):
    for n in ("experts", "counts", "tokens"):
        assert torch.equal(o[n].cpu(), r[n].cpu()), n
    w, rw = o["weights"].double().cpu(), r["weights"].cpu()
    assert ((w - rw).abs() <= W * rw.abs() + math.exp(-40) * 2).all()
    s, rs = o["stats"].double().cpu(), r["stats"].cpu()
    assert torch.equal(s[..., 0], rs[..., 0])
    assert ((s[..., 1] - rs[..., 1]).abs() <= W * rs[..., 1]).all()
    loss, rl = o["loss"].double().cpu(), r["loss"].cpu()
    assert ((loss[:, 0] - rl[:, 0]).abs() <= (W + (T + 100) * U32) * rl[:, 0]).all()
    # a lse of FLT_MAX squared is infinite in 32 bits
    lse = (r["stats"][..., 0] + torch.log(r["stats"][..., 1].clamp(min=1))).cpu() * \
        r["valid"].cpu()
    n = r["tokens"].cpu().clamp(min=1).double()
    tol = (T + 100) * U32 * rl[:, 1] + 2 * (lse.abs() * (70 * U32 + 4 * U32 * lse.abs())).sum(-1) / n
    big = rl[:, 1] > 3e38
    assert torch.isinf(loss[big, 1]).all()
    assert ((loss[:, 1] - rl[:, 1]).abs() <= tol)[~big].all()


SHAPES = [
    # G, T, E, k, dtype
    (1, 1, 1, 1, "f32"), (1, 1, 256, 8, "bf16"), (2, 3, 5, 5, "f16"), (1, 33, 31, 4, "f32"),
    (3, 17, 33, 2, "bf16"), (2, 64, 60, 4, "f16"), (4, 100, 64, 6, "f32"), (2, 41, 100, 32, "bf16"),
    (1, 300, 129, 3, "f16"), (8, 96, 256, 8, "f32"), (2, 50, 257, 8, "bf16"), (1, 40, 512, 10, "f32"),
    (1, 21, 999, 1, "f16"), (2, 9, 1024, 32, "f32"), (700, 3, 16, 2, "f32"),
]


@pytest.mark.parametrize("G,T,E,k,dt", SHAPES)
@pytest.mark.parametrize("kind", ["plain", "ties", "holes"])
def test_forward(G, T, E, k, dt, kind):
    l, mask = make(G, T, E, dt, G + 7 * T + E, kind)
    for renorm, scale in ((1, 1.0), (0, 2.5)):
        _, o = forward(l, mask, k, dt, renorm, scale)
        check_forward(o, ref.route(l, mask, k, renorm, scale), E, k, T)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_infinite_and_huge_logits(dt):
    l, _ = make(2, 24, 40, dt, 5, "infinite")
    _, o = forward(l, None, 4, dt, 1)
    check_forward(o, ref.route(l, None, 4, 1, 1.0), 40, 4, 24)


def test_many_tokens_and_equal_bits():
    """A group that many CTAs share; the same inputs give the same bits."""
    l, _ = make(1, 20000, 64, "bf16", 8)
    _, a = forward(l, None, 6, "bf16", 1)
    _, b = forward(l, None, 6, "bf16", 1)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    idx = torch.sort(l.float(), dim=-1, descending=True, stable=True)[1][..., :6]
    assert torch.equal(a["experts"].cpu().long(), idx)
    assert torch.equal(a["counts"].cpu().long()[0], torch.bincount(idx.reshape(-1), minlength=64))
    p = torch.softmax(l.double(), -1).sum(1)
    want = 64 / (6 * 20000 ** 2) * (a["counts"].cpu().double() * p).sum(-1)
    assert abs(a["loss"][0, 0].item() - want.item()) <= (W + 20100 * U32) * want.item()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("E,k", [(256, 8), (256, 9), (256, 20), (128, 12), (200, 32), (512, 20)])
def test_neighbouring_experts_win(dt, E, k):
    """All of one lane's experts are chosen, and more: descending, ascending and equal runs."""
    l = torch.zeros(1, 24, E)
    for t in range(24):
        s = 8 * t % (E - k)
        run = torch.arange(k).float()
        l[0, t, s:s + k] = 2 + (run, run.flip(0), torch.zeros(k))[t % 3]
    l = l.to(DTYPES[dt])
    _, o = forward(l, None, k, dt, 1)
    check_forward(o, ref.route(l, None, k, 1, 1.0), E, k, 24)


def test_empty_groups():
    """No tokens, or none valid: zero counts and losses."""
    for T, mask in ((0, None), (6, torch.zeros(3, 6, dtype=torch.uint8))):
        l = torch.zeros(3, T, 10)
        _, o = forward(l, mask, 2, "f32", 1)
        assert not o["counts"].any() and not o["tokens"].any() and not o["loss"].any()
        assert (o["experts"] == -1).all() and not o["weights"].any() and not o["stats"].any()
    abi.moe_route(None, 8, None, 2, 0, 5, 8, 2, 1, 1.0, *[None] * 7)  # G = 0: nothing to do


def back(l, f, k, dt, renorm, scale, dw, dl, ld=None, ldd=None, inplace=False, buf=None):
    G, T, E = l.shape
    ldd = ldd or E
    out = buf if inplace else torch.full((G * T * ldd,), 7.0, dtype=l.dtype, device="cuda")
    abi.moe_route_backward(buf.data_ptr(), ld or E, CODES[dt], G, T, E, k, renorm, scale,
                           *[f[n].data_ptr() for n in ("experts", "counts", "tokens", "stats")],
                           None if dw is None else dw.data_ptr(),
                           None if dl is None else dl.data_ptr(), out.data_ptr(), ldd)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("G,T,E,k,dt", SHAPES)
@pytest.mark.parametrize("kind", ["plain", "holes"])
@pytest.mark.parametrize("renorm,scale", [(1, 1.0), (0, 2.5)])
def test_backward(G, T, E, k, dt, kind, renorm, scale):
    l, mask = make(G, T, E, dt, G + 3 * T + E, kind)
    buf, f = forward(l, mask, k, dt, renorm, scale)
    r = ref.route(l, mask, k, renorm, scale)
    g = torch.Generator().manual_seed(1)
    dw, dl = torch.randn(G, T, k, generator=g), torch.randn(G, 2, generator=g)
    if kind == "holes":
        dl[:, 1] *= 1e-3  # rows of the type's lowest value: lse itself is near the largest float
    for use_w, use_l in ((1, 1), (1, 0), (0, 1)):
        got = back(l, f, k, dt, renorm, scale, dw.cuda() if use_w else None,
                   dl.cuda() if use_l else None, buf=buf).view(G, T, E).double().cpu()
        d, mag = ref.route_grad(ref.clean(l), r["experts"], r["counts"], r["tokens"], r["valid"], k,
                                renorm, scale, dw * use_w, dl * use_l)
        assert torch.isfinite(got).all()
        tol = 2 * W * mag + ref.U_OUT[dt] * d.abs() + ref.TINY[dt]
        assert ((got - d).abs() <= tol).all(), ((got - d).abs() / tol).max()
        assert not got[~r["valid"]].any()


def test_backward_against_differences():
    """<gradient, direction> against a central difference of the 64-bit scalar."""
    G, T, E, k = 2, 30, 40, 4
    l, _ = make(G, T, E, "f32", 77)
    g = torch.Generator().manual_seed(2)
    dw, dl = torch.randn(G, T, k, generator=g), torch.randn(G, 2, generator=g)
    v = torch.randn(G, T, E, generator=g).double()
    for renorm in (1, 0):
        buf, f = forward(l, None, k, "f32", renorm)
        got = back(l, f, k, "f32", renorm, 1.0, dw.cuda(), dl.cuda(), buf=buf)
        got = got.view(G, T, E).double().cpu()
        r = ref.route(l, None, k, renorm, 1.0)
        args = (r["experts"], r["counts"], r["tokens"], r["valid"], k, renorm, 1.0, dw, dl)
        h = 1e-6
        diff = (ref.route_scalar(l.double() + h * v, *args) -
                ref.route_scalar(l.double() - h * v, *args)) / (2 * h)
        _, mag = ref.route_grad(l.double(), *args)
        tol = ((2 * W + 2.0 ** -23) * mag * v.abs()).sum() + 1e-6
        assert abs((got * v).sum() - diff) <= tol


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_strides_and_in_place(dt):
    """Padded rows (also of odd length) are read and written in place of
    dense ones, what lies between the rows stays, and dlogits may be the
    logits."""
    G, T, E, k = 2, 37, 48, 4
    l, _ = make(G, T, E, dt, 4)
    g = torch.Generator().manual_seed(6)
    dw, dl = torch.randn(G, T, k, generator=g).cuda(), torch.randn(G, 2, generator=g).cuda()
    buf, f = forward(l, None, k, dt, 1)
    want = back(l, f, k, dt, 1, 1.0, dw, dl, buf=buf).view(G * T, E)
    for ld in (49, 56, 64):
        buf2, f2 = forward(l, None, k, dt, 1, ld=ld)
        for n in f:
            assert torch.equal(f[n], f2[n]), n
        out = back(l, f, k, dt, 1, 1.0, dw, dl, ld=ld, ldd=ld + 3, buf=buf2).view(G * T, ld + 3)
        assert torch.equal(out[:, :E], want) and (out[:, E:] == 7).all()
        same = back(l, f, k, dt, 1, 1.0, dw, dl, ld=ld, ldd=ld, inplace=True, buf=buf2)
        same = same.view(G * T, ld)
        assert torch.equal(same[:, :E], want) and (same[:, E:] == 7).all()


def test_offsets_past_32_bits():
    G, T, E, k, ld = 2, 35000, 8, 2, 40000  # 2.8e9 elements
    buf = torch.empty(G * T, ld, dtype=torch.float16, device="cuda")
    g = torch.Generator().manual_seed(9)
    l = torch.randn(G, T, E, generator=g).half()
    buf[:, :E] = l.view(-1, E).cuda()
    dense, f = forward(l, None, k, "f16", 1)
    o = {n: torch.empty_like(v) for n, v in f.items()}
    ws = torch.empty(abi.moe_route_workspace(G, T, E), dtype=torch.uint8, device="cuda")
    abi.moe_route(buf.data_ptr(), ld, None, 0, G, T, E, k, 1, 1.0,
                  *[o[n].data_ptr() for n in ("experts", "weights", "counts", "tokens", "stats",
                                             "loss")], ws.data_ptr())
    for n in f:
        assert torch.equal(o[n], f[n]), n
    dw, dl = torch.randn(G, T, k, generator=g).cuda(), torch.ones(G, 2, device="cuda")
    want = back(l, f, k, "f16", 1, 1.0, dw, dl, buf=dense).view(G * T, E)
    got = back(l, f, k, "f16", 1, 1.0, dw, dl, ld=ld, ldd=ld, inplace=True, buf=buf.view(-1))
    assert torch.equal(got.view(G * T, ld)[:, :E], want)


def test_experts_out_of_range_are_ignored():
    """Saved choices that name no expert add nothing and read nothing."""
    l, _ = make(1, 4, 8, "f32", 3)
    buf, f = forward(l, None, 2, "f32", 0)
    dw = torch.ones(1, 4, 2, device="cuda")
    bad = dict(f, experts=f["experts"].clone())
    bad["experts"][0, :, 1] = 1 << 30
    got = back(l, bad, 2, "f32", 0, 1.0, dw, None, buf=buf)
    bad["experts"][0, :, 1] = -1
    want = back(l, bad, 2, "f32", 0, 1.0, dw, None, buf=buf)
    assert torch.equal(got, want)


def test_graph_capture_and_side_stream():
    l, mask = make(4, 200, 64, "bf16", 11, "holes")
    _, want = forward(l, mask, 4, "bf16", 1)
    st = torch.cuda.Stream()
    _, o = forward(l, mask, 4, "bf16", 1, stream=st)
    for n in want:
        assert torch.equal(o[n], want[n]), n
    lc, mc = l.cuda(), mask.cuda()
    ws = torch.empty(abi.moe_route_workspace(4, 200, 64), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    for v in o.values():
        v.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        abi.moe_route(lc.data_ptr(), 64, mc.data_ptr(), 1, 4, 200, 64, 4, 1, 1.0,
                      *[o[n].data_ptr() for n in ("experts", "weights", "counts", "tokens", "stats",
                                                 "loss")], ws.data_ptr())
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(o[n], want[n]), n
