"""GPU parity of moe_block_norm and moe_block_norm_backward against 64-bit
references.  The forward bounds (exo, eh) and the gradients' term magnitudes
come from moe_refs: with u = 2^-24, a value that is a sum of products whose
magnitudes add up to mag, each reached through at most 400 roundings (the
row sums have at most 100 dependent additions, and three of them feed one
another), errs by at most 400 u mag; a column sum over T tokens adds T more.
The outputs' rounding to their type comes on top."""
import pytest
import torch

import moe_refs as ref
from moe_refs import CODES, DTYPES, TINY, U32, U_OUT
from symmetric_memory_moe_gb300 import abi

pytestmark = pytest.mark.gpu

EPS = 1e-6
POISON = 7.0


def make(T, D, k, dt, seed, post=True, pre=True, optional=True, drop=False, spare=0):
    """Inputs as moe_refs.norm takes them, on the GPU; spare: rows of y that no token names."""
    g = torch.Generator().manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=g)

    yrows = T * k + spare
    rows = None
    if drop or spare:
        rows = torch.randperm(yrows, generator=g)[:T * k].view(T, k).to(torch.int32)
    if drop:
        lost = torch.rand(T, k, generator=g)
        rows[lost < 0.15] = -1
        rows[(lost >= 0.15) & (lost < 0.2)] = yrows  # one past the end
        rows[T // 2] = -1
    y = r(yrows, D).to(DTYPES[dt])
    i = dict(x=r(T, D).to(DTYPES[dt]), y=y, rows=rows,
             weights=torch.softmax(r(T, k), -1) if optional else None,
             gate=r(T) if optional else None, res=r(D) if optional else None,
             w_post=r(D) if post else None, w_pre=r(D) if pre else None)
    i = {n: None if v is None else v.cuda() for n, v in i.items()}
    i["k"] = k
    if drop:  # a row that nothing names may hold anything
        live = (i["rows"] >= 0) & (i["rows"] < yrows)
        keep = torch.zeros(yrows, dtype=torch.bool, device="cuda")
        keep[i["rows"][live].long()] = True
        i["y"][~keep] = float("nan")
    return i


def spread(t, ld):
    """t's rows, ld elements apart, poison between them."""
    buf = torch.full((t.shape[0], ld), POISON, dtype=t.dtype, device="cuda")
    buf[:, :t.shape[1]] = t
    return buf


def ptr(t):
    return None if t is None else t.data_ptr()


def forward(i, dt, ld=None, ldy=None, stream=None, inplace=False):
    T, D = i["x"].shape
    ld, ldy = ld or D, ldy or D
    x = spread(i["x"], ld)
    y = None if i["y"] is None else spread(i["y"], ldy)
    xo = None if y is None else (x if inplace else torch.full_like(x, POISON))
    h = None if i["w_pre"] is None else torch.full_like(x, POISON)
    rstd = torch.full((T, 2), 9.0, device="cuda")
    torch.cuda.synchronize()
    abi.moe_block_norm(ptr(x), ld, ptr(y), ldy, ptr(i["rows"]), 0 if y is None else len(y),
                       ptr(i["weights"]), ptr(i["gate"]), ptr(i["res"]), ptr(i["w_post"]),
                       ptr(i["w_pre"]), EPS, CODES[dt], T, D, i["k"], ptr(xo), ptr(h), ptr(rstd),
                       stream=stream)
    torch.cuda.synchronize()
    for o in (xo, h):
        if o is not None:
            assert (o[:, D:] == POISON).all()
    return (None if xo is None else xo[:, :D].contiguous(),
            None if h is None else h[:, :D].contiguous(), rstd)


def near(got, want, err, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    bad = (got - want).abs() > err
    assert not bad.any(), (what, int(bad.sum()), float(((got - want).abs() / err).max()))


def check_forward(i, dt, xo, h, rstd):
    r = ref.norm(i, EPS)
    if xo is not None:
        near(xo, r["xo"], r["exo"] + U_OUT[dt] * (r["xo"].abs() + r["exo"]) + TINY[dt], "xo")
    if h is not None:
        near(h, r["h"], r["eh"] + U_OUT[dt] * (r["h"].abs() + r["eh"]) + TINY[dt], "h")
    # the cancellation in a token's sum enters its norm: as eh, relative to it
    near(rstd[:, 0], r["rstd"][:, 0], 3e-5 * r["rstd"][:, 0], "rstd of y")
    near(rstd[:, 1], r["rstd"][:, 1], 3e-5 * r["rstd"][:, 1], "rstd of xo")


SHAPES = [
    # T, D, k, dtype
    (1, 1, 1, "f32"), (3, 7, 2, "bf16"), (5, 8, 3, "f16"), (2, 64, 8, "bf16"), (17, 200, 4, "f32"),
    (9, 999, 2, "f16"), (4, 999, 5, "f32"), (31, 1000, 8, "bf16"), (6, 2048, 8, "f32"),
    (5, 2056, 1, "bf16"), (3, 4099, 3, "bf16"), (40, 7168, 8, "bf16"), (2, 8192, 32, "f16"),
    (2, 8200, 2, "f32"), (3, 16384, 4, "bf16"), (2, 16383, 2, "f16"), (700, 96, 2, "f32"),
]


@pytest.mark.parametrize("T,D,k,dt", SHAPES)
@pytest.mark.parametrize("post,drop", [(True, False), (False, True), (True, True)])
def test_forward(T, D, k, dt, post, drop):
    i = make(T, D, k, dt, T + D + k, post=post, drop=drop, spare=3 if drop else 0)
    check_forward(i, dt, *forward(i, dt))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [48, 333])
def test_forward_without_the_optional_parts(dt, D):
    T, k = 11, 3
    for kw in (dict(optional=False), dict(pre=False), dict(optional=False, post=False, pre=False)):
        i = make(T, D, k, dt, 5, **kw)
        check_forward(i, dt, *forward(i, dt))
    i = make(T, D, k, dt, 6)  # the norm before the block alone
    i = dict(i, y=None, rows=None, weights=None, gate=None, res=None, w_post=None, k=0)
    check_forward(i, dt, *forward(i, dt))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_strides_streams_and_in_place(dt):
    T, D, k = 13, 264, 4
    i = make(T, D, k, dt, 8, drop=True, spare=2)
    want = forward(i, dt)
    st = torch.cuda.Stream()
    for ld, ldy in ((264, 272), (272, 264), (265, 264), (264, 267), (280, 288)):
        got = forward(i, dt, ld, ldy, stream=st)
        check_forward(i, dt, *got)
        if ld % 8 == 0 and ldy % 8 == 0:
            for a, b in zip(got, want):
                assert torch.equal(a, b)
    for a, b in zip(forward(i, dt, inplace=True), want):
        assert torch.equal(a, b)


def test_empty_and_zero_tokens():
    abi.moe_block_norm(None, 8, 16, 8, None, 0, None, None, None, None, None, EPS, 1, 0, 8, 2,
                       None, None, None)
    i = make(6, 40, 2, "f32", 1)
    i["x"].zero_()
    i["y"].zero_()
    xo, h, rstd = forward(i, "f32")
    assert not xo.any() and not h.any() and torch.isfinite(rstd).all()


def back(i, dt, f, dxo, dh, ld=None, ldy=None, inplace=False, grads=True):
    T, D = i["x"].shape
    ld, ldy, k = ld or D, ldy or D, i["k"]
    xo, _, rstd = f
    t = {n: None if v is None else spread(v, ld)
         for n, v in dict(x=i["x"], xo=xo, dxo=dxo, dh=dh).items()}
    y = None if i["y"] is None else spread(i["y"], ldy)
    dx = t["dxo"] if inplace else torch.full_like(t["x"], POISON)
    dy = None if y is None else torch.full_like(y, POISON)
    o = dict(dweights=i["weights"], dgate=i["gate"], dres=i["res"], dw_post=i["w_post"],
             dw_pre=i["w_pre"])
    o = {n: torch.full_like(v, 9.0) if v is not None and grads else None for n, v in o.items()}
    ws = torch.empty(abi.moe_block_norm_workspace(T, D), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)  # NaN: needs no initialisation
    torch.cuda.synchronize()
    abi.moe_block_norm_backward(
        ptr(t["dxo"]), ptr(t["dh"]), ptr(t["x"]), ptr(t["xo"]), ld, ptr(y), ldy, ptr(i["rows"]),
        0 if y is None else len(y), ptr(i["weights"]), ptr(i["gate"]), ptr(i["res"]),
        ptr(i["w_post"]), ptr(i["w_pre"]), ptr(rstd), CODES[dt], T, D, k, ptr(dx), ptr(dy),
        *[ptr(o[n]) for n in ("dweights", "dgate", "dres", "dw_post", "dw_pre")], ws.data_ptr())
    torch.cuda.synchronize()
    for b in (dx, dy):
        if b is not None:
            assert (b[:, D:] == POISON).all()
    o["dx"], o["dy"] = dx[:, :D], None if dy is None else dy[:, :D]
    return o


def check_back(i, dt, f, dxo, dh, o):
    T = i["x"].shape[0]
    r = ref.norm_grad(i, f[0] if f[0] is not None else i["x"], f[2], dxo, dh)
    for n, v in o.items():
        if v is None:
            continue
        want, mag = r[n], r[n + "_mag"]
        if n == "dy":
            free = torch.isnan(want[:, 0])
            assert (v[free] == POISON).all()  # rows that no token names are left alone
            v, want, mag = v[~free], want[~free], mag[~free]
        err = 400 * U32 * mag
        if n in ("dx", "dy"):
            err = err + U_OUT[dt] * want.abs() + TINY[dt]
        if n in ("dres", "dw_post", "dw_pre"):
            err = err + T * U32 * mag
        near(v, want, err + 1e-37, n)


@pytest.mark.parametrize("T,D,k,dt", SHAPES)
@pytest.mark.parametrize("post,drop", [(True, False), (False, True), (True, True)])
def test_backward(T, D, k, dt, post, drop):
    i = make(T, D, k, dt, T + D + k + 1, post=post, drop=drop, spare=3 if drop else 0)
    f = forward(i, dt)
    g = torch.Generator().manual_seed(3)
    dxo, dh = (torch.randn(T, D, generator=g).to(DTYPES[dt]).cuda() for _ in range(2))
    check_back(i, dt, f, dxo, dh, back(i, dt, f, dxo, dh))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [48, 333])
def test_backward_without_the_optional_parts(dt, D):
    T, k = 11, 3
    g = torch.Generator().manual_seed(3)
    dxo, dh = (torch.randn(T, D, generator=g).to(DTYPES[dt]).cuda() for _ in range(2))
    for kw, a, b in ((dict(optional=False), dxo, dh), (dict(pre=False), dxo, None),
                     (dict(), None, dh), (dict(optional=False, post=False, pre=False), dxo, None)):
        i = make(T, D, k, dt, 5, **kw)
        f = forward(i, dt)
        check_back(i, dt, f, a, b, back(i, dt, f, a, b))
        o = back(i, dt, f, a, b, grads=False)
        check_back(i, dt, f, a, b, o)
    i = make(T, D, k, dt, 6)  # the norm before the block alone
    i = dict(i, y=None, rows=None, weights=None, gate=None, res=None, w_post=None, k=0)
    f = forward(i, dt)
    for a in (dxo, None):
        check_back(i, dt, f, a, dh, back(i, dt, f, a, dh))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_backward_strides_and_in_place(dt):
    T, D, k = 13, 264, 4
    i = make(T, D, k, dt, 8, drop=True, spare=2)
    f = forward(i, dt)
    g = torch.Generator().manual_seed(3)
    dxo, dh = (torch.randn(T, D, generator=g).to(DTYPES[dt]).cuda() for _ in range(2))
    want = back(i, dt, f, dxo, dh)
    for ld, ldy in ((264, 272), (272, 264), (265, 264), (264, 267)):
        got = back(i, dt, f, dxo, dh, ld, ldy)
        check_back(i, dt, f, dxo, dh, got)
    same = back(i, dt, f, dxo, dh, inplace=True)
    for n in want:
        assert torch.equal(same[n], want[n]), n


def test_backward_of_many_tokens_gives_equal_bits():
    i = make(3000, 520, 3, "bf16", 12, drop=True)
    f = forward(i, "bf16")
    g = torch.Generator().manual_seed(3)
    dxo, dh = (torch.randn(3000, 520, generator=g).bfloat16().cuda() for _ in range(2))
    a, b = (back(i, "bf16", f, dxo, dh) for _ in range(2))
    for n in a:
        assert torch.equal(a[n], b[n]), n
    check_back(i, "bf16", f, dxo, dh, a)


def test_backward_of_no_tokens_gives_empty_sums():
    g = [torch.full((48,), 9.0, device="cuda") for _ in range(3)]
    w = torch.ones(48, device="cuda")
    ws = torch.empty(abi.moe_block_norm_workspace(0, 48), dtype=torch.uint8, device="cuda")
    abi.moe_block_norm_backward(None, ptr(ws), None, None, 48, ptr(ws), 48, None, 0, None, None,
                                ptr(w), ptr(w), ptr(w), None, 2, 0, 48, 1, None, None, None, None,
                                *[ptr(t) for t in g], ptr(ws))
    for t in g:
        assert not t.any()


ODD = [  # T, D, k, dtype: rows that start in the middle of a word, at the ring's edges
    (5, 1, 2, "bf16"), (4, 31, 3, "f16"), (6, 63, 2, "bf16"), (3, 255, 8, "f16"),
    (7, 257, 4, "bf16"), (3, 511, 3, "f16"), (2, 2047, 8, "bf16"), (3, 2049, 2, "f16"),
    (2, 4097, 8, "bf16"), (2, 7167, 8, "bf16"), (2, 8191, 4, "f16"), (2, 16383, 3, "bf16"),
    (5, 33, 2, "f32"), (3, 7167, 8, "f32"), (900, 65, 3, "bf16"), (5, 37, 32, "bf16"),
    (6, 129, 29, "f16"), (5, 40, 30, "bf16"), (400, 7168, 8, "bf16"), (400, 515, 5, "f16"),
]


@pytest.mark.parametrize("D,dt", [(33, "bf16"), (515, "f16"), (3001, "bf16"), (77, "f32")])
def test_odd_rows_in_place(D, dt):
    i = make(19, D, 3, dt, D)
    want = forward(i, dt)
    for a, b in zip(forward(i, dt, inplace=True), want):
        assert torch.equal(a, b)
    g = torch.Generator().manual_seed(3)
    dxo, dh = (torch.randn(19, D, generator=g).to(DTYPES[dt]).cuda() for _ in range(2))
    a, b = (back(i, dt, want, dxo, dh, inplace=p) for p in (False, True))
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("T,D,k,dt", ODD)
def test_odd_rows(T, D, k, dt):
    i = make(T, D, k, dt, T + D, drop=True, spare=3)
    g = torch.Generator().manual_seed(3)
    dxo, dh = (torch.randn(T, D, generator=g).to(DTYPES[dt]).cuda() for _ in range(2))
    for ld, ldy in ((D, D), (D + 1, D + 2), (D + 3, D + 1)):
        f = forward(i, dt, ld, ldy)
        check_forward(i, dt, *f)
        check_back(i, dt, f, dxo, dh, back(i, dt, f, dxo, dh, ld, ldy))


def test_backward_against_differences():
    """<gradients, directions> against a central difference of the 64-bit scalar."""
    T, D, k = 20, 96, 3
    i = make(T, D, k, "f32", 21)
    f = forward(i, "f32")
    g = torch.Generator().manual_seed(3)
    dxo, dh = (torch.randn(T, D, generator=g).cuda() for _ in range(2))
    o = back(i, "f32", f, dxo, dh)
    names = dict(x="dx", y="dy", weights="dweights", gate="dgate", res="dres", w_post="dw_post",
                 w_pre="dw_pre")
    d = {n: i[n].double() for n in names}
    have = torch.ones(T, k, dtype=torch.bool, device="cuda")

    def scalar(j):
        return ref.norm_scalar(j["x"], j["y"].view(T, k, D), j["weights"], j["gate"], j["res"],
                               j["w_post"], j["w_pre"], have, EPS, dxo.double(), dh.double())

    r = ref.norm_grad(i, f[0], f[2], dxo, dh)
    for n, grad in names.items():
        v = torch.randn(i[n].shape, generator=g).double().cuda()
        step = 1e-6
        diff = (scalar(dict(d, **{n: d[n] + step * v})) -
                scalar(dict(d, **{n: d[n] - step * v}))) / (2 * step)
        # the saved xo and rstd are 32-bit roundings: a few hundred u of the terms
        tol = ((800 * U32) * r[grad + "_mag"] * v.abs()).sum() + 1e-5
        assert abs((o[grad].double() * v).sum() - diff) <= tol, n


def test_offsets_past_32_bits():
    T, D, k, ldy = 7, 64, 2, 1 << 20
    yrows = 2100  # 2.2e9 elements
    y = torch.empty(yrows, ldy, dtype=torch.bfloat16, device="cuda")
    i = make(T, D, k, "bf16", 2)
    rows = (yrows - 1 - torch.arange(T * k, device="cuda")).view(T, k).to(torch.int32)
    y[rows.flatten().long(), :D] = i["y"]
    want = forward(i, "bf16")
    xo, h = torch.empty_like(i["x"]), torch.empty_like(i["x"])
    rstd = torch.empty(T, 2, device="cuda")
    abi.moe_block_norm(ptr(i["x"]), D, ptr(y), ldy, ptr(rows), yrows, ptr(i["weights"]),
                       ptr(i["gate"]), ptr(i["res"]), ptr(i["w_post"]), ptr(i["w_pre"]), EPS, 1, T,
                       D, k, ptr(xo), ptr(h), ptr(rstd))
    for a, b in zip((xo, h, rstd), want):
        assert torch.equal(a, b)


def test_graph_capture():
    i = make(24, 512, 4, "bf16", 30, drop=True)
    want = forward(i, "bf16")
    xo, h = torch.zeros_like(i["x"]), torch.zeros_like(i["x"])
    rstd = torch.zeros(24, 2, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        abi.moe_block_norm(ptr(i["x"]), 512, ptr(i["y"]), 512, ptr(i["rows"]), len(i["y"]),
                           ptr(i["weights"]), ptr(i["gate"]), ptr(i["res"]), ptr(i["w_post"]),
                           ptr(i["w_pre"]), EPS, 1, 24, 512, 4, ptr(xo), ptr(h), ptr(rstd))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((xo, h, rstd), want):
        assert torch.equal(a, b)
