"""The experts of a mixture-of-experts block, as cases to measure.

* ``ffn``: the gated feed-forward of every expert on the rows that the
  all-to-all brought it, y = (act(x Wg) * (x Wu)) Wd, and its gradients;
* ``quant``: rows to microscaled 4-bit floating point and back;
* ``linear``: the experts' projection with 4-bit weights and 4-bit rows, the
  rows quantised in the call (with ``act``: the gated product of their two
  halves, as the second projection of the feed-forward takes them).

``run`` computes them in their plain form (elementary torch operations in 32
bits), or, where ``own`` is true, by the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
CODES = {"f16": 0, "bf16": 1}
ACTS = {"none": -1, "silu": 0, "gelu": 1}
FORMATS = {"mx": 0, "nv": 1}     # 32 values to a power of two, 16 to an e4m3 number
BLOCK = {"mx": 32, "nv": 16}


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one decoding step of a small block: 16 tokens, 2 choices each, latency only
        dict(name="ffn: one decoding step", op="ffn", back=False, n=32, E=32, D=1024, F=512,
             act="silu", dtype="bf16", tail=False, closed=False),
        # a decoding step of 64 requests: 8 of 256 experts each, the 32 experts of one of 8 PEs
        dict(name="ffn: 64 requests", op="ffn", back=False, n=64, E=32, D=7168, F=2048, act="silu",
             dtype="bf16", tail=False, closed=False),
        # a training step: the rows of 4096 tokens' 8 choices on one PE's experts
        dict(name="ffn: training step", op="ffn", back=False, n=32768, E=32, D=7168, F=2048,
             act="silu", dtype="bf16", tail=False, closed=False),
        # odd sizes, experts without rows, a buffer that is not full
        dict(name="ffn: odd sizes", op="ffn", back=False, n=1531, E=5, D=1000, F=328, act="gelu",
             dtype="f16", tail=True, closed=True),
        # a training step's gradients, all of them
        dict(name="ffn: training step backward", op="ffn", back=True, n=16384, E=32, D=4096,
             F=2048, act="silu", dtype="bf16", tail=False, closed=False),
        # few rows per expert: the weights and their gradients are all there is to move
        dict(name="ffn: short sequences backward", op="ffn", back=True, n=512, E=16, D=2048,
             F=1408, act="silu", dtype="bf16", tail=False, closed=True),
        dict(name="ffn: odd sizes backward", op="ffn", back=True, n=1531, E=5, D=1000, F=328,
             act="gelu", dtype="f16", tail=True, closed=True),
        # rows of 64 requests on their way into the 4-bit projection
        dict(name="quant: 64 requests", op="quant", n=64, k=7168, fmt="nv", dtype="bf16",
             gscale=False),
        # a prompt's rows
        dict(name="quant: prompt", op="quant", n=32768, k=7168, fmt="mx", dtype="bf16",
             gscale=False),
        # gate and up projections of a decoding step, 4-bit experts
        dict(name="linear: 64 requests", op="linear", n=64, E=32, k=7168, m=4096, act="none",
             fmt="nv", dtype="bf16", gscale=True, tail=False, closed=False),
        # the second projection of a prompt, fed with the two halves of the first
        dict(name="linear: prompt", op="linear", n=32768, E=32, k=2048, m=7168, act="silu",
             fmt="nv", dtype="bf16", gscale=True, tail=False, closed=False),
        # odd sizes, blocks of 32
        dict(name="linear: odd sizes", op="linear", n=1531, E=5, k=1056, m=1000, act="none",
             fmt="mx", dtype="f16", gscale=False, tail=True, closed=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "quant", "linear"])
    dtype = rng.choice(sorted(DTYPES))
    if op == "quant":
        k = 32 * _log(rng, 1, 256)
        return dict(op=op, n=_log(rng, 1, min(32768, (1 << 28) // (2 * k))), k=k,
                    fmt=rng.choice(sorted(FORMATS)), dtype=dtype, gscale=rng.random() < 0.5)
    E = _log(rng, 1, 64)
    holes = dict(tail=rng.random() < 0.5, closed=E > 1 and rng.random() < 0.5)
    if op == "linear":
        k, m = 32 * _log(rng, 1, 224), 8 * _log(rng, 1, 896)
        E = max(1, min(E, (1 << 29) // (k * m)))
        return dict(op=op, n=_log(rng, 1, min(32768, (1 << 38) // (k * m))), E=E, k=k, m=m,
                    act=rng.choice(["none", "silu", "gelu"]), fmt=rng.choice(sorted(FORMATS)),
                    dtype=dtype, gscale=rng.random() < 0.5, **dict(holes, closed=E > 1 and
                                                                   holes["closed"]))
    D, F = 8 * _log(rng, 4, 896), 8 * _log(rng, 4, 352)
    E = max(1, min(E, (1 << 28) // (D * F)))
    back = rng.random() < 0.5
    return dict(op=op, back=back, n=_log(rng, 1, min(32768, (1 << 36) // (D * F))), E=E, D=D, F=F,
                act=rng.choice(["silu", "gelu"]), dtype=dtype,
                **dict(holes, closed=E > 1 and holes["closed"]))


def _used(n, E):
    """Experts that n rows reach, on average, when they spread evenly."""
    return E * (1 - (1 - 1 / E) ** n)


def _rows(c):
    """Rows that belong to an expert."""
    return c["n"] - c["n"] // 5 if c["tail"] else c["n"]


def work(case):
    c = case
    if c["op"] == "quant":
        bits = 4 + 8 / BLOCK[c["fmt"]]      # written, read again, and the values both ways
        return {"bytes": c["n"] * c["k"] * (4 + 2 * bits / 8), "flops": 0}
    if c["op"] == "linear":
        n, k, m, bits = _rows(c), c["k"], c["m"], 4 + 8 / BLOCK[c["fmt"]]
        wide = k if c["act"] == "none" else 2 * k
        return {"bytes": 2 * n * (wide + m) + _used(n, c["E"]) * k * m * bits / 8,
                "flops": 2 * n * k * m}
    n, D, F = _rows(c), c["D"], c["F"]
    if c["back"]:
        return {"bytes": 2 * (3 * n * D + 2 * n * F + (_used(n, c["E"]) + c["E"]) * 3 * D * F),
                "flops": 12 * n * D * F}
    return {"bytes": 2 * (2 * n * (D + F) + _used(n, c["E"]) * 3 * D * F), "flops": 6 * n * D * F}


# ----------------------------------------------------------------- inputs --
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="cuda").normal_(generator=g)


def _counts(c, g):
    """Rows of each expert, of uneven popularity as a router makes them; int32 [E]."""
    E = c["E"]
    like = torch.exp(0.4 * _randn(g, E))
    if c["closed"]:
        like[torch.randperm(E, generator=g, device="cuda")[:max(1, E // 4)]] = 0
    of = torch.multinomial(like, _rows(c), replacement=True, generator=g)
    return torch.bincount(of, minlength=E).to(torch.int32)


def _pack(x, fmt, g):
    """Codes [rows, k / 2] (the even element low) and scales [rows, k / block, filled up to whole
    16 bytes], uint8, of x [rows, k] in 32 bits or more."""
    rows, k = x.shape
    code, scale = _to_codes(x, fmt, g)
    code = code.view(rows, k // 2, 2)
    wide = torch.zeros(rows, -(-scale.shape[1] // 16) * 16, dtype=torch.uint8, device=x.device)
    wide[:, :scale.shape[1]] = scale
    return code[..., 0] | code[..., 1] << 4, wide


def _gscale(x):
    """A tensor's own scale: its largest value at 6 times e4m3's largest, to a power of two."""
    top = x.abs().amax().float().clamp(min=1e-30) / 2688
    return torch.exp2(torch.ceil(torch.log2(top))).reshape(1)


def prepare(case, seed):
    c, g, dt = case, _gen(seed), DTYPES[case["dtype"]]
    s = dict(case=c)
    n = c["n"]
    if c["op"] == "quant":
        s["x"] = _randn(g, n, c["k"], dtype=dt)
        s["x"][:, :: 97] *= 8                    # a few columns stand out, as activations' do
        s["gscale"] = _gscale(s["x"]) if c["gscale"] else None
        s["values"] = torch.empty_like(s["x"])
    elif c["op"] == "linear":
        E, k, m = c["E"], c["k"], c["m"]
        s["counts"] = _counts(c, g)
        s["most"] = int(s["counts"].max())       # the host's plan knows the fullest expert
        s["x"] = _randn(g, n, k if c["act"] == "none" else 2 * k, dtype=dt)
        packed, s["gw"] = [], torch.ones(E, device="cuda") if c["gscale"] else None
        for e in range(E):
            w = _randn(g, m, k) * k ** -0.5
            if c["gscale"]:
                s["gw"][e] = _gscale(w)
            packed.append(_pack(w, c["fmt"], s["gw"][e] if c["gscale"] else None))
        s["wc"], s["ws"] = (torch.stack(p) for p in zip(*packed))
        gate, up = s["x"][:, :k], s["x"][:, -k:]
        s["gx"] = _gscale(gate if c["act"] == "none" else gate * up) if c["gscale"] else None
        s["y"] = torch.zeros(n, m, dtype=dt, device="cuda")
    else:
        E, D, F = c["E"], c["D"], c["F"]
        s["counts"] = _counts(c, g)
        s["most"] = int(s["counts"].max())
        s["x"] = _randn(g, n, D, dtype=dt)
        s["w_gu"] = _randn(g, E, D, 2 * F, dtype=dt).mul_(D ** -0.5)
        s["w_d"] = _randn(g, E, F, D, dtype=dt).mul_(F ** -0.5)
        if c["back"]:
            gu = _apart(s, _together(s, s["x"]) @ s["w_gu"].float())
            s["gu"] = gu.to(dt)                  # what the forward pass kept
            del gu
            s["dy"] = _randn(g, n, D, dtype=dt)
            s["dx"] = torch.zeros(n, D, dtype=dt, device="cuda")
            s["dw_gu"], s["dw_d"] = torch.empty_like(s["w_gu"]), torch.empty_like(s["w_d"])
        else:
            s["gu"] = torch.zeros(n, 2 * F, dtype=dt, device="cuda")
            s["y"] = torch.zeros(n, D, dtype=dt, device="cuda")
    if own:  # the workspace, the packed rows' buffers and the heap handle that a program keeps
        from symmetric_memory_moe_gb300 import abi
        from symmetric_memory_moe_gb300.torch_heap import TorchSymmHeap
        if c["op"] == "ffn":
            size = abi.moe_expert_workspace(n, c["E"], c["D"], c["F"], c["back"])
            s["scratch"] = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
        else:
            lds = -(-c["k"] // BLOCK[c["fmt"]] // 16) * 16
            s["xc"] = torch.empty(n, c["k"] // 2, dtype=torch.uint8, device="cuda")
            s["xs"] = torch.zeros(n, lds, dtype=torch.uint8, device="cuda")
        if c["op"] != "quant":
            s["heap"] = TorchSymmHeap(1, 0)
    return s


# ------------------------------------------------------------ plain forms --
def _place(s):
    """Each row's place in a [E * most] table of rows by expert; one past it for rows of none."""
    c = s["case"]
    end = s["counts"].long().cumsum(0)
    row = torch.arange(c["n"], device="cuda")
    e = torch.searchsorted(end, row, right=True)
    start = torch.cat([end.new_zeros(1), end])[e]
    return torch.where(e < c["E"], e * s["most"] + row - start, c["E"] * s["most"])


def _together(s, rows):
    """[E, most, width] in 32 bits: each expert's rows, zeros behind them."""
    E, most = s["case"]["E"], s["most"]
    t = torch.zeros(E * most + 1, rows.shape[1], device="cuda")
    t[_place(s)] = rows.float()
    return t[:-1].view(E, most, -1)


def _apart(s, table):
    """The rows [n, width] back from the table, zeros where a row is no expert's."""
    flat = table.reshape(-1, table.shape[-1])
    return torch.cat([flat, flat.new_zeros(1, flat.shape[1])])[_place(s)]


def _act(name, g):
    """act(g) and its derivative."""
    if name == "silu":
        p = 1 / (1 + torch.exp(-g))
        return g * p, p * (1 + g * (1 - p))
    half = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
    return g * half, half + g * torch.exp(-0.5 * g * g) * (0.5 / math.pi) ** 0.5


def _plain_ffn(s):
    c, dt = s["case"], s["x"].dtype
    gu = _together(s, s["x"]) @ s["w_gu"].float()
    gate, up = gu.split(c["F"], -1)
    y = (_act(c["act"], gate)[0] * up) @ s["w_d"].float()
    return dict(gu=_apart(s, gu).to(dt), y=_apart(s, y).to(dt))


def _plain_ffn_back(s):
    c, dt = s["case"], s["x"].dtype
    dy, x = _together(s, s["dy"]), _together(s, s["x"])
    gate, up = _together(s, s["gu"]).split(c["F"], -1)
    a, da = _act(c["act"], gate)
    dh = dy @ s["w_d"].float().transpose(1, 2)
    dgu = torch.cat([dh * up * da, dh * a], -1)
    return dict(dx=_apart(s, dgu @ s["w_gu"].float().transpose(1, 2)).to(dt),
                dw_gu=(x.transpose(1, 2) @ dgu).to(dt),
                dw_d=((a * up).transpose(1, 2) @ dy).to(dt))


def _to_codes(x, fmt, g):
    """Codes uint8 [rows, k] (sign in bit 3) and scales uint8 [rows, k / block]."""
    b = x.float().view(x.shape[0], -1, BLOCK[fmt])
    top = b.abs().amax(-1)
    if fmt == "mx":   # the smallest power of two that 6 of reach the largest value
        m, e = torch.frexp(top)
        e = torch.where(top > 0, e - 3 + (m > 0.75).int(), -127).clamp(-127, 127)
        scale, unit = (e + 127).to(torch.uint8), torch.ldexp(torch.ones_like(top).double(), e)
    else:
        one = torch.ones(1, device=x.device) if g is None else g
        s8 = (top / (6 * one)).clamp(max=448).to(torch.float8_e4m3fn)
        scale, unit = s8.view(torch.uint8), (s8.float() * one).double()
    q = (b.double() / torch.where(unit > 0, unit, 1.0)[..., None]).float()  # next to a border: 64 bits
    q = torch.where(unit[..., None] > 0, q, 0.0)
    a = q.abs()       # ties go to the even code
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
            + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5).byte())
    return (code | (torch.signbit(q).byte() << 3)).view(x.shape), scale


def _from_codes(code, scale, fmt, g):
    """What codes [.., k] and scales [.., k / block] stand for, in 32 bits."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=code.device)
    v = torch.cat([table, -table])[code.int()]
    if fmt == "mx":
        unit = torch.where(scale == 0, 2.0 ** -127, (scale.int() << 23).view(torch.float32))
    else:
        unit = scale.contiguous().view(torch.float8_e4m3fn).float()
    if g is not None:
        unit = unit * g
    return (v.unflatten(-1, (-1, BLOCK[fmt])) * unit[..., None]).flatten(-2)


def _plain_quant(s):
    c = s["case"]
    code, scale = _to_codes(s["x"], c["fmt"], s["gscale"])
    return dict(values=_from_codes(code, scale, c["fmt"], s["gscale"]).to(s["x"].dtype))


def _unpacked(s):
    """The weights [E, m, k] in 32 bits."""
    c = s["case"]
    code = torch.stack([s["wc"] & 15, s["wc"] >> 4], -1).flatten(-2)
    gw = s["gw"][:, None, None] if s["gw"] is not None else None
    return _from_codes(code, s["ws"][..., :c["k"] // BLOCK[c["fmt"]]], c["fmt"], gw)


def _plain_linear(s):
    c = s["case"]
    x = s["x"].float()
    if c["act"] != "none":
        gate, up = x.split(c["k"], -1)
        x = _act(c["act"], gate)[0] * up
    code, scale = _to_codes(x, c["fmt"], s["gx"])
    x = _from_codes(code, scale, c["fmt"], s["gx"])
    y = _together(s, x) @ _unpacked(s).transpose(1, 2)
    return dict(y=_apart(s, y).to(s["y"].dtype))


# -------------------------------------------------------------------- run --
def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "ffn":
        return _plain_ffn_back(s) if c["back"] else _plain_ffn(s)
    return _plain_quant(s) if c["op"] == "quant" else _plain_linear(s)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _run_own(s, c):
    from symmetric_memory_moe_gb300 import abi
    dt, n = CODES[c["dtype"]], c["n"]
    if c["op"] == "ffn":
        E, D, F, act = c["E"], c["D"], c["F"], ACTS[c["act"]]
        if c["back"]:
            abi.moe_expert_ffn_backward(
                s["heap"].handle, _ptr(s["dy"]), D, _ptr(s["x"]), D, _ptr(s["gu"]),
                _ptr(s["counts"]), _ptr(s["w_gu"]), _ptr(s["w_d"]), act, dt, n, E, D, F,
                _ptr(s["dx"]), D, _ptr(s["dw_gu"]), _ptr(s["dw_d"]), _ptr(s["scratch"]))
            return {k: s[k] for k in ("dx", "dw_gu", "dw_d")}
        abi.moe_expert_ffn(s["heap"].handle, _ptr(s["x"]), D, _ptr(s["counts"]), _ptr(s["w_gu"]),
                           _ptr(s["w_d"]), act, dt, n, E, D, F, _ptr(s["gu"]), _ptr(s["y"]), D,
                           _ptr(s["scratch"]))
        return {k: s[k] for k in ("gu", "y")}
    k, fmt, kc, ks = c["k"], FORMATS[c["fmt"]], s["xc"].shape[1], s["xs"].shape[1]

    def to_pack(g):  # blocks of 32 are packed without a tensor's own scale
        return _ptr(g) if c["fmt"] == "nv" else None

    if c["op"] == "quant":
        abi.moe_fp4_quantize(_ptr(s["x"]), k, ACTS["none"], dt, fmt, to_pack(s["gscale"]), n,
                             k, _ptr(s["xc"]), kc, _ptr(s["xs"]), ks)
        abi.moe_fp4_dequantize(_ptr(s["xc"]), kc, _ptr(s["xs"]), ks, fmt, _ptr(s["gscale"]), n, k,
                               dt, _ptr(s["values"]), k)
        return dict(values=s["values"])
    abi.moe_fp4_quantize(_ptr(s["x"]), s["x"].shape[1], ACTS[c["act"]], dt, fmt, to_pack(s["gx"]),
                         n, k, _ptr(s["xc"]), kc, _ptr(s["xs"]), ks)
    abi.moe_fp4_expert_matmul(s["heap"].handle, _ptr(s["xc"]), kc, _ptr(s["xs"]), ks,
                              _ptr(s["wc"]), kc, _ptr(s["ws"]), ks, _ptr(s["counts"]),
                              _ptr(s["gx"]), _ptr(s["gw"]), fmt, dt, n, c["E"], k, c["m"],
                              _ptr(s["y"]), c["m"])
    return dict(y=s["y"])


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    """The operators' definitions in 64 bits, one expert after the other."""
    c, s = case, prepare(case, seed)
    if c["op"] == "quant":
        return dict(values=_exact_rounded(s["x"].double(), c["fmt"], s["gscale"]))
    n, ends = c["n"], s["counts"].cumsum(0).tolist()
    runs = [(e, ([0] + ends)[e], ends[e]) for e in range(c["E"])]

    def zeros(*shape):
        return torch.zeros(*shape, dtype=torch.float64, device="cuda")

    if c["op"] == "linear":
        x, y = s["x"].double(), zeros(n, c["m"])
        if c["act"] != "none":
            x = _exact_act(c["act"], x[:, :c["k"]])[0] * x[:, c["k"]:]
        x = _exact_rounded(x, c["fmt"], s["gx"])
        for e, a, b in runs:
            w = _exact_values(s["wc"][e], s["ws"][e], c["fmt"], c["k"])
            y[a:b] = x[a:b] @ w.t() * (1.0 if s["gw"] is None else s["gw"][e].double())
        return dict(y=y)
    F = c["F"]
    if not c["back"]:
        gu, y = zeros(n, 2 * F), zeros(n, c["D"])
        for e, a, b in runs:
            gu[a:b] = s["x"][a:b].double() @ s["w_gu"][e].double()
            h = _exact_act(c["act"], gu[a:b, :F])[0] * gu[a:b, F:]
            y[a:b] = h @ s["w_d"][e].double()
        return dict(gu=gu, y=y)
    dx, dw_gu, dw_d = zeros(n, c["D"]), zeros(*s["w_gu"].shape), zeros(*s["w_d"].shape)
    for e, a, b in runs:
        dy, gu = s["dy"][a:b].double(), s["gu"][a:b].double()
        f, df = _exact_act(c["act"], gu[:, :F])
        dw_d[e] = (f * gu[:, F:]).t() @ dy
        dh = dy @ s["w_d"][e].double().t()
        for at, d in ((0, dh * gu[:, F:] * df), (F, dh * f)):
            dw_gu[e][:, at:at + F] = s["x"][a:b].double().t() @ d
            dx[a:b] += d @ s["w_gu"][e][:, at:at + F].double().t()
    return dict(dx=dx, dw_gu=dw_gu, dw_d=dw_d)


def _exact_act(name, g):
    if name == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * (1 - p)
    p = torch.special.ndtr(g)       # the normal distribution's, whose density is p's derivative
    return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def _exact_rounded(x, fmt, g):
    """x [rows, k] at the nearest 4-bit values of its blocks' scales."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    b = x.reshape(len(x), -1, BLOCK[fmt])
    top = b.abs().amax(-1, keepdim=True)
    if fmt == "mx":
        unit = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-300) / 6)).clamp(-127, 127))
        unit = torch.where(top > 6 * unit, 2 * unit, unit)     # log2's own rounding
        unit = torch.where(top <= 3 * unit, unit / 2, unit).clamp(min=2.0 ** -127)
    else:
        one = 1.0 if g is None else g.double()
        s8 = (top / (6 * one)).clamp(max=448).float().to(torch.float8_e4m3fn)
        unit = s8.double() * one
    q = b.abs() / torch.where(unit > 0, unit, 1.0)
    q = torch.where(unit > 0, q, 0.0)
    lo = (q[..., None] >= grid).sum(-1) - 1                    # the value below, and above
    hi = (lo + 1).clamp(max=7)
    down, up = q - grid[lo], grid[hi] - q
    at = torch.where((up < down) | ((up == down) & (lo % 2 == 1)), hi, lo)
    return (torch.sign(b) * grid[at] * unit).reshape(x.shape)


def _exact_values(codes, scales, fmt, k):
    """[rows, k] of packed rows, from the fields of each code."""
    code = torch.stack([codes % 16, codes // 16], -1).reshape(len(codes), k).long()
    sign, exponent, half = code // 8, code // 2 % 4, code % 2
    size = torch.where(exponent == 0, 0.5 * half, (1 + 0.5 * half) * 2.0 ** (exponent - 1))
    v = size.double() * (1 - 2 * sign)
    s = scales[:, :k // BLOCK[fmt]].long()
    if fmt == "mx":
        unit = 2.0 ** (s - 127).double()
    else:
        e, m = s // 8, (s % 8).double()
        unit = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7).double())
    return v * unit.repeat_interleave(BLOCK[fmt], -1)
