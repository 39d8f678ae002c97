"""64-bit references of the experts' feed-forward and of 4-bit rows, written
from their definitions in include/symm_a2a.h, with the magnitudes that the
tests' error bounds are made of.  Nothing of the library is used."""
import math

import torch

U23 = 2.0 ** -23
SLOPE = 1.13  # of both activations, at most: silu 1.0998, gelu 1.1290


def act(name, g):
    """act(g) and its derivative."""
    if name == "silu":
        p = torch.sigmoid(g)
        return g * p, p * (1 + g * (1 - p))
    p = torch.special.ndtr(g)
    return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def act_error(g):
    """Bounds on a 32-bit evaluation of act(g) and its derivative: exponentials of x are within
    (2 + 1.2 |x|) ulp with |x| at most |g| or g^2 / 2 (where exp(-g^2 / 2) |g| x is below 1), Phi
    within 5 ulp, and at most 6 further roundings."""
    r = (13 + 1.2 * g.abs()) * U23
    return r * g.abs(), r * (1 + g.abs())


def runs(counts):
    ends = torch.cumsum(counts.long(), 0).tolist()
    return list(zip(range(len(ends)), [0] + ends[:-1], ends))


def ffn(x, counts, w_gu, w_d, name, u_out, tiny):
    """gu, y and their bounds for a 32-bit evaluation whose sums of k terms err by k 2^-23 of the
    sum of magnitudes, and whose h, gu and y are rounded to the type once."""
    F = w_d.shape[1]
    out = {k: [] for k in ("gu", "y", "egu", "ey")}
    for e, a, b in runs(counts):
        X, G, Wd = x[a:b].double(), w_gu[e].double(), w_d[e].double()
        gu = X @ G
        eg = (G.shape[0] + 8) * U23 * (X.abs() @ G.abs())
        g, u = gu[:, :F], gu[:, F:]
        f, _ = act(name, g)
        h = f * u
        ef = SLOPE * eg[:, :F] + act_error(g)[0]
        eh = ef * u.abs() + (f.abs() + ef) * eg[:, F:]
        eh = eh + u_out * (h.abs() + eh) + tiny
        y = h @ Wd
        ey = eh @ Wd.abs() + (F + 8) * U23 * ((h.abs() + eh) @ Wd.abs())
        for k, v in (("gu", gu), ("y", y), ("egu", eg * (1 + u_out) + u_out * gu.abs() + tiny),
                     ("ey", ey * (1 + u_out) + u_out * y.abs() + tiny)):
            out[k].append(v)
    return {k: torch.cat(v) for k, v in out.items()}


def ffn_grad(dy, x, gu, counts, w_gu, w_d, name, u_out, tiny):
    """dx, dw_gu, dw_d from the saved gu, and their bounds, as ``ffn``."""
    E, F, D = w_d.shape
    o = dict(dx=[], edx=[], dw_gu=[], edw_gu=[], dw_d=[], edw_d=[])
    for e, a, b in runs(counts):
        Y, X, GU = dy[a:b].double(), x[a:b].double(), gu[a:b].double()
        G, Wd = w_gu[e].double(), w_d[e].double()
        g, u = GU[:, :F], GU[:, F:]
        f, df = act(name, g)
        ef, edf = act_error(g)
        dh = Y @ Wd.t()
        edh = (D + 8) * U23 * (Y.abs() @ Wd.abs().t())

        def product(p, ep, q, eq):  # of two factors with errors
            return p * q, ep * q.abs() + (p.abs() + ep) * eq

        def rounded(v, ev):
            return v, ev + u_out * (v.abs() + ev) + tiny

        h, eh = rounded(*product(f, ef, u, 4 * U23 * u.abs()))
        t, et = product(dh, edh, u, 4 * U23 * u.abs())
        dg, edg = rounded(*product(t, et, df, edf + 4 * U23 * df.abs()))
        du, edu = rounded(*product(dh, edh, f, ef + 4 * U23 * f.abs()))
        d, ed = torch.cat([dg, du], 1), torch.cat([edg, edu], 1)
        n = b - a

        def summed(v, ev, k, mag):
            ev = ev + (k + 8) * U23 * mag
            return v, ev * (1 + u_out) + u_out * v.abs() + tiny

        for name_, (v, ev) in (
                ("dx", summed(d @ G.t(), ed @ G.abs().t(), 2 * F, (d.abs() + ed) @ G.abs().t())),
                ("dw_gu", summed(X.t() @ d, X.abs().t() @ ed, n, X.abs().t() @ (d.abs() + ed))),
                ("dw_d", summed(h.t() @ Y, eh.t() @ Y.abs(), n, (h.abs() + eh).t() @ Y.abs()))):
            o[name_].append(v)
            o["e" + name_].append(ev)
    cat = {k: torch.cat(v) if k.endswith("dx") else torch.stack(v) for k, v in o.items()}
    return cat


# ------------------------------------------------------------ 4-bit rows --
GRID = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
BLOCK = {"mx": 32, "nv": 16}


def nearest(q):
    """Codes 0 .. 7 of magnitudes q in 64 bits: the nearest value, ties to the even code."""
    grid = GRID.to(q.device)
    lo = (torch.bucketize(q, grid, right=True) - 1).clamp(0, 7)
    hi = (lo + 1).clamp(max=7)
    down, up = q - grid[lo], grid[hi] - q
    return torch.where((up < down) | ((up == down) & (lo % 2 == 1)), hi, lo)


def unit_of(scale, fmt, g):
    """What a block's scale byte stands for, with the tensor's own scale g (None: 1)."""
    if fmt == "mx":
        u = torch.ldexp(torch.ones(scale.shape, dtype=torch.float64), scale.cpu().int() - 127)
        u[scale.cpu() == 255] = math.nan
        u = u.to(scale.device)
        return u if g is None else (u.float() * g).double()
    u = scale.contiguous().view(torch.float8_e4m3fn).float()
    return (u if g is None else u * g).double()


def quantize(x, fmt, g):
    """Codes [n, k] uint8 (sign in bit 3) and scales [n, k / block] uint8 of x in 64 bits."""
    b = x.double().unflatten(-1, (-1, BLOCK[fmt]))
    top = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    top = torch.where(bad, 0.0, top)
    if fmt == "mx":
        s = torch.full_like(top, -127, dtype=torch.int64)
        for e in range(-126, 128):  # the smallest that reaches the largest value
            s = torch.where(top > 6 * 2.0 ** (e - 1), e, s)
        scale = (s + 127).to(torch.uint8)
        scale[bad] = 255
    else:
        six = 6 * (torch.ones(1, device=x.device) if g is None else g)
        scale = (top.float() / six).clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8)
        scale = torch.where(bad, torch.full_like(scale, 0x7f), scale)
    unit = unit_of(scale, fmt, None if fmt == "mx" else g)[..., None]
    q = (b / unit).float().double()  # the quotient is rounded to 32 bits
    code = nearest(torch.where((unit > 0) & ~bad[..., None], q.abs(), 0.0))
    code = torch.where(torch.signbit(b) & ~bad[..., None] & (unit > 0), code + 8, code)
    return code.flatten(-2).to(torch.uint8), scale


def values(code, scale, fmt, g):
    """What codes and scales stand for, in 64 bits."""
    v = GRID.to(code.device)[(code & 7).long()] * torch.where(code > 7, -1.0, 1.0)
    return (v.unflatten(-1, (-1, BLOCK[fmt])) * unit_of(scale, fmt, g)[..., None]).flatten(-2)


def pack(code):
    c = code.unflatten(-1, (-1, 2))
    return c[..., 0] | (c[..., 1] << 4)


def unpack(codes):
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
