"""64-bit references of the MoE block operators, written from their
definitions in include/symm_a2a.h, with the magnitudes that the tests'
error bounds are made of.  Plain tensors in, plain tensors out, on any
device; nothing of the library is used."""
import math

import torch

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"f16": 0, "bf16": 1, "f32": 2}
U32 = 2.0 ** -24                                        # one rounding of a float
U_OUT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -23}
TINY = {"f16": 2.0 ** -24, "bf16": 1e-38, "f32": 1e-37}  # half-precision subnormal step
FLT_MAX = torch.finfo(torch.float32).max


def clean(logits):
    l = logits.double()
    l = torch.where(torch.isnan(l), -math.inf, l)
    return l.clamp(max=FLT_MAX)


def route(logits, mask, k, renorm, scale):
    """logits [G, T, E], mask [G, T] or None."""
    l = clean(logits)
    G, T, E = l.shape
    valid = (l > -math.inf).any(-1)
    if mask is not None:
        valid &= mask != 0
    m = torch.where(valid, l.amax(-1), 0.0)
    e = torch.where(valid[..., None], torch.exp(l - m[..., None]), 0.0)
    s = e.sum(-1)
    p = e / torch.where(valid, s, 1.0)[..., None]
    experts = torch.full((G, T, k), -1, dtype=torch.int32)
    lc, vc = l.cpu(), valid.cpu()
    for g in range(G):
        for t in range(T):
            if not vc[g, t]:
                continue
            row = lc[g, t].tolist()
            order = sorted((i for i in range(E) if row[i] > -math.inf), key=lambda i: (-row[i], i))
            for j, i in enumerate(order[:k]):
                experts[g, t, j] = i
    experts = experts.to(l.device)
    weights, loss, counts, n = soft(l, experts, valid, p, s, m, k, renorm, scale)
    return dict(experts=experts, weights=weights, counts=counts.to(torch.int32),
                tokens=n.to(torch.int32), stats=torch.stack([m, s], -1), loss=loss, p=p,
                valid=valid)


def soft(l, experts, valid, p, s, m, k, renorm, scale):
    E = l.shape[-1]
    ok = experts >= 0
    idx = experts.clamp(min=0).long()
    u = torch.where(ok, p.gather(-1, idx), 0.0)
    tot = u.sum(-1) if renorm else torch.ones_like(u[..., 0])
    weights = scale * u / torch.where(valid, tot, 1.0)[..., None]
    hot = torch.zeros_like(p).scatter_add_(-1, idx, ok.double())
    counts, n = hot.sum(1), valid.sum(-1)
    n1 = n.clamp(min=1).double()
    lse = torch.where(valid, m + torch.log(torch.where(valid, s, 1.0)), 0.0)
    loss = torch.stack([E / (k * n1 ** 2) * (counts * p.sum(1)).sum(-1),
                        (lse ** 2).sum(-1) / n1], -1)
    return weights, loss, counts, n


def route_scalar(l, experts, counts, n, valid, k, renorm, scale, dweights, dloss):
    """The scalar whose gradient moe_route_backward returns, of 64-bit logits
    (finite or -inf) with the choice and the counts held fixed."""
    E = l.shape[-1]
    safe = torch.where(valid[..., None], l, 0.0)
    p = torch.softmax(safe, -1) * valid[..., None]
    lse = torch.logsumexp(safe, -1) * valid
    ok = experts >= 0
    u = torch.where(ok, p.gather(-1, experts.clamp(min=0).long()), 0.0)
    tot = u.sum(-1, keepdim=True) if renorm else torch.ones_like(u[..., :1])
    w = scale * u / torch.where(valid[..., None], tot, 1.0)
    n1 = n.clamp(min=1).double()
    balance = E / (k * n1 ** 2) * (counts.double() * p.sum(1)).sum(-1)
    z = (lse ** 2).sum(-1) / n1
    return (w * dweights.double()).sum() + (balance * dloss[:, 0].double()).sum() + \
        (z * dloss[:, 1].double()).sum()


def route_grad(l, experts, counts, n, valid, k, renorm, scale, dweights, dloss):
    """The gradient's formula and, second, the sum of the magnitudes of its terms."""
    E = l.shape[-1]
    safe = torch.where(valid[..., None], l, 0.0)
    p = torch.softmax(safe, -1) * valid[..., None]
    lse = torch.logsumexp(safe, -1) * valid
    n1 = n.clamp(min=1).double()[:, None]
    a = (dloss[:, :1].double() * counts.double() * E / k / n1 ** 2)[:, None, :].expand_as(p)
    ok = experts >= 0
    idx = experts.clamp(min=0).long()
    dw = torch.where(ok, scale * dweights.double(), 0.0)
    u = torch.where(ok, p.gather(-1, idx), 0.0)
    cz = (2 * dloss[:, 1:].double() / n1)[..., None]
    if not renorm:
        a = a.scatter_add(-1, idx, dw)
    d = p * (a - (p * a).sum(-1, keepdim=True) + cz * lse[..., None])
    mag = p * (a.abs() + (p * a.abs()).sum(-1, keepdim=True) + cz.abs() * (lse.abs() + 1)[..., None])
    if renorm:
        q = u / torch.where(valid, u.sum(-1), 1.0)[..., None]
        mean = (q * dw).sum(-1, keepdim=True)
        d = d.scatter_add(-1, idx, torch.where(ok, q * (dw - mean), 0.0))
        mag = mag.scatter_add(-1, idx, q * (dw.abs() + (q * dw.abs()).sum(-1, keepdim=True)))
    return d, mag


# ------------------------------------------------------------------- norm --
def gather(y, rows, yrows, T, k):
    """[T, k, D] rows (0 where dropped) and which are there."""
    if rows is None:
        rows = torch.arange(T * k, device=y.device).view(T, k)
    rows = rows.long()
    have = (rows >= 0) & (rows < yrows)
    return torch.where(have[..., None], y.double()[rows.clamp(0, yrows - 1)], 0.0), have, rows


def norm(i, eps):
    """i: dict of x [T, D], y [yrows, D] or None, rows, weights, gate, res,
    w_post, w_pre (None where absent), k.  Returns xo, h, rstd and the bounds
    exo, eh on the error of a 32-bit evaluation (before its last rounding):
    sums of at most 100 dependent additions each."""
    x = i["x"].double()
    T, D = x.shape
    one = torch.ones(T, 1, dtype=torch.float64, device=x.device)
    r1 = one
    exo = torch.zeros_like(x)
    if i["y"] is not None:
        Y, have, _ = gather(i["y"], i["rows"], i["y"].shape[0], T, i["k"])
        w = torch.where(have, i["weights"].double() if i["weights"] is not None else 1.0, 0.0)
        y = (w[..., None] * Y).sum(1)
        ey = (i["k"] + 1) * U32 * (w[..., None] * Y).abs().sum(1)
        wp, d1 = 1.0, 0.0
        if i["w_post"] is not None:
            r1 = 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
            d1 = (y.abs() * ey).sum(-1, keepdim=True) / ((y * y).sum(-1, keepdim=True) + D * eps) \
                + 100 * U32
            wp = i["w_post"].double()
        gate = i["gate"].double()[:, None] if i["gate"] is not None else 1.0
        res = i["res"].double() if i["res"] is not None else 1.0
        u = gate * wp * y * r1
        xo = res * x + u
        exo = abs(gate * wp) * r1 * (ey + y.abs() * d1) + 6 * U32 * (u.abs() + (res * x).abs())
    else:
        xo = x
    out = dict(xo=xo, exo=exo, h=None, rstd=torch.cat([r1, one], 1))
    if i["w_pre"] is not None:
        r2 = 1 / torch.sqrt((xo * xo).mean(-1, keepdim=True) + eps)
        d2 = (xo.abs() * exo).sum(-1, keepdim=True) / ((xo * xo).sum(-1, keepdim=True) + D * eps) \
            + 100 * U32
        wpre = i["w_pre"].double()
        h = xo * r2 * wpre
        out.update(h=h, eh=wpre.abs() * r2 * (exo + xo.abs() * d2) + 4 * U32 * h.abs(),
                   rstd=torch.cat([r1, r2], 1))
    return out


def norm_grad(i, z, rstd, dxo, dh):
    """The gradients' formulas at the saved xo (z) and rstd; beside each, the
    sum of the magnitudes of its terms (name + "_mag")."""
    z = z.double()
    x = i["x"].double()
    T, D = z.shape
    r1, r2 = rstd.double()[:, :1], rstd.double()[:, 1:]
    zero = torch.zeros_like(z)
    dz = dxo.double() if dxo is not None else zero
    mz = dz.abs()
    o = {}
    if dh is not None:
        q = dh.double() * i["w_pre"].double()
        dz = dz + r2 * (q - z * r2 ** 2 * (q * z).mean(-1, keepdim=True))
        mz = mz + r2 * (q.abs() + z.abs() * r2 ** 2 * (q * z).abs().mean(-1, keepdim=True))
        o["dw_pre"] = (dh.double() * z * r2).sum(0)
        o["dw_pre_mag"] = (dh.double() * z * r2).abs().sum(0)
    res = i["res"].double() if i["res"] is not None else torch.ones(D, dtype=torch.float64,
                                                                  device=z.device)
    o["dx"], o["dx_mag"] = res * dz, res.abs() * mz
    if i["y"] is None:
        return o
    o["dres"], o["dres_mag"] = (dz * x).sum(0), (mz * x.abs()).sum(0)
    Y, have, rows = gather(i["y"], i["rows"], i["y"].shape[0], T, i["k"])
    w = torch.where(have, i["weights"].double() if i["weights"] is not None else 1.0, 0.0)
    y, ay = (w[..., None] * Y).sum(1), (w[..., None] * Y).abs().sum(1)
    post = i["w_post"] is not None
    wp = i["w_post"].double() if post else torch.ones_like(res)
    gate = i["gate"].double()[:, None] if i["gate"] is not None else torch.ones_like(r1)
    n, an = y * r1, ay * r1
    o["dgate"], o["dgate_mag"] = (dz * n * wp).sum(-1), (mz * an * wp.abs()).sum(-1)
    o["dw_post"] = (gate * dz * n).sum(0)
    o["dw_post_mag"] = (gate.abs() * mz * an).sum(0)
    dn, mdn = gate * dz * wp, gate.abs() * mz * wp.abs()
    if post:
        dy = r1 * (dn - n * (dn * n).mean(-1, keepdim=True))
        mdy = r1 * (mdn + an * (mdn * an).mean(-1, keepdim=True))
    else:
        dy, mdy = dn, mdn
    o["dweights"] = (dy[:, None] * Y).sum(-1)
    o["dweights_mag"] = (mdy[:, None] * Y.abs()).sum(-1)
    o["dy"] = torch.full(i["y"].shape, math.nan, dtype=torch.float64, device=z.device)
    o["dy_mag"] = torch.zeros_like(o["dy"])
    t, j = have.nonzero(as_tuple=True)
    o["dy"][rows[t, j]] = w[t, j, None] * dy[t]
    o["dy_mag"][rows[t, j]] = w[t, j, None].abs() * mdy[t]
    return o


def norm_scalar(x, Y, w, gate, res, w_post, w_pre, have, eps, dxo, dh):
    """<dxo, xo> + <dh, h> of 64-bit inputs; Y [T, k, D]."""
    y = (torch.where(have, w, 0.0)[..., None] * Y).sum(1)
    u = w_post * y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) if w_post is not None else y
    xo = res * x + gate[:, None] * u
    h = w_pre * xo / torch.sqrt((xo * xo).mean(-1, keepdim=True) + eps)
    return (xo * dxo).sum() + (h * dh).sum()
