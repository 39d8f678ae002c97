"""The operators around the all-to-all of a mixture-of-experts block, as cases to measure.

* ``route``: the router's choice of k experts per token, its weights, the
  per-expert counts and the balance and z losses, and the gradient of all of
  it with respect to the logits;
* ``norm``: the weighted sum of a token's expert rows, the norm after the
  block, its gate and residual scale, and the norm before the next block, in
  one pass, and its gradients;
* ``adapter``: a shared projection with a low-rank adapter per request.

``run`` computes them in their plain form (elementary torch operations in 32
bits), or, where ``own`` is true, by the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CODES = {"f16": 0, "bf16": 1, "f32": 2}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
FLT_MAX = torch.finfo(torch.float32).max
EPS = 1e-6


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # the router of one decoding step: 8 tokens, latency only
        dict(name="route, one decoding step", op="route", back=False, G=1, T=8, E=256, k=8,
             dtype="f32", renorm=True, holes=False),
        # a training step's router: 8 PEs of 4096 tokens, 256 experts
        dict(name="route, training step", op="route", back=False, G=8, T=4096, E=256, k=8,
             dtype="bf16", renorm=True, holes=False),
        # its gradient, logits kept in 32 bits
        dict(name="route, training step, backward", op="route", back=True, G=8, T=4096, E=256, k=8,
             dtype="f32", renorm=True, holes=False),
        # padded sequences of odd length, few experts, some of them closed
        dict(name="route, padded sequences", op="route", back=False, G=3, T=1531, E=60, k=4,
             dtype="f16", renorm=False, holes=True),
        # one decoding step: 16 tokens, each with 8 expert rows of 7168
        dict(name="norm, one decoding step", op="norm", back=False, T=16, D=7168, k=8,
             dtype="bf16", post=True, holes=False),
        # a training step: 8192 tokens and their 65,536 expert rows
        dict(name="norm, training step", op="norm", back=False, T=8192, D=7168, k=8,
             dtype="bf16", post=True, holes=False),
        # its gradients
        dict(name="norm, training step, backward", op="norm", back=True, T=4096, D=7168, k=8,
             dtype="bf16", post=True, holes=False),
        # odd width and count, dropped rows, 32 bits
        dict(name="norm, dropped rows, backward", op="norm", back=True, T=1531, D=999, k=2,
             dtype="f32", post=True, holes=True),
        # one request, one token: the weight matrix is all there is to read
        dict(name="adapters, one token", op="adapter", T=1, K=8192, N=8192, R=4, r=16,
             dtype="bf16", runs=1),
        # one token each of 64 requests
        dict(name="adapters, 64 requests", op="adapter", T=64, K=7168, N=2048, R=32, r=16,
             dtype="bf16", runs=64),
        # prompts of 8 requests, 8192 tokens in all
        dict(name="adapters, prompts", op="adapter", T=8192, K=4096, N=4096, R=8, r=32,
             dtype="bf16", runs=8),
        # odd sizes, some requests without an adapter
        dict(name="adapters, odd sizes", op="adapter", T=333, K=1000, N=2056, R=5, r=8,
             dtype="f16", runs=9),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "norm", "adapter"])
    if op == "route":
        E = _log(rng, 8, 512)
        return dict(op=op, back=rng.random() < 0.5, G=rng.randint(1, 8), T=_log(rng, 1, 4096), E=E,
                    k=rng.randint(1, min(8, E)), dtype=rng.choice(sorted(DTYPES)),
                    renorm=rng.random() < 0.5, holes=rng.random() < 0.5)
    if op == "norm":
        back, D, k = rng.random() < 0.5, _log(rng, 64, 8192), rng.randint(1, 8)
        dtype = rng.choice(sorted(DTYPES))
        row = (2 * k + 5 if back else k + 3) * D * BYTES[dtype]
        return dict(op=op, back=back, T=_log(rng, 1, min(8192, (1 << 30) // row)), D=D, k=k,
                    dtype=dtype, post=rng.random() < 0.75, holes=rng.random() < 0.5)
    K, N = 8 * _log(rng, 8, 1024), 8 * _log(rng, 8, 1024)
    T = _log(rng, 1, min(8192, (1 << 36) // (K * N)))
    return dict(op=op, T=T, K=K, N=N, R=rng.randint(1, 32), r=8 * rng.randint(1, 8),
                dtype=rng.choice(["bf16", "f16"]), runs=_log(rng, 1, T))


def work(case):
    c = case
    if c["op"] == "route":
        n, es = c["G"] * c["T"], BYTES[c["dtype"]]
        side = n * (8 * c["k"] + 8) + c["G"] * (c["E"] * 4 + 12)
        if c["back"]:
            return {"bytes": 2 * n * c["E"] * es + side, "flops": 8 * n * c["E"]}
        return {"bytes": n * c["E"] * es + n + side, "flops": 6 * n * c["E"]}
    if c["op"] == "norm":
        T, D, k, es = c["T"], c["D"], c["k"], BYTES[c["dtype"]]
        if c["back"]:
            return {"bytes": (2 * k + 5) * T * D * es + T * (12 * k + 16) + 24 * D,
                    "flops": (6 * k + 30) * T * D}
        return {"bytes": (k + 3) * T * D * es + T * (8 * k + 12) + 12 * D,
                "flops": (2 * k + 10) * T * D}
    T, K, N, r, es = c["T"], c["K"], c["N"], c["r"], BYTES[c["dtype"]]
    used = min(c["R"], c["runs"])
    return {"bytes": es * (T * K + K * N + used * r * (K + N) + T * N) + 4 * T,
            "flops": 2 * T * K * N + 2 * T * r * (K + N)}


# ----------------------------------------------------------------- inputs --
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)


def _route_inputs(c, seed):
    g = _gen(seed)
    G, T, E, dt = c["G"], c["T"], c["E"], DTYPES[c["dtype"]]
    # experts of uneven popularity, as a router in training has them
    logits = (1.5 * _randn(g, G, T, E) + _randn(g, E)).to(dt)
    mask = torch.ones(G, T, dtype=torch.uint8, device="cuda")
    if c["holes"]:
        keep = (T * (0.4 + 0.6 * _rand(g, G, 1))).long().clamp(min=1)
        mask = (torch.arange(T, device="cuda") < keep).to(torch.uint8)
        logits[:, :, (_rand(g, E) < 0.1) & (torch.arange(E, device="cuda") >= c["k"])] = -math.inf
        logits[~mask.bool()] = math.nan  # what stands in padding must not matter
        if T >= 4:
            logits[:, T // 2] = -math.inf  # a row that its mask leaves empty
    return logits, mask


def _norm_inputs(c, seed):
    g = _gen(seed)
    T, D, k, dt = c["T"], c["D"], c["k"], DTYPES[c["dtype"]]
    x = _randn(g, T, D).to(dt)
    y = torch.empty(T * k, D, dtype=dt, device="cuda").normal_(generator=g)
    rows = torch.randperm(T * k, generator=g, device="cuda").view(T, k).to(torch.int32)
    if c["holes"]:
        drop = _rand(g, T, k) < 0.1      # rows dropped on the way
        if T < 64:
            drop[:, :2] = False
        rows[drop] = -1
        if T >= 4:
            rows[T // 2] = -1            # a token whose rows were all dropped
    # one row per token needs no weight: the norm would take it out again
    return dict(x=x, y=y, rows=rows, weights=torch.softmax(_randn(g, T, k), -1) if k > 1 else None,
                gate=torch.sigmoid(_randn(g, T)), res=1 + 0.1 * _randn(g, D),
                w_post=1 + 0.1 * _randn(g, D) if c["post"] else None,
                w_pre=1 + 0.1 * _randn(g, D))


def _adapter_inputs(c, seed):
    g = _gen(seed)
    T, K, N, R, r, dt = c["T"], c["K"], c["N"], c["R"], c["r"], DTYPES[c["dtype"]]
    x = _randn(g, T, K).to(dt)
    w = torch.empty(K, N, dtype=dt, device="cuda").normal_(generator=g).mul_(K ** -0.5)
    a = (_randn(g, R, K, r) * K ** -0.5).to(dt)
    b = (_randn(g, R, r, N) * r ** -0.5).to(dt)
    scale = 0.5 + _rand(g, R)
    # `runs` requests of consecutive tokens; about one in sixteen has no adapter
    start = torch.zeros(T, dtype=torch.int64, device="cuda")
    start[torch.randperm(T, generator=g, device="cuda")[:c["runs"] - 1]] = 1
    start[0] = 0
    of_run = torch.randint(0, R, (c["runs"],), generator=g, device="cuda")
    if c["runs"] > 1:
        of_run[_rand(g, c["runs"]) < 1 / 16] = -1
    return dict(x=x, w=w, a=a, b=b, scale=scale, ids=of_run[start.cumsum(0)].to(torch.int32))


def prepare(case, seed):
    c, dev = case, "cuda"
    s = dict(case=c)
    if c["op"] == "route":
        G, T, E, k = c["G"], c["T"], c["E"], c["k"]
        s["logits"], s["mask"] = _route_inputs(c, seed)
        if c["back"]:
            s.update(_plain_route(s))  # what the forward pass left
            g = _gen(seed + 1)
            s["dweights"], s["dloss"] = _randn(g, G, T, k), 0.5 + _rand(g, G, 2)
            s["dlogits"] = torch.empty_like(s["logits"])
        else:
            s["experts"] = torch.empty(G, T, k, dtype=torch.int32, device=dev)
            s["weights"] = torch.empty(G, T, k, device=dev)
            s["counts"] = torch.empty(G, E, dtype=torch.int32, device=dev)
            s["tokens"] = torch.empty(G, dtype=torch.int32, device=dev)
            s["stats"], s["loss"] = torch.empty(G, T, 2, device=dev), torch.empty(G, 2, device=dev)
    elif c["op"] == "norm":
        T, D, k = c["T"], c["D"], c["k"]
        s.update(_norm_inputs(c, seed))
        if c["back"]:
            f = _plain_norm(s)
            s["xo"], s["rstd"] = f["xo"], f["rstd"]
            g = _gen(seed + 1)
            s["dxo"], s["dh"] = (_randn(g, T, D).to(s["x"].dtype) for _ in range(2))
            s["dx"], s["dy"] = torch.empty_like(s["x"]), torch.zeros_like(s["y"])
            s["dweights"] = torch.empty(T, k, device=dev) if k > 1 else None
            s["dgate"] = torch.empty(T, device=dev)
            s["dres"], s["dw_post"], s["dw_pre"] = torch.zeros(3, D, device=dev)
        else:
            s["xo"], s["h"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
            s["rstd"] = torch.empty(T, 2, device=dev)
    else:
        s.update(_adapter_inputs(c, seed))
        s["y"] = torch.empty(c["T"], c["N"], dtype=s["x"].dtype, device=dev)
    if own:  # the workspace and the heap handle that a user's program keeps
        from symmetric_memory_moe_gb300 import abi
        from symmetric_memory_moe_gb300.torch_heap import TorchSymmHeap
        if c["op"] == "route":
            size = abi.moe_route_workspace(c["G"], c["T"], c["E"])
        elif c["op"] == "norm":
            size = abi.moe_block_norm_workspace(c["T"], c["D"])
        else:
            size = abi.moe_adapter_workspace(c["T"], c["K"], c["N"], c["r"])
            s["heap"] = TorchSymmHeap(1, 0)
        s["ws"] = torch.empty(max(size, 1), dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------ plain forms --
def _plain_route(s):
    c = s["case"]
    k = c["k"]
    l = s["logits"].float()
    l = torch.where(torch.isnan(l), -math.inf, l).clamp(max=FLT_MAX)
    m = l.amax(-1)
    valid = s["mask"].bool() & (m > -math.inf)
    m = torch.where(valid, m, 0.0)
    e = torch.where(valid[..., None], torch.exp(l - m[..., None]), 0.0)
    z = torch.where(valid, e.sum(-1), 1.0)
    p = e / z[..., None]
    top, idx = torch.sort(l, dim=-1, descending=True, stable=True)
    top, idx = top[..., :k], idx[..., :k]
    ok = valid[..., None] & (top > -math.inf)
    chosen = torch.where(ok, e.gather(-1, idx), 0.0)
    total = chosen.sum(-1) if c["renorm"] else z
    weights = chosen / torch.where(valid, total, 1.0)[..., None]
    counts = torch.zeros(c["G"], c["E"], device=l.device)
    counts.scatter_add_(1, idx.reshape(c["G"], -1), ok.reshape(c["G"], -1).float())
    n = valid.sum(-1)
    n1 = n.clamp(min=1).float()
    balance = (counts * p.sum(1)).sum(-1) * (c["E"] / k) / (n1 * n1)
    lse = torch.where(valid, m + torch.log(z), 0.0)
    return dict(experts=torch.where(ok, idx, -1).to(torch.int32), weights=weights,
                counts=counts.to(torch.int32), tokens=n.to(torch.int32),
                stats=torch.stack([m, torch.where(valid, z, 0.0)], -1),
                loss=torch.stack([balance, (lse * lse).sum(-1) / n1], -1))


def _plain_route_back(s):
    c = s["case"]
    l = s["logits"].float()
    l = torch.where(torch.isnan(l), -math.inf, l).clamp(max=FLT_MAX)
    m, z = s["stats"].unbind(-1)
    valid = s["experts"][..., 0] >= 0
    z1 = torch.where(valid, z, 1.0)
    p = torch.where(valid[..., None], torch.exp(l - m[..., None]) / z1[..., None], 0.0)
    n1 = s["tokens"].clamp(min=1).float()[:, None]
    dbalance, dz = s["dloss"][:, :1], s["dloss"][:, 1:]
    a = (dbalance * s["counts"].float() * (c["E"] / c["k"]) / (n1 * n1))[:, None, :].expand_as(p)
    ok = s["experts"] >= 0
    idx = s["experts"].clamp(min=0).long()
    dw = torch.where(ok, s["dweights"], 0.0)
    if c["renorm"]:
        u = torch.where(ok, p.gather(-1, idx), 0.0)
        u = u / torch.where(valid, u.sum(-1), 1.0)[..., None]
        d = p * (a - (p * a).sum(-1, keepdim=True))
        d = d.scatter_add(-1, idx, u * (dw - (u * dw).sum(-1, keepdim=True)))
    else:
        a = a.scatter_add(-1, idx, dw)
        d = p * (a - (p * a).sum(-1, keepdim=True))
    lse = torch.where(valid, m + torch.log(z1), 0.0)
    d = d + p * (2 * dz * lse / n1)[..., None]
    return d.to(s["logits"].dtype)


def _slots(s):
    """Row indices (one past the end for absent ones) and their weights, 0 for absent ones."""
    have = (s["rows"] >= 0) & (s["rows"] < s["y"].shape[0])
    idx = torch.where(have, s["rows"], s["y"].shape[0]).long()
    return have, idx, torch.where(have, s["weights"] if s["weights"] is not None else 1.0, 0.0)


def _rows(s, have, idx):
    rows = s["y"][idx.clamp(max=s["y"].shape[0] - 1)].float()
    return torch.where(have[..., None], rows, 0.0)


def _plain_norm(s):
    x = s["x"].float()
    have, idx, w = _slots(s)
    y = (w[..., None] * _rows(s, have, idx)).sum(1)
    r1 = torch.rsqrt((y * y).mean(-1) + EPS)
    u = y * r1[:, None] * s["w_post"] if s["w_post"] is not None else y
    xo = s["res"] * x + s["gate"][:, None] * u
    r2 = torch.rsqrt((xo * xo).mean(-1) + EPS)
    h = xo * r2[:, None] * s["w_pre"]
    dt = s["x"].dtype
    return dict(xo=xo.to(dt), h=h.to(dt),
                rstd=torch.stack([r1 if s["w_post"] is not None else torch.ones_like(r1), r2], -1))


def _plain_norm_back(s):
    x, z, dxo, dh = (s[n].float() for n in ("x", "xo", "dxo", "dh"))
    r1, r2 = s["rstd"][:, :1], s["rstd"][:, 1:]
    g = dh * s["w_pre"]
    dz = dxo + r2 * (g - z * r2 * r2 * (g * z).mean(-1, keepdim=True))
    have, idx, w = _slots(s)
    rows = _rows(s, have, idx)
    y = (w[..., None] * rows).sum(1)
    gate = s["gate"][:, None]
    out = dict(dw_pre=(dh * z * r2).sum(0), dres=(dz * x).sum(0))
    if s["w_post"] is not None:
        n = y * r1
        out["dgate"] = (dz * n * s["w_post"]).sum(-1)
        out["dw_post"] = (gate * dz * n).sum(0)
        dn = gate * dz * s["w_post"]
        dy = r1 * (dn - n * (dn * n).mean(-1, keepdim=True))
    else:
        out["dgate"] = (dz * y).sum(-1)
        dy = gate * dz
    if s["weights"] is not None:
        out["dweights"] = (dy[:, None] * rows).sum(-1)
    d = torch.zeros(s["y"].shape[0] + 1, x.shape[1], device=x.device)
    d[idx.reshape(-1)] = (w[..., None] * dy[:, None]).reshape(-1, x.shape[1])
    out["dy"], out["dx"] = d[:-1].to(s["y"].dtype), (s["res"] * dz).to(s["x"].dtype)
    return out


def _plain_adapter(s):
    c = s["case"]
    x = s["x"].float()
    a = s["a"].float().permute(1, 0, 2).reshape(c["K"], -1)
    mine = s["ids"][:, None] == torch.arange(c["R"], device=x.device)  # [T, R]
    h = (x @ a).view(c["T"], c["R"], c["r"]) * s["scale"][:, None]
    h = torch.where(mine[..., None], h, 0.0).view(c["T"], -1)
    y = x @ s["w"].float() + h @ s["b"].float().view(-1, c["N"])
    return dict(y=y.to(s["x"].dtype))


# -------------------------------------------------------------------- run --
def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "route":
        return dict(dlogits=_plain_route_back(s)) if c["back"] else _plain_route(s)
    if c["op"] == "norm":
        return _plain_norm_back(s) if c["back"] else _plain_norm(s)
    return _plain_adapter(s)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _run_own(s, c):
    from symmetric_memory_moe_gb300 import abi
    dt, ws = CODES[c["dtype"]], s["ws"].data_ptr()
    if c["op"] == "route":
        G, T, E, k = c["G"], c["T"], c["E"], c["k"]
        if c["back"]:
            abi.moe_route_backward(_ptr(s["logits"]), E, dt, G, T, E, k, c["renorm"], 1.0,
                                   _ptr(s["experts"]), _ptr(s["counts"]), _ptr(s["tokens"]),
                                   _ptr(s["stats"]), _ptr(s["dweights"]), _ptr(s["dloss"]),
                                   _ptr(s["dlogits"]), E)
            return dict(dlogits=s["dlogits"])
        abi.moe_route(_ptr(s["logits"]), E, _ptr(s["mask"]), dt, G, T, E, k, c["renorm"], 1.0,
                      _ptr(s["experts"]), _ptr(s["weights"]), _ptr(s["counts"]),
                      _ptr(s["tokens"]), _ptr(s["stats"]), _ptr(s["loss"]), ws)
        return {n: s[n] for n in ("experts", "weights", "counts", "tokens", "stats", "loss")}
    if c["op"] == "norm":
        T, D, k = c["T"], c["D"], c["k"]
        if c["back"]:
            abi.moe_block_norm_backward(
                _ptr(s["dxo"]), _ptr(s["dh"]), _ptr(s["x"]), _ptr(s["xo"]), D, _ptr(s["y"]), D,
                _ptr(s["rows"]), T * k, _ptr(s["weights"]), _ptr(s["gate"]), _ptr(s["res"]),
                _ptr(s["w_post"]), _ptr(s["w_pre"]), _ptr(s["rstd"]), dt, T, D, k, _ptr(s["dx"]),
                _ptr(s["dy"]), _ptr(s["dweights"]), _ptr(s["dgate"]), _ptr(s["dres"]),
                _ptr(s["dw_post"]) if c["post"] else None, _ptr(s["dw_pre"]), ws)
            names = ["dw_pre", "dres", "dgate", "dy", "dx"]
            names += (["dw_post"] if c["post"] else []) + (["dweights"] if k > 1 else [])
            return {n: s[n] for n in names}
        abi.moe_block_norm(_ptr(s["x"]), D, _ptr(s["y"]), D, _ptr(s["rows"]), T * k,
                           _ptr(s["weights"]), _ptr(s["gate"]), _ptr(s["res"]), _ptr(s["w_post"]),
                           _ptr(s["w_pre"]), EPS, dt, T, D, k, _ptr(s["xo"]), _ptr(s["h"]),
                           _ptr(s["rstd"]))
        return {n: s[n] for n in ("xo", "h", "rstd")}
    abi.moe_adapter_matmul(s["heap"].handle, _ptr(s["x"]), c["K"], _ptr(s["w"]), c["N"],
                           _ptr(s["a"]), _ptr(s["b"]), _ptr(s["scale"]), _ptr(s["ids"]), dt,
                           c["T"], c["K"], c["N"], c["R"], c["r"], _ptr(s["y"]), c["N"], ws)
    return dict(y=s["y"])


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    """The operators' definitions in 64 bits."""
    c = case
    s = prepare(c, seed)
    if c["op"] == "route":
        return _exact_route(c, s)
    if c["op"] == "norm":
        return _exact_norm_back(c, s) if c["back"] else _exact_norm(c, s)
    ids = s["ids"].cpu()
    x = s["x"].double()
    y = x @ s["w"].double()
    for a in sorted(set(ids.tolist()) - {-1}):  # each request's tokens with its own adapter
        t = (ids == a).nonzero().flatten().to(x.device)
        y[t] += s["scale"][a].double() * ((x[t] @ s["a"][a].double()) @ s["b"][a].double())
    return dict(y=y)


def _exact_route(c, s):
    E, k = c["E"], c["k"]
    l = s["logits"].double()
    l[torch.isnan(l)] = -math.inf
    live = s["mask"].bool() & (l > -math.inf).any(-1)
    l[~live] = 0.0
    p = torch.softmax(l, -1)
    lse = torch.logsumexp(l, -1)
    if not c["back"]:
        # a token's choice: the k largest, the lower index first among equals
        order = torch.argsort(-l, dim=-1, stable=True)[..., :k]
        ok = live[..., None] & (torch.gather(l, -1, order) > -math.inf)
        w = torch.gather(p, -1, order) * ok
        if c["renorm"]:
            w = w / w.sum(-1, keepdim=True).masked_fill(~live[..., None], 1.0)
        hot = torch.zeros_like(p).scatter_(-1, order, ok.double())
        n = live.sum(-1).double().clamp(min=1)
        share, mean_p = hot.sum(1) / (k * n)[:, None], (p * live[..., None]).sum(1) / n[:, None]
        loss = torch.stack([E * (share * mean_p).sum(-1), (lse ** 2 * live).sum(-1) / n], -1)
        top = l.amax(-1)
        stats = torch.stack([top, torch.exp(lse - top)], -1) * live[..., None]
        return dict(experts=None, weights=w, counts=None, tokens=None, stats=stats, loss=loss)
    # the gradient by the softmax's Jacobian, applied to dL/dp
    n = live.sum(-1).double().clamp(min=1)[:, None]
    up = torch.zeros_like(p) + (s["dloss"][:, :1].double() * E * s["counts"].double()
                                / (k * n * n))[:, None, :]
    ok = s["experts"] >= 0
    idx = torch.where(ok, s["experts"], 0).long()
    dw = s["dweights"].double() * ok
    if c["renorm"]:
        pc = torch.gather(p, -1, idx) * ok
        tot = pc.sum(-1, keepdim=True).masked_fill(~live[..., None], 1.0)
        dp = dw / tot - ((dw * pc).sum(-1, keepdim=True) / tot ** 2)
        up.scatter_add_(-1, idx, dp * ok)
    else:
        up.scatter_add_(-1, idx, dw)
    d = p * up - p * (p * up).sum(-1, keepdim=True)
    d = d + p * (2 * s["dloss"][:, 1:].double() * lse / n)[..., None]
    return dict(dlogits=d * live[..., None])


def _exact_sum(s):
    """Each token's weighted rows, one slot after the other."""
    T, k = s["rows"].shape
    y = torch.zeros(T, s["x"].shape[1], dtype=torch.float64, device=s["x"].device)
    for j in range(k):
        r = s["rows"][:, j].long()
        w = s["weights"][:, j].double() if k > 1 else 1.0
        y += torch.where(r >= 0, w, 0.0)[:, None] * s["y"][r].double()
    return y


def _exact_norm(c, s):
    y = _exact_sum(s)
    one = torch.ones(len(y), dtype=torch.float64, device=y.device)
    r1 = 1 / torch.sqrt(y.square().sum(-1) / c["D"] + EPS) if c["post"] else one
    u = torch.einsum("td,t,d->td", y, r1, s["w_post"].double()) if c["post"] else y
    xo = s["x"].double() * s["res"].double() + u * s["gate"].double()[:, None]
    r2 = 1 / torch.sqrt(xo.square().sum(-1) / c["D"] + EPS)
    h = torch.einsum("td,t,d->td", xo, r2, s["w_pre"].double())
    return dict(xo=xo, h=h, rstd=torch.stack([r1, r2], -1))


def _exact_norm_back(c, s):
    D = c["D"]
    z, dh, x = s["xo"].double(), s["dh"].double(), s["x"].double()
    r1, r2 = s["rstd"].double().unbind(-1)
    zn = z * r2[:, None]
    g = dh * s["w_pre"].double()
    dz = s["dxo"].double() + r2[:, None] * (g - zn * ((g * zn).sum(-1) / D)[:, None])
    y, gate = _exact_sum(s), s["gate"].double()
    out = dict(dw_pre=(dh * zn).sum(0), dres=(dz * x).sum(0), dx=dz * s["res"].double())
    if c["post"]:
        yn, wp = y * r1[:, None], s["w_post"].double()
        out["dgate"] = torch.einsum("td,td,d->t", dz, yn, wp)
        out["dw_post"] = torch.einsum("td,td,t->d", dz, yn, gate)
        q = torch.einsum("td,d,t->td", dz, wp, gate)
        dy = r1[:, None] * (q - yn * ((q * yn).sum(-1) / D)[:, None])
    else:
        out["dgate"] = (dz * y).sum(-1)
        dy = dz * gate[:, None]
    out["dy"] = torch.zeros(s["y"].shape, dtype=torch.float64, device=x.device)
    if c["k"] > 1:
        out["dweights"] = torch.zeros(c["T"], c["k"], dtype=torch.float64, device=x.device)
    for j in range(c["k"]):
        r = s["rows"][:, j].long()
        t = (r >= 0).nonzero().flatten()
        out["dy"][r[t]] = (s["weights"][t, j].double()[:, None] if c["k"] > 1 else 1.0) * dy[t]
        if c["k"] > 1:
            out["dweights"][t, j] = (dy[t] * s["y"][r[t]].double()).sum(-1)
    return out
