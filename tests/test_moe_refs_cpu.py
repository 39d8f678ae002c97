"""The 64-bit references that the MoE operators' GPU tests compare against:
their gradients agree with central differences of the forward definitions."""
import pytest
import torch

import moe_refs as ref


@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_agrees_with_differences(renorm):
    g = torch.Generator().manual_seed(3)
    G, T, E, k = 2, 5, 7, 3
    l = torch.randn(G, T, E, generator=g, dtype=torch.float64)
    l[0, 1, 2] = -float("inf")
    l[1, 3] = -float("inf")
    f = ref.route(l, None, k, renorm, 1.7)
    dw = torch.randn(G, T, k, generator=g, dtype=torch.float64)
    dl = torch.randn(G, 2, generator=g, dtype=torch.float64)
    args = (f["experts"], f["counts"], f["tokens"], f["valid"], k, renorm, 1.7, dw, dl)
    d, mag = ref.route_grad(l, *args)
    assert (d.abs() <= mag * (1 + 1e-12)).all()
    eps = 1e-6
    for i in range(G * T * E):
        if not torch.isfinite(l.view(-1)[i]):
            assert d.view(-1)[i] == 0
            continue
        hi, lo = l.clone().view(-1), l.clone().view(-1)
        hi[i] += eps
        lo[i] -= eps
        diff = (ref.route_scalar(hi.view_as(l), *args) - ref.route_scalar(lo.view_as(l), *args)) / \
            (2 * eps)
        # a central difference errs by eps^2 |f'''| / 6 and by |f| 2^-52 / eps
        assert abs(diff - d.view(-1)[i]) < 1e-8


@pytest.mark.parametrize("post", [True, False])
def test_norm_gradient_agrees_with_differences(post):
    g = torch.Generator().manual_seed(4)
    T, D, k, eps = 3, 6, 2, 1e-3

    def r(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)

    rows = torch.tensor([[4, 0], [-1, 2], [5, 1]])
    i = dict(x=r(T, D), y=r(T * k, D), rows=rows, weights=r(T, k), gate=r(T), res=r(D),
             w_post=r(D) if post else None, w_pre=r(D), k=k)
    dxo, dh = r(T, D), r(T, D)
    f = ref.norm(i, eps)
    o = ref.norm_grad(i, f["xo"], f["rstd"], dxo, dh)

    def scalar(j):
        Y, have, _ = ref.gather(j["y"], j["rows"], T * k, T, k)
        return ref.norm_scalar(j["x"], Y, j["weights"], j["gate"], j["res"], j["w_post"],
                               j["w_pre"], have, eps, dxo, dh)

    step = 1e-6
    for name, grad in (("x", "dx"), ("y", "dy"), ("weights", "dweights"), ("gate", "dgate"),
                       ("res", "dres"), ("w_post", "dw_post"), ("w_pre", "dw_pre")):
        if i[name] is None:
            continue
        for n in range(i[name].numel()):
            hi, lo = dict(i), dict(i)
            hi[name], lo[name] = i[name].clone(), i[name].clone()
            hi[name].view(-1)[n] += step
            lo[name].view(-1)[n] -= step
            diff = (scalar(hi) - scalar(lo)) / (2 * step)
            got = o[grad].reshape(-1)[n]
            if torch.isnan(got):          # a row that no token names
                assert diff == 0
                continue
            # central difference: step^2 |f'''| / 6 (|f'''| up to ~1e3 here) and |f| 2^-52 / step
            assert abs(diff - got) < 1e-7 * max(1.0, float(abs(got))), (name, n)
