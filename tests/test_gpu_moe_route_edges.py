"""moe_route and moe_route_backward at the ends of their range."""
import math

import pytest
import torch

import moe_refs as ref
from moe_refs import DTYPES, U32
from symmetric_memory_moe_gb300 import abi
from test_gpu_moe_route import W, back, check_forward, forward, make

pytestmark = pytest.mark.gpu


def test_the_largest_number_of_tokens():
    """2^31 - 1 tokens of one expert: the last step of every warp's count leaves 31 bits.
    Every logit is 1 but the last one's 2, so p = 1 and lse is the logit.  A warp adds
    fewer than 2^20 ones and a CTA fewer than 2^23, exactly; joining at most 1024 CTAs
    rounds 1024 times."""
    T = (1 << 31) - 1
    logits = torch.ones(T, dtype=torch.float16, device="cuda")
    logits[-1] = 2
    experts = torch.full((T,), 9, dtype=torch.int32, device="cuda")
    weights, stats = torch.zeros(T, device="cuda"), torch.zeros(T, 2, device="cuda")
    counts, tokens = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    loss = torch.zeros(2, device="cuda")
    ws = torch.empty(abi.moe_route_workspace(1, T, 1), dtype=torch.uint8, device="cuda")
    abi.moe_route(logits.data_ptr(), 1, None, abi.SYMM_DTYPE_F16, 1, T, 1, 1, 1, 1.0,
                  *[t.data_ptr() for t in (experts, weights, counts, tokens, stats, loss)],
                  ws.data_ptr())
    assert int(counts) == T and int(tokens) == T
    assert not experts.any() and bool((weights == 1).all())
    assert bool((stats[:-1] == 1).all()) and stats[-1].tolist() == [2.0, 1.0]
    assert abs(loss[0] - 1) <= 1024 * U32 and abs(loss[1] - 1) <= 1024 * U32
    # dl = 2 lse / n dz with dz = n
    dloss = torch.tensor([0.0, float(T)], device="cuda")
    abi.moe_route_backward(logits.data_ptr(), 1, abi.SYMM_DTYPE_F16, 1, T, 1, 1, 1, 1.0,
                           *[t.data_ptr() for t in (experts, counts, tokens, stats)], None,
                           dloss.data_ptr(), logits.data_ptr(), 1)
    assert bool((logits[:-1] == 2).all()) and float(logits[-1]) == 4


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("E", [30, 64, 100, 256, 300])
def test_subnormal_logits_keep_their_order(dt, E):
    """Numbers below the type's smallest normal one, of both signs, and zeros of both signs."""
    g = torch.Generator().manual_seed(E)
    bits = torch.randint(0, 128 if dt == "bf16" else 1024, (2, 40, E), generator=g)
    sign = torch.randint(0, 2, bits.shape, generator=g) << 15
    l = (bits | sign).to(torch.int32).to(torch.int16).view(DTYPES[dt])
    _, o = forward(l, None, 8, dt, 1)
    check_forward(o, ref.route(l, None, 8, 1, 1.0), E, 8, 40)


@pytest.mark.parametrize("k", range(1, 12))
@pytest.mark.parametrize("E,dt", [(40, "f16"), (256, "bf16"), (256, "f32"), (20, "f32")])
@pytest.mark.parametrize("kind", ["ties", "holes"])
def test_every_number_of_choices(k, E, dt, kind):
    l, mask = make(2, 25, E, dt, k + E, kind)
    _, o = forward(l, mask, k, dt, 1)
    check_forward(o, ref.route(l, mask, k, 1, 1.0), E, k, 25)


@pytest.mark.parametrize("renorm", [1, 0])
@pytest.mark.parametrize("E", [8, 100, 300])
def test_z_gradient_of_the_largest_and_lowest_logits(E, renorm):
    """2 p lse dz / n with lse at either end of a float's range: infinite only where the
    gradient itself is, and 0 where p is."""
    top = torch.finfo(torch.float32).max
    l = torch.randn(2, 1, E, generator=torch.Generator().manual_seed(E))
    l[0, 0, 3] = math.inf
    l[1] = -top
    buf, f = forward(l, None, 2, "f32", renorm)
    dl = torch.tensor([[0.0, 1.0], [0.0, 2.0]], device="cuda")
    d = back(l, f, 2, "f32", renorm, 1.0, torch.zeros(2, 1, 2, device="cuda"), dl, buf=buf)
    d = d.view(2, E).double().cpu()
    want = torch.zeros(E, dtype=torch.float64)
    want[3] = math.inf                       # 2 FLT_MAX
    assert torch.equal(d[0], want)
    assert ((d[1] + 4 * top / E).abs() <= 2 * W * 4 * top / E).all()
