"""Rows to NV codes where the tensor's own scale is far too small for the values: the block's scale
stays at 448 and the quotient is far above 6, up to beyond the largest float.  The code is that
of 6 with the value's own sign; everything is compared bit for bit."""
import pytest
import torch

import expert_refs as ref
from moe_refs import DTYPES
from test_gpu_moe_fp4 import gscale, pack

pytestmark = pytest.mark.gpu


def saturating(n, k, dt, top):
    """Rows whose blocks hold magnitudes of every size up to `top`, both signs."""
    g = torch.Generator().manual_seed(n)
    x = top * torch.exp2(-40 * torch.rand(n, k, generator=g, dtype=torch.float64))
    x[:, ::16], x[:, 1::16], x[:, 2::16], x[:, 3::16] = top, -top, 0.0, -0.0
    x[:, 4::16] = -top / 2
    x *= torch.where(torch.rand(n, k, generator=g) < 0.5, -1.0, 1.0)
    return x.to(DTYPES[dt]).cuda()


@pytest.mark.parametrize("dt", ["bf16", "f32", "f16"])
@pytest.mark.parametrize("g", [1e-3, 2.0 ** -90, 2.0 ** -100, 1e-30, 3e-39, 0.0371, 1.0])
@pytest.mark.parametrize("n,k", [(1, 32), (37, 96)])
def test_largest_values_keep_their_sign(n, k, g, dt):
    x = saturating(n, k, dt, torch.finfo(DTYPES[dt]).max)
    codes, scales = pack(x, "nv", gscale(g))
    code, scale = ref.quantize(x, "nv", gscale(g))
    assert (scales[:, :k // 16] == scale).all()
    assert torch.equal(codes[:, :k // 2], ref.pack(code))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("power", [3, 10, 18, 19, 20, 21, 22, 60, 100, 126])
def test_quotients_of_every_size(power, dt):
    """Largest quotients about 2^power (powers where one way to divide gives way to another
    among them), with the small ones of their blocks."""
    g = 2.0 ** -9 / 448  # a block's scale at 448 makes the unit about 2^-9
    x = saturating(40, 64, dt, 2.0 ** (power - 9) * 1.1)
    codes, scales = pack(x, "nv", gscale(g))
    code, scale = ref.quantize(x, "nv", gscale(g))
    assert (scales[:, :4] == scale).all()
    assert torch.equal(codes[:, :32], ref.pack(code))


@pytest.mark.parametrize("name", ["silu", "gelu"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_gated_largest_values(name, sign):
    """act(1000) u = 1000 u, with u down to -3e35: beyond what 448 units of 1e-3 hold."""
    x = torch.full((3, 64), 1000.0, device="cuda")
    x[:, 32:] = sign * torch.logspace(0, 35.4, 32, device="cuda") * \
        torch.tensor([1.0, -1.0], device="cuda").repeat(16)
    codes, scales = pack(x, "nv", gscale(1e-3), name)
    code = ref.unpack(codes[:, :16])
    assert (scales[:, :2] == 0x7e).all()  # 448
    big = x[:, 32:].abs() * 1000 > 8 * 0.448
    want = torch.where(x[:, 32:] < 0, 15, 7).to(torch.uint8)
    assert big[:, 1:].all() and torch.equal(code[big], want[big])
