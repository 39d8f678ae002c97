"""moe_block_norm and its gradients where a token has one row and its weight matters."""
import pytest
import torch

from moe_refs import DTYPES
from test_gpu_moe_norm import back, check_back, check_forward, forward, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D,dt", [(7, 64, "bf16"), (300, 1000, "f32"), (33, 2049, "f16"),
                                    (3, 7168, "bf16")])
def test_one_weighted_row_without_a_norm_after_the_block(T, D, dt):
    """Without w_post the weight of a token's only row is not taken out again."""
    i = make(T, D, 1, dt, T + D, post=False, drop=T > 3, spare=2)
    g = torch.Generator().manual_seed(5)
    i["weights"] = (torch.randn(T, 1, generator=g) * 3).cuda()
    f = forward(i, dt)
    check_forward(i, dt, *f)
    dxo, dh = (torch.randn(T, D, generator=g).to(DTYPES[dt]).cuda() for _ in range(2))
    check_back(i, dt, f, dxo, dh, back(i, dt, f, dxo, dh))
