"""The experts' operators at the ends of their ranges: D and F of 2^17, rows of 2^17 values and
2^20 features in the 4-bit product, rows of 2^17 values to codes and back."""
import pytest
import torch

import expert_refs as ref
from moe_refs import TINY, U_OUT
from symmetric_memory_moe_gb300 import abi
from symmetric_memory_moe_gb300.torch_heap import TorchSymmHeap
from test_gpu_moe_expert import backward, forward, make, near, ptr
from test_gpu_moe_fp4 import CODES, FMTS, operands, pack, product, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def heap():
    h = TorchSymmHeap(1, 0)
    yield h
    h.close()


@pytest.mark.parametrize("n,E,D,F", [(70, 2, 1 << 17, 24), (70, 2, 24, 1 << 17),
                                     (3, 3, (1 << 17) - 8, 136), (300, 1, 136, (1 << 17) - 8)])
def test_feed_forward(heap, n, E, D, F):
    i = make(n, E, D, F, "bf16", "even")
    y, gu = forward(heap, i, "bf16", "silu")
    r = ref.ffn(i["x"], i["counts"], i["w_gu"], i["w_d"], "silu", U_OUT["bf16"], TINY["bf16"])
    near(gu, r["gu"], r["egu"], "gu")
    near(y, r["y"], r["ey"], "y")
    o = backward(heap, i, gu, "bf16", "silu")
    g = ref.ffn_grad(i["dy"], i["x"], gu, i["counts"], i["w_gu"], i["w_d"], "silu", U_OUT["bf16"],
                     TINY["bf16"])
    for k in ("dx", "dw_gu", "dw_d"):
        near(o[k], g[k], g["e" + k], k)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("n,E,k,m", [(40, 2, 1 << 17, 40), (200, 1, (1 << 17) - 32, 300),
                                     (40, 1, 32, 1 << 20), (40, 2, 64, (1 << 20) - 1)])
def test_product(heap, n, E, k, m, fmt):
    (xc, xs, x), (wc, ws, w), c = operands(n, E, k, m, fmt, "even")
    y = product(heap, xc, xs, wc, ws, c.cuda(), None, None, fmt, "bf16", k, m)
    for e, a, b in ref.runs(c):
        want, mag = x[a:b] @ w[e].t(), x[a:b].abs() @ w[e].abs().t()
        bound = U_OUT["bf16"] * want.abs() + (k + 8) * 2.0 ** -23 * mag + TINY["bf16"]
        near(y[a:b], want, bound * (1 + 2.0 ** -8), e)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_codes(fmt):
    k = 1 << 17
    x = rows(5, k, "bf16")
    codes, scales = pack(x, fmt)
    code, scale = ref.quantize(x, fmt, None)
    assert torch.equal(scales[:, :scale.shape[1]], scale)
    assert torch.equal(codes[:, :k // 2], ref.pack(code))
    y = torch.empty_like(x)
    abi.moe_fp4_dequantize(ptr(codes), codes.shape[1], ptr(scales), scales.shape[1], FMTS[fmt],
                           None, 5, k, CODES["bf16"], ptr(y), k)
    torch.cuda.synchronize()
    assert torch.equal(y, ref.values(code, scale, fmt, None).float().bfloat16())
