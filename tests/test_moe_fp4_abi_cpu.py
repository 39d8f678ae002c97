"""A tensor's own scale where rows are packed: MX takes none, so that the same scale given to
packing and unpacking cannot turn x into its multiple.  Host-side checks before any launch."""
import pytest

from symmetric_memory_moe_gb300 import abi
from test_moe_expert_abi_cpu import QUANT, E, P, code


@pytest.mark.parametrize("act", [abi.SYMM_ACT_NONE, abi.SYMM_ACT_SILU, abi.SYMM_ACT_GELU])
@pytest.mark.parametrize("dtype", [abi.SYMM_DTYPE_F16, abi.SYMM_DTYPE_BF16, abi.SYMM_DTYPE_F32])
def test_mx_refuses_a_tensors_scale(act, dtype):
    call = dict(QUANT, act=act, dtype=dtype, ldx=128, fmt=abi.SYMM_FP4_MX)
    assert code(abi.moe_fp4_quantize, **dict(call, gscale=4 * P)) == E
    assert b"gscale" in abi.lib().symm_last_error()


def test_no_rows_are_no_call():
    abi.moe_fp4_quantize(**dict(QUANT, n=0, fmt=abi.SYMM_FP4_MX, gscale=4 * P))
