"""Host-side arithmetic and checks of the MoE block operators at the ends of their ranges."""
from symmetric_memory_moe_gb300 import abi
from test_moe_abi_cpu import NORM, code


def test_route_workspace_at_the_largest_number_of_tokens():
    """As many partial sums at 2^31 - 1 tokens as at half of them."""
    for E in (1, 8, 1024):
        want = abi.moe_route_workspace(1, 1 << 30, E)
        for T in ((1 << 31) - 17, (1 << 31) - 16, (1 << 31) - 8, (1 << 31) - 1):
            assert abi.moe_route_workspace(1, T, E) == want, T


def test_norm_refuses_to_overwrite_its_rows():
    """xo may be x, but not y, whose rows other tokens still read."""
    assert code(abi.moe_block_norm, **dict(NORM, xo=NORM["y"])) == abi.SYMM_EINVAL
