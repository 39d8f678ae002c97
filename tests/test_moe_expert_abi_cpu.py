"""What the experts' operators refuse, and their workspace sizes: host-side
checks that come before any launch.  The pointers are never dereferenced."""
import ctypes

import pytest

from symmetric_memory_moe_gb300 import abi

P = 0x7F0000001000  # aligned, never touched
E = abi.SYMM_EINVAL
BF16 = abi.SYMM_DTYPE_BF16


@pytest.fixture(scope="module")
def heap():
    # a heap's host side alone: its base is only ever added to
    h = abi.symm_heap_init(P, 1 << 21, 1)
    yield h
    abi.symm_heap_destroy(h)


def code(fn, *args, **kw):
    with pytest.raises(abi.SymmError) as e:
        fn(*args, **kw)
    return e.value.code


FFN = dict(x=P, ldx=64, counts=P, w_gu=2 * P, w_d=3 * P, act=0, dtype=BF16, n=4, E=2, D=64, F=32,
           gu=4 * P, y=5 * P, ldy=64, workspace=6 * P, stream=0)


@pytest.mark.parametrize("bad", [
    dict(heap=None), dict(act=2), dict(act=-1), dict(dtype=2), dict(dtype=-1), dict(n=-1),
    dict(n=(1 << 24) + 1), dict(E=0), dict(E=1025), dict(D=0), dict(D=60), dict(D=4),
    dict(D=(1 << 17) + 8, ldx=1 << 18, ldy=1 << 18), dict(F=0), dict(F=12), dict(F=(1 << 17) + 8),
    dict(ldx=56), dict(ldx=68), dict(ldx=1 << 37), dict(ldy=63), dict(ldy=68), dict(ldy=1 << 37),
    dict(counts=None), dict(x=None), dict(w_gu=None), dict(w_d=None), dict(y=None),
    dict(workspace=None), dict(x=P + 2), dict(w_gu=P + 8), dict(w_d=P + 8), dict(counts=P + 2),
    dict(gu=P + 8), dict(y=P + 8), dict(workspace=P + 128), dict(y=P), dict(y=2 * P),
    dict(y=3 * P), dict(y=4 * P), dict(gu=P), dict(gu=2 * P), dict(gu=3 * P)])
def test_forward_refuses(heap, bad):
    assert code(abi.moe_expert_ffn, **dict(FFN, **dict(dict(heap=heap), **bad))) == E


def test_forward_of_no_rows(heap):
    abi.moe_expert_ffn(**dict(FFN, heap=heap, n=0, x=None, y=None, workspace=None))


BACK = dict(dy=P, lddy=64, x=2 * P, ldx=64, gu=3 * P, counts=P, w_gu=4 * P, w_d=5 * P, act=1,
            dtype=BF16, n=4, E=2, D=64, F=32, dx=6 * P, lddx=64, dw_gu=7 * P, dw_d=8 * P,
            workspace=9 * P, stream=0)


@pytest.mark.parametrize("bad", [
    dict(heap=None), dict(act=2), dict(dtype=2), dict(n=-1), dict(n=(1 << 24) + 1), dict(E=0),
    dict(E=1025), dict(D=60), dict(F=12), dict(lddy=56), dict(lddy=68), dict(ldx=56), dict(ldx=68),
    dict(lddx=63), dict(lddx=68), dict(lddx=1 << 37), dict(counts=None), dict(dy=None), dict(x=None),
    dict(gu=None), dict(w_gu=None), dict(w_d=None), dict(workspace=None), dict(dy=P + 2),
    dict(x=P + 2), dict(gu=P + 8), dict(dx=P + 8), dict(dw_gu=P + 2), dict(dw_d=P + 2),
    dict(workspace=P + 16), dict(dx=P), dict(dx=2 * P), dict(dx=3 * P), dict(dw_gu=4 * P),
    dict(dw_d=5 * P), dict(dw_gu=6 * P), dict(dw_d=6 * P), dict(dw_d=7 * P)])
def test_backward_refuses(heap, bad):
    assert code(abi.moe_expert_ffn_backward, **dict(BACK, **dict(dict(heap=heap), **bad))) == E


@pytest.mark.parametrize("n,E_,D,F,back,want", [
    (0, 1, 8, 8, False, 0), (1, 1, 8, 8, False, 256), (1, 1, 8, 8, True, 512),
    (100, 4, 64, 64, False, 12800), (100, 4, 64, 64, True, 12800 * 3),
    (1 << 24, 1024, 8, 1 << 17, True, (1 << 42) + (1 << 43))])
def test_workspace(n, E_, D, F, back, want):
    assert abi.moe_expert_workspace(n, E_, D, F, back) == want


def test_workspace_refuses():
    for bad in ((-1, 1, 8, 8), (1, 0, 8, 8), (1, 1, 12, 8), (1, 1, 8, 4)):
        assert code(abi.moe_expert_workspace, *bad) == E
    assert abi.lib().moe_expert_workspace(1, 1, 8, 8, 0, ctypes.POINTER(ctypes.c_size_t)()) == E


QUANT = dict(x=P, ldx=64, act=-1, dtype=BF16, fmt=0, gscale=P, n=4, k=64, codes=2 * P, ldc=32,
             scales=3 * P, lds=16, stream=0)


@pytest.mark.parametrize("bad", [
    dict(act=2), dict(act=-2), dict(dtype=3), dict(dtype=-1), dict(fmt=2), dict(fmt=-1),
    dict(n=-1), dict(n=(1 << 24) + 1), dict(k=0), dict(k=48),
    dict(k=(1 << 17) + 32, ldx=1 << 18, ldc=1 << 17, lds=1 << 14),
    dict(ldx=56), dict(ldx=68), dict(ldx=1 << 37), dict(act=0), dict(ldc=16), dict(ldc=40),
    dict(ldc=1 << 37), dict(lds=0), dict(lds=8), dict(lds=24), dict(lds=1 << 37), dict(x=None),
    dict(codes=None), dict(scales=None), dict(x=P + 8), dict(codes=P + 8), dict(scales=P + 8),
    dict(gscale=P + 2), dict(codes=P), dict(scales=P), dict(scales=2 * P)])
def test_quantize_refuses(bad):
    assert code(abi.moe_fp4_quantize, **dict(QUANT, **bad)) == E


DEQ = dict(codes=P, ldc=32, scales=2 * P, lds=16, fmt=1, gscale=None, n=4, k=64, dtype=BF16,
           y=3 * P, ldy=64, stream=0)


@pytest.mark.parametrize("bad", [
    dict(fmt=2), dict(dtype=3), dict(n=-1), dict(n=(1 << 24) + 1), dict(k=0), dict(k=40),
    dict(ldc=16), dict(ldc=33), dict(lds=0), dict(lds=20), dict(ldy=56), dict(ldy=65),
    dict(ldy=1 << 37), dict(codes=None), dict(scales=None), dict(y=None), dict(codes=P + 4),
    dict(scales=P + 4), dict(y=P + 8), dict(gscale=P + 1), dict(y=P), dict(y=2 * P)])
def test_dequantize_refuses(bad):
    assert code(abi.moe_fp4_dequantize, **dict(DEQ, **bad)) == E


MM = dict(xc=P, ldxc=32, xs=2 * P, ldxs=16, wc=3 * P, ldwc=32, ws=4 * P, ldws=16, counts=P,
          gx=None, gw=P, fmt=1, dtype=BF16, n=4, E=2, k=64, m=40, y=5 * P, ldy=40, stream=0)


@pytest.mark.parametrize("bad", [
    dict(heap=None), dict(fmt=2), dict(dtype=2), dict(n=-1), dict(n=(1 << 24) + 1), dict(E=0),
    dict(E=1025), dict(k=0), dict(k=48), dict(m=0), dict(m=(1 << 20) + 1, ldy=1 << 21),
    dict(ldxc=16), dict(ldxc=40), dict(ldxs=0), dict(ldxs=8), dict(ldwc=16), dict(ldwc=40),
    dict(ldws=0), dict(ldws=8), dict(ldy=39), dict(ldy=1 << 37), dict(counts=None), dict(xc=None),
    dict(xs=None), dict(wc=None), dict(ws=None), dict(y=None), dict(xc=P + 8), dict(xs=P + 8),
    dict(wc=P + 8), dict(ws=P + 8), dict(y=P + 1), dict(counts=P + 2), dict(gx=P + 2),
    dict(gw=P + 2), dict(y=P), dict(y=2 * P), dict(y=3 * P), dict(y=4 * P)])
def test_product_refuses(heap, bad):
    assert code(abi.moe_fp4_expert_matmul, **dict(MM, **dict(dict(heap=heap), **bad))) == E


def test_fp4_of_no_rows(heap):
    abi.moe_fp4_quantize(**dict(QUANT, n=0, x=None, codes=None, scales=None))
    abi.moe_fp4_dequantize(**dict(DEQ, n=0, codes=None, scales=None, y=None))
    abi.moe_fp4_expert_matmul(**dict(MM, heap=heap, n=0, xc=None, xs=None, wc=None, ws=None,
                                     y=None))
