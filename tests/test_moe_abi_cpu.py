"""What the MoE block operators refuse, and their workspace sizes: host-side
checks that come before any launch.  The pointers are never dereferenced."""
import pytest

from symmetric_memory_moe_gb300 import abi

P = 0x7F0000001000  # aligned, never touched
E = abi.SYMM_EINVAL
F32, BF16 = abi.SYMM_DTYPE_F32, abi.SYMM_DTYPE_BF16


def code(fn, *args, **kw):
    with pytest.raises(abi.SymmError) as e:
        fn(*args, **kw)
    return e.value.code


ROUTE = dict(logits=P, ld=8, mask=None, dtype=F32, G=2, T=4, E=8, k=2, renorm=1, scale=1.0,
             experts=P, weights=P, counts=P, tokens=P, stats=P, loss=P, workspace=P, stream=0)


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(dtype=-1), dict(G=-1), dict(T=-1), dict(G=1 << 16, T=1 << 15), dict(E=0),
    dict(E=1025, ld=1025), dict(k=0), dict(k=9), dict(E=64, ld=64, k=33), dict(ld=7),
    dict(ld=1 << 41), dict(scale=float("nan")), dict(scale=float("inf")), dict(logits=None),
    dict(experts=None), dict(weights=None), dict(counts=None), dict(tokens=None), dict(stats=None),
    dict(loss=None), dict(workspace=None), dict(logits=P + 2), dict(counts=P + 1),
    dict(workspace=P + 8)])
def test_route_refuses(bad):
    assert code(abi.moe_route, **dict(ROUTE, **bad)) == E


BACK = dict(logits=P, ld=8, dtype=F32, G=2, T=4, E=8, k=2, renorm=1, scale=1.0, experts=P, counts=P,
            tokens=P, stats=P, dweights=P, dloss=P, dlogits=P + 4096, ldd=8, stream=0)


@pytest.mark.parametrize("bad", [
    dict(dtype=9), dict(G=-1), dict(E=0), dict(k=0), dict(k=9), dict(ld=7), dict(ldd=7),
    dict(ldd=1 << 41), dict(scale=float("nan")), dict(logits=None), dict(experts=None),
    dict(counts=None), dict(tokens=None), dict(stats=None), dict(dlogits=None),
    dict(dlogits=P, ldd=9), dict(dlogits=P + 4097), dict(stats=P + 2), dict(dweights=P + 2)])
def test_route_backward_refuses(bad):
    assert code(abi.moe_route_backward, **dict(BACK, **bad)) == E


NORM = dict(x=P, ld=8, y=2 * P, ldy=8, rows=P, yrows=8, weights=P, gate=P, res=P, w_post=P,
            w_pre=P, eps=1e-6, dtype=BF16, T=4, D=8, k=2, xo=3 * P, h=4 * P, rstd=P, stream=0)


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(T=-1), dict(D=0), dict(D=16385, ld=16385, ldy=16385), dict(k=0),
    dict(k=33), dict(T=1 << 30, k=2), dict(ld=7), dict(ldy=7), dict(ld=1 << 41), dict(eps=0.0),
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(xo=None),
    dict(h=None), dict(w_pre=None), dict(y=None), dict(h=P), dict(h=3 * P), dict(h=2 * P),
    dict(x=P + 1), dict(xo=3 * P + 1), dict(rows=P + 2), dict(w_post=P + 1),
    dict(y=None, k=0), dict(y=None, k=0, rows=None, weights=None, gate=None, res=None, w_post=None),
    dict(y=None, k=0, rows=None, weights=None, gate=None, res=None, w_post=None, xo=None, h=None,
         w_pre=None)])
def test_norm_refuses(bad):
    assert code(abi.moe_block_norm, **dict(NORM, **bad)) == E


NBACK = dict(dxo=P, dh=2 * P, x=3 * P, xo=4 * P, ld=8, y=5 * P, ldy=8, rows=P, yrows=8, weights=P,
             gate=P, res=P, w_post=P, w_pre=P, rstd=P, dtype=BF16, T=4, D=8, k=2, dx=6 * P,
             dy=7 * P, dweights=P, dgate=P, dres=P, dw_post=P, dw_pre=P, workspace=P, stream=0)
ALONE = dict(y=None, k=0, rows=None, weights=None, gate=None, res=None, w_post=None, xo=None,
             dy=None, dweights=None, dgate=None, dres=None, dw_post=None)


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(T=-1), dict(D=0), dict(k=0), dict(k=33), dict(ld=7), dict(ldy=7),
    dict(dh=None), dict(w_pre=None), dict(w_post=None), dict(gate=None), dict(res=None),
    dict(weights=None), dict(x=None), dict(xo=None), dict(rstd=None), dict(dx=None), dict(dy=None),
    dict(workspace=None), dict(workspace=P + 8), dict(dx=3 * P), dict(dx=4 * P), dict(dx=2 * P),
    dict(dy=5 * P), dict(dy=6 * P), dict(dx=6 * P + 1), dict(dgate=P + 2), dict(y=None, k=0),
    dict(ALONE, dx=None), dict(ALONE, dy=P), dict(dxo=None, dh=None, w_pre=None, dw_pre=None)])
def test_norm_backward_refuses(bad):
    assert code(abi.moe_block_norm_backward, **dict(NBACK, **bad)) == E


def test_workspaces():
    for G, T, n in ((1, 1, 16), (8, 4096, 256), (0, 0, 1), (3, 1531, 60)):
        size = abi.moe_route_workspace(G, T, n)
        assert size % 16 == 0 and size >= (2 * n + 2) * 4 * G
    for bad in ((-1, 1, 8), (1, -1, 8), (1, 1, 0), (1, 1, 1025), (1 << 16, 1 << 15, 8)):
        assert code(abi.moe_route_workspace, *bad) == E
    for T, D in ((0, 8), (1, 1), (4096, 7168), (9, 16384)):
        size = abi.moe_block_norm_workspace(T, D)
        assert size % 16 == 0 and size >= 3 * D * 4
    for bad in ((-1, 8), (1, 0), (1, 16385)):
        assert code(abi.moe_block_norm_workspace, *bad) == E


def test_nothing_to_do_launches_nothing():
    abi.moe_route(**dict(ROUTE, G=0, logits=None, counts=None))
    abi.moe_route_backward(**dict(BACK, T=0, logits=None))
    abi.moe_block_norm(**dict(NORM, T=0, x=None, xo=None))
    abi.moe_block_norm_backward(**dict(NBACK, T=0, dres=None, dw_post=None, dw_pre=None, dx=None))


ADAPTER = dict(x=P, ldx=16, w=2 * P, ldw=24, a=3 * P, b=4 * P, scale=P, ids=P, dtype=BF16, T=4,
               k=16, n=24, R=2, r=8, y=5 * P, ldy=24, workspace=P - P % 256, stream=0)


@pytest.fixture
def heap():
    h = abi.symm_heap_init(0x7F0000000000, 4 << 20, 1)
    yield h
    abi.symm_heap_destroy(h)


@pytest.mark.parametrize("bad", [
    dict(dtype=F32), dict(dtype=7), dict(T=-1), dict(T=(1 << 24) + 1), dict(k=0), dict(k=12),
    dict(n=0), dict(n=20), dict(k=(1 << 20) + 8), dict(R=-1), dict(r=-8), dict(r=12), dict(r=136),
    dict(R=0), dict(r=0), dict(ldx=8), dict(ldx=20), dict(ldw=16), dict(ldw=28), dict(ldy=23),
    dict(ldx=1 << 40), dict(x=None), dict(w=None), dict(a=None), dict(b=None), dict(scale=None),
    dict(ids=None), dict(y=None), dict(workspace=None), dict(x=P + 8), dict(w=2 * P + 2),
    dict(a=3 * P + 8), dict(b=4 * P + 1), dict(y=5 * P + 1), dict(ids=P + 2), dict(scale=P + 1),
    dict(workspace=P - P % 256 + 64), dict(y=P), dict(y=2 * P), dict(y=3 * P), dict(y=4 * P)])
def test_adapter_refuses(heap, bad):
    assert code(abi.moe_adapter_matmul, heap, **dict(ADAPTER, **bad)) == E


def test_adapter_refuses_no_heap():
    assert code(abi.moe_adapter_matmul, None, **ADAPTER) == E


def test_adapter_workspace():
    for T, k, n, r in ((1, 8, 8, 8), (0, 8, 8, 0), (300, 4096, 1000, 64), (8192, 4096, 4096, 32)):
        assert abi.moe_adapter_workspace(T, k, n, r) >= T * r * 4
    for bad in ((-1, 8, 8, 8), (1, 7, 8, 8), (1, 8, 12, 8), (1, 8, 8, 4), (1, 8, 8, 256)):
        assert code(abi.moe_adapter_workspace, *bad) == E


def test_adapter_without_tokens_launches_nothing(heap):
    abi.moe_adapter_matmul(heap, **dict(ADAPTER, T=0, x=None, y=None, workspace=None))
