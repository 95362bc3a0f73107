"""Host-only checks of the expert-grouped products: argument refusals of the
C ABI (nothing is launched) and of the Python binding."""
import ctypes

import pytest

from second_order_optimizer_shampoo_b200 import _abi as A

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first
MIS = ctypes.c_void_p(0x10004)
ODD = ctypes.c_void_p(0x10008)


def rows(X=FAKE, off=FAKE, W=FAKE, trans=0, Y=FAKE, out=A.SHP_BF16, T=64, K=64, N=64, E=4):
    return A.lib().shp_grouped_matmul(X, off, W, trans, Y, out, T, K, N, E, None)


def wgrad(X=FAKE, B=FAKE, off=FAKE, G=FAKE, T=64, m=64, n=64, E=4, acc=0):
    return A.lib().shp_grouped_wgrad(X, B, off, G, T, m, n, E, acc, None)


@pytest.mark.parametrize("kw", [
    dict(X=None), dict(off=None), dict(W=None), dict(Y=None),
    dict(X=ODD), dict(W=ODD), dict(Y=ODD), dict(off=MIS),
    dict(out=A.SHP_3XTF32), dict(out=A.SHP_OZAKI), dict(out=9),
    dict(T=-1), dict(K=0), dict(N=0), dict(E=0), dict(K=60), dict(N=60)])
def test_grouped_matmul_refuses(kw):
    assert rows(**kw) == A.SHP_EINVAL


@pytest.mark.parametrize("kw", [
    dict(X=None), dict(B=None), dict(off=None), dict(G=None),
    dict(X=ODD), dict(B=ODD), dict(G=ODD), dict(off=MIS),
    dict(T=-1), dict(m=0), dict(n=0), dict(E=0), dict(m=60), dict(n=60)])
def test_grouped_wgrad_refuses(kw):
    assert wgrad(**kw) == A.SHP_EINVAL


def test_sizes_beyond_the_tile_coordinates():
    big = 2 ** 31
    for kw in (dict(T=big), dict(K=big), dict(N=big), dict(E=65536)):
        assert rows(**kw) == A.SHP_EUNSUPPORTED
    for kw in (dict(T=big), dict(m=big), dict(n=big), dict(E=65536)):
        assert wgrad(**kw) == A.SHP_EUNSUPPORTED
    # more tiles than 32 bits number
    assert rows(T=2 ** 30, N=2 ** 30) == A.SHP_EUNSUPPORTED
    assert wgrad(m=2 ** 24, n=2 ** 24, E=65535) == A.SHP_EUNSUPPORTED


def test_no_rows_launches_nothing():
    # X and Y of no rows may be null; nothing runs, so this passes without a GPU
    assert rows(X=None, Y=None, T=0) == A.SHP_OK


def test_binding_refuses():
    torch = pytest.importorskip("torch")
    from second_order_optimizer_shampoo_b200 import prism
    x = torch.zeros(8, 64, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int64)
    w = torch.zeros(2, 64, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # CPU tensors
        prism.shp_grouped_matmul(x, off, w)
    with pytest.raises(ValueError):
        prism.shp_grouped_wgrad(x, x, off)
