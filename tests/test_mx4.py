"""Host-only checks of the MXFP4 entry points: sizes and argument refusals."""
import ctypes

import pytest

from second_order_optimizer_shampoo_b200 import _abi as A

F = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10008)


def quant(X=F, st=A.SHP_TF32, rows=64, cols=64, batch=1, Q=F, S=F, Qt=F, St=F):
    return A.lib().shp_mx4_quantize(X, st, rows, cols, batch, Q, S, Qt, St, None)


def dequant(Q=F, S=F, rows=64, cols=64, batch=1, X=F, st=A.SHP_TF32):
    return A.lib().shp_mx4_dequantize(Q, S, rows, cols, batch, X, st, None)


def mm(Am=F, As=F, B=F, Bs=F, C=F, out=A.SHP_BF16, M=64, N=64, K=64, batch=1):
    return A.lib().shp_mx4_matmul(Am, As, B, Bs, C, out, M, N, K, batch, None)


def test_sizes():
    L = A.lib()
    assert L.shp_mx4_code_bytes(3, 33, 2) == 2 * 3 * 32
    assert L.shp_mx4_scale_bytes(129, 129, 2) == 2 * 2 * 2 * 512
    assert L.shp_mx4_code_bytes(1 << 20, 1 << 20, 4) == 4 << 39
    for bad in ((0, 8, 1), (8, 0, 1), (8, 8, 0), (-1, 8, 1), (2 ** 31, 8, 1)):
        assert L.shp_mx4_code_bytes(*bad) == 0
        assert L.shp_mx4_scale_bytes(*bad) == 0


@pytest.mark.parametrize("kw", [
    dict(X=None), dict(X=ODD), dict(Q=ODD), dict(S=ODD), dict(Qt=ODD), dict(St=ODD),
    dict(S=None), dict(Q=None), dict(St=None), dict(Qt=None),
    dict(Q=None, S=None, Qt=None, St=None), dict(st=A.SHP_3XTF32), dict(rows=0), dict(cols=0),
    dict(batch=0), dict(cols=62), dict(st=A.SHP_BF16, cols=60)])
def test_quantize_refuses(kw):
    assert quant(**kw) == A.SHP_EINVAL


@pytest.mark.parametrize("kw", [
    dict(Q=None), dict(S=None), dict(X=None), dict(Q=ODD), dict(S=ODD), dict(X=ODD),
    dict(st=A.SHP_OZAKI), dict(rows=0), dict(cols=-1), dict(batch=0)])
def test_dequantize_refuses(kw):
    assert dequant(**kw) == A.SHP_EINVAL


@pytest.mark.parametrize("kw", [
    dict(Am=None), dict(As=None), dict(B=None), dict(Bs=None), dict(C=None),
    dict(Am=ODD), dict(As=ODD), dict(B=ODD), dict(Bs=ODD), dict(C=ODD),
    dict(out=A.SHP_3XTF32), dict(M=0), dict(N=0), dict(K=0), dict(batch=0),
    dict(K=48), dict(N=60), dict(out=A.SHP_TF32, N=62)])
def test_matmul_refuses(kw):
    assert mm(**kw) == A.SHP_EINVAL


def test_beyond_the_coordinates():
    big = 2 ** 31
    assert quant(rows=big) == A.SHP_EUNSUPPORTED
    assert quant(cols=big) == A.SHP_EUNSUPPORTED
    assert quant(batch=1 << 30, rows=1024) == A.SHP_EUNSUPPORTED
    assert dequant(rows=big) == A.SHP_EUNSUPPORTED
    for kw in (dict(M=big), dict(N=big), dict(K=big), dict(batch=65536), dict(batch=65535, M=1 << 24, N=1 << 24)):
        assert mm(**kw) == A.SHP_EUNSUPPORTED


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    from second_order_optimizer_shampoo_b200 import prism
    q, s = torch.zeros(1, 64, 32, dtype=torch.uint8), torch.zeros(1, 1, 1, 512, dtype=torch.uint8)
    with pytest.raises(ValueError):
        prism.shp_mx4_quantize(torch.zeros(64, 64))
    with pytest.raises(ValueError):
        prism.shp_mx4_dequantize(q, s, 64)
    with pytest.raises(ValueError):
        prism.shp_mx4_matmul(q, s, q, s)
