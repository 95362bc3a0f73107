"""Results of the expert-layer and 4-bit calls that share memory with an operand
or another result are refused before anything is launched."""
import ctypes

import pytest

from second_order_optimizer_shampoo_b200 import _abi as A

BASE = 1 << 20


def p(offset):
    return ctypes.c_void_p(BASE + offset)


# X 64 x 128 bf16 at 0 (16384 bytes), W 2 x 128 x 64 at 16384 (32768), offsets at
# 49152 (24), free from 49280 on
@pytest.mark.parametrize("out", [A.SHP_BF16, A.SHP_TF32])
@pytest.mark.parametrize("Y", [0, 16384 - 16, 16384, 49152 - 16, 49152, 49152 + 16])
def test_grouped_matmul(Y, out):
    assert A.lib().shp_grouped_matmul(p(0), p(49152), p(16384), 0, p(Y), out, 64, 128, 64, 2, None) == A.SHP_EINVAL


def test_grouped_matmul_behind_the_end_of_the_result():
    # Y of 8192 bytes ends 16 bytes inside X
    X = ctypes.c_void_p(BASE)
    Y = ctypes.c_void_p(BASE - 8192 + 16)
    assert A.lib().shp_grouped_matmul(X, p(49152), p(16384), 0, Y, A.SHP_BF16, 64, 128, 64, 2, None) == A.SHP_EINVAL


# A 64 x 128 bf16 at 0 (16384), B 64 x 64 at 16384 (8192), offsets at 24576 (24)
@pytest.mark.parametrize("G", [0, 16384, 24576 - 16, 24576 + 16])
def test_grouped_wgrad(G):
    assert A.lib().shp_grouped_wgrad(p(0), p(16384), p(24576), p(G), 64, 128, 64, 2, 0, None) == A.SHP_EINVAL


# X 64 x 64 fp32 at 0 (16384), codes 2048, scales 512
@pytest.mark.parametrize("Q,S,Qt,St", [
    (16368, 20000, 24000, 28000), (16384, 16368 - 480, 24000, 28000), (16384, 18416, 24000, 28000),
    (16384, 20000, 18416, 28000), (16384, 20000, 24000, 26032), (16384, 20000, 24000, 0), (16384, 20000, 20496, 28000)])
def test_mx4_quantize(Q, S, Qt, St):
    assert A.lib().shp_mx4_quantize(p(0), A.SHP_TF32, 64, 64, 1, p(Q), p(S), p(Qt), p(St), None) == A.SHP_EINVAL


@pytest.mark.parametrize("X", [0, 2032, 4096, 4592])
def test_mx4_dequantize(X):
    assert A.lib().shp_mx4_dequantize(p(0), p(4096), 64, 64, 1, p(X), A.SHP_TF32, None) == A.SHP_EINVAL


# A, B 64 x 64 codes (2048), scales 512: at 0, 4096, 8192, 12288
@pytest.mark.parametrize("C", [0, 2032, 4096 + 496, 8192 + 2032, 12288])
def test_mx4_matmul(C):
    assert A.lib().shp_mx4_matmul(p(0), p(4096), p(8192), p(12288), p(C), A.SHP_BF16, 64, 64, 64, 1, None) == A.SHP_EINVAL


def test_sizes_beyond_64_bits_do_not_wrap():
    # W of 2^65 bytes, 0 in 64 bits, holds Y; X and the offsets lie elsewhere
    assert A.lib().shp_grouped_matmul(p(1 << 50), p(1 << 52), p(0), 0, p(1 << 40), A.SHP_BF16, 64, 1 << 30, 1 << 21,
                                      1 << 13, None) == A.SHP_EINVAL
