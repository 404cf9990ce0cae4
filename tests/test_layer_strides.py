"""Outputs of the operators around the packed product whose rows would lie over each other are refused (CPU)."""
import ctypes

import pytest

from test_layer_abi import A, B, C, bwd_args, distill_args, gemm_args, norm_args, pq  # noqa: F401

SHAPE = 2


def call(f, args, **over):
    for at, value in over.items():
        args[int(at[1:])] = value
    return f(*args)


@pytest.mark.parametrize("stride", [0, 1, 63, -1, -63])
def test_norm(pq, stride):
    lib = pq.lib
    assert call(lib.pq_rmsnorm, norm_args(pq), _8=stride) == SHAPE                                   # sum
    assert call(lib.pq_rmsnorm, norm_args(pq), _13=stride) == SHAPE                                  # y
    assert call(lib.pq_rmsnorm, norm_args(pq), _12=None, _14=C + 4096, _15=stride, _16=A) == SHAPE   # q
    assert call(lib.pq_rmsnorm_bwd, bwd_args(pq), _12=A + 4096, _13=stride) == SHAPE                 # dx
    assert call(lib.pq_quantize_rows, [pq.PQ_BF16, 3, 64, A, 64, C, stride, B, None]) == SHAPE


@pytest.mark.parametrize("stride", [0, 47, -47])
def test_product(pq, stride):
    assert call(pq.lib.pq_gemm_a8, gemm_args(pq), _13=stride) == SHAPE
    e = pq.pq_epilogue()
    e.other, e.other_stride = C, stride                     # in place: the same stride, and still no rows of their own
    assert call(pq.lib.pq_gemm_a8, gemm_args(pq, e), _13=stride) == SHAPE
    assert ctypes.sizeof(e) == 40


@pytest.mark.parametrize("stride", [0, 99, -99])
def test_distill(pq, stride):
    assert call(pq.lib.pq_distill, distill_args(pq), _15=stride) == SHAPE
    assert call(pq.lib.pq_distill_bwd, [pq.PQ_BF16, 3, 100, A, 100, 8, A, B, pq.PQ_F32, 2.0, A, B, C, C, stride, None]) == SHAPE
