"""CPU tests of the expert operators at their edges: sizes, counts and refusals."""
import ctypes

import pytest

import bit_weight_quantized_prepack_b200 as wq


@pytest.mark.parametrize("T,E,k,N", [(4, 8, 2, 32), (300, 8, 2, 4096), (1 << 20, 128, 8, 2048)])
def test_scratch_holds_the_pairs_unrounded(T, E, k, N):
    assert wq.wq_experts_scratch_bytes(T, E, k, N) == T * k * N * 4
    ok = ctypes.c_void_p(0x10000)  # never dereferenced: the call ends before a launch
    assert wq.lib.wq_gemm_w4a16_experts_combine(ok, ok, ok, ok, ok, ok, ok, ok, T * k * N * 4 - 1, T, E, k, N, 128, 128,
                                                None) == wq.WQ_ERR_INVALID_ARG
