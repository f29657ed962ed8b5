"""CPU tests of the expert operators at their edges: sizes, counts and refusals."""
import ctypes
import math
import os
import re

import pytest
import torch

import bit_weight_quantized_prepack_b200 as wq


@pytest.mark.parametrize("T,E,k,N", [(4, 8, 2, 32), (300, 8, 2, 4096), (1 << 20, 128, 8, 2048)])
def test_scratch_holds_the_pairs_unrounded(T, E, k, N):
    assert wq.wq_experts_scratch_bytes(T, E, k, N) == T * k * N * 4
    ok = ctypes.c_void_p(0x10000)  # never dereferenced: the call ends before a launch
    assert wq.lib.wq_gemm_w4a16_experts_combine(ok, ok, ok, ok, ok, ok, ok, ok, T * k * N * 4 - 1, T, E, k, N, 128, 128,
                                                None) == wq.WQ_ERR_INVALID_ARG


# ------------------------------------------------------------------ the stream whose memory outputs are
@pytest.mark.parametrize("stream,want", [(0, "default"), (4711, "external 4711")])
def test_outputs_belong_to_the_stream_of_the_handle(monkeypatch, stream, want):
    entered = []

    class Entered:
        def __init__(self, s):
            entered.append(s)

        def __enter__(self):
            return self

        def __exit__(self, *a):
            return False

    class External:
        def __new__(cls, handle, device=None):
            assert handle != 0, "torch would make a new stream for handle 0"
            return f"external {handle}"
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch.cuda, "stream", Entered)
    t = wq._empty_on(stream, torch.device("cpu"))(3, dtype=torch.float16, device="cpu")
    assert t.shape == (3,) and entered == [want]


# ------------------------------------------------------------------ more choices than experts of this device
def test_lists_and_products_take_more_choices_than_experts():
    L, P = wq.lib, ctypes.c_void_p
    ok, odd = P(0x10000), P(0x10002)  # never dereferenced: the misaligned pointer ends every call before a launch
    T, E, k, N, K, g = 5, 4, 8, 32, 128, 128
    assert wq.wq_experts_scratch_bytes(T, E, k, N) == T * k * N * 4
    assert L.wq_expert_lists(ok, T, E, k, ok, odd, None) == wq.WQ_ERR_MISALIGNED
    assert L.wq_gemm_w4a16_experts(ok, ok, ok, odd, ok, T, E, k, N, K, g, 0, None) == wq.WQ_ERR_MISALIGNED
    assert L.wq_gemm_w4a16_experts_combine(ok, ok, ok, odd, ok, ok, ok, ok, 1 << 20, T, E, k, N, K, g,
                                           None) == wq.WQ_ERR_MISALIGNED
    # 32 choices at most, and the routing chooses among E
    assert L.wq_expert_lists(ok, T, E, 33, ok, odd, None) == wq.WQ_ERR_UNSUPPORTED_SHAPE
    assert L.wq_route_experts(ok, 1, None, T, E, k, 0, 1, 1, 1, 1, 1.0, ok, ok, None, None,
                              None) == wq.WQ_ERR_INVALID_ARG


# ------------------------------------------------------------------ the factor of the weights
def test_the_scale_reaches_the_library_in_64_bits():
    # the weights are computed in 64 bits and rounded once, so their factor must not be rounded before
    at = [i for i, t in enumerate(wq.lib.wq_route_experts.argtypes) if t in (ctypes.c_float, ctypes.c_double)]
    assert len(at) == 1 and wq.lib.wq_route_experts.argtypes[at[0]] is ctypes.c_double
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "wq.h")).read()
    args = re.search(r"WQ_API int wq_route_experts\((.*?)\);", text, re.S).group(1).split(",")
    assert args[at[0]].split() == ["double", "scale"]


def test_the_bound_of_32_bit_scores_covers_its_terms():
    # terms of the softmax bound as the kernel's comment derives them, at the largest E
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "bit_weight_quantized_prepack_b200", "csrc", "wq_route.cu")).read()
    err = float(re.search(r"kSoftmaxErr = ([0-9.e-]+)f", text).group(1))
    E = 1024
    own = 2.0 ** -22
    total = 2.0 ** -23 * (2 + 1.7 * math.log(E)) + 37 * 2.0 ** -24
    quotient = 2.0 ** -22 + 2.0 ** -24
    assert own + total + quotient <= err


# ------------------------------------------------------------------ the C ABI
def test_header_and_library_have_the_expert_entry_points():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    declared = re.findall(r"^WQ_API\s+[\w\s\*]+?\b(wq_\w+)\s*\(", open(os.path.join(root, "include", "wq.h")).read(), flags=re.M)
    raw = ctypes.CDLL(wq.LIB_PATH)
    for name in ("wq_route_experts", "wq_expert_lists", "wq_prepacked_bytes_experts", "wq_prepack_experts",
                 "wq_unpack_experts", "wq_gemm_w4a16_experts", "wq_experts_scratch_bytes",
                 "wq_gemm_w4a16_experts_combine"):
        assert name in declared and hasattr(raw, name) and name in wq.__all__


def test_the_version_tells_of_the_changed_signature():
    assert wq.wq_version() >= 10100


@pytest.mark.parametrize("N", [2 ** 31 - 8, 2 ** 31 - 40, 2 ** 31 - 248])
def test_columns_whose_tiles_pass_an_int_are_refused(N):
    assert wq.wq_prepacked_bytes_experts(1, 128, N, 128) == 0
    ok = ctypes.c_void_p(0x10000)  # never dereferenced
    assert wq.lib.wq_gemm_w4a16_experts(ok, ok, ok, ctypes.c_void_p(0x10002), ok, 4, 1, 1, N, 128, 128, 0,
                                        None) == wq.WQ_ERR_UNSUPPORTED_SHAPE
    assert wq.wq_prepacked_bytes_experts(1, 128, 2 ** 31 - 256, 128) >= 64 * (2 ** 31 - 256)
