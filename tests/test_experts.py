"""CPU tests of the expert operators: the oracle's pins (hand-worked routing, lists and layout), the
host-side argument checks of the C ABI and the binding's refusals."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import bit_weight_quantized_prepack_b200 as wq
import oracle
from experts_check import experts_inputs


# ------------------------------------------------------------------ the oracle's pins
def test_route_softmax_by_hand():
    # softmax of (ln 1, ln 2, ln 4, ln 1) = (1, 2, 4, 1) / 8
    x = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    idx, w = oracle.route_experts(x, 2, renorm=False, scale=2.0)
    assert idx.tolist() == [[2, 1]]
    assert np.allclose(w, [[1.0, 0.5]], rtol=1e-15)
    idx, w = oracle.route_experts(x, 3)
    assert idx.tolist() == [[2, 1, 0]]  # experts 0 and 3 tie: the lower index
    assert np.allclose(w, [[4 / 7, 2 / 7, 1 / 7]], rtol=1e-15)


def test_route_bias_and_groups_by_hand():
    # sigmoid of 0 is 1/2 everywhere; the bias alone decides, the weights stay 1/2
    b = np.array([0.0, 0.3, 0.2, 0.2, 0.45, -0.4])
    idx, w = oracle.route_experts(np.zeros((1, 6)), 2, bias=b, score="sigmoid", renorm=False)
    assert idx.tolist() == [[4, 1]] and w.tolist() == [[0.5, 0.5]]
    # three groups of two: best member 0.8, 0.7, 0.95; sums of two 1.3, 1.4, 1.05
    idx, _ = oracle.route_experts(np.zeros((1, 6)), 2, bias=b, score="sigmoid", groups=3, top_groups=1)
    assert idx.tolist() == [[4, 5]]
    idx, _ = oracle.route_experts(np.zeros((1, 6)), 2, bias=b, score="sigmoid", groups=3, top_groups=1, group_top=2)
    assert idx.tolist() == [[2, 3]]


def test_route_leaves_out_what_is_not_finite():
    x = np.array([[math.nan, 1.0, -math.inf, 0.0], [math.nan, -math.inf, math.inf, math.nan]])
    idx, w = oracle.route_experts(x, 3, score="softmax")
    assert idx.tolist() == [[1, 3, -1], [-1, -1, -1]]
    assert w[0, 2] == 0 and w[1].tolist() == [0, 0, 0]
    assert math.isclose(w[0, 0], math.e / (1 + math.e), rel_tol=1e-15)
    idx, _ = oracle.route_experts(np.zeros((1, 3)), 2, bias=[0.0, -math.inf, 1.0])
    assert idx.tolist() == [[2, 0]]


def test_lists_by_hand():
    offsets, rows = oracle.expert_lists([[2, 0], [-1, 2], [0, 7]], 3)
    assert offsets.tolist() == [0, 2, 2, 4] and rows.tolist() == [1, 4, 0, 3]


def test_products_by_hand():
    # one expert of K = 128: codes 8 except two, scales 0.5
    Q = np.full((2, 16, 8), 0x88888888, dtype=np.uint32)
    Q[1, 0, 3] = 0x888888A8        # row 1: q = 10 -> weight 1.0
    Q[1, 1, 3] = 0x8888888F        # row 8: q = 15 -> weight 3.5
    s = np.full((2, 1, 8), 0.5, dtype=np.float16)
    A = np.zeros((1, 128), dtype=np.float16)
    A[0, 1], A[0, 8] = 2.0, -1.0
    y, ad = oracle.experts_product(A, Q.view(np.int32), s, 128, [[1, 0]])
    assert y[0].tolist() == [0, 0, 0, -1.5, 0, 0, 0, 0] and ad[0, 3] == 5.5 and not y[1].any()
    out = oracle.experts_combine(y, np.array([[1, 0]]), np.array([[2.0, 9.0]]))
    assert out[0, 3] == -3.0
    h = oracle.experts_gated(np.array([[0.0, math.log(3.0), 4.0, 2.0]]))
    assert h[0, 0] == 0 and math.isclose(h[0, 1], math.log(3.0) * 0.75 * 2.0, rel_tol=1e-15)


def _golden(golden_dir):
    for line in open(os.path.join(golden_dir, "experts_layout.txt")):
        if line.strip() and not line.startswith("#"):
            kind, shape, place, byte, half = (x.strip() for x in line.split("|"))
            yield kind, [int(v) for v in shape.split()], [int(v) for v in place.split()], int(byte), half


def test_layout_restatement_matches_the_hand_worked_offsets(golden_dir):
    n = 0
    for kind, (K, N, g, gated, e), (k, col), byte, half in _golden(golden_dir):
        Q = np.full((2, K // 8, N), 0x88888888, dtype=np.uint32)
        s = np.zeros((2, K // g, N), dtype=np.float16)
        if kind == "code":
            Q[e, k // 8, col] = (0x88888888 & ~(0xF << (4 * (k % 8)))) | (0x3 << (4 * (k % 8)))
        else:
            s[e, k, col] = 1.0
        buf = oracle.prepack_experts(Q.view(np.int32), s, g, bool(gated))
        ref = oracle.prepack_experts(np.full_like(Q, 0x88888888).view(np.int32), np.zeros_like(s), g, bool(gated))
        changed = np.flatnonzero(buf != ref).tolist()
        if kind == "code":
            assert changed == [byte] and buf[byte] == (0x83 if half == "lo" else 0x38), (k, col)
        else:
            assert changed == [byte + 1] and buf[byte + 1] == 0x3C, (k, col)
        n += 1
    assert n == 23


@pytest.mark.parametrize("E,K,N,g", [(1, 128, 8, 128), (3, 256, 40, 128), (2, 384, 296, 32), (5, 256, 200, 64),
                                     (2, 1280, 520, 640), (4, 512, 72, 512), (1024, 128, 16, 128)])
def test_sizes_agree_with_the_oracle(E, K, N, g):
    assert wq.wq_prepacked_bytes_experts(E, K, N, g) == oracle.prepacked_bytes_experts(E, K, N, g)


@pytest.mark.parametrize("E,K,N,g", [(0, 128, 8, 128), (1025, 128, 8, 128), (2, 100, 8, 100), (2, 128, 12, 128),
                                     (2, 256, 8, 48), (2, 384, 8, 256), (-1, 128, 8, 128)])
def test_unsupported_weights_have_no_size(E, K, N, g):
    assert wq.wq_prepacked_bytes_experts(E, K, N, g) == 0


# ------------------------------------------------------------------ host-side checks of the C ABI
def test_host_side_argument_checks():
    L, P = wq.lib, ctypes.c_void_p
    ok, odd = P(0x10000), P(0x10002)  # never dereferenced: every call below ends before a launch
    INV, UNS, MIS = wq.WQ_ERR_INVALID_ARG, wq.WQ_ERR_UNSUPPORTED_SHAPE, wq.WQ_ERR_MISALIGNED

    def route(T=4, E=8, k=2, fp32=1, score=0, groups=1, top_groups=1, group_top=1, renorm=1, logits=ok, idx=ok, w=ok,
              bias=None, offsets=None, rows=None):
        return L.wq_route_experts(logits, fp32, bias, T, E, k, score, groups, top_groups, group_top, renorm, 1.0, idx, w,
                                  offsets, rows, None)
    assert route(T=-1) == INV and route(E=0) == INV and route(k=0) == INV and route(k=9) == INV
    assert route(E=1025) == UNS and route(E=64, k=33) == UNS and route(T=(1 << 24) + 1) == UNS
    assert route(T=1 << 24, E=64, k=32) == UNS
    assert route(score=2) == INV and route(fp32=2) == INV and route(renorm=2) == INV and route(group_top=3) == INV
    assert route(groups=3) == INV and route(groups=4, top_groups=5) == INV and route(groups=0) == INV
    assert route(groups=8, top_groups=1, k=2) == INV and route(E=130, groups=65, top_groups=2) == UNS
    assert route(logits=None) == INV and route(idx=None) == INV and route(w=None) == INV
    assert route(offsets=ok) == INV and route(rows=ok) == INV
    assert route(logits=odd) == MIS and route(idx=odd) == MIS and route(w=odd) == MIS and route(bias=odd) == MIS
    assert route(offsets=odd, rows=ok) == MIS
    assert route(T=0, logits=None, idx=None, w=None) == wq.WQ_OK

    assert L.wq_expert_lists(ok, 4, 0, 2, ok, ok, None) == INV
    assert L.wq_expert_lists(None, 4, 8, 2, ok, ok, None) == INV
    assert L.wq_expert_lists(ok, 4, 8, 2, None, ok, None) == INV
    assert L.wq_expert_lists(ok, 4, 8, 2, ok, odd, None) == MIS

    assert L.wq_prepack_experts(ok, ok, 2, 256, 24, 128, 1, ok, None) == UNS      # gated: N % 16
    assert L.wq_prepack_experts(ok, ok, 2, 256, 24, 96, 0, ok, None) == INV
    assert L.wq_prepack_experts(ok, ok, 2, 256, 24, 128, 2, ok, None) == INV
    assert L.wq_prepack_experts(ok, None, 2, 256, 24, 128, 0, ok, None) == INV
    assert L.wq_prepack_experts(odd, ok, 2, 256, 24, 128, 0, ok, None) == MIS
    assert L.wq_unpack_experts(ok, 2, 256, 24, 128, 0, ok, P(0x10008), None) == MIS

    def gemm(A=ok, Wp=ok, offsets=ok, rows=ok, Y=ok, T=4, E=8, k=2, N=32, K=128, g=128, gated=0):
        return L.wq_gemm_w4a16_experts(A, Wp, offsets, rows, Y, T, E, k, N, K, g, gated, None)
    assert gemm(T=-1) == INV and gemm(k=0) == INV and gemm(E=0) == INV and gemm(K=100) == UNS and gemm(N=12) == UNS
    assert gemm(g=48) == INV and gemm(gated=1, N=24) == UNS and gemm(gated=3) == INV
    assert gemm(A=None) == INV and gemm(Wp=None) == INV and gemm(offsets=None) == INV and gemm(rows=None) == INV
    assert gemm(Y=None) == INV and gemm(A=P(0x10008)) == MIS and gemm(Y=P(0x10008)) == MIS and gemm(rows=odd) == MIS
    assert gemm(T=0, A=None, Y=None, offsets=None, rows=None) == wq.WQ_OK

    def comb(H=ok, idx=ok, w=ok, Y=ok, scratch=ok, nbytes=1 << 20, T=4, E=8, k=2, N=32, K=128, g=128):
        return L.wq_gemm_w4a16_experts_combine(H, ok, idx, w, ok, ok, Y, scratch, nbytes, T, E, k, N, K, g, None)
    need = wq.wq_experts_scratch_bytes(4, 8, 2, 32)
    assert need > 0 and comb(nbytes=need - 1) == INV and comb(scratch=None) == INV and comb(scratch=P(0x10004)) == MIS
    assert comb(idx=None) == INV and comb(w=None) == INV and comb(H=None) == INV and comb(w=odd) == MIS
    assert comb(T=0, H=None, idx=None, w=None, Y=None, scratch=None) == wq.WQ_OK
    assert wq.wq_experts_scratch_bytes(-1, 8, 2, 32) == 0 and wq.wq_experts_scratch_bytes(4, 64, 33, 32) == 0
    assert wq.wq_experts_scratch_bytes(4, 32, 2, 32) == 0  # few pairs: the form without scratch


# ------------------------------------------------------------------ the binding refuses before any call
class _Recorder:
    PURE = {"wq_prepacked_bytes_experts", "wq_experts_scratch_bytes", "wq_status_string"}

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name in self.PURE:
            return getattr(self.real, name)

        def f(*args):
            self.calls.append(name)
            return 0
        return f


@pytest.fixture
def rec(monkeypatch):
    r = _Recorder(wq.lib)
    monkeypatch.setattr(wq, "lib", r)
    return r


def _layer(**over):
    E, K, N, g, T, k = 4, 256, 48, 128, 3, 2
    d = {n: torch.from_numpy(v) for n, v in experts_inputs(E, K, N, g, T, k, seed=1).items()}
    d.update(Wp=torch.zeros(wq.wq_prepacked_bytes_experts(E, K, N, g), dtype=torch.uint8), N=N, g=g,
             H=torch.zeros((T * k, K), dtype=torch.float16), **{})
    d.update(over)
    return d


@pytest.mark.parametrize("over,err", [
    ({"A": torch.zeros(3 * 256, dtype=torch.float16)}, ValueError),
    ({"A": torch.zeros((3, 256), dtype=torch.bfloat16)}, TypeError),
    ({"A": torch.zeros((3, 512), dtype=torch.float16)[:, ::2]}, ValueError),
    ({"A": torch.zeros((4, 256), dtype=torch.float16)}, ValueError),          # 6 pairs over 4 rows
    ({"Wp": torch.zeros(100, dtype=torch.uint8)}, ValueError),
    ({"offsets": torch.zeros(5, dtype=torch.int64)}, TypeError),
    ({"rows": torch.zeros((3, 2), dtype=torch.int32)}, ValueError),
    ({"Y": torch.zeros((6, 40), dtype=torch.float16)}, ValueError),
    ({"g": 96}, wq.WqError), ({"N": 44}, wq.WqError),
    ({}, TypeError),                                                             # CPU tensors
])
def test_products_refuse(rec, over, err):
    d = _layer(**over)
    with pytest.raises(err):
        wq.wq_gemm_w4a16_experts(d["A"], d["Wp"], d["offsets"], d["rows"], d["N"], d["g"], Y=d.get("Y"))
    assert rec.calls == []


@pytest.mark.parametrize("over,err", [
    ({"H": torch.zeros((5, 256), dtype=torch.float16)}, ValueError),
    ({"w": torch.zeros((2, 3))}, ValueError), ({"w": torch.zeros((3, 2), dtype=torch.float64)}, TypeError),
    ({"idx": torch.zeros((6,), dtype=torch.int32)}, ValueError),
    ({"idx": torch.zeros((3, 2), dtype=torch.int64)}, TypeError),
    ({"rows": torch.zeros(7, dtype=torch.int32)}, ValueError),
    ({"Y": torch.zeros((6, 48), dtype=torch.float16)}, ValueError),
    ({"scratch": torch.zeros(8, dtype=torch.uint8)}, ValueError), ({"scratch": torch.zeros(999)}, TypeError),
    ({"idx": torch.zeros((3, 0), dtype=torch.int32)}, wq.WqError),
    ({}, TypeError),
])
def test_combine_refuses(rec, over, err):
    d = _layer(**over)
    with pytest.raises((err, ValueError) if "idx" in over else err):
        wq.wq_gemm_w4a16_experts_combine(d["H"], d["Wp"], d["idx"], d["w"], d["offsets"], d["rows"], d["N"], d["g"],
                                         Y=d.get("Y"), scratch=d.get("scratch"))
    assert rec.calls == []


def test_route_lists_and_prepack_refuse(rec):
    x = torch.zeros((3, 8))
    for bad in (dict(score="relu"), dict(bias=torch.zeros(7)), dict(idx=torch.zeros((3, 1), dtype=torch.int32)),
                dict(w=torch.zeros((2, 2)))):
        with pytest.raises(ValueError):
            wq.wq_route_experts(x, 2, **bad)
    with pytest.raises(TypeError):
        wq.wq_route_experts(x.bfloat16(), 2)
    with pytest.raises(TypeError):
        wq.wq_route_experts(x.bfloat16(), 2)
    with pytest.raises(ValueError):
        wq.wq_route_experts(x.t(), 2)
    with pytest.raises(wq.WqError):
        wq.wq_route_experts(x, 0)
    with pytest.raises(TypeError):
        wq.wq_expert_lists(torch.zeros((3, 2), dtype=torch.int64), 4)
    with pytest.raises(ValueError):
        wq.wq_expert_lists(torch.zeros((3, 2), dtype=torch.int32), 4, rows=torch.zeros(5, dtype=torch.int32))
    d = _layer()
    with pytest.raises(ValueError):
        wq.wq_prepack_experts(d["Q"][0], d["s"], 128)
    with pytest.raises(ValueError):
        wq.wq_prepack_experts(d["Q"], d["s"][:, :1].contiguous(), 128)
    with pytest.raises(wq.WqError):
        wq.wq_prepack_experts(d["Q"][:, :, :40].contiguous(), d["s"], 128, gated=True)
    with pytest.raises(wq.WqError):
        wq.wq_prepack_experts(d["Q"], d["s"], 0)
    assert rec.calls == []


@pytest.mark.parametrize("k", [9, 2 ** 30])
def test_route_refuses_more_choices_than_experts(rec, k):
    # before any output of that size is allocated
    with pytest.raises(wq.WqError):
        wq.wq_route_experts(torch.zeros((3, 8)), k)
    assert rec.calls == []
