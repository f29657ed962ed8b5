"""GPU tests of the expert operators against the fp64 oracle: routing, lists, the layout pass, the
products by expert, the combined down product, and the layer as a run of them."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

import bit_weight_quantized_prepack_b200 as wq  # noqa: E402
import oracle  # noqa: E402
from experts_check import combine_bound, experts_inputs, gated_bound, product_bound  # noqa: E402


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def f64(t):
    return t.double().cpu().numpy()


def status_ok():
    assert wq.wq_get_device_status() == wq.WQ_OK


# ------------------------------------------------------------------ routing
ROUTES = [
    # T, E, k, dtype, score, bias, groups, top_groups, group_top, renorm, scale
    (1, 8, 2, "fp16", "softmax", False, 1, 1, 1, True, 1.0),
    (1, 1, 1, "fp32", "sigmoid", True, 1, 1, 1, True, 1.0),
    (5, 128, 8, "fp16", "softmax", False, 1, 1, 1, True, 1.0),
    (33, 60, 4, "fp16", "softmax", False, 1, 1, 1, False, 1.0),
    (64, 256, 8, "fp32", "sigmoid", True, 8, 4, 2, True, 2.5),
    (7, 256, 8, "fp32", "softmax", True, 8, 3, 1, True, 1.0),
    (65, 72, 6, "fp16", "sigmoid", False, 4, 2, 2, False, 1.0),
    (19, 40, 10, "fp32", "softmax", False, 5, 2, 2, True, 0.5),
    (3, 33, 32, "fp32", "sigmoid", False, 1, 1, 1, True, 1.0),
    (9, 96, 32, "fp16", "softmax", True, 1, 1, 1, False, 1.0),
    (4, 512, 16, "fp32", "sigmoid", True, 64, 5, 2, True, 1.0),
    (5, 1024, 32, "fp16", "softmax", False, 1, 1, 1, True, 1.0),
    (3, 1024, 8, "fp32", "sigmoid", True, 32, 4, 1, True, 1.0),
    (300, 16, 1, "fp32", "softmax", True, 1, 1, 1, False, 1.0),
    (130, 200, 7, "fp32", "softmax", False, 8, 8, 1, True, 1.0),
]


def _check_route(x, k, bias, **kw):
    idx_ref, w_ref = oracle.route_experts(x.double().cpu().numpy(), k, bias=None if bias is None else f64(bias), **kw)
    idx, w, offsets, rows = wq.wq_route_experts(x, k, bias=bias, lists=True, **kw)
    assert np.array_equal(idx.cpu().numpy(), idx_ref)
    # fp32: half a step, and the 64-bit score's own error far below it
    assert np.all(np.abs(f64(w) - w_ref) <= 2.0 ** -24 * np.abs(w_ref) * 1.001 + 2.0 ** -149)
    o_ref, r_ref = oracle.expert_lists(idx_ref, x.shape[1])
    assert np.array_equal(offsets.cpu().numpy(), o_ref)
    assert np.array_equal(rows.cpu().numpy()[:r_ref.size], r_ref)


@pytest.mark.parametrize("T,E,k,dtype,score,bias,groups,top_groups,group_top,renorm,scale", ROUTES)
def test_route(T, E, k, dtype, score, bias, groups, top_groups, group_top, renorm, scale):
    gen = torch.Generator(device="cuda").manual_seed(T * 1000 + E)
    x = (torch.randn((T, E), generator=gen, device="cuda") * 2).to(torch.float16 if dtype == "fp16" else torch.float32)
    b = torch.randn(E, generator=gen, device="cuda") * 0.2 if bias else None
    _check_route(x, k, b, score=score, groups=groups, top_groups=top_groups, group_top=group_top, renorm=renorm,
                 scale=scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_ties_and_near_ties(score, bias, groups):
    # equal logits, logits one unit in the last place apart, and far ones whose scores vanish or saturate
    T, E, k = 12, 64, 6
    x = torch.zeros((T, E), dtype=torch.float32)
    x[1] = 1.0
    x[2, 40:] = float(np.nextafter(np.float32(0), np.float32(1)))
    x[3] = torch.where(torch.arange(E) % 3 == 0, float(np.nextafter(np.float32(1), np.float32(2))), 1.0)
    x[4] = torch.arange(E).float() * -30
    x[5] = torch.arange(E).float() * 30
    x[6, 10] = x[6, 50] = 5.0
    x[7] = -1.0e30
    x[7, 33] = -2.0e30
    x[8] = 3.0e38
    x[9] = -float(np.finfo(np.float32).max)
    x[10, ::2] = -0.0
    x[11] = torch.tensor(np.random.default_rng(0).integers(0, 3, E)).float()
    b = (torch.arange(E) % 4).float() * 0.25 if bias else None
    _check_route(x.cuda(), k, None if b is None else b.cuda(), score=score, groups=groups,
                 top_groups=min(groups, 2), group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_not_finite(score, groups):
    T, E, k = 6, 32, 5
    x = torch.randn((T, E), generator=torch.Generator().manual_seed(3))
    x[0] = math.nan
    x[1] = -math.inf
    x[2, 3:] = -math.inf
    x[3, ::2] = math.nan
    x[4, 5], x[4, 6] = math.inf, -math.inf
    b = torch.zeros(E)
    b[7], b[9], b[11] = -math.inf, math.nan, math.inf
    b[24:] = -math.inf
    for bias in (None, b.cuda()):
        for renorm in (True, False):
            _check_route(x.cuda(), k, bias, score=score, groups=groups, top_groups=min(groups, 2), renorm=renorm)


def test_route_empty_and_given_outputs():
    x = torch.zeros((0, 8), device="cuda")
    idx, w, offsets, rows = wq.wq_route_experts(x, 2, lists=True)
    assert idx.shape == (0, 2) and rows.numel() == 0 and offsets.tolist() == [0] * 9
    x = torch.randn((3, 8), device="cuda")
    idx = torch.empty((3, 2), dtype=torch.int32, device="cuda")
    w = torch.empty((3, 2), device="cuda")
    i2, w2 = wq.wq_route_experts(x, 2, idx=idx, w=w)
    assert i2 is idx and w2 is w
    _check_route(torch.randn((9, 9), device="cuda", dtype=torch.float16)[1:], 3, None)  # a 2-byte aligned slice


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (3, 5, 5), (257, 60, 4), (4096, 128, 8), (9001, 1000, 3),
                                   (70000, 8, 2), (33000, 300, 32)])
@pytest.mark.parametrize("kind", ["spread", "one", "padded"])
def test_lists(T, E, k, kind):
    rng = np.random.default_rng(T + E)
    idx = rng.integers(0, E, (T, k)).astype(np.int32)
    if kind == "one":
        idx[:] = E - 1
    if kind == "padded":
        idx[rng.random((T, k)) < 0.4] = -1
        idx[rng.random((T, k)) < 0.1] = E
        idx[0, 0] = 2 ** 31 - 1
        idx[-1, -1] = -2 ** 31
    rows = torch.full((T * k,), -7, dtype=torch.int32, device="cuda")
    offsets, rows = wq.wq_expert_lists(dev(idx), E, rows=rows)
    flat = idx.reshape(-1)
    ok = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(ok, flat, E).astype(np.int64), kind="stable")[:ok.sum()]
    assert np.array_equal(offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=E))]))
    got = rows.cpu().numpy()
    assert np.array_equal(got[:order.size], order)
    assert np.all(got[order.size:] == -7)  # left as they were


# ------------------------------------------------------------------ layout pass
@pytest.mark.parametrize("E,K,N,g,gated", [(1, 128, 8, 128, False), (3, 256, 40, 128, False), (2, 384, 296, 32, False),
                                           (5, 256, 208, 64, True), (2, 1280, 528, 640, True), (4, 512, 72, 512, False),
                                           (3, 256, 16, 256, True)])
def test_prepack_bytes_and_round_trip(E, K, N, g, gated):
    d = experts_inputs(E, K, N, g, 1, 1, seed=K + N)
    Q, s = dev(d["Q"]), dev(d["s"])
    Wp = torch.zeros(wq.wq_prepacked_bytes_experts(E, K, N, g), dtype=torch.uint8, device="cuda")
    wq.wq_prepack_experts(Q, s, g, gated=gated, Wp=Wp)
    assert np.array_equal(Wp.cpu().numpy(), oracle.prepack_experts(d["Q"], d["s"], g, gated))
    Q2, s2 = wq.wq_unpack_experts(Wp, E, K, N, g, gated=gated)
    assert torch.equal(Q2, Q) and torch.equal(s2.view(torch.int16), s.view(torch.int16))


# ------------------------------------------------------------------ products
PRODUCTS = [
    # E, K, N, g, T, k, skew, padded
    (1, 128, 8, 128, 1, 1, 0, 0),
    (4, 128, 16, 128, 1, 2, 0, 0),
    (8, 256, 48, 128, 1, 8, 0, 0),
    (8, 1024, 272, 128, 3, 2, 0, 0),
    (5, 384, 80, 32, 7, 3, 1, 0),
    (6, 640, 112, 64, 13, 4, 0, 0.3),
    (3, 512, 144, 512, 9, 2, 0, 0),
    (3, 1280, 48, 640, 5, 1, 0, 0),
    (4, 512, 96, 256, 33, 2, 2, 0),
    (2, 256, 304, 128, 50, 2, 0, 0.1),
    (7, 384, 176, 384, 64, 3, 1, 0),
    (40, 256, 64, 64, 100, 6, 2, 0),
    (3, 256, 144, 32, 129, 2, 0, 0.2),
    (2, 512, 272, 128, 300, 1, 0, 0),
    (5, 384, 400, 128, 700, 2, 1, 0.1),
    (2, 256, 144, 256, 515, 1, 3, 0),
    (130, 128, 16, 128, 1100, 4, 1, 0),
    (1024, 128, 16, 128, 50, 32, 0, 0),
    (3, 256, 528, 64, 1025, 3, 0, 0),
    (2, 384, 288, 32, 260, 1, 0, 0.1),
    (3, 640, 176, 64, 150, 2, 0, 0),
    (2, 768, 560, 256, 130, 1, 0, 0),
    (2, 128, 272, 128, 129, 1, 0, 0),
    (4, 1024, 1040, 128, 1030, 2, 2, 0),
    # few pairs of many experts
    (64, 768, 264, 128, 1, 8, 0, 0),
    (33, 384, 48, 32, 2, 4, 0, 0),
    (128, 256, 144, 64, 3, 8, 0, 0.4),
    (16, 512, 80, 512, 4, 1, 0, 0),
    (40, 1280, 72, 640, 5, 2, 0, 0.4),
    (1024, 128, 8, 128, 200, 1, 0, 0.1),
    # rows too long for two, or for one, of their places in shared memory
    (3, 11008, 72, 128, 5, 2, 0, 0),
    (4, 8192, 48, 64, 9, 3, 1, 0.2),
    (2, 16384, 48, 128, 3, 2, 0, 0),
]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("E,K,N,g,T,k,skew,padded", PRODUCTS)
def test_products(E, K, N, g, T, k, skew, padded, gated):
    if gated:
        N = (N + 15) // 16 * 16
    d = experts_inputs(E, K, N, g, T, k, seed=E * 7 + T, padded=padded, skew=skew)
    Wp = wq.wq_prepack_experts(dev(d["Q"]), dev(d["s"]), g, gated=gated)
    n_out = N // 2 if gated else N
    Y = torch.full((T * k, n_out), -77.0, dtype=torch.float16, device="cuda")
    args = (dev(d["A"]), Wp, dev(d["offsets"]), dev(d["rows"]), N, g)
    wq.wq_gemm_w4a16_experts(*args, gated=gated, Y=Y)
    status_ok()
    y, ad = oracle.experts_product(d["A"], d["Q"], d["s"], g, d["idx"])
    ref = oracle.experts_gated(y) if gated else y
    bound = (gated_bound if gated else product_bound)(y, ad, K)
    listed = ~np.isnan(y).all(1)
    got = f64(Y)
    assert np.all(got[~listed] == -77.0)
    err = np.abs(got - ref)[listed]
    assert np.all(err <= bound[listed]), (err / bound[listed]).max()
    Y2 = wq.wq_gemm_w4a16_experts(*args, gated=gated)
    assert torch.equal(Y2[torch.from_numpy(listed).cuda()], Y[torch.from_numpy(listed).cuda()])  # the same bits again


@pytest.mark.parametrize("E,K,N,g,T,k,skew,padded", PRODUCTS)
def test_combine(E, K, N, g, T, k, skew, padded):
    d = experts_inputs(E, K, N, g, T, k, seed=E * 5 + T, padded=padded, skew=skew, by_pair=True)
    Wp = wq.wq_prepack_experts(dev(d["Q"]), dev(d["s"]), g)
    args = (dev(d["A"]), Wp, dev(d["idx"]), dev(d["w"]), dev(d["offsets"]), dev(d["rows"]), N, g)
    # a scratch of NaN: nothing of what it held may enter
    scratch = torch.full((wq.wq_experts_scratch_bytes(T, E, k, N),), 255, dtype=torch.uint8, device="cuda")
    Y = wq.wq_gemm_w4a16_experts_combine(*args, scratch=scratch)
    status_ok()
    y, ad = oracle.experts_product(d["A"], d["Q"], d["s"], g, d["idx"], by_pair=True)
    ref = oracle.experts_combine(y, d["idx"], d["w"])
    # a bound for pairs that are rounded before the sum also holds where they are not
    bound = combine_bound(y, ad, d["idx"], d["w"], K)
    err = np.abs(f64(Y) - ref)
    assert np.all(err <= bound), (err / bound).max()
    assert torch.equal(wq.wq_gemm_w4a16_experts_combine(*args), Y)


def test_weights_come_back_exactly():
    # activations of one 1 per token: the products are the weights, exact in fp16 for scales of 2^-6
    E, K, N, g = 3, 256, 72, 128
    d = experts_inputs(E, K, N, g, 1, 1, seed=5)
    s = np.full_like(d["s"], 2.0 ** -6)
    Wp = wq.wq_prepack_experts(dev(d["Q"]), dev(s), g)
    for e in range(E):
        for reps in (1, 3):
            A = torch.eye(K, dtype=torch.float16, device="cuda").repeat(reps, 1)
            for T in (K * reps, 5):
                offsets, rows = wq.wq_expert_lists(torch.full((T, 1), e, dtype=torch.int32, device="cuda"), E)
                Y = wq.wq_gemm_w4a16_experts(A[:T].contiguous(), Wp, offsets, rows, N, g)
                W = oracle.dequant(oracle.unpack_codes(d["Q"][e]), s[e], g)
                assert np.array_equal(f64(Y), np.tile(W, (reps, 1))[:T])


@pytest.mark.parametrize("T", [2, 40, 600])
def test_not_finite_rows_stay_in_their_rows(T):
    E, K, N, g, k = 4, 256, 80, 128, 2
    d = experts_inputs(E, K, N, g, T, k, seed=T)
    bad = [0, T - 1]
    A = d["A"].copy()
    A[bad[0], 5], A[bad[1], 200] = np.inf, np.nan
    Wp = wq.wq_prepack_experts(dev(d["Q"]), dev(d["s"]), g)
    call = lambda a: wq.wq_gemm_w4a16_experts(dev(a), Wp, dev(d["offsets"]), dev(d["rows"]), N, g)  # noqa: E731
    Y, Y0 = call(A), call(d["A"])
    keep = [p for p in range(T * k) if p // k not in bad]
    assert torch.equal(Y[keep], Y0[keep])
    assert not torch.isfinite(Y[(T - 1) * k]).any()


@pytest.mark.parametrize("T,E", [(3, 4), (200, 4)])
def test_lists_that_lead_outside_are_refused_on_the_device(T, E):
    # entries of rows outside the pairs are skipped and reported; offsets are clamped and made non-decreasing
    K, N, g, k = 256, 48, 128, 2
    d = experts_inputs(E, K, N, g, T, k, seed=2)
    Wp = wq.wq_prepack_experts(dev(d["Q"]), dev(d["s"]), g)
    good = wq.wq_gemm_w4a16_experts(dev(d["A"]), Wp, dev(d["offsets"]), dev(d["rows"]), N, g)
    status_ok()
    rows = d["rows"].copy()
    lost = [int(rows[0]), int(rows[-1])]
    rows[0], rows[-1] = -1, T * k
    Y = torch.full((T * k, N), -77.0, dtype=torch.float16, device="cuda")
    wq.wq_gemm_w4a16_experts(dev(d["A"]), Wp, dev(d["offsets"]), dev(rows), N, g, Y=Y)
    assert wq.wq_get_device_status() == wq.WQ_ERR_INVALID_ARG
    status_ok()  # cleared
    keep = [p for p in range(T * k) if p not in lost]
    assert torch.equal(Y[keep], good[keep]) and bool((Y[lost] == -77.0).all())
    offsets = d["offsets"].copy()
    offsets[0], offsets[-1] = -5, 2 ** 31 - 1
    Y = wq.wq_gemm_w4a16_experts(dev(d["A"]), Wp, dev(offsets), dev(d["rows"]), N, g)
    assert torch.equal(Y, good)
    offsets[1:] = offsets[1:][::-1].copy()  # decreasing: only memory safety is promised
    wq.wq_gemm_w4a16_experts(dev(d["A"]), Wp, dev(offsets), dev(d["rows"]), N, g)
    status_ok()


def _layer(T, E, k, H, I, g, seed=0):
    up = experts_inputs(E, H, 2 * I, g, T, k, seed=seed)
    down = experts_inputs(E, I, H, g if I % g == 0 else I, T, k, seed=seed + 1)
    gd = g if I % g == 0 else I
    Wu = wq.wq_prepack_experts(dev(up["Q"]), dev(up["s"]), g, gated=True)
    Wd = wq.wq_prepack_experts(dev(down["Q"]), dev(down["s"]), gd)
    x = dev(up["A"])
    logits = torch.randn((T, E), generator=torch.Generator().manual_seed(seed)).cuda()

    def run(x=x, logits=logits, stream=None):
        idx, w, offsets, rows = wq.wq_route_experts(logits, k, lists=True, stream=stream)
        h = wq.wq_gemm_w4a16_experts(x, Wu, offsets, rows, 2 * I, g, gated=True, stream=stream)
        return wq.wq_gemm_w4a16_experts_combine(h, Wd, idx, w, offsets, rows, H, gd, stream=stream), idx, w, h
    return up, down, gd, x, logits, run


@pytest.mark.parametrize("T", [1, 6, 90, 500])
def test_a_layer(T):
    E, k, H, I, g = 8, 2, 512, 384, 128
    up, down, gd, x, logits, run = _layer(T, E, k, H, I, g, seed=T)
    y, idx, w, h = run()
    status_ok()
    idx_ref, w_ref = oracle.route_experts(f64(logits), k)
    assert np.array_equal(idx.cpu().numpy(), idx_ref)
    u, uad = oracle.experts_product(up["A"], up["Q"], up["s"], g, idx_ref)
    assert np.all(np.abs(f64(h) - oracle.experts_gated(u)) <= gated_bound(u, uad, H))
    # the down product of the h that it was given
    v, vad = oracle.experts_product(f64(h), down["Q"], down["s"], gd, idx_ref, by_pair=True)
    ref = oracle.experts_combine(v, idx_ref, w_ref)
    assert np.all(np.abs(f64(y) - ref) <= combine_bound(v, vad, idx_ref, w_ref, I) + 2.0 ** -23 * np.abs(ref))


@pytest.mark.parametrize("T", [1, 24, 500])
def test_layer_in_a_graph_and_on_other_streams(T):
    E, k, H, I, g = 8, 2, 512, 256, 64
    *_, x, logits, run = _layer(T, E, k, H, I, g, seed=9)
    want = run()[0].clone()
    x2, l2 = torch.randn_like(x), torch.randn_like(logits)
    want2 = run(x2, l2)[0].clone()
    # another stream, given as a Stream and as a handle, while the current one works too
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = []
    for i in range(6):
        outs.append((run(stream=s)[0], want))
        outs.append((run(x2, l2)[0], want2))
        outs.append((run(stream=s.cuda_stream)[0], want))
    torch.cuda.synchronize()
    for got, ref in outs:
        assert torch.equal(got, ref)
    # two graphs of the same calls, replayed at the same time on two streams
    graphs = []
    for xx, ll in ((x, logits), (x2, l2)):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            y = run(xx, ll)[0]
        graphs.append((gr, y))
    s2 = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        for (gr, _), st in zip(graphs, (s, s2)):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], want) and torch.equal(graphs[1][1], want2)
    # new contents in the captured inputs
    x.copy_(x2)
    logits.copy_(l2)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], want2)
    status_ok()


def test_empty_calls():
    E, K, N, g = 4, 128, 16, 128
    d = experts_inputs(E, K, N, g, 3, 2, seed=0)
    Wp = wq.wq_prepack_experts(dev(d["Q"]), dev(d["s"]), g)
    z = torch.zeros((0, K), dtype=torch.float16, device="cuda")
    off, rows = torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    assert wq.wq_gemm_w4a16_experts(z, Wp, off, rows, N, g).shape == (0, N)
    idx = torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    assert wq.wq_gemm_w4a16_experts_combine(z, Wp, idx, torch.zeros((0, 2), device="cuda"), off, rows, N, g).shape == (0, N)
    # every place padded: nothing is computed, the sums are zeros
    idx = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    off, rows = wq.wq_expert_lists(idx, E)
    Y = wq.wq_gemm_w4a16_experts_combine(torch.randn((6, K), device="cuda").half(), Wp, idx,
                                         torch.ones((3, 2), device="cuda"), off, rows, N, g)
    assert not Y.any()
    status_ok()


def test_memory_of_a_side_stream_stays_with_it():
    # what a call on another stream returned and the caller dropped must not be handed to the current
    # stream while that other stream may still write it
    x = torch.randn((4096, 256), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        out = wq.wq_route_experts(x, 8, lists=True, stream=stream)
        held = {t.data_ptr() for t in out}
        shapes = [(t.shape, t.dtype) for t in out]
        del out
        fresh = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype in shapes]
        assert not held & {t.data_ptr() for t in fresh}
    torch.cuda.synchronize()
    status_ok()


def test_layers_and_a_dense_product_at_the_same_time():
    # few pairs, few rows, many rows and a dense layer on four streams, unordered among each other
    runs = [_layer(T, 8, 2, 512, 256, 128, seed=T)[-1] for T in (1, 40, 700)]
    d = experts_inputs(1, 512, 2048, 128, 1, 1, seed=3)
    Wd = wq.wq_prepack(dev(d["Q"][0]), dev(d["s"][0]), 128)
    A = torch.randn((96, 512), device="cuda").half()
    runs.append(lambda stream=None: (wq.wq_gemm_w4a16(A, Wd, 2048, 128, stream=stream),))
    want = [r()[0].clone() for r in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for i, (r, st) in enumerate(zip(runs, streams)):
            with torch.cuda.stream(st):
                outs.append((i, r(stream=st)[0]))
    torch.cuda.synchronize()
    for i, y in outs:
        assert torch.equal(y, want[i])
    status_ok()


@pytest.mark.parametrize("T", [1, 30, 400])
def test_the_same_expert_twice(T):
    # choices of one token that name the same expert are pairs of their own
    E, K, N, g, k = 6, 384, 72, 128, 3
    d = experts_inputs(E, K, N, g, T, k, seed=T)
    idx = d["idx"].copy()
    idx[:, 1] = idx[:, 0]
    idx[::2, 2] = idx[::2, 0]
    w = np.random.default_rng(T).uniform(0.1, 1.0, (T, k)).astype(np.float32)
    H = (np.random.default_rng(T + 1).standard_normal((T * k, K)) * 0.5).astype(np.float16)
    Wp = wq.wq_prepack_experts(dev(d["Q"]), dev(d["s"]), g)
    offsets, rows = wq.wq_expert_lists(dev(idx), E)
    o_ref, r_ref = oracle.expert_lists(idx, E)
    assert np.array_equal(offsets.cpu().numpy(), o_ref) and np.array_equal(rows.cpu().numpy(), r_ref)
    y = wq.wq_gemm_w4a16_experts_combine(dev(H), Wp, dev(idx), dev(w), offsets, rows, N, g)
    v, vad = oracle.experts_product(H.astype(np.float64), d["Q"], d["s"], g, idx, by_pair=True)
    ref = oracle.experts_combine(v, idx, w.astype(np.float64))
    assert np.all(np.abs(f64(y) - ref) <= combine_bound(v, vad, idx, w.astype(np.float64), K))
    status_ok()
