"""GPU tests of the expert operators at their edges, against the fp64 oracle."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

import bit_weight_quantized_prepack_b200 as wq  # noqa: E402
import oracle  # noqa: E402
from experts_check import combine_bound_once, experts_inputs, gated_bound, product_bound  # noqa: E402


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------ the combined product rounds once
@pytest.mark.parametrize("large", [False, True])
@pytest.mark.parametrize("E,K,N,g,T,k,padded", [
    (64, 768, 264, 128, 1, 8, 0), (40, 1280, 72, 640, 5, 2, 0.4), (33, 384, 48, 32, 2, 4, 0),           # few pairs
    (8, 1024, 272, 128, 3, 2, 0), (6, 640, 112, 64, 13, 4, 0.3), (4, 512, 96, 512, 20, 2, 0),            # few rows
    (5, 384, 80, 32, 40, 3, 0.2),
    (2, 512, 272, 128, 128, 1, 0), (3, 640, 528, 64, 200, 2, 0.1), (2, 384, 96, 384, 90, 2, 0),          # many rows
    (4, 256, 1040, 32, 260, 4, 0.1)])
def test_combine_rounds_once(E, K, N, g, T, k, padded, large):
    d = experts_inputs(E, K, N, g, T, k, seed=E * 3 + T, padded=padded, by_pair=True)
    s, w = d["s"], d["w"]
    if large:  # products far beyond fp16's 65504, weights that bring their sums back
        s = (s.astype(np.float32) * 2.0 ** 17 / 8).astype(np.float16)
        w = (w * 2.0 ** -12).astype(np.float32)
    A = (d["A"] * (64 if large else 1)).astype(np.float16)
    Wp = wq.wq_prepack_experts(dev(d["Q"]), dev(s), g)
    Y = wq.wq_gemm_w4a16_experts_combine(dev(A), Wp, dev(d["idx"]), dev(w), dev(d["offsets"]), dev(d["rows"]), N, g)
    assert wq.wq_get_device_status() == wq.WQ_OK
    y, ad = oracle.experts_product(A, d["Q"], s, g, d["idx"], by_pair=True)
    if large:
        assert np.nanmax(np.abs(y)) > 4 * 65504
    ref = oracle.experts_combine(y, d["idx"], w)
    assert np.abs(ref).max() < 60000
    err, bound = np.abs(f64(Y) - ref), combine_bound_once(y, ad, d["idx"], w, K)
    assert np.all(err <= bound), np.nanmax(err / bound)


# ------------------------------------------------------------------ every count of rows of a tile
@pytest.mark.parametrize("K,N,g", [(256, 272, 128), (384, 272, 384), (128, 304, 64), (128, 272, 32)])
def test_every_row_count_of_an_expert(K, N, g):
    # n of 200 tokens take expert 0, the others expert 1: many rows an expert on average
    E, T = 2, 200
    d = experts_inputs(E, K, N, g, T, 1, seed=K + g)
    Wp = wq.wq_prepack_experts(dev(d["Q"]), dev(d["s"]), g)
    Wg = wq.wq_prepack_experts(dev(d["Q"]), dev(d["s"]), g, gated=True)
    A = dev(d["A"])
    per = [oracle.experts_product(d["A"], d["Q"], d["s"], g, np.full((T, 1), e)) for e in range(E)]
    rng = np.random.default_rng(0)
    for n in range(1, 129):
        idx = np.ones((T, 1), dtype=np.int32)
        idx[rng.permutation(T)[:n]] = 0
        offsets, rows = wq.wq_expert_lists(dev(idx), E)
        y, ad = (np.where(idx == 0, per[0][i], per[1][i]) for i in (0, 1))
        for gated, wp, ref, bound in ((False, Wp, y, product_bound(y, ad, K)),
                                      (True, Wg, oracle.experts_gated(y), gated_bound(y, ad, K))):
            got = f64(wq.wq_gemm_w4a16_experts(A, wp, offsets, rows, N, g, gated=gated))
            assert np.all(np.abs(got - ref) <= bound), (n, gated)
    assert wq.wq_get_device_status() == wq.WQ_OK


# ------------------------------------------------------------------ the default stream by its handle
def test_the_default_stream_by_its_handle():
    # what a call on stream 0 returned and the caller dropped goes to later work of the default stream only
    x = torch.randn((4096, 256), device="cuda")
    side = [torch.cuda.Stream() for _ in range(40)]  # more than torch keeps of them: all are in here
    for handle in (0, torch.cuda.default_stream().cuda_stream):
        want = wq.wq_route_experts(x, 8, lists=True)
        torch.cuda.synchronize()
        out = wq.wq_route_experts(x, 8, lists=True, stream=handle)
        held = {t.data_ptr() for t in out}
        shapes = [(t.shape, t.dtype) for t in out]
        del out
        for s in side:
            with torch.cuda.stream(s):
                assert not held & {torch.empty(shape, dtype=dtype, device="cuda").fill_(-3).data_ptr()
                                   for shape, dtype in shapes}
        outs = []
        for i in range(20):
            outs.append(wq.wq_route_experts(x, 8, lists=True, stream=handle))
            with torch.cuda.stream(side[i]):
                for shape, dtype in shapes:
                    torch.empty(shape, dtype=dtype, device="cuda").fill_(-3)
        torch.cuda.synchronize()
        for got in outs:
            assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------ routing
def _check_route(x, k, bias=None, **kw):
    idx_ref, w_ref = oracle.route_experts(x.double().cpu().numpy(), k, bias=None if bias is None else f64(bias), **kw)
    idx, w, offsets, rows = wq.wq_route_experts(x, k, bias=bias, lists=True, **kw)
    assert np.array_equal(idx.cpu().numpy(), idx_ref)
    # fp32: half a step, and the 64-bit score's own error far below it
    assert np.all(np.abs(f64(w) - w_ref) <= 2.0 ** -24 * np.abs(w_ref) * 1.001 + 2.0 ** -149)
    o_ref, r_ref = oracle.expert_lists(idx_ref, x.shape[1])
    assert np.array_equal(offsets.cpu().numpy(), o_ref)
    assert np.array_equal(rows.cpu().numpy()[:r_ref.size], r_ref)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("E", [32, 320])
def test_route_groups_whose_sums_pass_the_range_of_32_bits(score, sign, E):
    # biases of the type's lowest (largest) value: sums of two of them are told apart in 64 bits
    top = float(np.finfo(np.float32).max)
    b = torch.full((4, E // 4), -top)
    b[0, :], b[1, 2:4], b[2, 1], b[2, 5], b[3, 6:8] = -top, -2.0e38, -2.4e38, -2.6e38, 0.5
    b = (sign * b).reshape(-1).cuda()
    x = torch.randn((40, E), generator=torch.Generator().manual_seed(E)).cuda()
    for top_groups in (1, 2, 3):
        _check_route(x, 5, b, score=score, groups=4, top_groups=top_groups, group_top=2)


# ------------------------------------------------------------------ some of the experts of a layer
@pytest.mark.parametrize("T", [1, 9, 300, 2500])
@pytest.mark.parametrize("E", [1, 4])
def test_more_choices_than_experts_here(T, E):
    # 8 of 32 experts a token, E of them on this device
    K, N, g, k = 256, 80, 128, 8
    d = experts_inputs(32, K, N, g, T, k, seed=T + E, by_pair=True)
    idx = d["idx"] - 8
    Q, s = d["Q"][8:8 + E], d["s"][8:8 + E]
    Wp = wq.wq_prepack_experts(dev(Q), dev(s), g)
    offsets, rows = wq.wq_expert_lists(dev(idx), E)
    here = (idx >= 0) & (idx < E)
    o_ref, r_ref = oracle.expert_lists(np.where(here, idx, -1), E)
    assert np.array_equal(offsets.cpu().numpy(), o_ref) and np.array_equal(rows.cpu().numpy()[:r_ref.size], r_ref)
    seen = np.where(here, idx, -1)
    A = d["A"][:T]
    Y = torch.full((T * k, N), -77.0, dtype=torch.float16, device="cuda")
    wq.wq_gemm_w4a16_experts(dev(A), Wp, offsets, rows, N, g, Y=Y)
    y, ad = oracle.experts_product(A, Q, s, g, seen)
    listed = here.reshape(-1)
    assert np.all(f64(Y)[~listed] == -77.0)
    assert np.all(np.abs(f64(Y) - y)[listed] <= product_bound(y, ad, K)[listed])
    out = wq.wq_gemm_w4a16_experts_combine(dev(d["A"]), Wp, dev(idx), dev(d["w"]), offsets, rows, N, g)
    y, ad = oracle.experts_product(d["A"], Q, s, g, seen, by_pair=True)
    ref = oracle.experts_combine(y, seen, d["w"])
    assert np.all(np.abs(f64(out) - ref) <= combine_bound_once(y, ad, seen, d["w"], K))
    assert wq.wq_get_device_status() == wq.WQ_OK


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_with_a_scale_that_32_bits_do_not_hold(score, renorm):
    # 2.446 is off by 0.68 * 2^-24 of itself in fp32: more than half of a weight's own rounding again
    x = torch.randn((500, 64), generator=torch.Generator().manual_seed(1)).cuda()
    for scale in (2.446, 0.1, 16.0 / 3):
        _check_route(x, 6, score=score, renorm=renorm, scale=scale)


# ------------------------------------------------------------------ the gate over its whole range
@pytest.mark.parametrize("E,T", [(64, 9), (4, 30), (2, 300)])  # few pairs, few rows, many rows
def test_gated_over_the_whole_range_of_the_gate(E, T):
    # rows of one 1 make the sums the weights themselves, exact in fp32: gates from -110 to 110, ups to
    # 59904 so that what a gate of -24 leaves is still above fp16's smallest
    K, N, g = 128, 64, 128
    rng = np.random.default_rng(E)
    q = rng.integers(0, 16, (E, K, N))
    q[:, :, N // 2:] = rng.choice([0, 1, 15], (E, K, N // 2))
    Q = np.zeros((E, K // 8, N), dtype=np.uint32)
    for j in range(8):
        Q |= q[:, j::8].astype(np.uint32) << np.uint32(4 * j)
    s = np.empty((E, 1, N), dtype=np.float16)
    s[:, 0, :N // 2] = 13.75 * 2.0 ** -rng.integers(0, 8, (E, N // 2))
    s[:, 0, N // 2:] = 7486.0 * 2.0 ** -rng.integers(0, 10, (E, N // 2))
    A = np.zeros((T, K), dtype=np.float16)
    A[np.arange(T), rng.integers(0, K, T)] = 1.0
    idx = rng.integers(0, E, (T, 1)).astype(np.int32)
    Wp = wq.wq_prepack_experts(dev(Q.view(np.int32)), dev(s), g, gated=True)
    offsets, rows = wq.wq_expert_lists(dev(idx), E)
    got = f64(wq.wq_gemm_w4a16_experts(dev(A), Wp, offsets, rows, N, g, gated=True))
    y, _ = oracle.experts_product(A, Q.view(np.int32), s, g, idx)
    gate = y[:, :N // 2]
    assert gate.min() < -100 and gate.max() > 90
    ref = oracle.experts_gated(y)
    # fp32's quotient and product of such ups may also pass below the normal range: 2^-100 covers it
    rel = (8 + 1.18 * np.abs(gate)) * 2.0 ** -23
    over = np.abs(ref) * (1 + 2.0 ** -10) >= 65504
    bound = rel * np.abs(ref) + np.maximum(2.0 ** -11 * np.abs(ref) * (1 + 2.0 ** -10), 2.0 ** -25) + 2.0 ** -100
    assert np.all(np.abs(got - ref)[~over] <= bound[~over])
    assert np.all(np.abs(got[over]) >= 65400) and np.all(np.sign(got[over]) == np.sign(ref[over]))


# ------------------------------------------------------------------ sizes on both sides of each switch of kernel
@pytest.mark.parametrize("K", [4992, 5120, 9984, 10112, 11136, 11264])
@pytest.mark.parametrize("g", [128, 0])
def test_the_longest_rows_of_each_form(K, g):
    # 3 experts, 12 pairs: 8-row tiles with two places for the rows (K up to 4992), one (9984 with 24 warps, 11136
    # with 16), none (the many-rows kernel)
    g = g or K
    E, N, T, k = 3, 72, 6, 2
    d = experts_inputs(E, K, N, g, T, k, seed=K, by_pair=True)
    Wp = wq.wq_prepack_experts(dev(d["Q"]), dev(d["s"]), g)
    lists = dev(d["offsets"]), dev(d["rows"])
    got = f64(wq.wq_gemm_w4a16_experts(dev(d["A"][:T]), Wp, *lists, N, g))
    y, ad = oracle.experts_product(d["A"][:T], d["Q"], d["s"], g, d["idx"])
    assert np.all(np.abs(got - y) <= product_bound(y, ad, K))
    out = f64(wq.wq_gemm_w4a16_experts_combine(dev(d["A"]), Wp, dev(d["idx"]), dev(d["w"]), *lists, N, g))
    y, ad = oracle.experts_product(d["A"], d["Q"], d["s"], g, d["idx"], by_pair=True)
    assert np.all(np.abs(out - oracle.experts_combine(y, d["idx"], d["w"])) <= combine_bound_once(y, ad, d["idx"], d["w"], K))
    assert wq.wq_get_device_status() == wq.WQ_OK


# ------------------------------------------------------------------ offsets beyond 2^31 elements
def _weights_on_the_device(E, K, N, g, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    Q = torch.randint(-2 ** 31, 2 ** 31, (E, K // 8, N), generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    s = ((0.5 + torch.rand((E, K // g, N), generator=gen, device="cuda")) * (0.22 / K ** 0.5)).to(torch.float16)
    return Q, s


def _some(T):
    """Tokens at both ends and around the middle."""
    return [0, 1, T // 2 - 1, T // 2, T - 2, T - 1]


@pytest.mark.parametrize("E,K,N,g,T,k", [
    (2, 128, 16400, 128, 65552, 2),     # many rows: outputs and scratch of 2^31 elements and more
    (2, 16512, 64, 128, 65052, 2),      # many rows: the pairs' activations
    (1024, 128, 150000, 64, 7168, 2)])  # few rows: outputs, and 9.8 GB of weights
def test_offsets_beyond_32_bits(E, K, N, g, T, k):
    assert max(T * k * N, T * k * K) > 2 ** 31
    Q, s = _weights_on_the_device(E, K, N, g, seed=N)
    Wp = wq.wq_prepack_experts(Q, s, g)
    gen = torch.Generator(device="cuda").manual_seed(1)
    H = torch.randn((T * k, K), generator=gen, device="cuda", dtype=torch.float16)
    idx = torch.rand((T, E), generator=gen, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
    w = torch.rand((T, k), generator=gen, device="cuda") + 0.05
    lists = wq.wq_expert_lists(idx, E)
    up = wq.wq_gemm_w4a16_experts(H[:T], Wp, *lists, N, g)
    picked = _some(T)
    pi = idx[picked].cpu().numpy()
    used = sorted(set(pi.reshape(-1).tolist()))
    where = np.vectorize(used.index)(pi)
    q_, s_ = Q[used].cpu().numpy(), s[used].cpu().numpy()
    got = f64(up.view(T, k, N)[picked]).reshape(-1, N)
    y, ad = oracle.experts_product(H[picked].cpu().numpy(), q_, s_, g, where)
    assert np.all(np.abs(got - y) <= product_bound(y, ad, K))
    del up
    out = wq.wq_gemm_w4a16_experts_combine(H, Wp, idx, w, *lists, N, g)
    h = H.view(T, k, K)[picked].reshape(-1, K).cpu().numpy()
    y, ad = oracle.experts_product(h, q_, s_, g, where, by_pair=True)
    wn = w[picked].cpu().numpy()
    assert np.all(np.abs(f64(out[picked]) - oracle.experts_combine(y, where, wn)) <= combine_bound_once(y, ad, where, wn, K))
    assert wq.wq_get_device_status() == wq.WQ_OK


# ------------------------------------------------------------------ no memory but what the caller gives
@pytest.mark.parametrize("T", [1, 24, 500])
def test_calls_with_given_outputs_leave_the_free_memory(T):
    E, K, N, g, k = 8, 256, 256, 128, 2
    d = experts_inputs(E, K, N, g, T, k, seed=T, by_pair=True)
    Q, s, H = dev(d["Q"]), dev(d["s"]), dev(d["A"])
    Wp = torch.zeros(wq.wq_prepacked_bytes_experts(E, K, N, g), dtype=torch.uint8, device="cuda")
    x = torch.randn((T, E), device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, w, offsets, rows = torch.empty((T, k), **i32), torch.empty((T, k), device="cuda"), torch.empty(E + 1, **i32), \
        torch.empty(T * k, **i32)
    up = torch.empty((T * k, N), dtype=torch.float16, device="cuda")
    Y = torch.empty((T, N), dtype=torch.float16, device="cuda")
    scratch = torch.empty(max(16, wq.wq_experts_scratch_bytes(T, E, k, N)), dtype=torch.uint8, device="cuda")
    for turn in range(3):
        torch.cuda.synchronize()
        before = torch.cuda.mem_get_info()[0], torch.cuda.memory_allocated()
        wq.wq_prepack_experts(Q, s, g, Wp=Wp)
        wq.wq_route_experts(x, k, idx=idx, w=w)
        wq.wq_expert_lists(idx, E, offsets=offsets, rows=rows)
        wq.wq_gemm_w4a16_experts(H[:T], Wp, offsets, rows, N, g, Y=up)
        wq.wq_gemm_w4a16_experts_combine(H, Wp, idx, w, offsets, rows, N, g, Y=Y, scratch=scratch)
        torch.cuda.synchronize()
        if turn:  # the first calls on a device load the library's device code
            assert (torch.cuda.mem_get_info()[0], torch.cuda.memory_allocated()) == before


# ------------------------------------------------------------------ calls at the limits
def test_the_most_pairs_that_a_call_takes():
    # 2^24 tokens, 16 choices: 2^28 pairs
    E, K, N, g, T, k = 16, 128, 8, 128, 1 << 24, 16
    gen = torch.Generator(device="cuda").manual_seed(2)
    logits = torch.randn((T, E), generator=gen, device="cuda", dtype=torch.float16)
    idx, w, offsets, rows = wq.wq_route_experts(logits, k, lists=True)
    for t0 in (0, T // 2, T - 64):
        ref, w_ref = oracle.route_experts(f64(logits[t0:t0 + 64]), k)
        assert np.array_equal(idx[t0:t0 + 64].cpu().numpy(), ref)
        assert np.all(np.abs(f64(w[t0:t0 + 64]) - w_ref) <= 2.0 ** -24 * 1.001 * w_ref + 2.0 ** -149)
    flat = idx.view(-1)
    for e in range(E):  # every token takes every expert once
        assert int(offsets[e]) == e * T
        assert torch.equal(rows[e * T:(e + 1) * T].long(), torch.nonzero(flat == e).view(-1))
    assert int(offsets[E]) == E * T
    d = experts_inputs(E, K, N, g, 1, 1, seed=4)
    A = torch.randn((T, K), generator=gen, device="cuda", dtype=torch.float16)
    Y = wq.wq_gemm_w4a16_experts(A, wq.wq_prepack_experts(dev(d["Q"]), dev(d["s"]), g), offsets, rows, N, g)
    assert wq.wq_get_device_status() == wq.WQ_OK
    for t0 in (0, T // 3, T - 64):
        y, ad = oracle.experts_product(A[t0:t0 + 64].cpu().numpy(), d["Q"], d["s"], g, idx[t0:t0 + 64].cpu().numpy())
        assert np.all(np.abs(f64(Y[t0 * k:(t0 + 64) * k]) - y) <= product_bound(y, ad, K))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_in_one_launch_at_its_largest(score):
    gen = torch.Generator().manual_seed(6)
    x, b = torch.randn((16, 1024), generator=gen).cuda(), (torch.randn(1024, generator=gen) * 0.1).cuda()
    _check_route(x, 8, b, score=score, groups=64, top_groups=9, group_top=2)
    _check_route(x[:4].contiguous(), 32, b, score=score)


@pytest.mark.parametrize("E,T", [(64, 3), (4, 9), (3, 200)])  # few pairs, few rows, many rows
def test_rows_of_padded_places_are_not_read(E, T):
    K, N, g, k = 384, 80, 128, 3
    d = experts_inputs(E, K, N, g, T, k, seed=E, by_pair=True)
    rng = np.random.default_rng(T)
    idx = np.where(rng.random((T, k)) < 0.4, -1, d["idx"])
    idx[T - 1] = -1
    H, w = d["A"].copy(), d["w"].copy()
    H[idx.reshape(-1) < 0] = np.nan
    w[idx < 0] = np.nan
    Wp = wq.wq_prepack_experts(dev(d["Q"]), dev(d["s"]), g)
    lists = wq.wq_expert_lists(dev(idx), E)
    out = f64(wq.wq_gemm_w4a16_experts_combine(dev(H), Wp, dev(idx), dev(w), *lists, N, g))
    y, ad = oracle.experts_product(d["A"], d["Q"], d["s"], g, idx, by_pair=True)
    assert np.all(np.abs(out - oracle.experts_combine(y, idx, d["w"])) <= combine_bound_once(y, ad, idx, d["w"], K))
    assert not out[T - 1].any()


def test_calls_from_several_threads():
    import threading
    E, K, N, g, k = 8, 512, 256, 128, 2
    work = []
    for i, T in enumerate((1, 20, 400, 33)):
        d = experts_inputs(E, K, N, g, T, k, seed=i, by_pair=True)
        Wp = wq.wq_prepack_experts(dev(d["Q"]), dev(d["s"]), g)
        x, H = torch.randn((T, E), device="cuda"), dev(d["A"])

        def one(stream=None, x=x, H=H, Wp=Wp):
            idx, w, *lists = wq.wq_route_experts(x, k, lists=True, stream=stream)
            return wq.wq_gemm_w4a16_experts_combine(H, Wp, idx, w, *lists, N, g, stream=stream)
        work.append((one, one(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[] for _ in work]
    threads = [threading.Thread(target=lambda i=i: outs[i].extend(work[i][0](stream=work[i][2]) for _ in range(30)))
               for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for (_, want, _), got in zip(work, outs):
        assert len(got) == 30 and all(torch.equal(y, want) for y in got)
    assert wq.wq_get_device_status() == wq.WQ_OK
