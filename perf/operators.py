"""What is measured of the expert operators: routing tokens to experts, the experts' 4-bit products.

Three operators of a sparse-expert layer with 4-bit weights:

* ``route``: scores, choice of ``top_k`` experts per token, their weights, and the lists of
  (token, choice) pairs by expert;
* ``up``: each pair's token row times its expert's weight, for gate/up weights with
  ``silu(gate) * up`` applied;
* ``down``: each pair's row times its expert's weight, summed over a token's choices with the
  routing weights.

Codes are packed 8 per int32 along K, ``w = (q - 8) * s`` with one fp16 scale per group of ``g``
rows and column (``g == K``: per column). A pair is ``p = t * top_k + j``.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------------- cases
def _route(T, E, k, dtype, score, bias, groups, top_groups, group_top, renorm, scale):
    return {"op": "route", "T": T, "E": E, "k": k, "dtype": dtype, "score": score, "bias": bias, "groups": groups,
            "top_groups": top_groups, "group_top": group_top, "renorm": renorm, "scale": scale}


def _up(T, E, k, K, N, g, gated, skew):
    return {"op": "up", "T": T, "E": E, "k": k, "K": K, "N": N, "g": g, "gated": gated, "skew": skew}


def _down(T, E, k, K, N, g, skew, padded):
    return {"op": "down", "T": T, "E": E, "k": k, "K": K, "N": N, "g": g, "skew": skew, "padded": padded}


def listed():
    out = []

    def add(name, case):
        out.append(dict(case, name=name))

    # one token of a decode step: 128 small experts, softmax scores renormalised over the choice
    add("route_decode_1", _route(1, 128, 8, "fp16", "softmax", False, 1, 1, 1, True, 1.0))
    # a decode batch: sigmoid scores with a balancing bias, 4 of 8 groups by their two best
    add("route_batch_64", _route(64, 256, 8, "fp32", "sigmoid", True, 8, 4, 2, True, 2.5))
    # a short prompt, few experts, an odd count of both, weights not renormalised
    add("route_prompt_1000", _route(1000, 60, 4, "fp16", "softmax", False, 1, 1, 1, False, 1.0))
    # a long prefill of the grouped router
    add("route_prefill_8192", _route(8192, 256, 8, "fp32", "sigmoid", True, 8, 4, 2, True, 2.5))
    # decode of one token: 8 of 128 small experts, gate and up in one product
    add("up_decode_1", _up(1, 128, 8, 2048, 1536, 128, True, 0.5))
    # a decode batch over mid-sized experts with a ragged count, small groups, no gate
    add("up_batch_24", _up(24, 60, 6, 4096, 1400, 64, False, 1.0))
    # a decode batch over 8 wide experts (the 4096 x 22016 layer in each), per-column scales
    add("up_wide_16", _up(16, 8, 2, 4096, 22016, 4096, True, 0.5))
    # prefill of 4096 tokens over 128 small experts: about 256 rows each
    add("up_prefill_4096", _up(4096, 128, 8, 2048, 1536, 128, True, 0.5))
    # decode of one token, the way back
    add("down_decode_1", _down(1, 128, 8, 768, 2048, 128, 0.5, 0.0))
    # a decode batch with padded places, small groups, odd width
    add("down_batch_40", _down(40, 60, 6, 1408, 4104, 32, 1.0, 0.15))
    # a short prompt over 8 wide experts (the 11008 x 4096 layer in each)
    add("down_wide_300", _down(300, 8, 2, 11008, 4096, 128, 0.5, 0.0))
    # prefill of 4096 tokens, the way back
    add("down_prefill_4096", _down(4096, 128, 8, 768, 2048, 128, 0.5, 0.02))
    return out


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "up", "down"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(max(1, 8 // groups), 256 // groups)
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(10, E // groups * top_groups))
        T = _log_int(rng, 1, 8192)
        return _route(T, E, k, rng.choice(["fp16", "fp32"]), rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5,
                      groups, top_groups, rng.choice([1, 2]), rng.random() < 0.7, rng.choice([1.0, 2.5]))
    while True:
        E = rng.choice([8, 16, 40, 60, 64, 128])
        k = rng.randint(1, 8)
        T = _log_int(rng, 1, 4096)
        K = 128 * rng.randint(2, 40)
        g = rng.choice([32, 64, 128, 128, K])
        gated = op == "up" and rng.random() < 0.6
        N = 16 * rng.randint(16, 256) if gated else 8 * rng.randint(32, 512)
        if E * K * N > 8 * 4096 * 22016 or T * k * K * N > 4096 * 8 * 768 * 2048:
            continue
        skew = rng.choice([0.0, 0.5, 1.0, 2.0])
        if op == "up":
            return _up(T, E, k, K, N, g, gated, skew)
        return _down(T, E, k, K, N, g, skew, rng.choice([0.0, 0.1, 0.3]))


# ---------------------------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(1000003 * seed + 17)


def _route_inputs(case, seed):
    gen = _generator(seed)
    T, E = case["T"], case["E"]
    # router outputs: some experts are liked more by every token
    liked = torch.randn(E, generator=gen, device=DEV) * 0.7
    logits = torch.randn((T, E), generator=gen, device=DEV) * 1.5 + liked
    logits = logits.to(torch.float16 if case["dtype"] == "fp16" else torch.float32)
    bias = torch.randn(E, generator=gen, device=DEV) * 0.1 if case["bias"] else None
    return logits, bias


def _choices(case, gen):
    """idx int32 [T, k]: distinct experts per token, popular ones more often; and pair lists."""
    T, E, k = case["T"], case["E"], case["k"]
    liked = torch.randn(E, generator=gen, device=DEV) * case["skew"]
    key = liked - torch.log(-torch.log(torch.rand((T, E), generator=gen, device=DEV).clamp(1e-6, 1 - 1e-6)))
    idx = torch.sort(key, dim=1, descending=True).indices[:, :k].to(torch.int32)
    if case.get("padded"):
        # places of a padded batch: a token that takes no expert
        idx[torch.rand(T, generator=gen, device=DEV) < case["padded"]] = -1
    flat = idx.reshape(-1).long()
    order = torch.argsort(torch.where(flat < 0, E, flat), stable=True)
    counts = torch.bincount(torch.where(flat < 0, E, flat), minlength=E + 1)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(counts[:E], 0)
    return idx.contiguous(), offsets, order.to(torch.int32)


def _product_inputs(case, seed):
    gen = _generator(seed)
    T, E, k, K, N, g = (case[x] for x in ("T", "E", "k", "K", "N", "g"))
    idx, offsets, rows = _choices(case, gen)
    Q = torch.randint(-2 ** 31, 2 ** 31, (E, K // 8, N), generator=gen, device=DEV, dtype=torch.int64).to(torch.int32)
    # scales of a quantised weight whose entries have a deviation of about 1 / sqrt(K)
    s = (0.5 + torch.rand((E, K // g, N), generator=gen, device=DEV)) * (0.22 / math.sqrt(K))
    x = torch.randn((T if case["op"] == "up" else T * k, K), generator=gen, device=DEV).to(torch.float16)
    w = torch.rand((T, k), generator=gen, device=DEV) + 0.05
    w = w / w.sum(1, keepdim=True)
    return {"x": x, "Q": Q, "s": s.to(torch.float16), "idx": idx, "offsets": offsets, "rows": rows, "w": w}


def prepare(case, seed):
    if case["op"] == "route":
        logits, bias = _route_inputs(case, seed)
        return {"case": case, "logits": logits, "bias": bias}
    state = dict(_product_inputs(case, seed), case=case)
    if own:
        import bit_weight_quantized_prepack_b200 as wq
        # the weights a program holds: laid out once, the checkpoint's codes dropped
        state["Wp"] = wq.wq_prepack_experts(state.pop("Q"), state.pop("s"), case["g"],
                                            gated=case["op"] == "up" and case["gated"])
    return state


# ---------------------------------------------------------------------------------- plain forms
def _plain_route(state):
    case, logits = state["case"], state["logits"]
    T, E, k = case["T"], case["E"], case["k"]
    # 64 bits: two experts' scores can lie closer than 32 bits hold
    x = logits.double()
    if case["score"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    c = p + state["bias"].double() if state["bias"] is not None else p
    order_by = c if state["bias"] is not None else x
    G = case["groups"]
    if case["top_groups"] < G:
        members = min(case["group_top"], E // G)
        value = c.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :members].sum(2)
        best = value.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        stays = torch.zeros((T, G), dtype=torch.bool, device=x.device)
        stays.scatter_(1, best, True)
        order_by = torch.where(stays.repeat_interleave(E // G, 1), order_by, -math.inf)
    idx = order_by.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, idx)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = (w * case["scale"]).float()
    flat = idx.reshape(-1)
    rows = torch.argsort(flat, stable=True)
    offsets = torch.searchsorted(flat[rows], torch.arange(E + 1, device=x.device))
    return idx.to(torch.int32), w, offsets.to(torch.int32), rows.to(torch.int32)


_SHIFTS = tuple(range(0, 32, 4))


def _plain_weight(Q, s, g):
    """fp32 [K, N] of one expert."""
    K, N = Q.shape[0] * 8, Q.shape[1]
    q = torch.stack([(Q >> sh) & 15 for sh in _SHIFTS], 1).reshape(K, N)
    w = (q - 8).float().view(K // g, g, N) * s.float()[:, None, :]
    return w.view(K, N)


def _plain_products(state, a_of_pair):
    """fp32 [pairs, N], rows of pairs without an expert zero."""
    case = state["case"]
    ends = state["offsets"].tolist()
    y = torch.zeros((case["T"] * case["k"], case["N"]), dtype=torch.float32, device=DEV)
    for e in range(case["E"]):
        if ends[e + 1] > ends[e]:
            pairs = state["rows"][ends[e]:ends[e + 1]].long()
            y[pairs] = state["x"][pairs // a_of_pair].float() @ _plain_weight(state["Q"][e], state["s"][e], case["g"])
    return y


def _plain_up(state):
    case = state["case"]
    y = _plain_products(state, case["k"])
    if case["gated"]:
        gate, up = y[:, :case["N"] // 2], y[:, case["N"] // 2:]
        y = gate / (1.0 + torch.exp(-gate)) * up
    return y.to(torch.float16)


def _plain_down(state):
    case = state["case"]
    y = _plain_products(state, 1).view(case["T"], case["k"], case["N"])
    return (y * state["w"][:, :, None]).sum(1).to(torch.float16)


# ---------------------------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if not own:
        return {"route": _plain_route, "up": _plain_up, "down": _plain_down}[case["op"]](state)
    import bit_weight_quantized_prepack_b200 as wq
    if case["op"] == "route":
        return wq.wq_route_experts(state["logits"], case["k"], bias=state["bias"], score=case["score"],
                                   groups=case["groups"], top_groups=case["top_groups"], group_top=case["group_top"],
                                   renorm=case["renorm"], scale=case["scale"], lists=True)
    if case["op"] == "up":
        return wq.wq_gemm_w4a16_experts(state["x"], state["Wp"], state["offsets"], state["rows"], case["N"], case["g"],
                                        gated=case["gated"])
    return wq.wq_gemm_w4a16_experts_combine(state["x"], state["Wp"], state["idx"], state["w"], state["offsets"],
                                            state["rows"], case["N"], case["g"])


def work(case):
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "route":
        nbytes = T * E * (2 if case["dtype"] == "fp16" else 4) + (4 * E if case["bias"] else 0)
        nbytes += 8 * T * k + 4 * (E + 1) + 4 * T * k
        return {"bytes": nbytes, "flops": 4 * T * E}
    K, N, g = case["K"], case["N"], case["g"]
    pairs = T * k * (1 - case.get("padded", 0.0))
    # experts that at least one pair takes, were the choice even
    active = E * (1 - (1 - 1 / E) ** pairs) if T > 1 else k
    nbytes = active * (K * N / 2 + 2 * (K // g) * N) + 8 * T * k + 4 * E
    if case["op"] == "up":
        nbytes += 2 * T * K + 2 * T * k * (N // 2 if case["gated"] else N)
    else:
        nbytes += 2 * pairs * K + 2 * T * N + 4 * T * k
    return {"bytes": int(nbytes), "flops": int(2 * pairs * K * N)}


# ---------------------------------------------------------------------------------- in 64 bits
def _exact_route(case, seed):
    logits, bias = _route_inputs(case, seed)
    x = logits.cpu().double().numpy()
    b = None if bias is None else bias.cpu().double().numpy()
    import numpy as np
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    if case["score"] == "softmax":
        shifted = np.exp(x - np.max(x, axis=1)[:, None])
        p = shifted / np.sum(shifted, axis=1)[:, None]
    else:
        p = 1.0 / (1.0 + np.exp(-x))
    c = p if b is None else p + b[None, :]
    key = x if b is None else c
    allowed = np.ones((T, E), dtype=bool)
    if case["top_groups"] < G:
        size = E // G
        value = np.zeros((T, G))
        for j in range(G):
            part = -np.sort(-c[:, j * size:(j + 1) * size], axis=1)
            value[:, j] = part[:, :case["group_top"]].sum(axis=1)
        rank = np.argsort(-value, axis=1, kind="stable")
        allowed[:] = False
        for r in range(case["top_groups"]):
            cols = rank[:, r:r + 1] * size + np.arange(size)[None, :]
            np.put_along_axis(allowed, cols, True, axis=1)
    idx = np.argsort(np.where(allowed, -key, np.inf), axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(p, idx, axis=1)
    if case["renorm"]:
        w = w / w.sum(axis=1)[:, None]
    flat = idx.ravel()
    rows = np.concatenate([np.flatnonzero(flat == e) for e in range(E)])
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])])
    whole = [torch.from_numpy(a.astype(np.int32)).to(DEV) for a in (idx, offsets, rows)]
    return whole[0], torch.from_numpy(w * case["scale"]).to(DEV), whole[1], whole[2]


def _exact_products(case, seed):
    d = _product_inputs(case, seed)
    T, k, K, N, g = (case[x] for x in ("T", "k", "K", "N", "g"))
    flat = d["idx"].reshape(-1)
    y = torch.zeros((T * k, N), dtype=torch.float64, device=DEV)
    group_of_row = torch.arange(K, device=DEV) // g
    place = torch.arange(K, device=DEV) % 8 * 4
    for e in range(case["E"]):
        pairs = torch.nonzero(flat == e).flatten()
        if pairs.numel() == 0:
            continue
        words = d["Q"][e].long().repeat_interleave(8, dim=0)
        code = torch.bitwise_and(torch.bitwise_right_shift(words, place[:, None]), 15).double()
        weight = (code - 8.0) * d["s"][e].double()[group_of_row]
        token = pairs if case["op"] == "down" else torch.div(pairs, k, rounding_mode="floor")
        y.index_copy_(0, pairs, torch.matmul(d["x"].double()[token], weight))
    return d, y


def exact(case, seed):
    if case["op"] == "route":
        return _exact_route(case, seed)
    d, y = _exact_products(case, seed)
    if case["op"] == "up":
        if not case["gated"]:
            return y
        half = case["N"] // 2
        return y[:, half:] * y[:, :half] * torch.sigmoid(y[:, :half])
    return torch.einsum("tkn,tk->tn", y.view(case["T"], case["k"], case["N"]), d["w"].double())
