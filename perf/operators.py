"""Measured cases of the expert operators: routing and its gradient, the 8-bit integer product, and
the experts' products, each in a plain form, through the framework, and in 64 bits.

Sizes: d = 4096 and d_i = 14336 are this repository's layer; 1792 = 14336 / 8 channels an expert, so that
8 experts a token cost what the dense layer does.
"""
import math

import torch

own = False

DEV = "cuda:0"


def listed():
    return [
        # one token of a serving step: latency
        _route("route_decode_t1", 1, 64, 8, "softmax", False, 1, 1, 1, "float32"),
        # sigmoid scores with balance biases, 4 of 8 groups, a prefill chunk; some experts masked off
        _route("route_grouped_t4096", 4096, 256, 8, "sigmoid", True, 8, 4, 2, "float32", masked=3),
        # a long prefill or a training batch with an odd number of experts, bf16 logits
        _route("route_long_t32768", 32768, 160, 6, "softmax", False, 1, 1, 1, "bfloat16"),
        # gradients of the grouped sigmoid router's renormalised weights
        _route_bwd("route_backward_t4096", 4096, 256, 8, "sigmoid", True, False, "float32"),
        # softmax router with a balance loss on its scores: a dense gradient, bf16 logits
        _route_bwd("route_backward_long_t32768", 32768, 128, 8, "softmax", False, True, "bfloat16"),
        # one token through the layer's up projection: the weight stream
        _linear("linear_i8_decode_t1", 1, 4096, 14336, "bfloat16"),
        # a batch of decode streams through the down projection
        _linear("linear_i8_batch_t64", 64, 14336, 4096, "bfloat16"),
        # ragged: a short prompt, odd output width, float32 out
        _linear("linear_i8_ragged_t301", 301, 1040, 999, "float32"),
        # prefill
        _linear("linear_i8_prefill_t4096", 4096, 4096, 14336, "bfloat16"),
        # one token, 8 of 64 experts: their weights only
        _experts("experts_i8_decode_t1", 1, 64, 8, 4096, 1792),
        # a decode batch that touches nearly every expert with few rows each
        _experts("experts_i8_batch_t61", 61, 64, 8, 4096, 1792),
        # prefill, about 512 rows an expert
        _experts("experts_i8_prefill_t4096", 4096, 64, 8, 4096, 1792),
    ]


def _route(name, T, E, k, score, bias, groups, top_groups, group_top, dtype, masked=0, renorm=True):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "score": score, "bias": bias,
            "groups": groups, "top_groups": top_groups, "group_top": group_top, "dtype": dtype,
            "masked": masked, "renorm": renorm, "scale": 2.5 if score == "sigmoid" else 1.0}


def _route_bwd(name, T, E, k, score, renorm, dense, dtype):
    return {"name": name, "op": "route_bwd", "T": T, "E": E, "k": k, "score": score,
            "renorm": renorm, "dense": dense, "dtype": dtype,
            "scale": 2.5 if score == "sigmoid" else 1.0}


def _linear(name, T, K, N, out):
    return {"name": name, "op": "linear", "T": T, "K": K, "N": N, "out": out}


def _experts(name, T, E, k, d, f):
    return {"name": name, "op": "experts", "T": T, "E": E, "k": k, "d": d, "f": f}


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "linear", "experts"])
    if op in ("route", "route_bwd"):
        E = _log_int(rng, 4, 512)
        T = min(_log_int(rng, 1, 32768), 32768 * 160 // E)
        k = rng.randint(1, min(E, 16))
        score = rng.choice(["softmax", "sigmoid"])
        dtype = rng.choice(["float32", "bfloat16"])
        renorm = rng.random() < 0.6
        if op == "route_bwd":
            c = _route_bwd("", T, E, k, score, renorm, rng.random() < 0.4, dtype)
        else:
            groups = rng.choice([g for g in (1, 1, 2, 4, 8, 16) if E % g == 0 and E // g >= 2])
            top = rng.randint(1, groups)
            k = min(k, top * (E // groups))
            c = _route("", T, E, k, score, rng.random() < 0.5, groups, top, rng.choice([1, 2]),
                       dtype, rng.choice([0, 0, 1, E // 4]), renorm)
    elif op == "linear":
        K, N = 16 * _log_int(rng, 4, 896), _log_int(rng, 64, 14336)
        T = max(1, min(_log_int(rng, 1, 8192), 4096 * 4096 * 14336 // (K * N)))
        c = _linear("", T, K, N, rng.choice(["float32", "bfloat16"]))
    else:
        d, f = 16 * _log_int(rng, 16, 256), 16 * _log_int(rng, 8, 112)
        E = _log_int(rng, 2, 64)
        c = _experts("", _log_int(rng, 1, 4096), E, rng.randint(1, min(E, 8)), d, f)
    del c["name"]
    return c


def work(case):
    c = case
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        el = 4 if c["dtype"] == "float32" else 2
        return {"bytes": T * E * el + 8 * T * k + (4 * E if c["bias"] else 0), "flops": 6 * T * E}
    if c["op"] == "route_bwd":
        T, E, k = c["T"], c["E"], c["k"]
        el = 4 if c["dtype"] == "float32" else 2
        dense = 4 * T * E if c["dense"] else 0
        # what the sigmoid's gradient cannot do without is the chosen logits only
        read = T * E * el if c["score"] == "softmax" else T * k * el
        return {"bytes": read + T * E * el + dense + 8 * T * k, "flops": 8 * T * E}
    if c["op"] == "linear":
        T, K, N = c["T"], c["K"], c["N"]
        return {"bytes": 2 * T * K + N * K + 4 * N + T * N * (4 if c["out"] == "float32" else 2),
                "flops": 2 * T * K * N}
    T, E, k, d, f = c["T"], c["E"], c["k"], c["d"], c["f"]
    used = E * (1 - (1 - k / E) ** T)  # experts that some token chose, on average
    return {"bytes": int(used * (3 * d * f + 8 * f + 4 * d)) + 4 * T * d + 8 * T * k,
            "flops": 6 * T * k * d * f}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    c, g = case, _gen(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    if c["op"] in ("route", "route_bwd"):
        T, E, k = c["T"], c["E"], c["k"]
        logits = randn(T, E) * 1.5
        s = {"case": c}
        if c["op"] == "route":
            if c["masked"]:  # experts that are switched off
                off = torch.randperm(E, generator=g, device=DEV)[:c["masked"]]
                logits[:, off] = float("-inf")
            # biases move in equal steps in training
            s["bias"] = torch.round(randn(E) * 20) / 1000 if c["bias"] else None
        else:
            s["dweights"] = randn(T, k)
            s["dscores"] = randn(T, E) * 0.1 if c["dense"] else None
            # the forward's choice: any k experts of a row, here the largest logits
            s["experts"] = torch.topk(logits.to(getattr(torch, c["dtype"])).float(), k,
                                      dim=1).indices.to(torch.int32)
        s["logits"] = logits.to(getattr(torch, c["dtype"]))
        return s
    if c["op"] == "linear":
        T, K, N = c["T"], c["K"], c["N"]
        wq, ws = _int8_weights(g, (N,), K)
        return {"case": c, "x": randn(T, K).to(torch.bfloat16), "wq": wq, "ws": ws}
    T, E, k, d, f = c["T"], c["E"], c["k"], c["d"], c["f"]
    s = {"case": c, "x": randn(T, d).to(torch.bfloat16)}
    for n, rows, cols in (("g", f, d), ("u", f, d), ("d", d, f)):
        s["W" + n], s["s" + n] = _int8_weights(g, (E, rows), cols)
    # a router's choice: some experts are liked more than others
    liked = randn(E) * 0.5
    top = torch.topk(randn(T, E) + liked, k, dim=1)
    s["experts"] = top.indices.to(torch.int32)
    s["weights"] = torch.softmax(top.values, dim=1)
    return s


def _int8_weights(g, rows, cols):
    """Weights as a quantised N(0, 1/cols) matrix has them: a row's largest value is 127."""
    q = torch.randint(-90, 91, (*rows, cols), generator=g, device=DEV, dtype=torch.int8)
    q[..., 0] = 127
    s = (torch.rand(rows, generator=g, device=DEV) + 0.5) / (52 * math.sqrt(cols))
    return q, s


# ------------------------------------------------------------------ one pass
def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    if c["op"] == "route":
        return _plain_route(state, c)
    if c["op"] == "route_bwd":
        return _plain_route_bwd(state, c)
    if c["op"] == "linear":
        xq, sx = _plain_quantize(state["x"])
        y = _plain_product(xq, sx, state["wq"], state["ws"])
        return y.to(getattr(torch, c["out"]))
    return _plain_experts(state, c)


def _run_own(state, c):
    import predictor_gated_channel_b200 as sfn
    if c["op"] == "route":
        experts, weights, _ = sfn.route_experts(
            state["logits"], c["k"], bias=state["bias"], score=c["score"], groups=c["groups"],
            top_groups=c["top_groups"], group_top=c["group_top"], renormalize=c["renorm"],
            scale=c["scale"])
        return experts, weights
    if c["op"] == "route_bwd":
        return sfn.route_experts_backward(
            state["logits"], state["experts"], state["dweights"], dscores=state["dscores"],
            score=c["score"], renormalize=c["renorm"], scale=c["scale"])
    if c["op"] == "linear":
        return sfn.linear_i8(state["x"], state["wq"], state["ws"],
                             out_dtype=getattr(torch, c["out"]))
    return sfn.experts_i8_forward(state["x"], state["experts"], state["weights"],
                                  state["Wg"], state["sg"], state["Wu"], state["su"],
                                  state["Wd"], state["sd"])


def _plain_scores(logits, score):
    if score == "softmax":
        m = logits.amax(dim=1, keepdim=True)
        m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
        e = torch.exp(logits - m)
        z = e.sum(dim=1, keepdim=True)
        return torch.where(z > 0, e / z, torch.zeros_like(e))
    return 1 / (1 + torch.exp(-logits))


def _plain_route(state, c):
    # the choice in 64 bits: scores next to one another must not change places
    logits = state["logits"].double()
    T, E = logits.shape
    choice = _plain_scores(logits, c["score"])
    if state["bias"] is not None:
        choice = choice + state["bias"].double()
    choice = choice.masked_fill(torch.isneginf(logits), float("-inf"))
    if c["groups"] > 1:
        per = choice.view(T, c["groups"], E // c["groups"])
        best = per.sort(dim=2, descending=True).values[:, :, :c["group_top"]]
        none = torch.isneginf(best)
        group = best.masked_fill(none, 0.0).sum(dim=2).masked_fill(none.all(dim=2), float("-inf"))
        order = group.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        kept = torch.zeros((T, c["groups"]), dtype=torch.bool, device=logits.device)
        kept.scatter_(1, order, True)
        choice = per.masked_fill(~kept.unsqueeze(2), float("-inf")).view(T, E)
    top = choice.sort(dim=1, descending=True, stable=True)
    value, experts = top.values[:, :c["k"]], top.indices[:, :c["k"]]
    empty = torch.isneginf(value)
    scores = _plain_scores(state["logits"].float(), c["score"])
    weights = scores.gather(1, experts).masked_fill(empty, 0.0)
    if c["renorm"]:
        total = weights.sum(dim=1, keepdim=True)
        weights = torch.where(total > 0, weights / total, torch.zeros_like(weights))
    return experts.to(torch.int32).masked_fill(empty, -1), weights * c["scale"]


def _plain_route_bwd(state, c):
    logits = state["logits"].float()
    s = _plain_scores(logits, c["score"])
    at = state["experts"].long()
    dw = state["dweights"]
    if c["renorm"]:
        chosen = s.gather(1, at)
        total = chosen.sum(dim=1, keepdim=True)
        mean = (dw * chosen).sum(dim=1, keepdim=True) / total
        dw = (dw - mean) / total
    ds = torch.zeros_like(s).scatter_add_(1, at, dw * c["scale"])
    if state["dscores"] is not None:
        ds = ds + state["dscores"]
    if c["score"] == "softmax":
        dl = s * (ds - (s * ds).sum(dim=1, keepdim=True))
    else:
        dl = ds * s * (1 - s)
    return dl.to(state["logits"].dtype)


def _plain_quantize(x):
    x = x.float()
    amax = x.abs().amax(dim=-1, keepdim=True)
    q = torch.where(amax > 0, torch.round(x * 127 / amax), torch.zeros_like(x))
    return q.clamp(-127, 127), amax / 127


def _plain_product(xq, sx, wq, ws):
    # float32 holds these sums exactly up to 2^24
    return torch.matmul(xq, wq.float().transpose(-1, -2)) * sx * ws.unsqueeze(-2)


def _plain_experts(state, c):
    x, experts, weights = state["x"], state["experts"], state["weights"]
    T, E, k, d = c["T"], c["E"], c["k"], c["d"]
    slot_expert = experts.reshape(-1).long()
    order = torch.sort(slot_expert, stable=True).indices
    counts = torch.bincount(slot_expert, minlength=E)
    first = torch.cumsum(counts, 0) - counts
    place = torch.arange(T * k, device=x.device) - first[slot_expert[order]]
    cap = int(counts.max())
    # rows of each expert side by side, the shorter lists filled up with zeros
    xq, sx = _plain_quantize(x)
    token = order // k
    at = (slot_expert[order], place)
    rows = torch.zeros((E, cap, d), device=x.device)
    rows[at] = xq[token]
    scale = torch.zeros((E, cap, 1), device=x.device)
    scale[at] = sx[token]
    g = _plain_product(rows, scale, state["Wg"], state["sg"])
    u = _plain_product(rows, scale, state["Wu"], state["su"])
    h = (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)
    hq, sh = _plain_quantize(h)
    o = _plain_product(hq, sh, state["Wd"], state["sd"])
    by_slot = torch.empty((T * k, d), device=x.device)
    by_slot[order] = o[at]
    y = (by_slot.view(T, k, d) * weights.unsqueeze(2)).sum(dim=1)
    return y.to(torch.bfloat16)


# ------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "route":
        return _exact_route(s, c)
    if c["op"] == "route_bwd":
        return _exact_route_bwd(s, c)
    if c["op"] == "linear":
        return _exact_linear(s["x"], s["wq"], s["ws"])
    x, y = s["x"], torch.zeros(s["x"].shape, dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        token, slot = torch.nonzero(s["experts"] == e, as_tuple=True)
        if token.numel() == 0:
            continue
        g = _exact_linear(x[token], s["Wg"][e], s["sg"][e])
        u = _exact_linear(x[token], s["Wu"][e], s["su"][e])
        h = (g * torch.special.expit(g) * u).to(torch.bfloat16)
        o = _exact_linear(h, s["Wd"][e], s["sd"][e])
        y.index_add_(0, token, o * s["weights"][token, slot].double().unsqueeze(1))
    return y


def _exact_linear(x, wq, ws):
    x = x.double()
    amax = x.abs().max(dim=1).values
    unit = torch.where(amax > 0, amax, torch.ones_like(amax)).unsqueeze(1)
    q = torch.round(127 * x / unit)
    return (q @ wq.double().T) * (amax / 127).unsqueeze(1) * ws.double()


def _exact_route(s, c):
    logits = s["logits"].double()
    scores = (torch.softmax(logits, dim=1) if c["score"] == "softmax"
              else torch.special.expit(logits))
    choice = scores if s["bias"] is None else scores + s["bias"].double()
    choice = torch.where(logits == float("-inf"), logits, choice)
    T, E = logits.shape
    size = E // c["groups"]
    if c["groups"] > 1:
        marks = []
        for i in range(c["groups"]):
            part = choice[:, i * size:(i + 1) * size]
            first, where = part.max(dim=1)
            if c["group_top"] == 2:
                second = part.scatter(1, where.unsqueeze(1), float("-inf")).max(dim=1).values
                first = torch.where(second > float("-inf"), first + second, first)
            marks.append(first)
        marks = torch.stack(marks, dim=1)
        for _ in range(c["groups"] - c["top_groups"]):
            # drop the worst of the groups that stay; of equal ones the last
            worst = marks.nan_to_num(nan=float("inf")).flip(1).min(dim=1).indices
            worst = c["groups"] - 1 - worst
            marks.scatter_(1, worst.unsqueeze(1), float("nan"))
        off = torch.isnan(marks).repeat_interleave(size, dim=1)
        choice = torch.where(off, torch.full_like(choice, float("-inf")), choice)
    experts, values = [], []
    for _ in range(c["k"]):
        best = choice.max(dim=1, keepdim=True).values
        at = (choice == best).to(torch.int8).argmax(dim=1, keepdim=True)
        dead = best == float("-inf")
        experts.append(torch.where(dead, torch.full_like(at, -1), at))
        values.append(torch.where(dead, torch.zeros_like(best), scores.gather(1, at)))
        choice = choice.scatter(1, at, float("-inf"))
    w = torch.cat(values, dim=1)
    if c["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / torch.where(total > 0, total, 1.0), 0.0)
    return torch.cat(experts, dim=1).to(torch.int32), w * c["scale"]


def _exact_route_bwd(s, c):
    logits = s["logits"].double().requires_grad_(True)
    scores = (torch.softmax(logits, dim=1) if c["score"] == "softmax"
              else torch.sigmoid(logits))
    w = scores.gather(1, s["experts"].long())
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    loss = (w * c["scale"] * s["dweights"].double()).sum()
    if s["dscores"] is not None:
        loss = loss + (scores * s["dscores"].double()).sum()
    loss.backward()
    return logits.grad
