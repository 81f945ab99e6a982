"""The expert operators at the edges of their definition: infinite ties, scores far below a
row's largest, saturated scores, rows that are no numbers, and results that must not depend on
the tokens beside them.

Tolerances as in test_gpu_experts.py."""
import math

import numpy as np
import pytest
import torch

import predictor_gated_channel_b200 as sfn
from predictor_gated_channel_b200 import _capi
from predictor_gated_channel_b200 import build as sfn_build
from test_gpu_experts import (BF16, DEV, U, expert_weights, rand, ref_experts, ref_quantize,
                              ref_route, ref_scores, weights_i8)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    sfn_build.build()
    _capi.lib()


# ---------------------------------------------------------- experts' products
@pytest.mark.parametrize("T,E,k,d,f", [(300, 4, 2, 4096, 1792), (1500, 3, 2, 272, 208),
                                       (40, 16, 4, 400, 240), (700, 5, 2, 144, 4096)])
def test_experts_token_by_itself(T, E, k, d, f):
    """A token's bits are the same alone, among a few (streams) and among many
    (tiles, pairs): what follows the exact integer sums is the same arithmetic."""
    W = expert_weights(T, E, f, d)
    x = rand(T, T, d).to(torch.bfloat16).to(DEV)
    g = torch.Generator().manual_seed(T)
    experts = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    experts[2, 0] = -1
    weights = torch.rand((T, k), generator=g).to(DEV)
    experts = experts.to(DEV)
    y = sfn.experts_i8_forward(x, experts, weights, **W)
    for first, n in ((0, 1), (1, 5), (T - 1, 1), (T // 2, 32 // k), (3, 37)):
        rows = slice(first, first + n)
        part = sfn.experts_i8_forward(x[rows].contiguous(), experts[rows].contiguous(),
                                      weights[rows].contiguous(), **W)
        assert torch.equal(part, y[rows]), (first, n)


# ------------------------------------------------------------------- choices
def offset_view(t, by):
    """The same values `by` elements into an allocation: no 16-byte loads."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    view = buf[by:].view(t.shape)
    view.copy_(t)
    return view


@pytest.mark.parametrize("where", ["logits", "bias"])
@pytest.mark.parametrize("T,E,groups,top", [
    (200, 64, 1, 1), (200, 128, 1, 1), (200, 256, 1, 1), (200, 512, 1, 1), (200, 1024, 1, 1),
    (200, 96, 1, 1), (200, 64, 8, 5), (200, 160, 8, 5), (200, 192, 4, 3), (200, 256, 8, 5),
    (200, 384, 16, 9), (200, 100, 5, 3), (2100, 64, 1, 1), (2100, 256, 1, 1), (2100, 64, 4, 3),
    (2100, 160, 8, 5), (2100, 256, 2, 2), (16500, 64, 1, 1), (16500, 250, 1, 1),
])
def test_route_infinite_ties(T, E, groups, top, where):
    """More +inf logits (or biases) than slots: equal ones to the lower index,
    wherever they lie among a lane's values and in any batch and alignment."""
    g = torch.Generator().manual_seed(T + E)
    rows = torch.cat([torch.arange(120), torch.arange(T - 60, T)])
    for trial in range(3):
        logits = torch.randn((T, E), generator=g)
        bias = None
        if where == "logits":
            at = torch.rand((T, E), generator=g).argsort(1)[:, :4]
            if trial == 0:   # neighbours
                at = torch.randint(0, E - 3, (T, 1), generator=g) + torch.arange(4)[None, :]
            logits.scatter_(1, at, math.inf)
        else:
            bias = torch.zeros(E)
            first = int(torch.randint(0, E - 3, (1,), generator=g))
            bias[first:first + 4 if trial == 0 else first + 1] = math.inf
            bias[torch.randperm(E, generator=g)[:4 * (trial > 0)]] = math.inf
        b = None if bias is None else bias.to(DEV)
        for k, gtop in ((1, 1), (2, 1), (3, 2 if bias is not None and groups > 1 else 1)):
            re, _, _ = ref_route(logits[rows], k, bias, "sigmoid", groups, top, gtop)
            for dtype in (torch.float32, torch.bfloat16):
                if dtype == torch.bfloat16:
                    re, _, _ = ref_route(logits[rows].to(dtype), k, bias, "sigmoid", groups, top,
                                         gtop)
                x = logits.to(dtype).to(DEV)
                for view in (x, offset_view(x, 1)):
                    e, _, _ = sfn.route_experts(view, k, bias=b, score="sigmoid", groups=groups,
                                                top_groups=top, group_top=gtop)
                    assert np.array_equal(e.cpu()[rows].numpy(), re), (k, dtype, trial)


@pytest.mark.parametrize("E,groups", [(64, 8), (48, 6), (256, 8), (100, 5)])
def test_route_group_sums_past_the_range(E, groups):
    """Sums of two scores that pass float32's range (finite biases near its end)
    are told apart: the larger sum stays, not the lower group."""
    T, size = 20, E // groups
    logits = rand(E, T, E)
    bias = torch.zeros(E)
    bias[size:size + 2] = 2.9e38
    bias[3 * size + 1:3 * size + 3] = 3.3e38
    bias[4 * size:4 * size + 2] = 3.1e38
    for top in (1, 2):
        for score in ("softmax", "sigmoid"):
            e, _, _ = sfn.route_experts(logits.to(DEV), 2, bias=bias.to(DEV), score=score,
                                        groups=groups, top_groups=top, group_top=2)
            re, _, _ = ref_route(logits, 2, bias, score, groups, top, 2)
            assert np.array_equal(e.cpu().numpy(), re)
            assert (e[:, 0] // size == 3).all()


# ------------------------------------------------------------------- weights
@pytest.mark.parametrize("T,E,k,groups,gtop,bias", [
    (50, 64, 8, 1, 1, False), (50, 100, 5, 1, 1, True), (50, 256, 8, 8, 2, True),
    (2100, 64, 8, 1, 1, False), (2100, 250, 3, 1, 1, False), (17000, 64, 4, 1, 1, True),
])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_weights_of_tiny_scores(T, E, k, groups, gtop, bias, dtype):
    """Sigmoid scores below float32's range still share their weight as the
    definition says, down to where float64 has them as 0."""
    logits = rand(E, T, E, scale=2.0) - 95.0   # about the end of the range, and past it
    logits[1::3] -= 200.0
    logits[2::7] = -690.0 - logits[2::7].abs() / 50   # not below -709
    logits[3] = torch.finfo(dtype).min         # a mask of the lowest value
    logits[4, : E // 2] = -math.inf
    logits = logits.to(dtype)
    b = torch.round(rand(3, E) * 20) / 1000 if bias else None
    rows = torch.cat([torch.arange(40), torch.arange(T - 10, T)])
    e, w, _ = sfn.route_experts(logits.to(DEV), k, bias=None if b is None else b.to(DEV),
                                score="sigmoid", groups=groups, top_groups=max(1, groups // 2),
                                group_top=gtop, scale=1.5)
    re, rw, _ = ref_route(logits[rows], k, b, "sigmoid", groups, max(1, groups // 2), gtop, True,
                          1.5)
    assert np.array_equal(e.cpu()[rows].numpy(), re)
    assert np.allclose(w.cpu()[rows].double().numpy(), rw, rtol=100 * U, atol=1e-37)
    assert (w[3] == 0).all() and (w[0].sum() - 1.5).abs() < 1e-5


@pytest.mark.parametrize("T", [9, 17000])
def test_route_weights_far_below_the_largest(T):
    """Experts that a bias sends a token to, far below the row's largest logit:
    weights as the softmax's ratios have them at gaps of 90 and 200, and 0 where
    float64 has the scores as 0 (a mask of the lowest value)."""
    E, k = 64, 4
    for gap, zero in ((90.0, False), (200.0, False), (float(torch.finfo(torch.float32).max), True)):
        logits = rand(T, T, E)
        logits[:, 20:] -= gap
        bias = torch.zeros(E)
        bias[:20] = -math.inf
        e, w, _ = sfn.route_experts(logits.to(DEV), k, bias=bias.to(DEV))
        re, rw, _ = ref_route(logits[:9], k, bias)
        assert np.array_equal(e.cpu()[:9].numpy(), re)
        assert np.allclose(w.cpu()[:9].double().numpy(), rw, rtol=100 * U, atol=1e-37)
        assert (w == 0).all() if zero else ((w.sum(1) - 1).abs() < 1e-5).all()


# ------------------------------------------------------------------ gradients
def parts_of_gradient(logits, experts, dw, score):
    """In 64 bits: the row's scores, the chosen experts' shares n and v, the gradient of
    the chosen logits through the renormalised weights."""
    l = logits.double()
    s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    at, there = experts.long().clamp(min=0), experts >= 0
    n = s.gather(1, at) * there
    total = n.sum(1, keepdim=True)
    n = n / torch.where(total > 0, total, torch.ones_like(total))
    v = n * (dw.double() - (n * dw.double()).sum(1, keepdim=True))
    if score == "sigmoid":
        v = v * torch.sigmoid(-l).gather(1, at)
    return s, n, v, at


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dense", ["none", "zeros", "random"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [50, 9000])
def test_route_backward_of_tiny_scores(T, score, dense, dtype):
    """Chosen logits far below an unchosen one (softmax; a bias or a group choice
    does that) or far down the sigmoid: the gradient of the renormalised weights
    depends on the chosen logits alone, and is finite.

    v is right to 322 u n max |dw| scale: a share to 40 u, the differences from one
    slot's dw (at most 2 max |dw|) to u, their mean to 80 u."""
    E, k = 64, 6
    gaps = torch.tensor([60.0, 88.0, 90.0, 100.0, 104.0, 120.0, 300.0])
    logits = rand(T, T, E)
    experts = torch.stack([torch.randperm(E - 1, generator=torch.Generator().manual_seed(t))[:k]
                           for t in range(200)]).repeat(T // 200 + 1, 1)[:T]
    low = -gaps[torch.arange(T) % len(gaps)][:, None]
    logits = logits.scatter(1, experts, (logits + low).gather(1, experts)).to(dtype)
    experts = experts.to(torch.int32)
    experts[::5, 2] = -1
    dw = rand(7, T, k)
    ds = None if dense == "none" else rand(8, T, E) * (dense == "random")
    got = sfn.route_experts_backward(logits.to(DEV), experts.to(DEV), dw.to(DEV), scale=1.5,
                                     dscores=None if ds is None else ds.to(DEV), score=score)
    s, n, v, at = parts_of_gradient(logits, experts, dw, score)
    big = dw.double().abs().amax(1, keepdim=True)
    ref = torch.zeros_like(s).scatter_add(1, at, 1.5 * v * (experts >= 0))
    tol = torch.zeros_like(s).scatter_add(1, at, 1.5 * 322 * U * n * big)
    if ds is not None:
        d = ds.double()
        if score == "softmax":
            ref += s * (d - (s * d).sum(1, keepdim=True))
        else:
            ref += s * torch.sigmoid(-logits.double()) * d
        tol += 200 * U * s * d.abs().amax(1, keepdim=True)
    tol += 1e-37
    if dtype == torch.bfloat16:
        tol += BF16 * ref.abs()
    assert ((got.cpu().double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [60, 9000])
def test_route_backward_large_weight_gradient_of_a_small_score(T, score, dense):
    """One slot (the first, as biases can have it) with a large dweights and next
    to no weight must not cost the others their precision.

    A share n is right to 40 u (the exponential 4 u, its argument up to 25 u, sum
    and quotient 10 u), the differences from the largest score's dw (of which n is
    at least 1 / k: it is at most k M, M = sum n |dw|) to u each, and their mean to
    80 u of sum n |by| <= (k + 1) M: below 1000 u n_i (|dw_i| + M) in all."""
    E, k = 96, 8
    logits = rand(T, T, E, scale=0.5)
    experts = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:k]
                           for t in range(200)]).repeat(T // 200 + 1, 1)[:T]
    logits.scatter_(1, experts[:, :1], -20.0)
    dw = rand(7, T, k)
    dw[:, 0] = 1e6
    ds = torch.zeros((T, E)) if dense else None
    got = sfn.route_experts_backward(logits.to(DEV), experts.to(torch.int32).to(DEV), dw.to(DEV),
                                     dscores=None if ds is None else ds.to(DEV), score=score)
    l = logits.double()
    s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    n = s.gather(1, experts)
    n = n / n.sum(1, keepdim=True)
    mean_abs = (n * dw.double().abs()).sum(1, keepdim=True)
    v = n * (dw.double() - (n * dw.double()).sum(1, keepdim=True))
    if score == "sigmoid":
        v = v * (1 - s.gather(1, experts))
    ref = torch.zeros_like(l).scatter(1, experts, v)
    tol = torch.zeros_like(l).scatter(1, experts, 1000 * U * n * (dw.double().abs() + mean_abs))
    assert ((got.cpu().double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("T,E", [(50, 64), (50, 33), (50, 1000), (9000, 100), (9000, 256)])
def test_route_backward_of_rows_that_are_no_numbers(T, E, dense, dtype):
    """A NaN or +inf logit makes its softmax row's scores and weights NaN, and so
    its gradients, chosen or not; the other rows are what they are without it."""
    k = 4
    logits = rand(T, T, E).to(dtype)
    experts = torch.topk(logits[:, : E - 1].float(), k, dim=1).indices.to(torch.int32)
    dw = rand(7, T, k).to(DEV)
    ds = torch.zeros((T, E), device=DEV) if dense else None
    clean = sfn.route_experts_backward(logits.to(DEV), experts.to(DEV), dw, dscores=ds)
    bad = {3: (E - 1, math.nan), 7: (E - 1, math.inf), 11: (int(experts[11, 0]), math.nan),
           T - 1: (int(experts[T - 1, 1]), math.inf)}
    for t, (e, value) in bad.items():
        logits[t, e] = value
    got = sfn.route_experts_backward(logits.to(DEV), experts.to(DEV), dw, dscores=ds)
    rows = torch.zeros(T, dtype=torch.bool, device=DEV)
    rows[list(bad)] = True
    assert torch.isnan(got[rows]).all()
    assert torch.equal(got[~rows], clean[~rows])


def choose_by_logits(logits, k, score, groups, top):
    """No bias, groups by the sum of their two largest scores (float64, ties to the
    lower group), the experts of those that stay by their logits."""
    l, s = logits.double().numpy(), ref_scores(logits, score)
    T, E = l.shape
    size = E // groups
    out = np.full((T, k), -1, dtype=np.int32)
    for t in range(T):
        marks = []
        for g in range(groups):
            best = sorted((s[t, e] for e in range(g * size, (g + 1) * size) if l[t, e] > -np.inf),
                          reverse=True)[:2]
            marks.append(sum(best) if best else -np.inf)
        keep = sorted(range(groups), key=lambda g: (-marks[g], g))[:top]
        order = sorted((e for e in range(E) if e // size in keep and l[t, e] > -np.inf),
                       key=lambda e: (-l[t, e], e))[:k]
        out[t, :len(order)] = order
    return out


@pytest.mark.parametrize("T,E,k,groups,top", [(60, 64, 8, 8, 3), (60, 256, 8, 8, 4),
                                              (60, 160, 6, 8, 4), (60, 48, 4, 6, 3),
                                              (60, 100, 5, 5, 2), (60, 384, 31, 16, 9),
                                              (3000, 64, 8, 4, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_by_logits_within_summed_groups(T, E, k, groups, top, score, dtype):
    """Without a bias experts are ranked by their logits whatever scores the groups:
    where float64 has the scores as equal (1 far up the sigmoid, 0 far below a
    softmax row's largest), where they tie, and where nothing is special."""
    g = torch.Generator().manual_seed(E)
    logits = torch.randn((T, E), generator=g) * 1.5
    whole = torch.round(logits * 4)
    logits[::3] = whole[::3] + 45.0                        # sigmoid: all 1
    logits[1::6] = whole[1::6] - 800.0                     # sigmoid: all 0
    logits[1::6, ::7] = 0.0                                # softmax: 0 but for these
    logits[2::9] = whole[2::9] / 8
    logits[5, E // groups + 1:] = -math.inf
    logits = logits.to(dtype)
    e, _, _ = sfn.route_experts(logits.to(DEV), k, score=score, groups=groups, top_groups=top,
                                group_top=2)
    rows = torch.cat([torch.arange(60), torch.arange(T - 30, T)])
    assert np.array_equal(e.cpu()[rows].numpy(),
                          choose_by_logits(logits[rows], k, score, groups, top))


# --------------------------------------------------------------- quantisation
@pytest.mark.parametrize("largest", [1.0, 127.0, 127 * 2.0 ** -9, 254 * 3.0, 0.3, 1e-29, 3.0e38,
                                     1.3e-38, 1e-31, 2.0 ** -140, 5.1e36])
def test_quantize_float32_next_to_half_way(largest):
    """float32 values as close to half way between two integers as they come, on
    both sides, and exactly half way: the integer of the definition, for every row
    length's kernel.  (The reference divides in float64, whose rounding of 2^-46 is
    far below the 2^-33 that a quotient is away from half way if it is not on it.)"""
    amax = torch.tensor(largest, dtype=torch.float32)
    halves = (torch.arange(-127, 127).double() + 0.5) * amax.double() / 127
    x = halves.float()
    near = [x, torch.nextafter(x, torch.tensor(math.inf)), torch.nextafter(x, -torch.tensor(math.inf))]
    near += [torch.nextafter(near[1], torch.tensor(math.inf)), amax[None],
             (torch.arange(-127, 128).double() * amax.double() / 127).float()]
    values = torch.cat(near)
    values = values[values.abs() <= amax]
    for K in (64, 1024, 4096, 40960):
        g = torch.Generator().manual_seed(K)
        rows = max(3, 4000 // K)
        row = values[torch.randint(0, values.numel(), (rows, K), generator=g)]
        row[:, 3] = -amax
        q, s = sfn.quantize_rows_i8(row.to(DEV))
        rq, _ = ref_quantize(row)
        assert torch.equal(q.cpu().double(), rq)


@pytest.mark.parametrize("T,K,N", [(1, 64, 40), (2, 1088, 135), (3, 4096, 64), (4, 7344, 126),
                                   (2, 8400, 541), (1, 40960, 16)])
def test_few_tokens_quantise_as_many_do(T, K, N):
    """float32 tokens of values next to half way between two integers: the stream
    of few tokens, which quantises in its own kernel, has the integers of the
    definition too (the products are then the same bits)."""
    g = torch.Generator().manual_seed(K)
    amax = torch.rand(T, 1, generator=g) * 5 + 0.1
    halves = (torch.randint(-127, 127, (T, K), generator=g).double() + 0.5) * amax.double() / 127
    x = halves.float()
    away = torch.where(torch.rand(T, K, generator=g) < 0.5, math.inf, -math.inf)
    x = torch.where(torch.rand(T, K, generator=g) < 0.5, torch.nextafter(x, away), x)
    x = x.clamp(-amax, amax)
    x[:, :1] = amax
    wq, sw = weights_i8(5, N, K)
    rq, rs = ref_quantize(x)
    q, s = sfn.quantize_rows_i8(x.to(DEV))
    assert torch.equal(q.cpu().double(), rq)
    y = sfn.linear_i8(x.to(DEV), wq.to(DEV), sw.to(DEV))
    assert torch.equal(y, sfn.matmul_i8(q, s, wq.to(DEV), sw.to(DEV), out_dtype=torch.float32))
    ref = (rq @ wq.double().T) * rs[:, None] * sw.double()
    # the exact sum's conversion and two scalings, and the scale's own rounding
    assert ((y.cpu().double() - ref).abs() <= 5 * U * ref.abs()).all()


@pytest.mark.parametrize("T,E,k,d,f", [(8, 2, 2, 4096, 1792), (16, 2, 2, 4096, 1792),
                                       (8, 1, 1, 2048, 4096), (12, 1, 1, 2048, 4096),
                                       (3, 8, 8, 4096, 1792)])
def test_experts_that_slots_share(T, E, k, d, f):
    """Few slots, several of the same expert: streams up to some bytes of weights
    read again, tiles past them, with the same bits as a token by itself."""
    W = expert_weights(T, E, f, d)
    x = rand(T, T, d).to(torch.bfloat16).to(DEV)
    g = torch.Generator().manual_seed(T)
    experts = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    experts = experts.to(torch.int32).to(DEV)
    weights = torch.rand((T, k), generator=g).to(DEV)
    y = sfn.experts_i8_forward(x, experts, weights, **W)
    for t in (0, T // 2, T - 1):
        one = sfn.experts_i8_forward(x[t:t + 1], experts[t:t + 1].contiguous(),
                                     weights[t:t + 1].contiguous(), **W)
        assert torch.equal(one, y[t:t + 1])


@pytest.mark.parametrize("size", [2.0 ** 40, 2.0 ** 100])
@pytest.mark.parametrize("T", [9, 2100, 17000])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_weights_beside_a_larger_logit_next_in_line(T, score, size):
    """Experts that the selection scores leave out by a tie (a bias that swallows
    the scores, in float32 or in float64 too), with logits far above the chosen:
    the weights are the chosen ones' alone."""
    E, k = 64, 4
    logits = rand(T, T, E) - (150.0 if score == "sigmoid" else 0.0)
    logits[:, 4:6] += 150.0
    for groups, others in ((1, size), (8, size), (1, 0.0)):
        bias = torch.full((E,), size)
        bias[6:] = others
        e, w, _ = sfn.route_experts(logits.to(DEV), k, bias=bias.to(DEV), score=score,
                                    groups=groups, top_groups=groups)
        re, rw, _ = ref_route(logits[:9], k, bias, score, groups, groups)
        assert np.array_equal(e.cpu()[:9].numpy(), re)
        # float64 tells scores beside 2^40 apart, but not beside 2^100
        assert size == 2.0 ** 40 or (e == torch.arange(4, device=DEV)).all()
        assert np.allclose(w.cpu()[:9].double().numpy(), rw, rtol=100 * U, atol=1e-37)
        assert ((w.sum(1) - 1).abs() < 1e-5).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E", [(12, 64), (12, 33), (12, 600), (9000, 64), (17000, 100)])
def test_route_softmax_rows_of_nothing_but_nan(T, E, dtype):
    """A NaN makes its row's scores NaN also where nothing else is left of it: all
    NaN, or NaN and masked experts (which, at -inf, rank above a NaN and are empty
    slots).  With a bias and without, scores written, and the dense gradient."""
    k = 3
    logits = rand(T, T, E).to(dtype)
    logits[1] = math.nan
    logits[4] = -math.inf
    logits[4, 7] = math.nan
    logits[9, 5] = math.nan
    bad = [1, 4, 9]
    good = torch.ones(T, dtype=torch.bool)
    good[bad] = False
    for bias in (None, torch.linspace(0, 1, E)):
        b = None if bias is None else bias.to(DEV)
        for renorm in (False, True):
            for want in (False, True):
                e, w, s = sfn.route_experts(logits.to(DEV), k, bias=b, renormalize=renorm,
                                            want_scores=want)
                assert e[1].tolist() == [0, 1, 2] and (e[4] == -1).all()
                assert torch.isnan(w[1]).all() and (w[4] == 0).all() and torch.isnan(w[9]).all()
                assert torch.isfinite(w[good]).all()
                if want:
                    assert torch.isnan(s[bad]).all() and torch.isfinite(s[good]).all()
            dw, ds = rand(5, T, k).to(DEV), rand(6, T, E).to(DEV)
            got = sfn.route_experts_backward(logits.to(DEV), e, dw, dscores=ds, renormalize=renorm)
            assert torch.isnan(got[bad]).all() and torch.isfinite(got[good]).all()
            got = sfn.route_experts_backward(logits.to(DEV), e, dw, renormalize=renorm)
            assert torch.isnan(got[bad]).all() and torch.isfinite(got[good]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E", [(9000, 160), (9000, 200), (8193, 256), (70, 256)])
def test_route_backward_of_any_alignment(T, E, score, dtype):
    """Dense gradients with 16-byte loads and without, around the sizes where the
    kernels change (tolerances as in test_route_backward_of_tiny_scores)."""
    k = 6
    logits = rand(E, T, E, scale=2.0).to(dtype)
    experts = torch.topk(logits.float(), k, dim=1).indices.to(torch.int32)
    experts[::5, 2] = -1
    dw, ds = rand(7, T, k), rand(8, T, E)
    s, n, v, at = parts_of_gradient(logits, experts, dw, score)
    big, d = dw.double().abs().amax(1, keepdim=True), ds.double()
    ref = torch.zeros_like(s).scatter_add(1, at, v * (experts >= 0))
    tol = torch.zeros_like(s).scatter_add(1, at, 322 * U * n * big)
    if score == "softmax":
        ref += s * (d - (s * d).sum(1, keepdim=True))
    else:
        ref += s * torch.sigmoid(-logits.double()) * d
    tol += 200 * U * s * d.abs().amax(1, keepdim=True) + 1e-37
    if dtype == torch.bfloat16:
        tol += BF16 * ref.abs()
    for by in (0, 1):
        out = offset_view(torch.empty(T, E, dtype=dtype, device=DEV), by)
        got = sfn.route_experts_backward(offset_view(logits.to(DEV), by), experts.to(DEV),
                                         dw.to(DEV), dscores=offset_view(ds.to(DEV), by),
                                         score=score, dlogits=out)
        assert got.data_ptr() == out.data_ptr()
        assert ((got.cpu().double() - ref).abs() <= tol).all()


# ------------------------------------------------- scales at the end of the range
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,N,K", [(1, 300, 4096), (2, 129, 1040), (4, 64, 64), (64, 256, 8192),
                                   (300, 200, 1040), (2100, 7200, 144)])
def test_products_of_rows_with_the_lowest_value(T, N, K, dtype):
    """A row that holds its type's lowest value (a mask) has a scale near 2^121: the
    integer sum times it passes float32's range, the product with the channel's
    scale, which is finite, does not.  Channels of zeros give 0 there."""
    x = rand(T, T, K).to(dtype)
    x[0, 3] = torch.finfo(dtype).min
    x[T - 1, K - 1] = torch.finfo(dtype).min / 2
    wq, sw = weights_i8(5, N, K)
    wq[1], sw[1] = 0, 0.0
    sw[2] = 0.0
    sw = sw * 1e-2
    q, s = sfn.quantize_rows_i8(x.to(DEV))
    rq, rs = ref_quantize(x)
    assert torch.equal(q.cpu().double(), rq)
    ref = (rq @ wq.double().T) * rs[:, None] * sw.double()
    assert (ref.abs() < 3e38).all() and ref.abs().max() > 1e33
    for out in (torch.float32, torch.bfloat16):
        y = sfn.linear_i8(x.to(DEV), wq.to(DEV), sw.to(DEV), out_dtype=out)
        tol = 5 * U + (BF16 if out == torch.bfloat16 else 0)
        assert ((y.cpu().double() - ref).abs() <= tol * ref.abs() + 1e-37).all()
        z = sfn.matmul_i8(q, s, wq.to(DEV), sw.to(DEV), out_dtype=out)
        assert torch.equal(z, y)


@pytest.mark.parametrize("T", [3, 300])
def test_experts_of_rows_with_the_lowest_value(T):
    E, k, d, f = 4, 2, 256, 112
    W = expert_weights(2, E, f, d)
    W["sg"] *= 1e-30
    W["su"] *= 1e-30
    x = rand(T, T, d).to(torch.bfloat16)
    x[1, 3] = torch.finfo(torch.bfloat16).min
    x = x.to(DEV)
    experts = (torch.arange(k * T, device=DEV) % E).to(torch.int32).view(T, k)
    weights = torch.rand((T, k), generator=torch.Generator().manual_seed(1)).to(DEV)
    y = sfn.experts_i8_forward(x, experts, weights, **W)
    ref, room = ref_experts(x, experts, weights, W)
    assert ref[1].abs().max() > 1e3 and torch.isfinite(y).all()
    assert ((y[1].double() - ref[1]).abs() <= (BF16 + 100 * U) * ref[1].abs() + room[1]).all()
