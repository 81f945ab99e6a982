"""Routing to experts and its gradient, the product in 8-bit integers and the
experts' products, against plain implementations in 64 bits.

Tolerances, from the arithmetic:
  * experts (indices) are equal, ties included: the choice is exact.
  * float32 scores and weights: an exponential (2 ulp), a sum of up to 1024
    terms (32 in a row, then a tree: 37 roundings) and two quotients, each
    rounding at most u = 2^-24 relative, and for softmax the argument's rounding
    u |l - m|, |l - m| <= 40 here: below 100 u = 6e-6 relative.
  * bf16 results: half a step, 2^-8 relative, on top of the float32 error.
  * the 8-bit product: the sum is exact; the conversion of it, two scalings and
    (float32 x) the scale's own rounding: 4 u relative; plus 2^-8 for bf16.
    x in bf16 quantises to the same integers in any precision; x in float32 may
    round 127 x / amax the other way within 2 u * 127 of half way, which the
    reference removes by quantising with the kernel's own public operator,
    itself tested to one step.
"""
import math

import numpy as np
import pytest
import torch

import predictor_gated_channel_b200 as sfn
from predictor_gated_channel_b200 import _capi
from predictor_gated_channel_b200 import build as sfn_build

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
BF16 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    sfn_build.build()
    _capi.lib()


def rand(seed, *shape, scale=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale


# ------------------------------------------------------------------ routing
def ref_scores(logits, score):
    l = logits.double().numpy()
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1 / (1 + np.exp(-l))
    m = l.max(axis=1, keepdims=True)
    m = np.where(np.isneginf(m), 0.0, m)
    e = np.exp(l - m)
    z = e.sum(axis=1, keepdims=True)
    return np.where(z > 0, e / np.where(z > 0, z, 1), 0.0)


def ref_route(logits, k, bias=None, score="softmax", groups=1, top_groups=1, group_top=1,
              renormalize=True, scale=1.0):
    """Row by row, from the definition."""
    l = logits.double().numpy()
    T, E = l.shape
    s = ref_scores(logits, score)
    b = np.zeros(E) if bias is None else bias.double().numpy()
    # without a bias the ranking is the logits'
    c = l.copy() if bias is None and (groups == 1 or group_top == 1) else s + b
    c[np.isneginf(l) | np.isneginf(b)[None, :]] = -np.inf
    experts = np.full((T, k), -1, dtype=np.int32)
    weights = np.zeros((T, k))
    size = E // groups
    for t in range(T):
        order = list(range(E))
        if groups > 1:
            marks = []
            for g in range(groups):
                best = sorted(c[t, g * size:(g + 1) * size], reverse=True)[:group_top]
                best = [v for v in best if v > -np.inf]
                marks.append(sum(best) if best else -np.inf)
            keep = sorted(range(groups), key=lambda g: (-marks[g], g))[:top_groups]
            order = [e for e in order if e // size in keep]
        order = sorted(order, key=lambda e: (-c[t, e], e))[:k]
        for i, e in enumerate(order):
            if c[t, e] > -np.inf:
                experts[t, i] = e
                weights[t, i] = s[t, e]
        if renormalize and weights[t].sum() > 0:
            weights[t] /= weights[t].sum()
    return experts, weights * scale, s


ROUTE = [
    # T, E, k, score, bias, groups, top_groups, group_top, renorm, dtype
    (1, 64, 8, "softmax", False, 1, 1, 1, True, torch.float32),
    (1, 1, 1, "sigmoid", True, 1, 1, 1, True, torch.float32),
    (5, 7, 7, "softmax", False, 1, 1, 1, False, torch.bfloat16),
    (33, 33, 2, "sigmoid", False, 1, 1, 1, False, torch.float32),
    (130, 256, 8, "sigmoid", True, 8, 4, 2, True, torch.float32),
    (130, 256, 8, "sigmoid", True, 8, 4, 2, True, torch.bfloat16),
    (67, 160, 6, "softmax", False, 8, 3, 1, True, torch.bfloat16),
    (67, 160, 6, "softmax", True, 32, 5, 2, False, torch.float32),
    (19, 96, 32, "softmax", True, 3, 2, 1, True, torch.float32),
    (19, 1000, 32, "sigmoid", True, 10, 7, 2, True, torch.float32),
    (3, 1024, 4, "softmax", False, 1, 1, 1, True, torch.float32),
    (700, 513, 5, "sigmoid", False, 1, 1, 1, True, torch.bfloat16),
]


@pytest.mark.parametrize("T,E,k,score,bias,groups,top,gtop,renorm,dtype", ROUTE)
def test_route(T, E, k, score, bias, groups, top, gtop, renorm, dtype):
    logits = rand(T + E, T, E, scale=2.0).to(dtype)
    if E > 8:  # masks, exact ties, a row that the mask leaves empty
        logits[0, E // 2:] = -math.inf
        if T > 4:
            logits[1] = -math.inf
            logits[2] = 0.25
            logits[3, ::2] = torch.finfo(dtype).min
    b = torch.round(rand(3, E) * 20) / 1000 if bias else None
    got = sfn.route_experts(logits.to(DEV), k, bias=None if b is None else b.to(DEV),
                            score=score, groups=groups, top_groups=top, group_top=gtop,
                            renormalize=renorm, scale=1.5, want_scores=True)
    e, w, s = (t.cpu() for t in got)
    re, rw, rs = ref_route(logits, k, b, score, groups, top, gtop, renorm, 1.5)
    assert np.array_equal(e.numpy(), re)
    assert np.allclose(w.double().numpy(), rw, rtol=100 * U, atol=1e-37)
    assert np.allclose(s.double().numpy(), rs, rtol=100 * U, atol=1e-37)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_decides_neighbours_exactly(score):
    """Scores closer to one another than float32 can tell: many logits far up
    (or down) the sigmoid, with biases a few units in the last place apart."""
    T, E, k = 400, 128, 8
    g = torch.Generator().manual_seed(11)
    logits = rand(5, T, E, scale=0.01) + (9.0 if score == "sigmoid" else 0.0)
    logits += torch.randint(0, 3, (T, E), generator=g) * 1e-6
    bias = torch.randint(0, 4, (E,), generator=g) * 2.0 ** -24
    e, w, _ = sfn.route_experts(logits.to(DEV), k, bias=bias.to(DEV), score=score, groups=8,
                                top_groups=3, group_top=2)
    re, rw, _ = ref_route(logits, k, bias, score, 8, 3, 2)
    assert np.array_equal(e.cpu().numpy(), re)


def test_route_nan_and_inf():
    logits = rand(1, 4, 40)
    logits[0, 3] = math.nan
    logits[1, 5] = math.inf
    logits[2] = math.nan
    e, w, _ = sfn.route_experts(logits.to(DEV), 4)
    assert 3 not in e[0].tolist() and torch.isnan(w[0]).all()
    assert e[1, 0].item() == 5 and torch.isnan(w[1]).all()
    assert e[2].tolist() == [0, 1, 2, 3]
    assert torch.isfinite(w[3]).all()
    e, w, _ = sfn.route_experts(logits.to(DEV), 4, score="sigmoid", renormalize=False)
    assert 3 not in e[0].tolist() and torch.isfinite(w[0]).all()
    assert e[1, 0].item() == 5 and w[1, 0].item() == 1.0


def ref_route_bwd(logits, experts, dw, ds, score, renormalize, scale):
    l = logits.double().requires_grad_(True)
    s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    at = experts.long()
    w = s.gather(1, at.clamp(min=0)) * (at >= 0)
    if renormalize:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    loss = (w * scale * dw.double()).sum()
    if ds is not None:
        loss = loss + (s * ds.double()).sum()
    return torch.autograd.grad(loss, l)[0], s.detach()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 64, 8), (37, 33, 5), (9, 1000, 32), (3, 1, 1)])
def test_route_backward(T, E, k, score, renorm, dense, dtype):
    logits = rand(T + E, T, E, scale=2.0).to(dtype)
    experts = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:k]
                           for t in range(T)]).to(torch.int32)
    if k > 3:
        experts[0, 2] = -1
        experts[-1, 3] = experts[-1, 1]  # the same expert twice
    dw, ds = rand(7, T, k), rand(8, T, E) if dense else None
    got = sfn.route_experts_backward(logits.to(DEV), experts.to(DEV), dw.to(DEV),
                                     dscores=None if ds is None else ds.to(DEV), score=score,
                                     renormalize=renorm, scale=1.5)
    assert got.dtype == dtype
    ref, s = ref_route_bwd(logits, experts, dw, ds, score, renorm, 1.5)
    # each gradient is a difference of terms of at most max |ds| (the sum of
    # their magnitudes), each right to 100 u, times the score (<= 1)
    chosen = (s.gather(1, experts.long().clamp(min=0)) * (experts >= 0)).sum(1, keepdim=True)
    unit = 1.5 * dw.abs().double().amax(1, keepdim=True) * 2
    if renorm:
        unit = unit / chosen.clamp(min=1e-30)
    if ds is not None:
        unit = unit + 2 * ds.abs().double().amax(1, keepdim=True)
    tol = 100 * U * unit * s + (BF16 * ref.abs() if dtype == torch.bfloat16 else 0) + 1e-37
    assert ((got.cpu().double() - ref).abs() <= tol).all()


def test_route_gradient_by_differences():
    """Central differences through the forward kernel itself, at a choice that
    does not change."""
    T, E, k, h = 4, 24, 5, 2.0 ** -7
    logits = rand(2, T, E)
    dw = rand(3, T, k)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            e0, _, _ = sfn.route_experts(logits.to(DEV), k, score=score, renormalize=renorm)
            g = sfn.route_experts_backward(logits.to(DEV), e0, dw.to(DEV), score=score,
                                           renormalize=renorm).cpu()
            for t, e in ((0, int(e0[0, 0])), (1, int(e0[1, 4])), (2, 7)):
                vals = []
                for sign in (1, -1):
                    l = logits.clone()
                    l[t, e] += sign * h
                    ei, w, _ = sfn.route_experts(l.to(DEV), k, score=score, renormalize=renorm)
                    # the forward orders by score: weights by expert
                    by = dict(zip(ei[t].tolist(), w[t].cpu().double().tolist()))
                    if set(by) != set(e0[t].tolist()):
                        break
                    vals.append(sum(by[x] * float(dw[t, i])
                                    for i, x in enumerate(e0[t].tolist())))
                if len(vals) == 2:
                    diff = (vals[0] - vals[1]) / (2 * h)
                    # curvature: third derivatives of these scores are below 1 in
                    # magnitude each, h^2 / 6 sum |dw|; rounding: 100 u sum |dw| / h
                    room = (h * h + 100 * U / h) * float(dw[t].abs().sum())
                    assert abs(diff - float(g[t, e])) <= room


# ------------------------------------------------------------- 8-bit product
def ref_quantize(x):
    x = x.double()
    amax = x.abs().amax(-1, keepdim=True)
    q = torch.where(amax > 0, torch.round(127 * x / amax.clamp(min=1e-300)), torch.zeros_like(x))
    return q, (amax / 127).squeeze(-1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,K", [(1, 16), (3, 4096), (130, 208), (5, 14336), (2, 40960), (9, 1040)])
def test_quantize_rows(T, K, dtype):
    x = rand(T + K, T, K).to(dtype)
    x[0, 1::3] = 0
    x[0, 0], x[0, 5] = 2.0, 1.0   # amax / 2 is exactly half way: 63.5 -> 64
    x[0] = x[0].clamp(-2, 2)
    q, s = (t.cpu() for t in sfn.quantize_rows_i8(x.to(DEV)))
    rq, rs = ref_quantize(x)
    assert q[0, 5].item() == 64 and q[0, 0].item() == 127
    off = (q.double() - rq).abs()
    if dtype == torch.bfloat16:
        assert off.max() == 0
    else:  # at most one step, and only within 127 * 2 u of half way
        v = (127 * x.double() / x.double().abs().amax(-1, keepdim=True))
        near = (v - torch.floor(v) - 0.5).abs() <= 254 * U
        assert off.max() <= 1 and not (off.bool() & ~near).any()
    assert torch.allclose(s.double(), rs, rtol=2 * U, atol=0)


def test_quantize_rows_extremes():
    K = 64
    x = rand(4, 8, K)
    x[0] = 0
    x[1] *= 3e38 / x[1].abs().max()
    x[2] *= 1e-38 / x[2].abs().max()
    x[3] *= 1e-42
    x[4, 7] = math.inf
    x[5, 9] = math.nan
    x[6, :] = -1.0
    x[7] *= 1e-31 / x[7].abs().max()
    q, s = (t.cpu() for t in sfn.quantize_rows_i8(x.to(DEV)))
    assert s[0] == 0 and (q[0] == 0).all()
    for r in (4, 5):
        assert torch.isnan(s[r]) and (q[r] == 0).all()
    assert (q[6] == -127).all()
    for r in (1, 2, 3, 7):
        rq, _ = ref_quantize(x[r:r + 1])
        assert (q[r].double() - rq[0]).abs().max() <= 1 and q[r].abs().max() == 127


def weights_i8(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-127, 128, shape, generator=g, dtype=torch.int8)
    s = (torch.rand(shape[:-1], generator=g) + 0.5) * 1e-2
    return q, s


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,N,K", [(1, 1, 16), (1, 128, 4096), (2, 129, 144), (5, 999, 1040),
                                   (16, 256, 128), (17, 300, 256), (61, 77, 496),
                                   (64, 4096, 1024), (129, 130, 272), (256, 128, 640),
                                   (257, 1000, 512), (301, 999, 1040), (520, 385, 14336)])
def test_matmul_i8(T, N, K, out):
    xq, sx = weights_i8(1, T, K)
    wq, sw = weights_i8(2, N, K)
    xq[0], wq[0] = 127, 127      # the largest sums
    wq[-1] = -127
    y = sfn.matmul_i8(xq.to(DEV), sx.to(DEV), wq.to(DEV), sw.to(DEV), out_dtype=out)
    acc = (xq.double() @ wq.double().T)
    ref = acc * sx.double()[:, None] * sw.double()
    tol = 4 * U + (BF16 if out == torch.bfloat16 else 0)
    assert y.shape == (T, N) and y.dtype == out
    assert ((y.cpu().double() - ref).abs() <= tol * ref.abs()).all()


def test_matmul_i8_longest_sum():
    K = 131072
    xq = torch.full((3, K), 127, dtype=torch.int8)
    wq = torch.full((2, K), -127, dtype=torch.int8)
    one = torch.ones(3)
    y = sfn.matmul_i8(xq.to(DEV), one.to(DEV), wq.to(DEV), one[:2].to(DEV).contiguous(),
                      out_dtype=torch.float32)
    assert ((y.cpu().double() + 127 * 127 * K).abs() <= U * 127 * 127 * K).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,N,K", [(1, 14336, 4096), (2, 100, 2064), (3, 257, 14336), (4, 64, 64),
                                   (7, 1000, 4096), (64, 512, 4096), (300, 200, 1040)])
def test_linear_i8(T, N, K, dtype):
    x = rand(T, T, K).to(dtype).to(DEV)
    wq, sw = (t.to(DEV) for t in weights_i8(5, N, K))
    y = sfn.linear_i8(x, wq, sw)
    q, s = sfn.quantize_rows_i8(x)
    ref = (q.double() @ wq.double().T) * s.double()[:, None] * sw.double()
    tol = 4 * U + (BF16 if dtype == torch.bfloat16 else 0)
    assert y.dtype == dtype
    assert ((y.double() - ref).abs() <= tol * ref.abs()).all()
    # bit for bit the composition, on guarded outputs
    buf = torch.full((T + 2, N), 7.0, dtype=dtype, device=DEV)
    if (N * buf.element_size()) % 16 == 0:
        sfn.linear_i8(x, wq, sw, out=buf[1:T + 1])
        assert torch.equal(buf[1:T + 1], y) and (buf[0] == 7).all() and (buf[-1] == 7).all()
    assert torch.equal(sfn.matmul_i8(q, s, wq, sw, out_dtype=dtype), y)


def test_linear_i8_nan_row_is_loud():
    x = rand(1, 5, 64).to(torch.bfloat16)
    x[3, 2] = math.inf
    wq, sw = weights_i8(5, 40, 64)
    y = sfn.linear_i8(x.to(DEV), wq.to(DEV), sw.to(DEV))
    assert torch.isnan(y[3]).all() and torch.isfinite(y[[0, 1, 2, 4]]).all()


# ---------------------------------------------------------- experts' products
def ref_experts(x, experts, weights, W):
    """Row by row in 64 bits, from the definition."""
    T, d = x.shape
    y = torch.zeros((T, d), dtype=torch.float64, device=x.device)
    room = torch.zeros_like(y)

    def product(v, wq, s):
        q, sv = ref_quantize(v)
        return (q @ wq.double().T) * sv[:, None] * s.double()

    for e in range(W["Wg"].shape[0]):
        t, i = torch.nonzero(experts == e, as_tuple=True)
        if t.numel() == 0:
            continue
        g = product(x[t], W["Wg"][e], W["sg"][e])
        u = product(x[t], W["Wu"][e], W["su"][e])
        h = (g * torch.sigmoid(g) * u).to(torch.bfloat16)
        o = product(h, W["Wd"][e], W["sd"][e])
        w = weights[t, i].double()[:, None]
        y.index_add_(0, t, w * o)
        # h is float32 before it is rounded to bf16: where that rounding falls
        # the other way (a few u of half way), h moves by a bf16 step and its
        # integer by at most one, a step sh = amax / 127 of the row against one
        # weight of at most 127 sd; a few such elements are allowed for
        _, sh = ref_quantize(h)
        room.index_add_(0, t, w.abs() * 4 * 127 * sh[:, None] * W["sd"][e].double())
    return y, room


def expert_weights(seed, E, f, d):
    W = {}
    for n, shape in (("g", (E, f, d)), ("u", (E, f, d)), ("d", (E, d, f))):
        W["W" + n], W["s" + n] = (t.to(DEV) for t in weights_i8(seed, *shape))
        W["s" + n] *= 1 / math.sqrt(shape[-1])
        seed += 1
    return W


EXPERTS = [
    # T, E, k, d, f
    (1, 4, 2, 64, 32), (1, 64, 8, 256, 112), (2, 8, 8, 128, 48), (3, 3, 1, 4096, 1792),
    (5, 16, 4, 272, 144), (8, 2, 2, 64, 128), (17, 7, 3, 144, 80), (61, 64, 8, 256, 128),
    (130, 5, 2, 384, 272), (300, 4, 4, 128, 256), (1000, 16, 2, 208, 96),
]


@pytest.mark.parametrize("T,E,k,d,f", EXPERTS)
def test_experts_i8(T, E, k, d, f):
    W = expert_weights(T, E, f, d)
    x = rand(T, T, d).to(torch.bfloat16).to(DEV)
    g = torch.Generator().manual_seed(T + E)
    experts = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    weights = torch.rand((T, k), generator=g)
    if T > 2:
        experts[0] = -1                       # a token without experts
        experts[1, k - 1] = experts[1, 0]     # the same expert twice
        experts[2, 0] = -1
        x[1] = 0
    experts, weights = experts.to(DEV), weights.to(DEV)
    buf = torch.full((T + 2, d), 7.0, dtype=torch.bfloat16, device=DEV)
    sfn.experts_i8_forward(x, experts, weights, y=buf[1:T + 1], **W)
    y = buf[1:T + 1].double()
    ref, room = ref_experts(x, experts, weights, W)
    assert (buf[0] == 7).all() and (buf[-1] == 7).all()
    assert ((y - ref).abs() <= (BF16 + 100 * U) * ref.abs() + room).all()
    # the bf16 rounding of y alone: at most 2^-8 everywhere
    assert (y - ref).norm() <= BF16 * ref.norm()
    if T > 2:
        assert (y[0] == 0).all() and (y[1] == 0).all()


def test_experts_i8_skewed():
    """Every token to one expert, and experts that nobody chose."""
    T, E, k, d, f = 200, 9, 2, 128, 64
    W = expert_weights(3, E, f, d)
    x = rand(1, T, d).to(torch.bfloat16).to(DEV)
    experts = torch.tensor([[8, 2]], dtype=torch.int32).repeat(T, 1).to(DEV)
    weights = torch.rand((T, k), generator=torch.Generator().manual_seed(1)).to(DEV)
    y = sfn.experts_i8_forward(x, experts, weights, **W)
    ref, room = ref_experts(x, experts, weights, W)
    assert ((y.double() - ref).abs() <= (BF16 + 100 * U) * ref.abs() + room).all()
    none = torch.full_like(experts, -1)
    assert (sfn.experts_i8_forward(x, none, weights, **W) == 0).all()


def test_route_then_experts():
    """A router's output straight into the experts' products, quantised
    weights included, in a captured graph that is replayed on new inputs."""
    T, E, k, d, f = 23, 32, 4, 256, 112
    wr = rand(1, E, d, scale=1 / 16).to(DEV)
    full = [rand(s, *sh, scale=1 / math.sqrt(sh[-1])).to(torch.bfloat16).to(DEV)
            for s, sh in ((2, (E, f, d)), (3, (E, f, d)), (4, (E, d, f)))]
    W = {}
    for n, m in zip("gud", full):
        W["W" + n], W["s" + n] = sfn.quantize_rows_i8(m)
    bias = (rand(5, E) * 0.01).to(DEV)
    x = rand(6, T, d).to(torch.bfloat16).to(DEV)

    def layer():
        logits = x.float() @ wr.T
        e, w, _ = sfn.route_experts(logits, k, bias=bias, score="sigmoid", groups=4,
                                    top_groups=2, group_top=2, scale=2.5)
        return e, w, sfn.experts_i8_forward(x, e, w, **W)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        e, w, y = layer()
    for seed in (7, 8):
        x.copy_(rand(seed, T, d).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        ref, room = ref_experts(x, e, w, W)
        assert ((y.double() - ref).abs() <= (BF16 + 100 * U) * ref.abs() + room).all()
        e2, w2, y2 = layer()
        assert torch.equal(e, e2) and torch.equal(w, w2) and torch.equal(y, y2)
        # against the unquantised experts: 8-bit steps of 1/127 of a row's
        # largest value on three products
        dense = torch.zeros((T, d), dtype=torch.float64, device=DEV)
        for t in range(T):
            for i in range(k):
                q = int(e[t, i])
                h = torch.nn.functional.silu(full[0][q].double() @ x[t].double()) \
                    * (full[1][q].double() @ x[t].double())
                dense[t] += float(w[t, i]) * (full[2][q].double() @ h)
        # each operand's rounding is uniform within half a step of amax / 127 and
        # amax is below 5 standard deviations here (h: below 12): relative errors of
        # 5 / (127 sqrt 12) (four of them) and 12 / (127 sqrt 12) (one), independent
        assert (y.double() - dense).norm() / dense.norm() <= 2 * math.sqrt(4 * 0.0114**2 + 0.0273**2)
