"""The expert operators where their kernels change form: CTA pairs, split K slices, streams of
few tokens, wide SwiGLU tiles, packed keys that cannot decide, rows of other lengths; and calls as
a program makes them: captured, on other streams, two at once.

Tolerances as in test_gpu_experts.py: the integer sums are exact, so a product is right to the
conversion, the scalings (4 u) and its own rounding; choices are equal."""
import math

import numpy as np
import pytest
import torch

import predictor_gated_channel_b200 as sfn
from predictor_gated_channel_b200 import _capi
from predictor_gated_channel_b200 import build as sfn_build
from test_gpu_experts import (BF16, DEV, U, expert_weights, rand, ref_experts, ref_quantize,
                              ref_route, ref_route_bwd, weights_i8)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    sfn_build.build()
    _capi.lib()


def product(xq, sx, wq, sw):
    # float64 holds these integer sums exactly
    return (xq.double() @ wq.double().T) * sx.double()[:, None] * sw.double()


def close(y, ref, dtype):
    tol = 4 * U + (BF16 if dtype == torch.bfloat16 else 0)
    return ((y.double() - ref).abs() <= tol * ref.abs()).all()


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,N,K", [
    (2048, 7200, 144),      # CTA pairs: 8 x 29 tiles, a ragged last one
    (2303, 6912, 1040),     # pairs, rows that do not fill the last tile
    (4100, 4112, 256),      # pairs, an odd number of 128-channel halves
    (64, 256, 14336),       # eight CTAs share a tile's slices
    (33, 1000, 8208),       # shared slices, a ragged slice and tile
    (200, 384, 4096), (256, 130, 4112), (5, 17, 131072),
])
def test_product_forms(T, N, K, out):
    xq, sx = (t.to(DEV) for t in weights_i8(1, T, K))
    wq, sw = (t.to(DEV) for t in weights_i8(2, N, K))
    y = sfn.matmul_i8(xq, sx, wq, sw, out_dtype=out)
    assert close(y, product(xq, sx, wq, sw), out)
    assert torch.equal(sfn.matmul_i8(xq, sx, wq, sw, out_dtype=out), y)


def test_product_of_the_lowest_values():
    K = 131056
    xq = torch.full((9, K), -128, dtype=torch.int8, device=DEV)
    wq = torch.full((130, K), -128, dtype=torch.int8, device=DEV)
    y = sfn.matmul_i8(xq, torch.ones(9, device=DEV), wq, torch.ones(130, device=DEV),
                      out_dtype=torch.float32)
    assert ((y.double() - 16384.0 * K).abs() <= U * 16384.0 * K).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,N,K", [(1, 1, 16), (1, 999, 40960), (2, 14337, 1040), (3, 4096, 4096),
                                   (4, 5000, 4096), (3, 148, 2048), (4, 147, 2064)])
def test_few_tokens(T, N, K, dtype):
    x = rand(T + K, T, K).to(dtype).to(DEV)
    wq, sw = (t.to(DEV) for t in weights_i8(5, N, K))
    q, s = sfn.quantize_rows_i8(x)
    y = sfn.linear_i8(x, wq, sw)
    assert close(y, product(q, s, wq, sw), dtype)
    assert torch.equal(y, sfn.matmul_i8(q, s, wq, sw, out_dtype=dtype))


def test_every_bf16_quantises_to_the_nearest():
    """Every finite bf16 up to amax, for amaxes that put many quotients exactly
    half way, and for the ends of the range."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    finite = bits[torch.isfinite(bits)]
    g = torch.Generator().manual_seed(1)
    amaxes = finite[torch.randint(0, finite.numel(), (60,), generator=g)].abs()
    ends = torch.tensor([2.0 ** -133, 2.0 ** -126, 1e-30, 1e30, 3.3e38, 1.0, 3.5, 4.0, 127.0])
    for amax in torch.cat([amaxes, ends.to(torch.bfloat16)]):
        if amax == 0:
            continue
        x = finite[finite.abs() <= amax]
        row = torch.zeros((1, (x.numel() + 15) // 16 * 16), dtype=torch.bfloat16)
        row[0, :x.numel()] = x
        q, _ = sfn.quantize_rows_i8(row.to(DEV))
        ref = torch.round(127 * row.double() / amax.double())
        assert torch.equal(q.cpu().double(), ref), amax


# ------------------------------------------------------------------ experts
@pytest.mark.parametrize("T,E,k,d,f", [
    (1500, 3, 2, 272, 208),    # 1000 rows an expert: pairs, the widest SwiGLU tile
    (700, 5, 2, 144, 4096),    # long h
    (64, 1, 1, 256, 128),      # one expert, one slot each
    (600, 8, 1, 4096, 16),     # the shortest h
    (16, 2, 2, 64, 48), (33, 3, 1, 64, 48),   # one slot more or less than the stream takes
    (32, 5, 1, 208, 1040), (1, 40, 32, 128, 64), (2, 33, 17, 128, 64),
])
def test_experts_forms(T, E, k, d, f):
    W = expert_weights(T, E, f, d)
    x = rand(T, T, d).to(torch.bfloat16).to(DEV)
    g = torch.Generator().manual_seed(T + E)
    experts = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    experts[T // 2, 0] = -1
    weights = torch.rand((T, k), generator=g)
    experts, weights = experts.to(DEV), weights.to(DEV)
    y = sfn.experts_i8_forward(x, experts, weights, **W).double()
    ref, room = ref_experts(x, experts, weights, W)
    assert ((y - ref).abs() <= (BF16 + 100 * U) * ref.abs() + room).all()
    # y's own rounding (at most 2^-8 anywhere); a slot's 2^-12 before the sum is
    # a sixteenth of that
    assert (y - ref).norm() <= (BF16 + 2.0 ** -12) * ref.norm()


def test_experts_scales_of_any_size():
    """Down scales over the whole range within one block of channels, zeros
    and a NaN among them: each touches its own channel only."""
    T, E, k, d, f = 300, 2, 1, 96, 64
    W = expert_weights(2, E, f, d)
    sd = W["sd"]
    sd[:, 1::8] *= 2.0 ** -9     # in range of a block: full precision
    sd[:, 2] = 0.0
    sd[0, 3] = math.nan
    sd[1, 40] *= -1.0
    sd[:, 64:] *= 1e-30          # a block of small ones, and one of large ones
    sd[:, 32:64] *= 1e25
    x = rand(3, T, d).to(torch.bfloat16).to(DEV)
    experts = (torch.arange(T, device=DEV) % E).to(torch.int32)[:, None].contiguous()
    weights = torch.rand((T, k), generator=torch.Generator().manual_seed(1)).to(DEV)
    y = sfn.experts_i8_forward(x, experts, weights, **W).double()
    ref, room = ref_experts(x, experts, weights, W)
    bad = torch.isnan(ref)
    assert torch.equal(torch.isnan(y), bad) and bad.any() and not bad[:, 4:].any()
    # room is a magnitude times the scale: of a negative scale, its magnitude
    ok = (y - ref).abs() <= (BF16 + 2.0 ** -11) * ref.abs() + room.abs()
    assert (ok | bad).all()


def test_experts_bad_row_is_loud():
    for T in (3, 200):
        W = expert_weights(2, 4, 64, 128)
        x = rand(3, T, 128).to(torch.bfloat16).to(DEV)
        x[1, 5] = math.inf
        experts = (torch.arange(2 * T, device=DEV) % 4).to(torch.int32).view(T, 2)
        y = sfn.experts_i8_forward(x, experts, torch.ones((T, 2), device=DEV), **W)
        assert torch.isnan(y[1]).all()
        assert torch.isfinite(y[0]).all() and torch.isfinite(y[2:]).all()


def test_index_past_the_experts_is_reported():
    import ctypes
    W = expert_weights(2, 4, 64, 128)
    for T in (3, 200):
        x = rand(3, T, 128).to(torch.bfloat16).to(DEV)
        experts = torch.zeros((T, 2), dtype=torch.int32, device=DEV)
        experts[1, 1] = 4
        weights = torch.ones((T, 2), device=DEV)
        y = sfn.experts_i8_forward(x, experts, weights, **W)
        torch.cuda.synchronize()
        bits = ctypes.c_uint(0)
        assert _capi.lib().sfn_device_errors(ctypes.byref(bits), 1) == _capi.SFN_OK
        assert bits.value == 2
        experts[1, 1] = -1
        assert torch.equal(y, sfn.experts_i8_forward(x, experts, weights, **W))


# ------------------------------------------------------------------ routing
@pytest.mark.parametrize("score,bias", [("softmax", False), ("softmax", True), ("sigmoid", True),
                                        ("sigmoid", False)])
@pytest.mark.parametrize("T,E,k,groups,top,gtop", [
    (300, 160, 8, 8, 4, 2),    # five experts a lane, in groups
    (300, 192, 6, 1, 1, 1), (300, 384, 31, 16, 9, 2), (300, 96, 32, 1, 1, 1),
    (300, 64, 8, 32, 8, 1), (20000, 64, 3, 1, 1, 1), (9000, 256, 8, 8, 4, 2),
    (300, 48, 4, 6, 3, 2),
])
def test_route_forms(T, E, k, groups, top, gtop, score, bias):
    """Values on a coarse grid, so that equal scores are everywhere: in a lane,
    across lanes, at the k-th place, between groups."""
    g = torch.Generator().manual_seed(E + k)
    logits = torch.round(torch.randn((T, E), generator=g) * 12) / 8
    logits[5] = torch.round(logits[5])      # and some rows with few values
    b = torch.round(torch.randn(E, generator=g) * 4) / 64 if bias else None
    rows = torch.cat([torch.arange(min(T, 300)), torch.arange(max(T - 100, 0), T)]).unique()
    re, rw, _ = ref_route(logits[rows], k, b, score, groups, top, gtop, True, 1.0)
    for dtype in (torch.float32, torch.bfloat16):   # the grid is exact in both
        e, w, _ = sfn.route_experts(logits.to(dtype).to(DEV), k,
                                    bias=None if b is None else b.to(DEV), score=score,
                                    groups=groups, top_groups=top, group_top=gtop)
        assert np.array_equal(e.cpu()[rows].numpy(), re)
        assert np.allclose(w.cpu()[rows].double().numpy(), rw, rtol=100 * U, atol=1e-37)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(64, 1), (160, 1), (256, 8), (100, 5)])
def test_route_scores_a_rounding_apart(E, groups, score):
    """Biases that cancel the scores to within a few 1e-8: the float32 scores
    cannot tell them apart, the definition can."""
    T, k = 60, 8
    g = torch.Generator().manual_seed(E)
    one = torch.randn(E, generator=g)
    logits = one[None, :].repeat(T, 1) + torch.randint(-2, 3, (T, E), generator=g) * 2.0 ** -23
    s = torch.softmax(one.double(), 0) if score == "softmax" else torch.sigmoid(one.double())
    bias = (0.9 - s).float()
    e, _, _ = sfn.route_experts(logits.to(DEV), k, bias=bias.to(DEV), score=score, groups=groups,
                                top_groups=max(1, groups // 2), group_top=2 if groups > 1 else 1)
    re, _, _ = ref_route(logits, k, bias, score, groups, max(1, groups // 2),
                         2 if groups > 1 else 1)
    assert np.array_equal(e.cpu().numpy(), re)


def test_route_biases_that_are_no_numbers():
    """A NaN bias ranks its expert below every number, +inf above, -inf takes it
    out; a softmax row with +inf has NaN scores, which rank equal: the lower
    indexes.  In rows few and many (other kernels), with and without groups."""
    E, k = 64, 4
    for T, groups, top in ((7, 1, 1), (7, 8, 8), (20000, 1, 1)):
        logits = rand(3, T, E)
        bias = torch.zeros(E)
        bias[5], bias[9], bias[11], bias[60] = math.nan, math.inf, -math.inf, math.inf
        for score in ("softmax", "sigmoid"):
            e, w, _ = sfn.route_experts(logits.to(DEV), k, bias=bias.to(DEV), score=score,
                                        groups=groups, top_groups=top)
            ok = bias.clone()
            ok[5] = -math.inf    # below every number: not among four of 62
            re, rw, _ = ref_route(logits[:50], k, ok, score, groups, top)
            assert np.array_equal(e.cpu()[:50].numpy(), re)
            assert (e[:, 0] == 9).all() and (e[:, 1] == 60).all()
            assert np.allclose(w.cpu()[:50].double().numpy(), rw, rtol=100 * U, atol=1e-37)
        logits[2, 7] = math.inf
        e, w, _ = sfn.route_experts(logits.to(DEV), k, bias=torch.zeros(E, device=DEV),
                                    groups=groups, top_groups=top)
        assert e[2].tolist() == [0, 1, 2, 3] and torch.isnan(w[2]).all()
        assert torch.isfinite(w[[0, 1, 3, 4, 5, 6]]).all()


@pytest.mark.parametrize("E", [5, 64, 160, 256, 600])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_backward_long(E, dtype):
    """More rows than the grid has warps, a balance gradient, empty slots."""
    T, k = 6000, min(E, 5)
    g = torch.Generator().manual_seed(E)
    logits = torch.randn((T, E), generator=g).to(dtype)
    experts = torch.topk(logits.float(), k, dim=1).indices.to(torch.int32)
    experts[::7, k - 1] = -1
    dw, ds = torch.randn((T, k), generator=g), torch.randn((T, E), generator=g)
    got = sfn.route_experts_backward(logits.to(DEV), experts.to(DEV), dw.to(DEV),
                                     dscores=ds.to(DEV), renormalize=False).cpu().double()
    s = torch.softmax(logits.double(), 1)
    full = ds.double().scatter_add(1, experts.long().clamp(min=0), dw.double() * (experts >= 0))
    ref = s * (full - (s * full).sum(1, keepdim=True))
    tol = 200 * U * s * 2 * full.abs().amax(1, keepdim=True) + 1e-37
    if dtype == torch.bfloat16:
        tol = tol + BF16 * ref.abs()
    assert ((got - ref).abs() <= tol).all()


@pytest.mark.parametrize("T,E,k,groups,top,bias", [
    (5000, 5, 3, 1, 1, False), (5000, 25, 6, 1, 1, False), (17000, 9, 2, 1, 1, True),
    (17000, 250, 8, 1, 1, True), (3000, 250, 8, 1, 1, False), (3000, 160, 8, 8, 4, False),
    (3001, 64, 4, 4, 2, False), (2050, 256, 8, 2, 1, False), (4099, 130, 1, 1, 1, False),
])
@pytest.mark.parametrize("grid", [True, False])
def test_route_many_rows(T, E, k, groups, top, bias, grid):
    """Eight lanes a row: lanes without values, odd row counts, ties (on a grid)
    and plain values, with masked rows among them."""
    g = torch.Generator().manual_seed(T + E)
    logits = torch.randn((T, E), generator=g) * 1.5
    if grid:
        logits = torch.round(logits * 8) / 8
    logits[7] = -math.inf
    logits[11, 1:] = -math.inf
    b = torch.round(torch.randn(E, generator=g) * 4) / 64 if bias else None
    rows = torch.cat([torch.arange(100), torch.arange(T - 60, T)])
    for dtype in (torch.float32, torch.bfloat16):
        x = logits.to(dtype)
        for score in ("softmax", "sigmoid"):
            for renorm in (True, False):
                e, w, _ = sfn.route_experts(x.to(DEV), k, bias=None if b is None else b.to(DEV),
                                            score=score, groups=groups, top_groups=top,
                                            renormalize=renorm, scale=1.5)
                re, rw, _ = ref_route(x[rows], k, b, score, groups, top, 1, renorm, 1.5)
                assert np.array_equal(e.cpu()[rows].numpy(), re)
                assert np.allclose(w.cpu()[rows].double().numpy(), rw, rtol=100 * U, atol=1e-37)


@pytest.mark.parametrize("T,E,k", [(9001, 5, 3), (8192, 64, 8), (9000, 100, 4), (8195, 128, 8),
                                   (8200, 256, 5)])
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True),
                                          ("sigmoid", True)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_backward_many_rows(T, E, k, score, renorm, dtype):
    g = torch.Generator().manual_seed(E)
    logits = torch.randn((T, E), generator=g).to(dtype)
    experts = torch.topk(logits.float(), k, dim=1).indices.to(torch.int32)
    experts[::7, k - 1] = -1
    experts[3::9, 1] = experts[3::9, 0]     # the same expert twice
    dw, ds = torch.randn((T, k), generator=g), torch.randn((T, E), generator=g)
    got = sfn.route_experts_backward(logits.to(DEV), experts.to(DEV), dw.to(DEV),
                                     dscores=ds.to(DEV), score=score, renormalize=renorm,
                                     scale=1.5)
    ref, s = ref_route_bwd(logits, experts, dw, ds, score, renorm, 1.5)
    chosen = (s.gather(1, experts.long().clamp(min=0)) * (experts >= 0)).sum(1, keepdim=True)
    unit = 1.5 * dw.abs().double().amax(1, keepdim=True) * 2
    if renorm:
        unit = unit / chosen.clamp(min=1e-30)
    # as in test_route_backward: terms of at most max |ds| each, right to 100 u
    unit = unit + 2 * ds.abs().double().amax(1, keepdim=True)
    tol = 100 * U * unit * s + (BF16 * ref.abs() if dtype == torch.bfloat16 else 0) + 1e-37
    assert ((got.cpu().double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("T", [50, 9000])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_backward_of_constant_weights(T, score):
    """Renormalised weights do not change where there is one expert, nor along
    a dweights that is the same for all slots: gradients of exactly 0.  What an
    empty slot's dweights holds does not matter."""
    E = 100
    logits = rand(T, T, E)
    for k in (1, 4):
        experts = torch.topk(logits, k, dim=1).indices.to(torch.int32)
        dw = rand(3, T, 1).repeat(1, k)
        experts[5] = -1
        dw[5] = math.nan
        if k > 1:
            experts[::3, 0] = -1
            dw[::3, 0] = math.inf
        for ds in (None, torch.zeros((T, E))):
            g = sfn.route_experts_backward(logits.to(DEV), experts.to(DEV), dw.to(DEV), score=score,
                                           dscores=None if ds is None else ds.to(DEV))
            assert (g == 0).all()


# ------------------------------------------------------- as a program calls them
def test_captured_and_replayed():
    """Every form of the product in one graph, with one workspace, replayed on
    new inputs."""
    shapes = [(1, 512, 1024), (64, 256, 8192), (2100, 7168, 256), (300, 500, 1040)]
    ws = torch.empty(max(sfn.linear_i8_workspace_bytes(T, K) for T, _, K in shapes),
                     dtype=torch.uint8, device=DEV)
    parts = []
    for i, (T, N, K) in enumerate(shapes):
        wq, sw = (t.to(DEV) for t in weights_i8(i, N, K))
        parts.append((rand(i, T, K).to(torch.bfloat16).to(DEV), wq, sw,
                      torch.empty((T, N), dtype=torch.bfloat16, device=DEV)))

    def run():
        for x, wq, sw, y in parts:
            sfn.linear_i8(x, wq, sw, out=y, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in (21, 22):
        for i, (x, wq, sw, y) in enumerate(parts):
            x.copy_(rand(seed + i, *x.shape))
            y.fill_(7.0)
        graph.replay()
        for x, wq, sw, y in parts:
            q, s = sfn.quantize_rows_i8(x)
            assert close(y, product(q, s, wq, sw), torch.bfloat16)


def test_two_streams_at_once():
    W = expert_weights(2, 8, 256, 512)
    wq, sw = (t.to(DEV) for t in weights_i8(5, 2048, 1024))
    x1, x2 = rand(1, 900, 512).to(torch.bfloat16).to(DEV), rand(2, 64, 1024).to(DEV)
    experts = torch.stack([torch.randperm(8, generator=torch.Generator().manual_seed(t))[:2]
                           for t in range(900)]).to(torch.int32).to(DEV)
    weights = torch.rand((900, 2), generator=torch.Generator().manual_seed(1)).to(DEV)
    y1 = sfn.experts_i8_forward(x1, experts, weights, **W)
    y2 = sfn.linear_i8(x2, wq, sw)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        z1 = sfn.experts_i8_forward(x1, experts, weights, **W, stream=a)
        z2 = sfn.linear_i8(x2, wq, sw, stream=b)
        torch.cuda.synchronize()
        assert torch.equal(z1, y1) and torch.equal(z2, y2)


def test_memory_of_another_stream_is_not_taken():
    """A block freed while its own stream still writes it must not become the
    output or scratch of a call on another stream."""
    T, N, K = 64, 4096, 4096
    x = rand(1, T, K).to(torch.bfloat16).to(DEV)
    wq, sw = (t.to(DEV) for t in weights_i8(5, N, K))
    want = sfn.linear_i8(x, wq, sw)
    logits = rand(2, 5000, 64).to(DEV)
    e0, w0, _ = sfn.route_experts(logits, 8)
    side = torch.cuda.Stream()
    for _ in range(5):
        blocks = [torch.empty_like(want), torch.empty_like(e0), torch.empty_like(w0),
                  torch.empty(sfn.linear_i8_workspace_bytes(T, K), dtype=torch.uint8, device=DEV)]
        torch.cuda.synchronize()
        torch.cuda._sleep(4_000_000)   # about 2 ms
        for b in blocks:
            b.fill_(7)
        del blocks, b
        y = sfn.linear_i8(x, wq, sw, stream=side)
        e, w, _ = sfn.route_experts(logits, 8, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(e, e0) and torch.equal(w, w0)


def test_weights_written_just_before():
    """Weights quantised on the stream right before the call that reads them:
    the product must not run ahead of them."""
    for T, N, K in ((1, 14336, 2048), (64, 512, 8192), (300, 4096, 1024), (2100, 7168, 256)):
        x = rand(1, T, K).to(torch.bfloat16).to(DEV)
        full = [rand(s, N, K).to(DEV) for s in (2, 3)]
        want = [sfn.linear_i8(x, *sfn.quantize_rows_i8(m)) for m in full]
        torch.cuda.synchronize()
        wq = torch.empty((N, K), dtype=torch.int8, device=DEV)
        sw = torch.empty(N, device=DEV)
        for i in range(10):
            sfn.quantize_rows_i8(full[i % 2], q=wq, scale=sw)
            y = sfn.linear_i8(x, wq, sw)
            assert torch.equal(y, want[i % 2])


def test_binding_refuses():
    x, i8 = torch.zeros(4, 64, device=DEV), torch.zeros((8, 64), dtype=torch.int8, device=DEV)
    s = torch.zeros(8, device=DEV)
    e = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    w3 = torch.zeros((2, 8, 64), dtype=torch.int8, device=DEV)
    for call in (lambda: sfn.route_experts(x.half(), 2),
                 lambda: sfn.route_experts(x[0], 1),
                 lambda: sfn.route_experts(x.T, 2),
                 lambda: sfn.route_experts(x, 2, bias=torch.zeros(63, device=DEV)),
                 lambda: sfn.route_experts(x, 2, bias=torch.zeros(64)),
                 lambda: sfn.route_experts(x, 2, score="relu"),
                 lambda: sfn.route_experts(x, 2, experts=e.long()),
                 lambda: sfn.route_experts_backward(x, e, torch.zeros((4, 3), device=DEV)),
                 lambda: sfn.route_experts_backward(x, e.long(), torch.zeros((4, 2), device=DEV)),
                 lambda: sfn.matmul_i8(i8, s[:8], i8[:, :32], s),
                 lambda: sfn.linear_i8(x, i8.float(), s),
                 lambda: sfn.linear_i8(x, i8, s[:7]),
                 lambda: sfn.linear_i8(x, i8, s, out=torch.zeros((4, 9), device=DEV)),
                 lambda: sfn.experts_i8_forward(x.to(torch.bfloat16), e, x[:, :2].contiguous(), w3, s,
                                                w3, s, w3, s)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(sfn.SfnError):
        sfn.route_experts(x, 65)
    with pytest.raises(sfn.SfnError):
        sfn.linear_i8(x[:, :40].contiguous(), i8[:, :40].contiguous(), s)
    with pytest.raises(sfn.SfnError):
        sfn.linear_i8(x, i8, s, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
