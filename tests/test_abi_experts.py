"""What the expert operators refuse, through the C ABI and through the binding (no GPU:
nothing here passes the checks of its arguments)."""
import math

import pytest
import torch

import predictor_gated_channel_b200 as sfn
from predictor_gated_channel_b200 import _capi
from predictor_gated_channel_b200 import build as sfn_build

FAKE = 1 << 20   # aligned, never dereferenced by a refused call
OK, INVALID, MISALIGNED = _capi.SFN_OK, _capi.SFN_ERR_INVALID_VALUE, _capi.SFN_ERR_MISALIGNED
UNSUPPORTED, WORKSPACE = _capi.SFN_ERR_UNSUPPORTED, _capi.SFN_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    sfn_build.build()
    return _capi.lib()


def route(L, logits=FAKE, dtype=1, bias=None, experts=FAKE, weights=FAKE, scores=None, T=4, E=64,
          k=8, score=0, groups=1, top=1, gtop=1, renorm=1, scale=1.0):
    return L.sfn_route_experts(logits, dtype, bias, experts, weights, scores, T, E, k, score,
                               groups, top, gtop, renorm, scale, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=65), INVALID),
    (dict(dtype=7), INVALID), (dict(score=2), INVALID), (dict(groups=0), INVALID),
    (dict(groups=3, top=1), INVALID),            # 64 is no multiple of 3
    (dict(groups=4, top=5), INVALID), (dict(groups=4, top=0), INVALID),
    (dict(groups=16, top=1, k=5), INVALID),      # 4 experts in the one group that stays
    (dict(groups=4, top=2, gtop=3), INVALID), (dict(scale=math.inf), INVALID),
    (dict(scale=math.nan), INVALID), (dict(E=1025, k=1), UNSUPPORTED),
    (dict(k=33), UNSUPPORTED), (dict(groups=64, top=64), UNSUPPORTED),
    (dict(logits=None), INVALID), (dict(experts=None), INVALID), (dict(weights=None), INVALID),
    (dict(logits=FAKE + 2), MISALIGNED), (dict(bias=FAKE + 2), MISALIGNED),
    (dict(experts=FAKE + 2), MISALIGNED), (dict(scores=FAKE + 1), MISALIGNED),
    (dict(T=0, logits=None, experts=None, weights=None), OK),
])
def test_route_refuses(L, kw, status):
    assert route(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(k=33), UNSUPPORTED),
    (dict(E=2000), UNSUPPORTED), (dict(score=-1), INVALID), (dict(scale=math.nan), INVALID),
    (dict(logits=None), INVALID), (dict(experts=None), INVALID), (dict(dw=None), INVALID),
    (dict(out=None), INVALID), (dict(dw=FAKE + 1), MISALIGNED), (dict(ds=FAKE + 2), MISALIGNED),
    (dict(T=0, logits=None, dw=None, out=None), OK),
])
def test_route_backward_refuses(L, kw, status):
    a = dict(logits=FAKE, experts=FAKE, dw=FAKE, ds=None, out=FAKE, T=4, E=64, k=8, score=0,
             scale=1.0)
    a.update(kw)
    assert L.sfn_route_experts_backward(a["logits"], 1, a["experts"], a["dw"], a["ds"], a["out"],
                                        a["T"], a["E"], a["k"], a["score"], 1, a["scale"],
                                        None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(K=24), MISALIGNED),
    (dict(K=131088), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED), (dict(xdt=3), INVALID),
    (dict(ydt=3), INVALID), (dict(x=None), INVALID), (dict(wq=None), INVALID),
    (dict(y=None), INVALID), (dict(x=FAKE + 8), MISALIGNED), (dict(wq=FAKE + 8), MISALIGNED),
    (dict(y=FAKE + 4), MISALIGNED), (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 16), WORKSPACE),
    (dict(ws_bytes=-256), WORKSPACE), (dict(T=0, x=None, y=None, ws=None, ws_bytes=0), OK),
])
def test_linear_refuses(L, kw, status):
    a = dict(x=FAKE, xdt=0, wq=FAKE, sw=FAKE, y=FAKE, ydt=0, T=8, N=256, K=512, ws=FAKE)
    need = L.sfn_linear_i8_workspace_bytes(8, 512)
    assert need > 0 and need % 256 == 0
    a["ws_bytes"] = need
    a.update(kw)
    if a["ws_bytes"] < 0:
        a["ws_bytes"] = need - 256
    assert L.sfn_linear_i8(a["x"], a["xdt"], a["wq"], a["sw"], a["y"], a["ydt"], a["T"], a["N"],
                           a["K"], a["ws"], a["ws_bytes"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(d=0), INVALID),
    (dict(d=24), MISALIGNED), (dict(f=40), MISALIGNED), (dict(E=1025), UNSUPPORTED),
    (dict(k=33), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED), (dict(ptr=0), INVALID),
    (dict(ptr=4), INVALID), (dict(ptr=9), INVALID), (dict(odd=0), MISALIGNED),
    (dict(odd=3), MISALIGNED), (dict(odd=7), MISALIGNED), (dict(ws=None), WORKSPACE),
    (dict(T=0, ws=None), OK),
])
def test_experts_refuse(L, kw, status):
    a = dict(T=8, E=4, k=2, d=256, f=128, ws=FAKE)
    need = L.sfn_experts_i8_workspace_bytes(8, 4, 2, 256, 128)
    assert need > 0 and need % 256 == 0
    a.update(kw)
    ptrs = [FAKE] * 10
    if "ptr" in kw:
        ptrs[kw["ptr"]] = None
    if "odd" in kw:
        ptrs[kw["odd"]] = FAKE + 8
    assert L.sfn_experts_i8_forward(*ptrs, a["T"], a["E"], a["k"], a["d"], a["f"], a["ws"], need,
                                    None) == status


def test_workspace_sizes_of_refused_shapes_are_zero(L):
    assert L.sfn_linear_i8_workspace_bytes(0, 512) == 0
    assert L.sfn_linear_i8_workspace_bytes(4, 24) == 0
    assert L.sfn_experts_i8_workspace_bytes(0, 4, 2, 256, 128) == 0
    assert L.sfn_experts_i8_workspace_bytes(4, 4, 2, 250, 128) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64)
    i8, s = torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8)
    for call in (lambda: sfn.route_experts(x, 2),
                 lambda: sfn.route_experts([[1.0, 2.0]], 1),
                 lambda: sfn.route_experts_backward(x, i8, x),
                 lambda: sfn.quantize_rows_i8(x),
                 lambda: sfn.matmul_i8(i8, s, i8, s),
                 lambda: sfn.linear_i8(x, i8, s),
                 lambda: sfn.experts_i8_forward(x, i8, x, i8, s, i8, s, i8, s)):
        with pytest.raises(ValueError):
            call()
