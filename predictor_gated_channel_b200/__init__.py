"""Predictor-gated bank-wise top-k sparse SwiGLU FFN forward on B200 (sm_100a), and the
operators of its coarse counterpart: routing to whole SwiGLU experts, the product in 8-bit
integers, and the experts' products.

Thin PyTorch-facing binding of the C ABI in ``include/sfn.h``: these functions
only check tensors and pass their device pointers and the current CUDA stream
to ``libsfn.so``; every step of the computation runs in the library's CUDA
kernels.  There is no CPU path: without the built library or a CUDA device
every call raises.

Method: "Continual LLM Upcycling: A Predictor-Gated Bank-Wise Sparsity
Training Recipe for Dense-to-Sparse LLMs" (arXiv 2606.10722), gist.science
summary, "1. Architectuur" and "3. Hardware Implicaties".
"""
from __future__ import annotations

import functools

from . import _capi
from ._capi import SfnError

__all__ = ["predict", "bank_topk", "sparse_ffn_forward", "dense4x_forward", "workspace_bytes",
           "route_experts", "route_experts_backward", "quantize_rows_i8", "matmul_i8",
           "linear_i8", "linear_i8_workspace_bytes", "experts_i8_forward",
           "experts_i8_workspace_bytes", "kernel_launch_count", "SfnError"]


_module = None


def _torch():
    global _module
    if _module is None:
        import torch
        _module = torch
    return _module


def _stream_ptr(stream, device):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


def _dev(t, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _elt(dtype):
    torch = _torch()
    if dtype == torch.bfloat16:
        return _capi.SFN_DTYPE_BF16
    if dtype == torch.float32:
        return _capi.SFN_DTYPE_F32
    raise ValueError(f"unsupported dtype {dtype}: bf16 or float32")


def kernel_launch_count() -> int:
    """Kernels libsfn has launched in this process."""
    return int(_capi.lib().sfn_kernel_launch_count())


def workspace_bytes(T: int, d: int, d_i: int, r: int, bank: int, k: int, dtype) -> int:
    return int(_capi.lib().sfn_workspace_bytes(T, d, d_i, r, bank, k, _elt(dtype)))


def predict(x, A, B, out=None, stream=None):
    """Predictor logits p = B (A x) per token -> float32 [T, d_i]."""
    torch = _torch()
    for n, t in (("x", x), ("A", A), ("B", B)):
        _dev(t, n)
    T, d = x.shape
    r, d_i = A.shape[0], B.shape[0]
    if A.shape != (r, d) or B.shape != (d_i, r) or not (x.dtype == A.dtype == B.dtype):
        raise ValueError("predict: x [T,d], A [r,d], B [d_i,r] of one dtype")
    if out is None:
        out = torch.empty((T, d_i), dtype=torch.float32, device=x.device)
    _dev(out, "out")
    fn = (_capi.lib().sfn_predict if _elt(x.dtype) == _capi.SFN_DTYPE_BF16
          else _capi.lib().sfn_predict_f32)
    _capi.check(fn(x.data_ptr(), A.data_ptr(), B.data_ptr(), out.data_ptr(), T, d, d_i, r,
                   _stream_ptr(stream, x.device)), "sfn_predict")
    return out


def bank_topk(logits, bank: int = 64, k: int = 16, out=None, stream=None):
    """Bank-wise hard top-k of float32 logits [T, d_i] -> int64 [T, d_i/bank]
    holding the uint64 mask bit patterns (bit i of word b = channel b*bank+i)."""
    torch = _torch()
    _dev(logits, "logits")
    if logits.dtype != torch.float32:
        raise ValueError("bank_topk: logits must be float32")
    T, d_i = logits.shape
    if out is None:
        out = torch.empty((T, max(d_i // max(bank, 1), 0)), dtype=torch.int64,
                          device=logits.device)
    _dev(out, "out")
    _capi.check(_capi.lib().sfn_bank_topk(logits.data_ptr(), out.data_ptr(), T, d_i, bank, k,
                                          _stream_ptr(stream, logits.device)), "sfn_bank_topk")
    return out


PATHS = {"auto": _capi.SFN_PATH_AUTO, "cuda_core": _capi.SFN_PATH_CUDA_CORE,
         "tensor": _capi.SFN_PATH_TENSOR}


def sparse_ffn_forward(x, A, B, Wg, Wu, Wd, bank: int = 64, k: int = 16, y=None, mask=None,
                       workspace=None, want_mask: bool = True, path: str = "auto",
                       stream=None):
    """The sparse FFN forward.  Wd is channel-major: Wd[j] = W_down[:, j].

    Returns (y [T, d] in x's dtype, mask int64 [T, d_i/bank] or None).  With
    ``workspace`` (a uint8 CUDA tensor of at least ``workspace_bytes(...)``)
    the call uses it as scratch instead of allocating stream-ordered memory.
    ``path`` ("auto", "cuda_core" or "tensor") picks the kernels; a bf16
    call with an explicit path always uses caller scratch (allocated here
    when ``workspace`` is None).
    """
    torch = _torch()
    names = ("x", "A", "B", "Wg", "Wu", "Wd")
    ts = (x, A, B, Wg, Wu, Wd)
    for n, t in zip(names, ts):
        _dev(t, n)
    if len({t.dtype for t in ts}) != 1:
        raise ValueError("sparse_ffn_forward: all inputs must share one dtype")
    elt = _elt(x.dtype)
    T, d = x.shape
    r, d_i = A.shape[0], B.shape[0]
    if (A.shape != (r, d) or B.shape != (d_i, r) or Wg.shape != (d_i, d)
            or Wu.shape != (d_i, d) or Wd.shape != (d_i, d)):
        raise ValueError("sparse_ffn_forward: shapes x [T,d], A [r,d], B [d_i,r], "
                         "Wg/Wu/Wd [d_i,d]")
    if y is None:
        y = torch.empty((T, d), dtype=x.dtype, device=x.device)
    _dev(y, "y")
    if mask is None and want_mask:
        mask = torch.empty((T, max(d_i // max(bank, 1), 0)), dtype=torch.int64,
                           device=x.device)
    mptr = None
    if mask is not None:
        _dev(mask, "mask")
        mptr = mask.data_ptr()
    st = _stream_ptr(stream, x.device)
    L = _capi.lib()
    args = [x.data_ptr(), A.data_ptr(), B.data_ptr(), Wg.data_ptr(), Wu.data_ptr(),
            Wd.data_ptr(), y.data_ptr(), mptr, T, d, d_i, r, bank, k]
    if path != "auto":
        if elt != _capi.SFN_DTYPE_BF16:
            raise ValueError("an explicit path is available for bf16 only")
        if workspace is None:
            nbytes = workspace_bytes(T, d, d_i, r, bank, k, x.dtype)
            workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=x.device)
        _dev(workspace, "workspace")
        _capi.check(L.sfn_sparse_ffn_forward_path(
            *args, PATHS[path], workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), st), "sfn_sparse_ffn_forward_path")
        return y, mask
    if workspace is None:
        fn = (L.sfn_sparse_ffn_forward if elt == _capi.SFN_DTYPE_BF16
              else L.sfn_sparse_ffn_forward_f32)
        _capi.check(fn(*args, st), "sfn_sparse_ffn_forward")
    else:
        _dev(workspace, "workspace")
        fn = (L.sfn_sparse_ffn_forward_ws if elt == _capi.SFN_DTYPE_BF16
              else L.sfn_sparse_ffn_forward_f32_ws)
        _capi.check(fn(*args, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                       st), "sfn_sparse_ffn_forward_ws")
    return y, mask


def bank_shard(n_banks: int, rank: int, world: int) -> tuple:
    """Banks [b0, b1) of shard ``rank`` of ``world``: contiguous, sizes differing by
    at most one, covering every bank once."""
    if not 0 <= rank < world:
        raise ValueError("bank_shard: rank outside [0, world)")
    return n_banks * rank // world, n_banks * (rank + 1) // world


def sparse_ffn_forward_partial(x, A, B, Wg, Wu, Wd, bank: int = 64, k: int = 16,
                               y_partial=None, mask=None, workspace=None, path: str = "auto",
                               stream=None):
    """One bank shard of the layer (bf16): B, Wg, Wu, Wd hold only the shard's
    rows.  Returns (y_partial float32 [T, d], mask int64 [T, shard banks]); the
    sum of y_partial over a partition of the banks is the layer's y before
    rounding."""
    torch = _torch()
    for n, t in (("x", x), ("A", A), ("B", B), ("Wg", Wg), ("Wu", Wu), ("Wd", Wd)):
        _dev(t, n)
    T, d = x.shape
    r, d_i = A.shape[0], B.shape[0]
    if y_partial is None:
        y_partial = torch.empty((T, d), dtype=torch.float32, device=x.device)
    if mask is None:
        mask = torch.empty((T, max(d_i // max(bank, 1), 0)), dtype=torch.int64,
                           device=x.device)
    if workspace is None:
        nbytes = workspace_bytes(T, d, d_i, r, bank, k, x.dtype)
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=x.device)
    L = _capi.lib()
    _capi.check(L.sfn_sparse_ffn_forward_partial(
        x.data_ptr(), A.data_ptr(), B.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), Wd.data_ptr(),
        y_partial.data_ptr(), mask.data_ptr(), T, d, d_i, r, bank, k, PATHS[path],
        workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _stream_ptr(stream, x.device)), "sfn_sparse_ffn_forward_partial")
    return y_partial, mask


def dense4x_forward(x, Wg, Wu, Wd, bank: int = 64, k: int = 16, y=None, mask=None,
                    workspace=None, stream=None):
    """The Dense-4x comparison (post-hoc amplitude top-k of the SwiGLU
    activation, no predictor).  bf16.  Returns (y [T, d], mask int64)."""
    torch = _torch()
    for n, t in (("x", x), ("Wg", Wg), ("Wu", Wu), ("Wd", Wd)):
        _dev(t, n)
    T, d = x.shape
    d_i = Wg.shape[0]
    if y is None:
        y = torch.empty((T, d), dtype=x.dtype, device=x.device)
    if mask is None:
        mask = torch.empty((T, max(d_i // max(bank, 1), 0)), dtype=torch.int64, device=x.device)
    L = _capi.lib()
    if workspace is None:
        nbytes = int(L.sfn_dense4x_workspace_bytes(T, d, d_i, bank, k))
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=x.device)
    _capi.check(L.sfn_dense4x_forward(x.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), Wd.data_ptr(),
                                      y.data_ptr(), mask.data_ptr(), T, d, d_i, bank, k,
                                      workspace.data_ptr(),
                                      workspace.numel() * workspace.element_size(),
                                      _stream_ptr(stream, x.device)), "sfn_dense4x_forward")
    return y, mask


def sparse_ffn_backward(x, A, B, Wg, Wu, Wd, dy, bank: int = 64, k: int = 16,
                        temperature: float = 1.0, want=("dx", "dA", "dB", "dWg", "dWu", "dWd"),
                        workspace=None, stream=None) -> dict:
    """Gradients of the layer for dy = dL/dy (bf16 inputs, float32 outputs),
    with the soft surrogate gradient of the bank top-k (see
    ``sfn_sparse_ffn_backward`` in include/sfn.h).  Returns a dict holding
    the gradients named in ``want`` and the forward's ``mask``."""
    torch = _torch()
    for n, t in (("x", x), ("A", A), ("B", B), ("Wg", Wg), ("Wu", Wu), ("Wd", Wd), ("dy", dy)):
        _dev(t, n)
    T, d = x.shape
    r = A.shape[0]
    d_i = B.shape[0]
    f32 = dict(dtype=torch.float32, device=x.device)
    shapes = {"dx": (T, d), "dA": (r, d), "dB": (d_i, r), "dWg": (d_i, d), "dWu": (d_i, d),
              "dWd": (d_i, d)}
    out = {n: torch.empty(shapes[n], **f32) for n in want}
    out["mask"] = torch.empty((T, max(d_i // max(bank, 1), 0)), dtype=torch.int64,
                              device=x.device)
    L = _capi.lib()
    if workspace is None:
        nbytes = int(L.sfn_backward_workspace_bytes(T, d, d_i, r, bank, k))
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=x.device)

    def ptr(n):
        return out[n].data_ptr() if n in out else None

    _capi.check(L.sfn_sparse_ffn_backward(
        x.data_ptr(), A.data_ptr(), B.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), Wd.data_ptr(),
        dy.data_ptr(), float(temperature), ptr("dx"), ptr("dA"), ptr("dB"), ptr("dWg"),
        ptr("dWu"), ptr("dWd"), out["mask"].data_ptr(), T, d, d_i, r, bank, k,
        workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _stream_ptr(stream, x.device)), "sfn_sparse_ffn_backward")
    return out


# ---------------------------------------------------------------- expert operators
SCORES = {"softmax": _capi.SFN_SCORE_SOFTMAX, "sigmoid": _capi.SFN_SCORE_SIGMOID}


# Few-token calls take a few microseconds on the GPU, about what the checks, the
# allocation of the outputs and the C call cost on the host: what is looked up
# per call is kept in tables.
_fns = {}
_elts = {}


def _arg(t, name, where, device, shape, dtype):
    """The pointer of a contiguous CUDA tensor on `device` of this shape and dtype."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.device == device and t.is_cuda
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _dev(t, name)
    if t.device != device:
        raise ValueError(f"{where}: {name} is on {t.device}, not on {device}")
    raise ValueError(f"{where}: {name} must be {list(shape)} of {dtype}, not "
                     f"{list(t.shape)} of {t.dtype}")


def _kind(dtype):
    elt = _elts.get(dtype)
    if elt is None:
        elt = _elts[dtype] = _elt(dtype)
    return elt


def _new(device, rows, cols, dtype):
    """A new [rows, cols] tensor (empty_strided: 1.5 us where empty takes 2.5)."""
    return _torch().empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _raw_stream(device):
    return _torch()._C._cuda_getCurrentRawStream(device.index)


def _on(stream, device, where):
    """`stream` as the current one: what a call allocates then belongs to it.
    (Memory from another stream's pool may still have work pending there.)"""
    if stream.device != device:
        raise ValueError(f"{where}: the stream is on {stream.device}, not on {device}")
    return _torch().cuda.stream(stream)


def _run(name, device, args):
    """One C call, its stream the last of `args`, with `device` current."""
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(_capi.lib(), name)
    torch = _torch()
    if torch._C._cuda_getDevice() == device.index:
        status = fn(*args)
    else:
        with torch.cuda.device(device):
            status = fn(*args)
    if status:
        _capi.check(status, name)


def _scratch(workspace, nbytes, device):
    if workspace is None:
        nbytes = max(nbytes, 1)
        workspace = _torch().empty_strided((nbytes,), (1,), dtype=_torch().uint8, device=device)
        return workspace.data_ptr(), nbytes, workspace
    _dev(workspace, "workspace")
    if workspace.device != device:
        raise ValueError(f"workspace is on {workspace.device}, not on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _score(score):
    kind = SCORES.get(score)
    if kind is None:
        raise ValueError(f"score must be one of {sorted(SCORES)}")
    return kind


def _matrix(t, name, where):
    try:
        shape = t.shape
        if len(shape) == 2 and t.is_cuda and t.is_contiguous():
            return shape
    except AttributeError:
        pass
    _dev(t, name)
    raise ValueError(f"{where}: {name} must have two dimensions")


def route_experts(logits, k: int, bias=None, score: str = "softmax", groups: int = 1,
                  top_groups: int = 1, group_top: int = 1, renormalize: bool = True,
                  scale: float = 1.0, experts=None, weights=None, scores=None,
                  want_scores: bool = False, stream=None):
    """Route tokens to experts (``sfn_route_experts`` in include/sfn.h).

    logits [T, E] float32 or bf16, bias float32 [E] or None.  Returns (experts
    int32 [T, k] in descending order of their selection scores, -1 for an empty
    slot; weights float32 [T, k]; scores float32 [T, E], or None unless
    ``scores`` or ``want_scores`` is given)."""
    torch = _torch()
    where = "route_experts"
    T, E = _matrix(logits, "logits", where)
    dev = logits.device
    if stream is not None:
        with _on(stream, dev, where):
            return route_experts(logits, k, bias, score, groups, top_groups, group_top, renormalize,
                                 scale, experts, weights, scores, want_scores)
    elt, kind, slots = _kind(logits.dtype), _score(score), k if k > 0 else 0
    bptr = None if bias is None else _arg(bias, "bias", where, dev, (E,), torch.float32)
    if experts is None:
        experts = _new(dev, T, slots, torch.int32)
        eptr = experts.data_ptr()
    else:
        eptr = _arg(experts, "experts", where, dev, (T, slots), torch.int32)
    if weights is None:
        weights = _new(dev, T, slots, torch.float32)
        wptr = weights.data_ptr()
    else:
        wptr = _arg(weights, "weights", where, dev, (T, slots), torch.float32)
    if scores is None and want_scores:
        scores = _new(dev, T, E, torch.float32)
    sptr = None if scores is None else _arg(scores, "scores", where, dev, (T, E),
                                            torch.float32)
    _run("sfn_route_experts", dev,
         (logits.data_ptr(), elt, bptr, eptr, wptr, sptr, T, E, k, kind, groups, top_groups,
          group_top, 1 if renormalize else 0, float(scale), _raw_stream(dev)))
    return experts, weights, scores


def route_experts_backward(logits, experts, dweights, dscores=None, score: str = "softmax",
                           renormalize: bool = True, scale: float = 1.0, dlogits=None,
                           stream=None):
    """Gradient of ``route_experts`` with respect to its logits, in their dtype,
    for dweights float32 [T, k] and, optionally, dscores float32 [T, E]."""
    torch = _torch()
    where = "route_experts_backward"
    T, E = _matrix(logits, "logits", where)
    dev = logits.device
    if stream is not None:
        with _on(stream, dev, where):
            return route_experts_backward(logits, experts, dweights, dscores, score, renormalize,
                                          scale, dlogits)
    elt, kind = _kind(logits.dtype), _score(score)
    k = _matrix(experts, "experts", where)[1]
    eptr = _arg(experts, "experts", where, dev, (T, k), torch.int32)
    wptr = _arg(dweights, "dweights", where, dev, (T, k), torch.float32)
    sptr = None if dscores is None else _arg(dscores, "dscores", where, dev, (T, E),
                                             torch.float32)
    if dlogits is None:
        dlogits = torch.empty_like(logits)
        lptr = dlogits.data_ptr()
    else:
        lptr = _arg(dlogits, "dlogits", where, dev, (T, E), logits.dtype)
    _run("sfn_route_experts_backward", dev,
         (logits.data_ptr(), elt, eptr, wptr, sptr, lptr, T, E, k, kind, 1 if renormalize else 0,
          float(scale), _raw_stream(dev)))
    return dlogits


def quantize_rows_i8(x, q=None, scale=None, stream=None):
    """8-bit quantisation of the rows of x (float32 or bf16, [..., K]; any
    leading dimensions, so that [E, N, K] weights go in one call).  Returns (q
    int8 [..., K], scale float32 [...])."""
    torch = _torch()
    where = "quantize_rows_i8"
    _dev(x, "x")
    if x.dim() < 1:
        raise ValueError(f"{where}: x must have a dimension")
    dev, lead, K = x.device, x.shape[:-1], x.shape[-1]
    if stream is not None:
        with _on(stream, dev, where):
            return quantize_rows_i8(x, q, scale)
    if q is None:
        q = torch.empty(x.shape, dtype=torch.int8, device=dev)
    if scale is None:
        scale = torch.empty(lead, dtype=torch.float32, device=dev)
    qptr = _arg(q, "q", where, dev, x.shape, torch.int8)
    sptr = _arg(scale, "scale", where, dev, lead, torch.float32)
    _run("sfn_quantize_rows_i8", dev, (x.data_ptr(), _kind(x.dtype), qptr, sptr, scale.numel(), K,
                                       _raw_stream(dev)))
    return q, scale


def matmul_i8(xq, x_scale, wq, w_scale, out=None, out_dtype=None, stream=None):
    """y[t][n] = x_scale[t] w_scale[n] sum_k xq[t][k] wq[n][k]: int8 xq [T, K]
    and wq [N, K], float32 scales [T] and [N].  y [T, N] in out_dtype (bf16
    unless given) or as ``out``."""
    torch = _torch()
    where = "matmul_i8"
    T, K = _matrix(xq, "xq", where)
    N = _matrix(wq, "wq", where)[0]
    dev = xq.device
    if stream is not None:
        with _on(stream, dev, where):
            return matmul_i8(xq, x_scale, wq, w_scale, out, out_dtype)
    if out is None:
        out = _new(dev, T, N, out_dtype or torch.bfloat16)
    ptrs = [_arg(xq, "xq", where, dev, (T, K), torch.int8),
            _arg(x_scale, "x_scale", where, dev, (T,), torch.float32),
            _arg(wq, "wq", where, dev, (N, K), torch.int8),
            _arg(w_scale, "w_scale", where, dev, (N,), torch.float32),
            _arg(out, "out", where, dev, (T, N), out_dtype or out.dtype)]
    _run("sfn_matmul_i8", dev, (*ptrs, _kind(out.dtype), T, N, K, _raw_stream(dev)))
    return out


@functools.lru_cache(maxsize=4096)
def linear_i8_workspace_bytes(T: int, K: int) -> int:
    return int(_capi.lib().sfn_linear_i8_workspace_bytes(T, K))


def linear_i8(x, wq, w_scale, out=None, out_dtype=None, workspace=None, stream=None):
    """x [T, K] (float32 or bf16), quantised row by row, times the int8 weight
    wq [N, K] with its scales [N].  y [T, N] in out_dtype (x's unless given) or
    as ``out``."""
    torch = _torch()
    where = "linear_i8"
    T, K = _matrix(x, "x", where)
    N = _matrix(wq, "wq", where)[0]
    dev = x.device
    if stream is not None:
        with _on(stream, dev, where):
            return linear_i8(x, wq, w_scale, out, out_dtype, workspace)
    wptr = _arg(wq, "wq", where, dev, (N, K), torch.int8)
    sptr = _arg(w_scale, "w_scale", where, dev, (N,), torch.float32)
    if out is None:
        out = _new(dev, T, N, out_dtype or x.dtype)
        yptr = out.data_ptr()
    else:
        yptr = _arg(out, "out", where, dev, (T, N), out_dtype or out.dtype)
    ws, nbytes, _keep = _scratch(workspace, linear_i8_workspace_bytes(T, K), dev)
    _run("sfn_linear_i8", dev, (x.data_ptr(), _kind(x.dtype), wptr, sptr, yptr, _kind(out.dtype), T,
                                N, K, ws, nbytes, _raw_stream(dev)))
    return out


@functools.lru_cache(maxsize=4096)
def experts_i8_workspace_bytes(T: int, E: int, k: int, d: int, f: int) -> int:
    return int(_capi.lib().sfn_experts_i8_workspace_bytes(T, E, k, d, f))


def experts_i8_forward(x, experts, weights, Wg, sg, Wu, su, Wd, sd, y=None, workspace=None,
                       stream=None):
    """y_t = sum_i weights[t][i] FFN_e(x_t), e = experts[t][i], with every
    product in 8-bit integers (``sfn_experts_i8_forward`` in include/sfn.h).

    x bf16 [T, d]; experts int32, weights float32 [T, k] from
    ``route_experts``; Wg, Wu int8 [E, f, d] with scales [E, f], Wd int8
    [E, d, f] with scales [E, d] from ``quantize_rows_i8``.  Returns y bf16
    [T, d]."""
    torch = _torch()
    where = "experts_i8_forward"
    T, d = _matrix(x, "x", where)
    _, k = _matrix(experts, "experts", where)
    dev = x.device
    if stream is not None:
        with _on(stream, dev, where):
            return experts_i8_forward(x, experts, weights, Wg, sg, Wu, su, Wd, sd, y, workspace)
    _dev(Wg, "Wg")
    if Wg.dim() != 3:
        raise ValueError(f"{where}: Wg must be [E, f, d]")
    E, f = Wg.shape[0], Wg.shape[1]
    if y is None:
        y = _new(dev, T, d, torch.bfloat16)
    i8, f32, bf16 = torch.int8, torch.float32, torch.bfloat16
    ptrs = [_arg(x, "x", where, dev, (T, d), bf16),
            _arg(experts, "experts", where, dev, (T, k), torch.int32),
            _arg(weights, "weights", where, dev, (T, k), f32),
            _arg(Wg, "Wg", where, dev, (E, f, d), i8), _arg(sg, "sg", where, dev, (E, f), f32),
            _arg(Wu, "Wu", where, dev, (E, f, d), i8), _arg(su, "su", where, dev, (E, f), f32),
            _arg(Wd, "Wd", where, dev, (E, d, f), i8), _arg(sd, "sd", where, dev, (E, d), f32),
            _arg(y, "y", where, dev, (T, d), bf16)]
    ws, nbytes, _keep = _scratch(workspace, experts_i8_workspace_bytes(T, E, k, d, f), dev)
    _run("sfn_experts_i8_forward", dev,
         (*ptrs, T, E, k, d, f, ws, nbytes, _raw_stream(dev)))
    return y
