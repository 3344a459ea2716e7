"""Thin PyTorch binding of the attention calls: softmax attention over all
pairs (``attn``) and the per-head norms with position rotation
(``qk_norm_rope``), forward, backward and as autograd functions.

Argument marshalling only, as in the FLARE binding: outputs and workspaces are
allocated with torch on the tensors' device, for the stream the call runs on,
and everything is computed in ``libflare.so``.
"""
from __future__ import annotations

import ctypes
import functools
import importlib
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._lib import FlareError

_f = importlib.import_module(__package__ + ".flare")


# the current stream's handle by device index (the short way where torch has it)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class _NoSwitch:
    """The tensors' device and the caller's stream are current already."""

    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_NO_SWITCH = _NoSwitch()


def _on(index: int, stream):
    """Makes the tensors' device, and ``stream`` when given, current: the
    call's buffers then belong to the stream that uses them."""
    if stream is not None:
        if stream.device.index != index:
            raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
        return torch.cuda.stream(stream)
    if torch.cuda.current_device() != index:
        return torch.cuda.device(index)
    return _NO_SWITCH


def _same(what: str, first, *ts) -> int:
    """Checks 4-D views with D contiguous, of one device and dtype; returns
    the device's index."""
    index, dtype = first.get_device(), first.dtype
    for t in (first, *ts):
        if t.get_device() != index or index < 0:
            raise ValueError(f"{what} tensors must live on one CUDA device")
        if t.dim() != 4 or t.stride(3) != 1:
            raise ValueError(f"{what} tensors must be [B,H,N,D] views with D contiguous")
        if t.dtype != dtype:
            raise ValueError(f"{what} tensors differ in dtype")
    return index


_ARRAYS = {n: ctypes.c_int64 * (3 * n) for n in (4, 6, 8)}


def _strides(*ts):
    """The flare_strides_t array of these tensors."""
    return _ARRAYS[len(ts)](*[s for t in ts for s in t.stride()[:3]])


def _shape(name: str, t, shape):
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")


def _output(name: str, t):
    """A caller's output: its history in autograd would be the old one's."""
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} needs a gradient, and this call records none")


# The library writes through raw pointers: autograd is told, so that a backward
# that saved an overwritten tensor reports it.
_written = torch.autograd.graph.increment_version


def _p(t):
    return None if t is None else t.data_ptr()


def _rows(name: str, t, shape, index: int):
    if t.dtype != torch.float32 or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor on the tensors' device")
    _shape(name, t, shape)


def _workspace(workspace, nbytes: int, like, where: str):
    if workspace is None:
        if nbytes == 0:
            raise FlareError(2, where)
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    if workspace.dtype != torch.uint8 or workspace.get_device() != like.get_device() \
            or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the tensors' device")
    return workspace


# ------------------------------------------------------------------ attention

@functools.lru_cache(maxsize=1024)
def _attn_bytes(backward: int, B, Hq, Hk, Nq, Nk, D, code: int, device: int) -> int:
    return int(_lib.load().flare_attn_workspace_size(backward, B, Hq, Hk, Nq, Nk, D, code))


def attn_workspace_size(backward: bool, B: int, Hq: int, Hk: int, Nq: int, Nk: int, D: int,
                        dtype: torch.dtype) -> int:
    """Workspace bytes of attn_fwd or attn_bwd on the current device (0:
    unsupported sizes)."""
    code = _lib.FLARE_F32 if dtype == torch.float32 else _lib.FLARE_BF16
    return int(_lib.load().flare_attn_workspace_size(int(bool(backward)), B, Hq, Hk, Nq, Nk, D,
                                                     code))


def attn_plan(backward: bool, B: int, Hq: int, Hk: int, Nq: int, Nk: int, D: int,
              dtype: torch.dtype, causal: bool = False):
    """How attn_fwd or attn_bwd cuts a call of these sizes on the current device
    (flare_attn_plan): (query tiles a CTA, heads a tile, parts of the keys), or
    (parts of dK and dV, parts of dQ, CTAs stay for several pieces)."""
    code = _lib.FLARE_F32 if dtype == torch.float32 else _lib.FLARE_BF16
    out = (ctypes.c_int64 * 3)()
    _lib.check(_lib.load().flare_attn_plan(int(bool(backward)), B, Hq, Hk, Nq, Nk, D, code,
                                           int(bool(causal)), out), "flare_attn_plan")
    return tuple(out)


def _attn_dims(q, k, v, *more):
    """The device's index and the sizes."""
    index = _same("attention", q, k, v, *more)
    B, Hq, Nq, D = q.shape
    _, Hk, Nk, _ = k.shape
    _shape("k", k, (B, Hk, Nk, D))
    _shape("v", v, k.shape)
    if Hk == 0 or Hq % Hk:
        raise ValueError(f"{Hq} query heads are not a multiple of {Hk} key heads")
    return index, B, Hq, Hk, Nq, Nk, D


def attn_fwd(q, k, v, scale: Optional[float] = None, *, causal: bool = False,
             q_lens: Optional[torch.Tensor] = None, k_lens: Optional[torch.Tensor] = None,
             save: bool = False, save_low: bool = False,
             workspace: Optional[torch.Tensor] = None,
             out: Optional[torch.Tensor] = None, stream=None):
    """Softmax attention softmax(scale q k^T) v.  Returns y, or (y, lse) when
    ``save`` (lse float32 [B,Hq,Nq], for attn_bwd), or (y, lse, y_low) when
    ``save_low``: y_low is what rounding y to bf16 left over (None in float32).

    q [B,Hq,Nq,D]; k, v [B,Hk,Nk,D] with Hq a multiple of Hk (the query heads
    of a key head are neighbours); D a multiple of 8 up to 128.  All may be
    any views with D contiguous and rows on 16-byte boundaries, k, v and q also
    expanded over batch or heads; y takes q's layout, or goes to ``out``, which
    must not overlap q, k or v.  ``q_lens``, ``k_lens`` (int32 [B] on the device):
    valid queries and keys; rows past them are never used and y is 0 there.
    ``causal``: query i sees keys j <= i + (keys - queries), counted with the
    lengths.  A query that sees no key gives 0; one that sees a logit of NaN or
    +inf gives NaN.  A length out of range is clamped; device_status(workspace)
    reports it to a caller who passes the workspace."""
    index, B, Hq, Hk, Nq, Nk, D = _attn_dims(q, k, v)
    code = _f._dtype_code(q)
    s = D ** -0.5 if scale is None else float(scale)
    if q_lens is not None:
        _f._seq_lens(q_lens, B, q.device)
    if k_lens is not None:
        _f._seq_lens(k_lens, B, q.device)
    with _on(index, stream):
        if out is None:
            y = torch.empty_like(q)
        else:
            y = out
            _same("attention", q, y)
            _shape("out", y, q.shape)
            _output("out", y)
        lse = low = None
        if save or save_low:
            lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
        if save_low and code == _lib.FLARE_BF16:
            # y's own strides, also where ``out`` is a slice of something larger
            low = torch.empty_like(y)
            if low.stride() != y.stride():
                raise ValueError("save_low takes an out without gaps")
        ws = _workspace(workspace, _attn_bytes(0, B, Hq, Hk, Nq, Nk, D, code, index), q,
                        "flare_attn_workspace_size")
        st = _lib.load().flare_attn_fwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), y.data_ptr(), _strides(q, k, v, y),
            _p(q_lens), _p(k_lens), B, Hq, Hk, Nq, Nk, D, code, s, 1 if causal else 0, _p(lse),
            _p(low), ws.data_ptr(), ws.numel(), _raw_stream(index))
    if st:
        _lib.check(st, "flare_attn_fwd")
    if out is not None:
        _written(out)
    if save_low:
        return y, lse, low
    return (y, lse) if save else y


def attn_bwd(q, k, v, y, dy, lse, scale: Optional[float] = None, *, causal: bool = False,
             q_lens: Optional[torch.Tensor] = None, k_lens: Optional[torch.Tensor] = None,
             need_dq: bool = True, need_dkv: bool = True, y_low: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients (dq, dk, dv) of attn_fwd for the upstream gradient dy, from
    its output y and lse (``save=True``); with ``y_low`` (``save_low=True``) the
    rounding of y does not enter the gradients.  ``need_dq`` / ``need_dkv``: what is
    not wanted is not computed and comes back as None."""
    index, B, Hq, Hk, Nq, Nk, D = _attn_dims(q, k, v, y, dy)
    _shape("y", y, q.shape)
    _shape("dy", dy, q.shape)
    _rows("lse", lse, (B, Hq, Nq), index)
    if y_low is not None:
        _same("attention", y, y_low)
        if y_low.shape != y.shape or y_low.stride() != y.stride():
            raise ValueError("y_low must be laid out as y")
    if not (need_dq or need_dkv):
        return None, None, None
    code = _f._dtype_code(q)
    s = D ** -0.5 if scale is None else float(scale)
    if q_lens is not None:
        _f._seq_lens(q_lens, B, q.device)
    if k_lens is not None:
        _f._seq_lens(k_lens, B, q.device)
    with _on(index, stream):
        dq = torch.empty_like(q) if need_dq else None
        dk = torch.empty_like(k) if need_dkv else None
        dv = torch.empty_like(v) if need_dkv else None
        ws = _workspace(workspace, _attn_bytes(1, B, Hq, Hk, Nq, Nk, D, code, index), q,
                        "flare_attn_workspace_size")
        strides = _strides(q, k, v, y, dy, dq if need_dq else q, dk if need_dkv else k,
                           dv if need_dkv else v)
        st = _lib.load().flare_attn_bwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), y.data_ptr(), _p(y_low), dy.data_ptr(),
            lse.data_ptr(), _p(dq), _p(dk), _p(dv), strides, _p(q_lens), _p(k_lens), B, Hq, Hk, Nq,
            Nk, D, code, s, 1 if causal else 0, ws.data_ptr(), ws.numel(), _raw_stream(index))
    if st:
        _lib.check(st, "flare_attn_bwd")
    return dq, dk, dv


# ---------------------------------------------------------- norms and rotation

@functools.lru_cache(maxsize=1024)
def _norm_bytes(B, Hq, Hk, N, D, code: int, device: int) -> int:
    return int(_lib.load().flare_qk_norm_rope_workspace_size(B, Hq, Hk, N, D, code))


def _norm_args(q, k, wq, wk, cos, sin, *more):
    """The device's index, sizes (B, Hq, Hk, N, D, R), the table's batch stride."""
    index = _same("query and key", q, k, *more)
    B, Hq, N, D = q.shape
    Hk = k.shape[1]
    _shape("k", k, (B, Hk, N, D))
    for name, w in (("wq", wq), ("wk", wk)):
        if w is not None:
            if w.dtype != q.dtype or w.get_device() != index or not w.is_contiguous():
                raise ValueError(
                    f"{name} must be a contiguous tensor of the heads' device and dtype")
            _shape(name, w, (D,))
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    if cos is None:
        return index, B, Hq, Hk, N, D, 0, 0
    half = cos.shape[-1]
    own = cos.dim() == 3
    shape = (B, N, half) if own else (N, half)
    _rows("cos", cos, shape, index)
    _rows("sin", sin, shape, index)
    if half == 0:
        raise ValueError("cos and sin are empty; leave them out for no rotation")
    return index, B, Hq, Hk, N, D, 2 * half, N * half if own else 0


def qk_norm_rope_fwd(q, k, wq=None, wk=None, cos=None, sin=None, *, eps: float = 1e-6,
                     interleaved: bool = False, out=None, stream=None):
    """Norm of every head of q [B,Hq,N,D] and k [B,Hk,N,D] and rotation by
    position in one pass: u = w x / sqrt(mean(x^2) + eps), then the first R
    elements of u turned in pairs by the token's angles.  Returns (qo, ko).

    wq, wk: [D] weights in the heads' dtype (None: ones).  cos, sin: float32
    [N, R/2], or [B, N, R/2] for positions of their own per batch element
    (None: no rotation); R a multiple of 16 up to D, which is a multiple of 8
    up to 128.  Pairs are (i, i + R/2), or (2i, 2i + 1) when ``interleaved``.
    q and k may be any views with D contiguous and rows on 16-byte boundaries;
    the outputs take their layout, or go to ``out`` = (qo, ko), which may be q and
    k themselves."""
    index, B, Hq, Hk, N, D, R, sb = _norm_args(q, k, wq, wk, cos, sin)
    code = _f._dtype_code(q)
    with _on(index, stream):
        if out is None:
            qo, ko = torch.empty_like(q), torch.empty_like(k)
        else:
            qo, ko = out
            _same("query and key", q, qo, ko)
            _shape("out[0]", qo, q.shape)
            _shape("out[1]", ko, k.shape)
            _output("out[0]", qo)
            _output("out[1]", ko)
        st = _lib.load().flare_qk_norm_rope_fwd(
            q.data_ptr(), k.data_ptr(), _p(wq), _p(wk), _p(cos), _p(sin), sb, qo.data_ptr(),
            ko.data_ptr(), _strides(q, k, qo, ko), B, Hq, Hk, N, D, R, 1 if interleaved else 0,
            code, eps, _raw_stream(index))
    if st:
        _lib.check(st, "flare_qk_norm_rope_fwd")
    if out is not None:
        _written((qo, ko))
    return qo, ko


def qk_norm_rope_bwd(q, k, wq, wk, cos, sin, dqo, dko, *, eps: float = 1e-6,
                     interleaved: bool = False, need_dw: bool = True,
                     workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients (dq, dk, dwq, dwk) of qk_norm_rope_fwd; dwq, dwk are None
    for weights that are None, or without ``need_dw``."""
    index, B, Hq, Hk, N, D, R, sb = _norm_args(q, k, wq, wk, cos, sin, dqo, dko)
    _shape("dqo", dqo, q.shape)
    _shape("dko", dko, k.shape)
    code = _f._dtype_code(q)
    with _on(index, stream):
        dq, dk = torch.empty_like(q), torch.empty_like(k)
        dwq = torch.empty_like(wq) if need_dw and wq is not None else None
        dwk = torch.empty_like(wk) if need_dw and wk is not None else None
        ws = _workspace(workspace, _norm_bytes(B, Hq, Hk, N, D, code, index), q,
                        "flare_qk_norm_rope_workspace_size")
        st = _lib.load().flare_qk_norm_rope_bwd(
            q.data_ptr(), k.data_ptr(), _p(wq), _p(wk), _p(cos), _p(sin), sb, dqo.data_ptr(),
            dko.data_ptr(), dq.data_ptr(), dk.data_ptr(), _p(dwq), _p(dwk),
            _strides(q, k, dqo, dko, dq, dk), B, Hq, Hk, N, D, R, 1 if interleaved else 0, code,
            eps, ws.data_ptr(), ws.numel(), _raw_stream(index))
    if st:
        _lib.check(st, "flare_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk


# -------------------------------------------------------------------- autograd

def _no_gradient(name: str, t):
    """Refuses an argument that the backward gives no gradient to."""
    if isinstance(t, torch.Tensor) and t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} gets no gradient; pass {name}.detach()")


def _grad_view(t: torch.Tensor) -> torch.Tensor:
    """An upstream gradient the library reads in place, else a contiguous copy."""
    if t.is_contiguous() and t.data_ptr() % 16 == 0:
        return t
    esz = t.element_size()
    ok = t.stride(-1) == 1 and t.data_ptr() % 16 == 0 and all(
        n == 1 or (s > 0 and (s * esz) % 16 == 0) for n, s in zip(t.shape[:3], t.stride()[:3]))
    # (contiguous() keeps a contiguous tensor, also where it is misaligned)
    return t if ok else t.clone(memory_format=torch.contiguous_format)


def _once(backward):
    """A backward that cannot be differentiated again.  Where no graph is
    built of it (the ordinary case) it runs without the wrapper's cost."""
    guarded = once_differentiable(backward)

    @functools.wraps(backward)
    def run(ctx, *grads):
        return guarded(ctx, *grads) if torch.is_grad_enabled() else backward(ctx, *grads)
    return run


class AttnFunction(torch.autograd.Function):
    """y = softmax attention (see attn_fwd); saves y and the row statistics,
    the backward recomputes the probabilities."""

    @staticmethod
    def forward(ctx, q, k, v, scale, causal, q_lens, k_lens):
        if not any(ctx.needs_input_grad):
            return attn_fwd(q, k, v, scale, causal=causal, q_lens=q_lens, k_lens=k_lens)
        y, lse, low = attn_fwd(q, k, v, scale, causal=causal, q_lens=q_lens, k_lens=k_lens,
                               save_low=True)
        ctx.save_for_backward(q, k, v, y, lse, low, q_lens, k_lens)
        ctx.scale, ctx.causal = scale, causal
        return y

    @staticmethod
    @_once
    def backward(ctx, dy):
        q, k, v, y, lse, low, q_lens, k_lens = ctx.saved_tensors
        need = ctx.needs_input_grad
        dq, dk, dv = attn_bwd(q, k, v, y, _grad_view(dy), lse, ctx.scale, causal=ctx.causal,
                              q_lens=q_lens, k_lens=k_lens, need_dq=need[0],
                              need_dkv=need[1] or need[2], y_low=low)
        return dq, dk, dv, None, None, None, None


class QkNormRopeFunction(torch.autograd.Function):
    """(qo, ko) = norms and rotation (see qk_norm_rope_fwd)."""

    @staticmethod
    def forward(ctx, q, k, wq, wk, cos, sin, eps, interleaved):
        ctx.save_for_backward(q, k, wq, wk, cos, sin)
        ctx.eps, ctx.interleaved = eps, interleaved
        return qk_norm_rope_fwd(q, k, wq, wk, cos, sin, eps=eps, interleaved=interleaved)

    @staticmethod
    @_once
    def backward(ctx, dqo, dko):
        q, k, wq, wk, cos, sin = ctx.saved_tensors
        need = ctx.needs_input_grad
        grads = qk_norm_rope_bwd(q, k, wq, wk, cos, sin, _grad_view(dqo), _grad_view(dko),
                                 eps=ctx.eps, interleaved=ctx.interleaved,
                                 need_dw=need[2] or need[3])
        return (*grads, None, None, None, None)


def attn(q, k, v, scale: Optional[float] = None, *, causal: bool = False,
         q_lens: Optional[torch.Tensor] = None,
         k_lens: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Softmax attention with autograd (arguments as attn_fwd).  Gradients go
    to q, k and v: a scale that needs one is refused.  Kept for the backward: q,
    k, v, y, lse, and in bf16 what rounding y left over, one more tensor of y's
    size, which takes the gradients' error from 0.0026 - 0.0028 to 0.0024;
    attn_fwd(save=True) and attn_bwd do without it, and take a workspace."""
    _no_gradient("scale", scale)
    if not torch.is_grad_enabled():   # a Function would not know, and save for a backward
        return attn_fwd(q, k, v, scale, causal=causal, q_lens=q_lens, k_lens=k_lens)
    return AttnFunction.apply(q, k, v, scale, causal, q_lens, k_lens)


def qk_norm_rope(q, k, wq=None, wk=None, cos=None, sin=None, *, eps: float = 1e-6,
                 interleaved: bool = False):
    """Per-head norms and position rotation with autograd (arguments as
    qk_norm_rope_fwd); returns (qo, ko).  Gradients go to q, k, wq and wk: cos
    and sin that need one are refused."""
    _no_gradient("cos", cos)
    _no_gradient("sin", sin)
    return QkNormRopeFunction.apply(q, k, wq, wk, cos, sin, eps, interleaved)
