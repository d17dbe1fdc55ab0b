"""Torch-facing wrappers of the operators around the NVFP4 linear layers in a transformer block's
training step: layer norm, attention and AdamW (include/nvfp4.h has their formulas).

As in :mod:`.api`, the functions only check and marshal arguments, launch on
``torch.cuda.current_stream()`` and raise :class:`NVFP4Error` for argument errors before anything is
launched; device-side errors land in the status word read by ``status_query``."""
from __future__ import annotations

import ctypes
from typing import Dict, List, Optional, Sequence, Tuple, Union

import torch

from . import _lib as L
from ._lib import NVFP4Error
from .api import _DT, _check_2d, _ptr, _stream, _workspace, dev_status


def _invalid(what: str) -> NVFP4Error:
    return NVFP4Error(L.ERR_INVALID_ARG, what)


def _on_current_device(t: torch.Tensor, name: str) -> None:
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise _invalid(f"{name} must be a tensor on the current CUDA device")


def _rows(t: torch.Tensor, name: str, shape, dtype) -> int:
    """Row pitch of a [rows, cols] operand that has to match ``shape`` and ``dtype``."""
    _check_2d(t, name)
    _on_current_device(t, name)
    if t.dtype != dtype:
        raise _invalid(f"{name} must be {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise NVFP4Error(L.ERR_SHAPE, f"{name} must be {list(shape)}")
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _vector(t: torch.Tensor, name: str, n: int, dtypes) -> None:
    _on_current_device(t, name)
    if t.dtype not in dtypes:
        raise _invalid(f"{name} must be one of {[str(d) for d in dtypes]}")
    if t.dim() != 1 or t.shape[0] != n:
        raise NVFP4Error(L.ERR_SHAPE, f"{name} must be [{n}]")
    if n > 1 and t.stride(0) != 1:
        raise _invalid(f"{name} must be contiguous")


# ----------------------------------------------------------------------------- layer norm

def layer_norm_forward(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
                       residual: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                       ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Layer norm of the rows of x [rows, cols], or of h = x + residual (rounded to x's type).
    x: float32 / bfloat16 with unit column stride; weight, bias: [cols], one type; the result is
    of ``out_dtype`` (x's type by default).  Returns (y, mean, rstd, h), h being x itself without
    a residual: mean, rstd and h are what :func:`layer_norm_backward` needs."""
    _check_2d(x, "x")
    R, C = x.shape
    if C < 1:
        raise NVFP4Error(L.ERR_SHAPE, "x has no columns")
    ldx = _rows(x, "x", (R, C), x.dtype)
    _vector(weight, "weight", C, tuple(_DT))
    if bias is not None:
        _vector(bias, "bias", C, (weight.dtype,))
    out_dtype = x.dtype if out_dtype is None else out_dtype
    if out_dtype not in _DT:
        raise _invalid("out_dtype must be float32 or bfloat16")
    h, ldr = None, 0
    if residual is not None:
        ldr = _rows(residual, "residual", (R, C), x.dtype)
        h = torch.empty((R, C), dtype=x.dtype, device=x.device)
    y = torch.empty((R, C), dtype=out_dtype, device=x.device)
    mean = torch.empty(R, dtype=torch.float32, device=x.device)
    rstd = torch.empty(R, dtype=torch.float32, device=x.device)
    st = L.lib().nvfp4_layer_norm_forward(_ptr(x), _DT[x.dtype], R, C, ldx, _ptr(residual), ldr, _ptr(weight),
                                          _ptr(bias), _DT[weight.dtype], eps, _ptr(y), _DT[out_dtype], C, _ptr(h), C,
                                          _ptr(mean), _ptr(rstd), _stream())
    L.check(st, "nvfp4_layer_norm_forward")
    return y, mean, rstd, x if h is None else h


def layer_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor,
                        rstd: torch.Tensor, dh: Optional[torch.Tensor] = None, bias: bool = True,
                        ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """Gradients of :func:`layer_norm_forward`: (dx, dweight, dbias), dx in h's type, the vectors in
    float32, dbias None unless ``bias``.  ``dh`` (h's type) is the gradient that reaches h along
    the residual path; it is added to dx, which then is the gradient of x and of the residual."""
    _check_2d(h, "h")
    R, C = h.shape
    if C < 1:
        raise NVFP4Error(L.ERR_SHAPE, "h has no columns")
    ldx = _rows(h, "h", (R, C), h.dtype)
    _check_2d(dy, "dy")
    lddy = _rows(dy, "dy", (R, C), dy.dtype)
    lddh = 0 if dh is None else _rows(dh, "dh", (R, C), h.dtype)
    _vector(weight, "weight", C, tuple(_DT))
    _vector(mean, "mean", R, (torch.float32,))
    _vector(rstd, "rstd", R, (torch.float32,))
    dx = torch.empty((R, C), dtype=h.dtype, device=h.device)
    dw = torch.empty(C, dtype=torch.float32, device=h.device)
    db = torch.empty(C, dtype=torch.float32, device=h.device) if bias else None
    lib = L.lib()
    ws = _workspace(int(lib.nvfp4_layer_norm_backward_workspace_bytes(R, C)))
    st = lib.nvfp4_layer_norm_backward(_ptr(dy), _DT[dy.dtype], lddy, _ptr(h), _DT[h.dtype], R, C, ldx, _ptr(weight),
                                       _DT[weight.dtype], _ptr(mean), _ptr(rstd), _ptr(dh), lddh, _ptr(dx), C,
                                       _ptr(dw), _ptr(db), ws.data_ptr(), ws.numel(), _stream())
    L.check(st, "nvfp4_layer_norm_backward")
    return dx, dw, db


# ----------------------------------------------------------------------------- attention

def _heads(t: torch.Tensor, name: str, tokens: Optional[int] = None, heads: Optional[int] = None,
           dim: Optional[int] = None) -> L.HeadsC:
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise NVFP4Error(L.ERR_SHAPE, f"{name} must be [tokens, heads, dim]")
    _on_current_device(t, name)
    if t.dtype != torch.bfloat16:
        raise NVFP4Error(L.ERR_UNSUPPORTED, f"{name} must be bfloat16")
    T, H, D = t.shape
    if (tokens is not None and T != tokens) or (heads is not None and H != heads) or (dim is not None and D != dim):
        raise NVFP4Error(L.ERR_SHAPE, f"{name} is {list(t.shape)}, expected {[tokens, heads, dim]}")
    if D > 1 and t.stride(2) != 1:
        raise _invalid(f"{name} must be contiguous along dim")
    return L.HeadsC(t.data_ptr() if T else None, t.stride(0), t.stride(1))


def _attention_shape(q, k, causal, scale, cu_q, cu_k) -> L.AttentionShapeC:
    if q.dim() != 3 or k.dim() != 3:
        raise NVFP4Error(L.ERR_SHAPE, "q and k must be [tokens, heads, dim]")
    if (cu_q is None) and (cu_k is not None):
        raise _invalid("cu_k needs cu_q")
    cu_k = cu_q if cu_k is None else cu_k
    nseq = 1
    for cu, name in ((cu_q, "cu_q"), (cu_k, "cu_k")):
        if cu is None:
            continue
        _on_current_device(cu, name)
        if cu.dtype != torch.int32 or cu.dim() != 1 or not cu.is_contiguous() or cu.shape[0] < 2:
            raise _invalid(f"{name} must be a contiguous int32 vector of at least two offsets")
        if cu.shape != cu_q.shape:
            raise NVFP4Error(L.ERR_SHAPE, "cu_q and cu_k differ in length")
        nseq = cu.shape[0] - 1
    scale = q.shape[2] ** -0.5 if scale is None else float(scale)
    return L.AttentionShapeC(q.shape[0], k.shape[0], q.shape[1], k.shape[1], q.shape[2], int(bool(causal)), scale, nseq,
                             _ptr(cu_q), _ptr(cu_k))


def attention_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
                      scale: Optional[float] = None, cu_q: Optional[torch.Tensor] = None,
                      cu_k: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                      ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of q [tq, heads, dim] over k, v [tk, kv_heads, dim] (bfloat16, dim a multiple of 8
    up to 128, the last axis contiguous, the other strides multiples of 8): slices of one fused
    projection's output need no copy.  ``cu_q`` / ``cu_k``: int32 offsets [sequences + 1] of packed
    sequences (``cu_k`` defaults to ``cu_q``); None: one sequence.  ``causal`` masks are aligned at
    the sequences' ends.  ``scale`` defaults to dim ** -0.5.  Returns (out [tq, heads, dim], lse
    [heads, tq] float32); a query that sees no key gets 0 and -inf."""
    shape = _attention_shape(q, k, causal, scale, cu_q, cu_k)
    T, H, D = q.shape
    if out is None:
        out = torch.empty((T, H, D), dtype=torch.bfloat16, device=q.device)
    args = [_heads(q, "q"), _heads(k, "k", dim=D), _heads(v, "v", k.shape[0], k.shape[1], D), _heads(out, "out", T, H, D)]
    lse = torch.empty((H, T), dtype=torch.float32, device=q.device)
    st = L.lib().nvfp4_attention_forward(ctypes.byref(shape), *(ctypes.byref(a) for a in args), _ptr(lse),
                                         dev_status(q.device).data_ptr(), _stream())
    L.check(st, "nvfp4_attention_forward")
    return out, lse


def attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                       lse: torch.Tensor, causal: bool = False, scale: Optional[float] = None,
                       cu_q: Optional[torch.Tensor] = None, cu_k: Optional[torch.Tensor] = None,
                       dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                       dv: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients (dq, dk, dv) of :func:`attention_forward`, the probabilities recomputed from q, k and
    lse.  dq, dk, dv may be given as strided views, such as the slices of one buffer that is the
    fused projection's dY.  Deterministic."""
    shape = _attention_shape(q, k, causal, scale, cu_q, cu_k)
    T, H, D = q.shape
    S, G = k.shape[0], k.shape[1]
    dq = torch.empty((T, H, D), dtype=torch.bfloat16, device=q.device) if dq is None else dq
    dk = torch.empty((S, G, D), dtype=torch.bfloat16, device=q.device) if dk is None else dk
    dv = torch.empty((S, G, D), dtype=torch.bfloat16, device=q.device) if dv is None else dv
    ins = [_heads(dout, "dout", T, H, D), _heads(q, "q"), _heads(k, "k", dim=D), _heads(v, "v", S, G, D),
           _heads(out, "out", T, H, D)]
    outs = [_heads(dq, "dq", T, H, D), _heads(dk, "dk", S, G, D), _heads(dv, "dv", S, G, D)]
    _on_current_device(lse, "lse")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (H, T) or not lse.is_contiguous():
        raise _invalid(f"lse must be contiguous float32 [{H}, {T}]")
    lib = L.lib()
    ws = _workspace(int(lib.nvfp4_attention_backward_workspace_bytes(ctypes.byref(shape))))
    st = lib.nvfp4_attention_backward(ctypes.byref(shape), *(ctypes.byref(a) for a in ins), _ptr(lse),
                                      *(ctypes.byref(a) for a in outs), ws.data_ptr(), ws.numel(),
                                      dev_status(q.device).data_ptr(), _stream())
    L.check(st, "nvfp4_attention_backward")
    return dq, dk, dv


# ----------------------------------------------------------------------------- AdamW

STATE_BLOCK = 128                       # elements of an 8-bit state with one scale


class AdamW:
    """AdamW over a list of parameters (float32 / bfloat16, contiguous, CUDA), updated in place by
    :meth:`step`, one launch for many tensors.

    ``bits=32`` keeps the moments ``m`` and ``v`` in float32.  ``bits=8`` keeps E4M3 codes of them
    (torch.float8_e4m3fn) with a float32 scale per 128 elements (``m_scale``, ``v_scale``; value =
    code * scale): meant for beta2 up to about 0.99, where the spread that stochastic rounding gives
    v stays below two fifths of v.  ``state`` takes such lists over from elsewhere (a checkpoint) and
    ``steps`` how many steps they have seen; the object's lists are what a checkpoint stores.
    ``weight_decay`` is one number or one per parameter."""

    def __init__(self, params: Sequence[torch.Tensor], bits: int = 32,
                 weight_decay: Union[float, Sequence[float]] = 0.1,
                 state: Optional[Dict[str, List[torch.Tensor]]] = None, steps: int = 0):
        if bits not in (8, 32):
            raise _invalid("bits must be 8 or 32")
        if steps < 0:
            raise _invalid("steps must not be negative")
        self.params, self.bits, self.steps = list(params), bits, int(steps)
        n = len(self.params)
        decay = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else [float(d) for d in weight_decay]
        if len(decay) != n:
            raise NVFP4Error(L.ERR_SHAPE, "weight_decay must be one number or one per parameter")
        for i, p in enumerate(self.params):
            _on_current_device(p, f"params[{i}]")
            if p.dtype not in _DT or not p.is_contiguous():
                raise _invalid(f"params[{i}] must be contiguous float32 or bfloat16")
        if self.params and any(p.device != self.params[0].device for p in self.params):
            raise _invalid("params must be on one device")
        names = ("m", "v") if bits == 32 else ("m", "v", "m_scale", "v_scale")
        if state is not None and (set(state) != set(names) or any(len(state[k]) != n for k in names)):
            raise NVFP4Error(L.ERR_SHAPE, f"state must hold lists of {n} tensors named {names}")
        self.state: Dict[str, List[torch.Tensor]] = {}
        for k in names:
            blocks, dtype = k.endswith("_scale"), torch.float32
            if bits == 8 and not blocks:
                dtype = torch.float8_e4m3fn
            if state is None:
                self.state[k] = [torch.zeros((p.numel() + STATE_BLOCK - 1) // STATE_BLOCK if blocks else p.shape,
                                             dtype=dtype, device=p.device) for p in self.params]
                continue
            self.state[k] = list(state[k])
            for i, (s, p) in enumerate(zip(self.state[k], self.params)):
                want = (p.numel() + STATE_BLOCK - 1) // STATE_BLOCK if blocks else p.numel()
                if s.device != p.device or s.dtype != dtype or s.numel() != want or not s.is_contiguous():
                    raise _invalid(f"state[{k!r}][{i}] must be contiguous {dtype} of {want} elements beside its parameter")
        self._kept = [list(self.params)] + [list(v) for v in self.state.values()]   # what the pointers below point to
        self._shapes = [p.shape for p in self.params]
        self._ptrs = [p.data_ptr() for p in self.params]
        self._tensors = (L.AdamWTensorC * max(n, 1))()
        for i, (p, d) in enumerate(zip(self.params, decay)):
            self._tensors[i] = L.AdamWTensorC(
                p.data_ptr(), None, self.state["m"][i].data_ptr(), self.state["v"][i].data_ptr(),
                self.state["m_scale"][i].data_ptr() if bits == 8 else None,
                self.state["v_scale"][i].data_ptr() if bits == 8 else None, p.numel(), _DT[p.dtype], 0, d, i)

    def step(self, grads: Sequence[Optional[torch.Tensor]], lr: float, betas: Tuple[float, float] = (0.9, 0.95),
             eps: float = 1e-8, grad_scale: Optional[torch.Tensor] = None, round: int = L.SR, sr_seed: int = 0) -> None:
        """One update.  ``grads``: one per parameter, of its shape, contiguous, float32 or bfloat16
        (None leaves that parameter and its state alone).  ``grad_scale``: a one-element float32 CUDA tensor
        that multiplies every gradient (loss scale, clipping) without a host read.  ``round`` (RNE
        or SR with ``sr_seed``) is how 8-bit states and bfloat16 parameters are rounded."""
        if len(grads) != len(self.params):
            raise NVFP4Error(L.ERR_SHAPE, f"{len(grads)} gradients for {len(self.params)} parameters")
        if not self.params:
            return
        dev = self.params[0].device
        if torch.cuda.current_device() != dev.index:
            raise _invalid("the parameters are not on the current CUDA device")
        if grad_scale is not None and (grad_scale.device != dev or grad_scale.dtype != torch.float32
                                       or grad_scale.numel() != 1):
            raise _invalid("grad_scale must be one float32 on the parameters' device")
        for i, (g, p, ptr, t, shape) in enumerate(zip(grads, self._kept[0], self._ptrs, self._tensors, self._shapes)):
            if p.data_ptr() != ptr:
                raise _invalid(f"params[{i}] has other storage than when the optimizer was made")
            if g is None:
                t.grad = None
                continue
            if g.shape != shape or g.dtype not in _DT or g.device != dev or not g.is_contiguous():
                raise _invalid(f"grads[{i}] must be contiguous float32 or bfloat16 {list(shape)} beside its parameter")
            t.grad, t.grad_dtype = g.data_ptr(), _DT[g.dtype]
        hp = L.AdamWParams(self.bits, round, self.steps + 1, lr, betas[0], betas[1], eps, sr_seed & (2**64 - 1))
        st = L.lib().nvfp4_adamw_step(self._tensors, len(self.params), ctypes.byref(hp), _ptr(grad_scale),
                                      dev_status(dev).data_ptr(), _stream())
        L.check(st, "nvfp4_adamw_step")
        self.steps += 1
