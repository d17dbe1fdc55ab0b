"""Torch-facing wrappers of the operators around the NVFP4 linear layers in a transformer block's
training step: layer norm, attention and AdamW (include/nvfp4.h has their formulas).

As in :mod:`.api`, the functions only check and marshal arguments, launch on
``torch.cuda.current_stream()`` and raise :class:`NVFP4Error` for argument errors before anything is
launched; device-side errors land in the status word read by ``status_query``."""
from __future__ import annotations

import ctypes
import functools
import itertools
import struct
import threading
from array import array
from typing import Dict, List, Optional, Sequence, Tuple, Union

import torch

from . import _lib as L
from ._lib import NVFP4Error
from . import api
from .api import _DT, _check_2d, _ptr, _workspace, dev_status


def _invalid(what: str) -> NVFP4Error:
    return NVFP4Error(L.ERR_INVALID_ARG, what)


# The calls here are short; what a wrapper costs on the host shows.  So arguments are compared against what they
# have to be in one go, and looked at one by one only when something is wrong.

def _here(dev: int) -> int:
    """The current stream of device ``dev``, which has to be the current device."""
    if dev != torch.cuda.current_device():
        raise _invalid("the tensors must be on the current CUDA device")
    return torch._C._cuda_getCurrentRawStream(dev)


def _on(t: torch.Tensor, name: str, dev: int) -> None:
    if not t.is_cuda or t.get_device() != dev:
        raise _invalid(f"{name} must be on CUDA device {dev}")


def _matrix(t: torch.Tensor, name: str, shape, dtype, dev: int) -> int:
    """Row pitch of a [rows, cols] operand of ``shape``, ``dtype`` and device ``dev``."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        _check_2d(t, name)
        _on(t, name, dev)
        if t.dtype != dtype:
            raise _invalid(f"{name} must be {dtype}")
        raise NVFP4Error(L.ERR_SHAPE, f"{name} must be {list(shape)}")
    pitch, unit = t.stride()
    if unit != 1 and shape[1] > 1:
        raise _invalid(f"{name} must have unit column stride")
    return pitch if shape[0] > 1 else max(shape[1], 1)


def _vector(t: torch.Tensor, name: str, n: int, dtypes, dev: int) -> int:
    """Address of a contiguous [n] operand."""
    if t.dtype not in dtypes:
        raise _invalid(f"{name} must be one of {[str(d) for d in dtypes]}")
    if t.dim() != 1 or t.shape[0] != n:
        raise NVFP4Error(L.ERR_SHAPE, f"{name} must be [{n}]")
    if not t.is_contiguous():
        raise _invalid(f"{name} must be contiguous")
    if t.get_device() != dev:
        _on(t, name, dev)
    return t.data_ptr()


def _status_ptr(dev: int) -> int:
    t = api._status.get(dev)
    return (dev_status(dev) if t is None else t).data_ptr()


_F32_ONLY = (torch.float32,)


# ----------------------------------------------------------------------------- layer norm

def layer_norm_forward(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
                       residual: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                       ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Layer norm of the rows of x [rows, cols], or of h = x + residual (rounded to x's type).
    x: float32 / bfloat16 with unit column stride; weight, bias: [cols], one type; the result is
    of ``out_dtype`` (x's type by default).  Returns (y, mean, rstd, h), h being x itself without
    a residual: mean, rstd and h are what :func:`layer_norm_backward` needs."""
    dtype, dev = x.dtype, x.get_device()
    if dtype not in _DT or x.dim() != 2 or dev < 0:
        _check_2d(x, "x")
    R, C = shape = x.shape
    if C < 1:
        raise NVFP4Error(L.ERR_SHAPE, "x has no columns")
    ldx = _matrix(x, "x", shape, dtype, dev)
    w = _vector(weight, "weight", C, _DT, dev)
    b = None if bias is None else _vector(bias, "bias", C, (weight.dtype,), dev)
    out_dtype = dtype if out_dtype is None else out_dtype
    if out_dtype not in _DT:
        raise _invalid("out_dtype must be float32 or bfloat16")
    stream = _here(dev)
    h, ldr = None, 0
    if residual is not None:
        ldr = _matrix(residual, "residual", shape, dtype, dev)
        h = torch.empty(shape, dtype=dtype, device=x.device)
    y = torch.empty(shape, dtype=out_dtype, device=x.device)
    mean = torch.empty(R, dtype=torch.float32, device=x.device)
    rstd = torch.empty(R, dtype=torch.float32, device=x.device)
    st = L.lib().nvfp4_layer_norm_forward(x.data_ptr(), _DT[dtype], R, C, ldx, _ptr(residual), ldr, w, b, _DT[weight.dtype],
                                          eps, y.data_ptr(), _DT[out_dtype], C, _ptr(h), C, mean.data_ptr(),
                                          rstd.data_ptr(), stream)
    if st:
        L.check(st, "nvfp4_layer_norm_forward")
    return y, mean, rstd, x if h is None else h


def layer_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor,
                        rstd: torch.Tensor, dh: Optional[torch.Tensor] = None, bias: bool = True,
                        ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """Gradients of :func:`layer_norm_forward`: (dx, dweight, dbias), dx in h's type, the vectors in
    float32, dbias None unless ``bias``.  ``dh`` (h's type) is the gradient that reaches h along
    the residual path; it is added to dx, which then is the gradient of x and of the residual."""
    dtype, dev = h.dtype, h.get_device()
    if dtype not in _DT or h.dim() != 2 or dev < 0:
        _check_2d(h, "h")
    R, C = shape = h.shape
    if C < 1:
        raise NVFP4Error(L.ERR_SHAPE, "h has no columns")
    if dy.dtype not in _DT:
        raise _invalid("dy must be float32 or bfloat16")
    ldx, lddy = _matrix(h, "h", shape, dtype, dev), _matrix(dy, "dy", shape, dy.dtype, dev)
    lddh = 0 if dh is None else _matrix(dh, "dh", shape, dtype, dev)
    w = _vector(weight, "weight", C, _DT, dev)
    m, s = _vector(mean, "mean", R, _F32_ONLY, dev), _vector(rstd, "rstd", R, _F32_ONLY, dev)
    stream = _here(dev)
    dx = torch.empty(shape, dtype=dtype, device=h.device)
    dw = torch.empty(C, dtype=torch.float32, device=h.device)
    db = torch.empty(C, dtype=torch.float32, device=h.device) if bias else None
    lib = L.lib()
    ws = _workspace(_norm_workspace(dev, R, C), (dev, stream))
    st = lib.nvfp4_layer_norm_backward(dy.data_ptr(), _DT[dy.dtype], lddy, h.data_ptr(), _DT[dtype], R, C, ldx, w,
                                       _DT[weight.dtype], m, s, _ptr(dh), lddh, dx.data_ptr(), C, dw.data_ptr(), _ptr(db),
                                       ws.data_ptr(), ws.numel(), stream)
    if st:
        L.check(st, "nvfp4_layer_norm_backward")
    return dx, dw, db


# ----------------------------------------------------------------------------- attention

# A call's descriptors (AttentionShapeC, then a HeadsC for each tensor) are packed in one go into memory of the calling
# thread; the library has read them when it returns.
_SHAPE, _SHAPE_BYTES, _HEADS_BYTES = "qqiiiifiPP", ctypes.sizeof(L.AttentionShapeC), ctypes.sizeof(L.HeadsC)
_PACK = {n: struct.Struct(_SHAPE + "Pqq" * n) for n in (4, 8)}
assert all(s.size == _SHAPE_BYTES + n * _HEADS_BYTES for n, s in _PACK.items())


class _Descriptors(threading.local):
    def __init__(self):
        self.memory = ctypes.create_string_buffer(_PACK[8].size)
        shape = ctypes.addressof(self.memory)
        self.at = [shape] + [shape + _SHAPE_BYTES + i * _HEADS_BYTES for i in range(8)]

    def pack(self, n: int, *fields) -> List[int]:
        """Addresses of the shape and of n tensors' descriptors."""
        try:
            _PACK[n].pack_into(self.memory, 0, *fields)
        except (struct.error, OverflowError) as e:
            raise _invalid(f"attention: {e}")
        return self.at


_descriptors = _Descriptors()


def _heads(t: torch.Tensor, name: str, shape, dev: int) -> Tuple[int, int, int]:
    """The fields of a HeadsC."""
    if t.shape != shape or t.dtype is not torch.bfloat16 or t.get_device() != dev:
        if t.dim() != 3:
            raise NVFP4Error(L.ERR_SHAPE, f"{name} must be [tokens, heads, dim]")
        _on(t, name, dev)
        if t.dtype != torch.bfloat16:
            raise NVFP4Error(L.ERR_UNSUPPORTED, f"{name} must be bfloat16")
        raise NVFP4Error(L.ERR_SHAPE, f"{name} is {list(t.shape)}, expected {list(shape)}")
    tokens, heads, unit = t.stride()
    if unit != 1 and shape[2] > 1:
        raise _invalid(f"{name} must be contiguous along dim")
    return t.data_ptr(), tokens, heads


# What the C entries return for a workspace depends on these alone.
@functools.lru_cache(maxsize=256)
def _attention_workspace(back: bool, dev: int, tq: int, tk: int, heads: int, kv_heads: int, dim: int, nseq: int) -> int:
    lib = L.lib()
    cu = None if nseq == 1 else 4                          # not read
    shape = ctypes.byref(L.AttentionShapeC(tq, tk, heads, kv_heads, dim, False, 1.0, nseq, cu, cu))
    return (lib.nvfp4_attention_backward_workspace_bytes if back else lib.nvfp4_attention_forward_workspace_bytes)(shape)


@functools.lru_cache(maxsize=256)
def _norm_workspace(dev: int, rows: int, cols: int) -> int:
    return L.lib().nvfp4_layer_norm_backward_workspace_bytes(rows, cols)


def _attention_shape(q, k, causal, scale, cu_q, cu_k, dev) -> Tuple:
    """The fields of an AttentionShapeC."""
    if q.dim() != 3 or k.dim() != 3:
        raise NVFP4Error(L.ERR_SHAPE, "q and k must be [tokens, heads, dim]")
    nseq = 1
    if cu_q is None:
        if cu_k is not None:
            raise _invalid("cu_k needs cu_q")
    else:
        cu_k = cu_q if cu_k is None else cu_k
        for cu, name in ((cu_q, "cu_q"), (cu_k, "cu_k")):
            if cu.dtype != torch.int32 or cu.dim() != 1 or not cu.is_contiguous() or cu.shape[0] < 2:
                raise _invalid(f"{name} must be a contiguous int32 vector of at least two offsets")
            _on(cu, name, dev)
        if cu_k.shape != cu_q.shape:
            raise NVFP4Error(L.ERR_SHAPE, "cu_q and cu_k differ in length")
        nseq = cu_q.shape[0] - 1
    T, H, D = q.shape
    if D < 1:
        raise NVFP4Error(L.ERR_SHAPE, "q has no elements along dim")
    return (T, k.shape[0], H, k.shape[1], D, bool(causal), D ** -0.5 if scale is None else scale, nseq,
            0 if cu_q is None else cu_q.data_ptr(), 0 if cu_k is None else cu_k.data_ptr())


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
    dev = q.get_device()
    shape = _attention_shape(q, k, causal, scale, cu_q, cu_k, dev)
    T, H, D = qs = q.shape
    ks = (k.shape[0], k.shape[1], D)
    a, b, c = _heads(q, "q", qs, dev), _heads(k, "k", ks, dev), _heads(v, "v", ks, dev)
    stream = _here(dev)
    if out is None:
        out = torch.empty(qs, dtype=torch.bfloat16, device=q.device)
    d = _heads(out, "out", qs, dev)
    lse = torch.empty((H, T), dtype=torch.float32, device=q.device)
    ws = _workspace(_attention_workspace(False, dev, T, ks[0], H, ks[1], D, shape[7]), (dev, stream))
    s, a, b, c, d, *_ = _descriptors.pack(4, *shape, *a, *b, *c, *d)
    st = L.lib().nvfp4_attention_forward_ws(s, a, b, c, d, lse.data_ptr(), ws.data_ptr(), ws.numel(), _status_ptr(dev),
                                            stream)
    if st:
        L.check(st, "nvfp4_attention_forward_ws")
    return out, lse


def attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                       lse: torch.Tensor, causal: bool = False, scale: Optional[float] = None,
                       cu_q: Optional[torch.Tensor] = None, cu_k: Optional[torch.Tensor] = None,
                       dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                       dv: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients (dq, dk, dv) of :func:`attention_forward`, the probabilities recomputed from q, k and
    lse.  dq, dk, dv may be given as strided views, such as the slices of one buffer that is the
    fused projection's dY.  Deterministic."""
    dev = q.get_device()
    shape = _attention_shape(q, k, causal, scale, cu_q, cu_k, dev)
    T, H, D = qs = q.shape
    ks = (k.shape[0], k.shape[1], D)
    a, b, c = _heads(dout, "dout", qs, dev), _heads(q, "q", qs, dev), _heads(k, "k", ks, dev)
    d, e = _heads(v, "v", ks, dev), _heads(out, "out", qs, dev)
    if lse.dtype != torch.float32 or lse.shape != (H, T) or not lse.is_contiguous():
        raise _invalid(f"lse must be contiguous float32 [{H}, {T}]")
    _on(lse, "lse", dev)
    stream = _here(dev)
    dq = torch.empty(qs, dtype=torch.bfloat16, device=q.device) if dq is None else dq
    dk = torch.empty(ks, dtype=torch.bfloat16, device=q.device) if dk is None else dk
    dv = torch.empty(ks, dtype=torch.bfloat16, device=q.device) if dv is None else dv
    ws = _workspace(_attention_workspace(True, dev, T, ks[0], H, ks[1], D, shape[7]), (dev, stream))
    s, a, b, c, d, e, f, g, h = _descriptors.pack(8, *shape, *a, *b, *c, *d, *e, *_heads(dq, "dq", qs, dev),
                                                  *_heads(dk, "dk", ks, dev), *_heads(dv, "dv", ks, dev))
    st = L.lib().nvfp4_attention_backward(s, a, b, c, d, e, lse.data_ptr(), f, g, h, ws.data_ptr(), ws.numel(),
                                          _status_ptr(dev), stream)
    if st:
        L.check(st, "nvfp4_attention_backward")
    return dq, dk, dv


# ----------------------------------------------------------------------------- AdamW

STATE_BLOCK = 128                       # elements of an 8-bit state with one scale
_data_ptr, _device, _contiguous = torch.Tensor.data_ptr, torch.Tensor.get_device, torch.Tensor.is_contiguous


class AdamW:
    """AdamW over a list of parameters (float32 / bfloat16, contiguous, CUDA), updated in place by
    :meth:`step`, one launch for many tensors.

    ``bits=32`` keeps the moments ``m`` and ``v`` in float32.  ``bits=8`` keeps E4M3 codes of them
    (torch.float8_e4m3fn) with a float32 scale per 128 elements (``m_scale``, ``v_scale``; value =
    code * scale): meant for beta2 up to about 0.99, where the spread that stochastic rounding gives
    v stays below two fifths of v.  ``state`` takes such lists over from elsewhere (a checkpoint) and
    ``steps`` how many steps they have seen: it takes over their memory, under tensors of its own in
    :attr:`state`, whose lists are what a checkpoint stores.  To go on from other tensors make another
    object: a step after a parameter or a state was replaced, or given other storage, is refused (new
    values are copied into them).
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
            _on(p, f"params[{i}]", torch.cuda.current_device())
            if p.dtype not in _DT or not p.is_contiguous():
                raise _invalid(f"params[{i}] must be contiguous float32 or bfloat16")
        if self.params and any(p.device != self.params[0].device for p in self.params):
            raise _invalid("params must be on one device")
        names = ("m", "v") if bits == 32 else ("m", "v", "m_scale", "v_scale")
        if state is not None and (set(state) != set(names) or any(len(state[k]) != n for k in names)):
            raise NVFP4Error(L.ERR_SHAPE, f"state must hold lists of {n} tensors named {names}")
        states: Dict[str, List[torch.Tensor]] = {}
        for k in names:
            blocks, dtype = k.endswith("_scale"), torch.float32
            if bits == 8 and not blocks:
                dtype = torch.float8_e4m3fn
            if state is None:
                states[k] = [torch.zeros((p.numel() + STATE_BLOCK - 1) // STATE_BLOCK if blocks else p.shape,
                                         dtype=dtype, device=p.device) for p in self.params]
                continue
            for i, (s, p) in enumerate(zip(state[k], self.params)):
                want = (p.numel() + STATE_BLOCK - 1) // STATE_BLOCK if blocks else p.numel()
                if s.device != p.device or s.dtype != dtype or s.numel() != want or not s.is_contiguous():
                    raise _invalid(f"state[{k!r}][{i}] must be contiguous {dtype} of {want} elements beside its parameter")
            states[k] = [s.detach() for s in state[k]]
        # What the descriptors point to.  Aliases keep the parameters' memory, whatever becomes of the tensors.  Nobody else has the
        # tensors of the states until `state` is read; from then on a step looks at them too.
        self._states, self._state_read = states, False
        self._aliases = [p.detach() for p in self.params]
        self._addresses = [p.data_ptr() for p in self.params]
        kept = [t for k in names for t in states[k]]
        self._kept_states, self._state_addresses = [t.detach() for t in kept], [t.data_ptr() for t in kept]
        spans = sorted((at, at + t.numel() * t.element_size())
                       for at, t in zip(self._addresses + self._state_addresses, self._aliases + kept) if t.numel())
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            raise _invalid("parameters and states must not share memory (a shared weight is one parameter, its gradients summed)")
        self._shapes = [p.shape for p in self.params]
        size, T = ctypes.sizeof(L.AdamWTensorC), L.AdamWTensorC
        memory = bytearray(size * max(n, 1))
        self._tensors = (T * max(n, 1)).from_buffer(memory)
        for i, (p, d) in enumerate(zip(self.params, decay)):
            self._tensors[i] = T(
                p.data_ptr(), None, states["m"][i].data_ptr(), states["v"][i].data_ptr(),
                states["m_scale"][i].data_ptr() if bits == 8 else None,
                states["v_scale"][i].data_ptr() if bits == 8 else None, p.numel(), _DT[p.dtype], 0, d, i)
        # the fields that change from step to step: every descriptor's gradient and its type
        self._grads = memoryview(memory).cast("Q")[T.grad.offset // 8::size // 8]
        self._grad_dtypes = memoryview(memory).cast("i")[T.grad_dtype.offset // 4::size // 4]

    @property
    def state(self) -> Dict[str, List[torch.Tensor]]:
        """The states, a list of tensors for each name."""
        self._state_read = True
        return self._states

    def _unchanged(self) -> bool:
        """Whether parameters and states are still at the addresses that the descriptors were made from."""
        try:
            return list(map(_data_ptr, self.params)) == self._addresses and (
                not self._state_read or
                list(map(_data_ptr, itertools.chain.from_iterable(self._states.values()))) == self._state_addresses)
        except TypeError:                                  # something that is no tensor
            return False

    def _marshalled(self, grads: Sequence[Optional[torch.Tensor]], dev: int) -> Tuple[array, array]:
        """The gradients' addresses (0 for None) and types."""
        try:
            kinds = [_DT[g.dtype] for g in grads]
            if [g.shape for g in grads] == self._shapes and all(map(_contiguous, grads)) and {*map(_device, grads)} == {dev}:
                return array("Q", map(_data_ptr, grads)), array("i", kinds)
        except (AttributeError, KeyError):                  # a None, or a type that is looked at below
            pass
        at, kinds = array("Q"), array("i")
        for i, (g, shape) in enumerate(zip(grads, self._shapes)):
            code = 0 if g is None else _DT.get(g.dtype)
            if g is not None and (code is None or g.shape != shape or g.get_device() != dev or not g.is_contiguous()):
                raise _invalid(f"grads[{i}] must be contiguous float32 or bfloat16 {list(shape)} beside its parameter")
            at.append(0 if g is None else g.data_ptr())
            kinds.append(code)
        return at, kinds

    def step(self, grads: Sequence[Optional[torch.Tensor]], lr: float, betas: Tuple[float, float] = (0.9, 0.95),
             eps: float = 1e-8, grad_scale: Optional[torch.Tensor] = None, round: int = L.SR, sr_seed: int = 0) -> None:
        """One update.  ``grads``: one per parameter, of its shape, contiguous, float32 or bfloat16
        (None leaves that parameter and its state alone).  ``grad_scale``: a one-element float32 CUDA tensor
        that multiplies every gradient (loss scale, clipping) without a host read.  ``round`` (RNE
        or SR with ``sr_seed``) is how 8-bit states and bfloat16 parameters are rounded.  The step's number is
        part of the launch: a step cannot be captured in a CUDA graph."""
        n = len(self._shapes)
        if len(grads) != n:
            raise NVFP4Error(L.ERR_SHAPE, f"{len(grads)} gradients for {n} parameters")
        if not self._unchanged():
            raise _invalid("a parameter or a state was replaced or has other storage than when the optimizer was made")
        if not n:
            return
        dev = self._aliases[0].get_device()
        stream = _here(dev)
        if torch.cuda.is_current_stream_capturing():
            raise NVFP4Error(L.ERR_UNSUPPORTED, "an AdamW step in a CUDA graph would be replayed with the same step number, and "
                                                "so with the same bias corrections and random bits")
        if grad_scale is not None and (grad_scale.get_device() != dev or grad_scale.dtype != torch.float32
                                       or grad_scale.numel() != 1):
            raise _invalid("grad_scale must be one float32 on the parameters' device")
        at, kinds = self._marshalled(grads, dev)
        self._grads[:], self._grad_dtypes[:] = at, kinds
        hp = L.AdamWParams(self.bits, round, self.steps + 1, lr, betas[0], betas[1], eps, sr_seed & (2**64 - 1))
        st = L.lib().nvfp4_adamw_step(self._tensors, n, hp, _ptr(grad_scale), _status_ptr(dev), stream)
        L.check(st, "nvfp4_adamw_step")
        self.steps += 1
