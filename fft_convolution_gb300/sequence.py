"""Tensor helpers of the sequence-model operators (``fft_layer_norm``,
``fft_clip_grad_norm``, ``fft_delta_rule`` and their kin in
``include/fft_gb300.h``): they check and marshal torch tensors, allocate
outputs and workspaces, and call the library.  Every call is asynchronous on
``stream`` (default: torch's current stream); what a call allocates belongs
to that stream.  Results carry no autograd graph: forward and backward calls
are the two halves of a torch.autograd.Function (examples/sequence_block.py).
Tensors that a call overwrites count as changed in place.
"""
from __future__ import annotations

import array
import contextlib
import struct

import torch

from . import FFT_ELEM_BF16, FFT_ELEM_F16, FFT_ELEM_F32, FFT_ELEM_F64, _check, _lib

_ELEM = {torch.float32: FFT_ELEM_F32, torch.float64: FFT_ELEM_F64,
         torch.bfloat16: FFT_ELEM_BF16, torch.float16: FFT_ELEM_F16}
_NULL = contextlib.nullcontext()
# fft_delta_desc: sizes, five strides of three, scale, type, whether to clear rows.
_DESC = struct.Struct("=6q15qd2i")


def _elem(t, what: str) -> int:
    code = _ELEM.get(t.dtype)
    if code is None:
        raise TypeError(f"{what}: float32, float64, bfloat16 or float16, got {t.dtype}")
    return code


# Handle of torch's current stream on a device: without building a Stream
# object, where torch offers that (it costs as much as a kernel launch).
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on(stream, device):
    """(context in which the call allocates and launches, stream handle).  The
    library works on the current device, so inside it that is the tensors'."""
    if stream is None:
        here = device.index == torch.cuda.current_device()
        return _NULL if here else torch.cuda.device(device), _current(device.index)
    if stream.device != device:
        raise ValueError(f"tensors on {device}, a stream of {stream.device}")
    return torch.cuda.stream(stream), stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _device(first, *others):
    """Every tensor given lies on one CUDA device, which it returns."""
    if not first.is_cuda:
        raise ValueError("the operators take CUDA tensors")
    device = first.device
    for t in others:
        if t is not None and t.device != device:
            raise ValueError(f"tensors on {device} and {t.device}")
    return device


# Tells autograd of tensors that the library has written: a backward pass that
# needs what was there before raises then instead of using what is there now.
_changed = torch.autograd.graph.increment_version


def _workspace(nbytes: int, device):
    return torch.empty(max(16, nbytes), dtype=torch.uint8, device=device)


# ---- layer normalisation -----------------------------------------------------------

def _rows(t):
    """`t` as rows of its last axis, at one stride: a view where the strides
    allow it, else a copy."""
    if t.is_contiguous():
        return t if t.dim() == 2 else t.view(-1, t.shape[-1])
    if t.dim() == 2 and (t.stride(1) == 1 or t.shape[1] == 1) and t.stride(0) >= t.shape[1]:
        return t
    t = t.reshape(-1, t.shape[-1])
    if t.stride(1) != 1 and t.shape[1] != 1 or t.stride(0) < t.shape[1]:
        t = t.contiguous()
    return t


def _vector(t, dim: int, what: str):
    if t is None:
        return None
    if t.dim() != 1 or t.shape[0] != dim:
        raise ValueError(f"{what} must hold {dim} elements")
    return t if t.is_contiguous() else t.contiguous()


def _row_stats(t, rows: int, dtype, what: str):
    if t.numel() != rows or t.dtype != (torch.float64 if dtype == torch.float64 else torch.float32):
        raise ValueError(f"{what} must hold one value per row, as layer_norm returned it")
    return t.contiguous()


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, out=None, stream=None):
    """(y, mean, rstd) of the rows along x's last axis (see fft_layer_norm):
    y = (x - mean) rstd weight + bias.  weight and bias: vectors of x's type,
    or float32 with 16-bit x.  mean and rstd (float32; float64 for float64
    x) have x's shape without its last axis."""
    dim = x.shape[-1]
    if dim == 0:
        raise ValueError("rows need at least one element")
    device = _device(x, weight, bias, out)
    code = _elem(x, "x")
    context, handle = _on(stream, device)
    with context:
        w, b = _vector(weight, dim, "weight"), _vector(bias, dim, "bias")
        if w is not None and b is not None and w.dtype != b.dtype:
            raise TypeError("weight and bias need one type")
        wcode = code if w is None and b is None else _elem(w if w is not None else b, "weight")
        x2 = _rows(x)
        rows = x2.shape[0]
        given = out
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=device)
        elif out.shape != x.shape or out.dtype != x.dtype or not out.is_contiguous():
            raise ValueError("out must be contiguous and like x")
        kind = torch.float64 if code == FFT_ELEM_F64 else torch.float32
        mean = torch.empty(x.shape[:-1], dtype=kind, device=device)
        rstd = torch.empty(x.shape[:-1], dtype=kind, device=device)
        rc = _lib.fft_layer_norm(x2.data_ptr(), max(dim, x2.stride(0)), _ptr(w), _ptr(b),
                                 out.data_ptr(), dim, mean.data_ptr(), rstd.data_ptr(), rows, dim,
                                 eps, code, wcode, handle)
    if rc:
        _check(rc, "fft_layer_norm")
    if given is not None:
        _changed(given)
    return out, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, bias: bool = True, stream=None):
    """(dx, dweight, dbias) from dy and layer_norm's x, weight, mean and rstd
    (see fft_layer_norm_backward).  dweight is None without a weight; dbias
    is None with bias=False.  dweight and dbias have the weight's type (x's
    without a weight)."""
    dim = x.shape[-1]
    if dy.shape != x.shape or dy.dtype != x.dtype or dim == 0:
        raise ValueError("dy must be like x")
    device = _device(x, dy, weight, mean, rstd)
    code = _elem(x, "x")
    context, handle = _on(stream, device)
    with context:
        w = _vector(weight, dim, "weight")
        wcode = code if w is None else _elem(w, "weight")
        wtype = x.dtype if w is None else w.dtype
        x2, dy2 = _rows(x), _rows(dy)
        rows = x2.shape[0]
        mean, rstd = (_row_stats(t, rows, x.dtype, n) for t, n in ((mean, "mean"), (rstd, "rstd")))
        dx = torch.empty(x.shape, dtype=x.dtype, device=device)
        dw = torch.empty(dim, dtype=wtype, device=device) if w is not None else None
        db = torch.empty(dim, dtype=wtype, device=device) if bias else None
        ws = None
        nbytes = 0
        if dw is not None or db is not None:
            nbytes = _lib.fft_layer_norm_workspace_bytes(rows, dim, code)
            ws = _workspace(nbytes, device)
        _check(_lib.fft_layer_norm_backward(
            dy2.data_ptr(), max(dim, dy2.stride(0)), x2.data_ptr(), max(dim, x2.stride(0)), _ptr(w),
            mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), dim, _ptr(dw), _ptr(db), rows, dim,
            code, wcode, _ptr(ws), nbytes, handle), "fft_layer_norm_backward")
    return dx, dw, db


# ---- gradient clipping ---------------------------------------------------------------

def _table(tensors, what: str):
    """Host arrays of the tensors' pointers, sizes and types, and their device."""
    of = torch.Tensor  # its functions mapped: a third faster than a call by name each
    device = tensors[0].device
    if device.type != "cuda" or set(map(of.get_device, tensors)) != {device.index}:
        raise ValueError(f"{what}: CUDA tensors of one device")
    if not all(map(of.is_contiguous, tensors)):
        raise ValueError(f"{what}: contiguous tensors")
    try:
        codes = array.array("i", [_ELEM[t.dtype] for t in tensors])
    except KeyError:
        raise TypeError(f"{what}: float32, float64, bfloat16 or float16") from None
    return (array.array("Q", list(map(of.data_ptr, tensors))),
            array.array("q", list(map(of.numel, tensors))), codes, device)


def _address(a) -> int:
    return a.buffer_info()[0]


def grad_norm(grads, stream=None):
    """The 2-norm over all elements of a sequence of contiguous CUDA tensors
    (types may differ), as a float32 tensor without axes on their device."""
    grads = list(grads)
    if not grads:
        raise ValueError("grad_norm needs at least one tensor")
    ptrs, numels, codes, device = _table(grads, "grads")
    context, handle = _on(stream, device)
    with context:
        norm = torch.empty((), dtype=torch.float32, device=device)
        nbytes = _lib.fft_grad_norm_workspace_bytes(len(grads))
        ws = _workspace(nbytes, device)
        _check(_lib.fft_grad_norm(len(grads), _address(ptrs), _address(numels), _address(codes),
                                  norm.data_ptr(), ws.data_ptr(), nbytes, handle), "fft_grad_norm")
    return norm


def clip_grad_norm(grads, max_norm: float, out=None, eps: float = 1e-6, stream=None):
    """Scales every tensor by min(1, max_norm / (norm + eps)), in place or
    into the tensors of `out` (same shapes and types), and returns the norm
    before the scaling (see grad_norm, fft_clip_grad_norm)."""
    grads = list(grads)
    if not grads:
        raise ValueError("clip_grad_norm needs at least one tensor")
    ptrs, numels, codes, device = _table(grads, "grads")
    outs = ptrs
    if out is not None:
        out = list(out)
        if len(out) != len(grads):
            raise ValueError("out needs one tensor for each of grads")
        outs, onumels, ocodes, odevice = _table(out, "out")
        if odevice != device or onumels != numels or ocodes != codes:
            raise ValueError("out must be like grads")
    context, handle = _on(stream, device)
    with context:
        norm = torch.empty((), dtype=torch.float32, device=device)
        nbytes = _lib.fft_grad_norm_workspace_bytes(len(grads))
        ws = _workspace(nbytes, device)
        _check(_lib.fft_clip_grad_norm(len(grads), _address(ptrs), _address(outs),
                                       _address(numels), _address(codes), max_norm, eps,
                                       norm.data_ptr(), ws.data_ptr(), nbytes, handle),
               "fft_clip_grad_norm")
    _changed(grads if out is None else out)
    return norm


# ---- the gated delta rule --------------------------------------------------------------

def _dense(t):
    return t if t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


def _delta_inputs(q, k, v, g, beta, scale, batch, packed: bool, clear: bool = False):
    """Checks the five inputs; returns q, k, v (elements of a head contiguous),
    fft_delta_desc, its head sizes and the device."""
    qs, vs, kind = q.shape, v.shape, q.dtype
    lead = 1 if packed else 2
    if len(qs) != lead + 2 or len(vs) != lead + 2 or k.shape != qs or vs[:lead] != qs[:lead]:
        raise ValueError("q, k: [batch, tokens, key heads, dk]; v: [batch, tokens, value heads, dv] "
                         "(packed rows: without the batch axis)")
    if g.shape != vs[:-1] or beta.shape != g.shape:
        raise ValueError("g and beta hold one value per token and value head")
    if k.dtype != kind or v.dtype != kind:
        raise TypeError("q, k and v need one type")
    if g.dtype != torch.float32 or beta.dtype != torch.float32:
        raise TypeError("g and beta are float32")
    device = _device(q, k, v, g, beta)
    q, k, v = _dense(q), _dense(k), _dense(v)
    if scale is None:
        scale = qs[-1] ** -0.5
    first = (0,) if packed else ()  # packed rows have no stride between sequences
    strides = [first + t.stride()[:lead + 1] for t in (q, k, v, g, beta)]
    desc = _DESC.pack(batch, qs[lead - 1], qs[-2], vs[-2], qs[-1], vs[-1], *strides[0], *strides[1],
                      *strides[2], *strides[3], *strides[4], scale, _elem(q, "q"), clear)
    return q, k, v, desc, (vs[-2], qs[-1], vs[-1]), device


def _packing(q, offsets):
    """(number of sequences, packed) of the inputs' leading axes."""
    if offsets is None:
        return q.shape[0], False
    if offsets.dim() != 1 or offsets.shape[0] < 1 or offsets.dtype not in (torch.int32, torch.int64):
        raise ValueError("offsets must be int32 or int64 [sequences + 1]")
    return offsets.shape[0] - 1, True


def _states(t, shape, what: str):
    if t is None:
        return None
    if t.dtype != torch.float32 or tuple(t.shape) != shape:
        raise ValueError(f"{what} must be float32 {list(shape)}")
    return t.contiguous()


def delta_rule(q, k, v, g, beta, scale=None, initial_state=None, offsets=None, out=None,
               stream=None):
    """(o, final state) of the gated delta rule over whole sequences (see
    fft_delta_rule).  q, k: [batch, tokens, key heads, dk]; v: [batch, tokens,
    value heads, dv]; g (log decay) and beta: float32 [batch, tokens, value
    heads].  With offsets (int32 [sequences + 1] on the device) the rows of
    all sequences are packed and the arrays have no batch axis; rows of no
    sequence are 0 in o (in `out`, if it is given, as they were).  scale:
    dk ** -0.5 by default.  States: float32 [sequences, value heads, dk, dv]."""
    batch, packed = _packing(q, offsets)
    context, handle = _on(stream, _device(q))
    with context:
        q, k, v, desc, sizes, device = _delta_inputs(q, k, v, g, beta, scale, batch, packed,
                                                     packed and out is None)
        _device(q, initial_state, offsets, out)
        if packed:
            offsets = offsets.to(torch.int32).contiguous()
        shape = (batch,) + sizes
        initial_state = _states(initial_state, shape, "initial_state")
        given = out
        if out is None:
            out = torch.empty(v.shape, dtype=v.dtype, device=device)
        elif out.shape != v.shape or out.dtype != v.dtype or not out.is_contiguous():
            raise ValueError("out must be contiguous and like v")
        final = torch.empty(shape, dtype=torch.float32, device=device)
        nbytes = _lib.fft_delta_rule_workspace_bytes(desc, packed)
        ws = _workspace(nbytes, device)
        _check(_lib.fft_delta_rule(desc, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                   g.data_ptr(), beta.data_ptr(), _ptr(offsets),
                                   _ptr(initial_state), out.data_ptr(), final.data_ptr(),
                                   ws.data_ptr(), nbytes, handle), "fft_delta_rule")
    if given is not None:
        _changed(given)
    return out, final


def delta_rule_backward(do, q, k, v, g, beta, scale=None, initial_state=None, offsets=None,
                        dfinal_state=None, stream=None):
    """(dq, dk, dv, dg, dbeta, dinitial_state) of delta_rule, from the gradient
    of o (like v) and of the final state (None: zero); the other arguments
    as in the forward call (see fft_delta_rule_backward).  Packed rows of no
    sequence have gradients of 0."""
    batch, packed = _packing(q, offsets)
    context, handle = _on(stream, _device(q))
    with context:
        q, k, v, desc, sizes, device = _delta_inputs(q, k, v, g, beta, scale, batch, packed, packed)
        _device(q, do, initial_state, dfinal_state, offsets)
        if do.shape != v.shape or do.dtype != v.dtype:
            raise ValueError("do must be like v")
        do = do.contiguous()
        if packed:
            offsets = offsets.to(torch.int32).contiguous()
        shape = (batch,) + sizes
        initial_state = _states(initial_state, shape, "initial_state")
        dfinal_state = _states(dfinal_state, shape, "dfinal_state")
        new = lambda like, dtype: torch.empty(like.shape, dtype=dtype, device=device)  # noqa: E731
        dq, dk, dv = new(q, q.dtype), new(k, q.dtype), new(v, q.dtype)
        dg, dbeta = new(g, torch.float32), new(g, torch.float32)
        dinitial = torch.empty(shape, dtype=torch.float32, device=device)
        nbytes = _lib.fft_delta_rule_backward_workspace_bytes(desc, packed)
        ws = _workspace(nbytes, device)
        _check(_lib.fft_delta_rule_backward(
            desc, do.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(),
            g.data_ptr(), beta.data_ptr(), _ptr(offsets), _ptr(initial_state), _ptr(dfinal_state),
            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dg.data_ptr(), dbeta.data_ptr(),
            dinitial.data_ptr(), ws.data_ptr(), nbytes, handle), "fft_delta_rule_backward")
    return dq, dk, dv, dg, dbeta, dinitial


def delta_rule_step(q, k, v, g, beta, state, slots=None, scale=None, out=None, stream=None):
    """One or a few tokens per sequence of the gated delta rule (see
    fft_delta_rule_step): returns o [batch, tokens, value heads, dv] and
    updates `state` (float32 [pool, value heads, dk, dv], contiguous) in
    place.  slots: int32 [batch], the state of each sequence (negative: idle,
    o is 0); by default sequence i has state i."""
    context, handle = _on(stream, _device(q))
    with context:
        q, k, v, desc, sizes, device = _delta_inputs(q, k, v, g, beta, scale, q.shape[0], False)
        _device(q, state, slots, out)
        if state.dtype != torch.float32 or not state.is_contiguous() or state.dim() != 4 or \
                state.shape[1:] != sizes:
            raise ValueError("state must be contiguous float32 [pool, value heads, dk, dv]")
        if slots is not None and (slots.dtype != torch.int32 or slots.shape != (q.shape[0],)
                                  or not slots.is_contiguous()):
            raise ValueError("slots must be contiguous int32 [batch]")
        given = out
        if out is None:
            out = torch.empty(v.shape, dtype=v.dtype, device=device)
        elif out.shape != v.shape or out.dtype != v.dtype or not out.is_contiguous():
            raise ValueError("out must be contiguous and like v")
        _check(_lib.fft_delta_rule_step(desc, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                        g.data_ptr(), beta.data_ptr(), state.data_ptr(), _ptr(slots),
                                        state.shape[0], out.data_ptr(), handle),
               "fft_delta_rule_step")
    _changed(state if given is None else [state, given])
    return out
