"""The operators around retention in a gated recurrent block.

gated_recurrence (with its backward and its single-token step) is a linear
recurrence whose decay is computed per token and channel, where retention's is
fixed per head; gated_norm and residual_norm are the norms after and before the
block's mixer, with their backward passes. Like the functions of the package's
front module these only check and marshal tensors for the C ABI
(include/retention_block.h states each operator); all computation runs in the
library's HIP kernels on the current stream of the tensors' device.

Tensors of activations are float32 or bfloat16 with a contiguous last
dimension; the others may be strided, so a slice of a fused projection or a
token-major tensor is taken as it is. Outputs are contiguous unless passed in,
and must not share memory with inputs or one another. None of the functions
takes part in autograd: the ``*_backward`` functions return the gradients.
"""

from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass
from typing import Optional, Union

import torch

from . import GroupNorm, RetentionError, _lib, _require, _require_workspace, _stream

FORMS = {"sigmoid": 0, "log": 1}
_CODES = {torch.float32: _lib.RET_F32, torch.bfloat16: _lib.RET_BF16}


@dataclass
class Norm:
    """A norm over the last dimension: eps, optional fp32 weight and bias on the
    device, and the form, layer (rms False) or root-mean-square."""

    eps: float = 1e-5
    weight: Optional[torch.Tensor] = None
    bias: Optional[torch.Tensor] = None
    rms: bool = False


NormLike = Union[Norm, GroupNorm]

# A decode step's call is bound by the host, so what is checked for every
# tensor is checked in one pass, and said in full only where it fails. torch's
# current stream is asked for as a number: a Stream object costs 2 us, a fifth
# of a step's whole host time.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _activations(t, name, dims):
    """``t`` is a device tensor of a supported dtype with one of ``dims`` dimensions, the last contiguous. Returns the
    dtype's code."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() not in dims:
        raise ValueError(f"{name} must have {' or '.join(map(str, dims))} dimensions, not {t.dim()}")
    if t.stride(-1) != 1:
        _last_contiguous(t, name)
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")
    return code


def _last_contiguous(t, name):
    if t.stride(-1) != 1 and t.size(-1) > 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    return t


def _same(t, name, like, dtype=None):
    """``t`` is a tensor of ``like``'s shape and device (and dtype, unless another is given), the last dimension
    contiguous."""
    dtype = dtype or like.dtype
    if (isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == like.shape and t.stride(-1) == 1
            and t.device == like.device):
        return t
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.device != like.device:
        raise ValueError(f"{name} must be on {like.device} (the inputs' device), not {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != like.shape:
        raise ValueError(f"{name} must have shape {tuple(like.shape)}, not {tuple(t.shape)}")
    return _last_contiguous(t, name)


def _f32(t, name, shape, device):
    """``t`` is a contiguous float32 tensor of this shape on ``device``."""
    if (isinstance(t, torch.Tensor) and t.dtype == torch.float32 and t.shape == shape and t.device == device
            and t.is_contiguous()):
        return t
    return _require(t, name, shape, torch.float32, device)


def _ints(*sizes):
    """Sizes that reach the C library as ints."""
    if max(sizes) >> 31:
        raise ValueError(f"a size of {max(sizes)} is too large")
    return sizes


def _new(like, dtype=None):
    return torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format)


def _output(t, name, like, dtype=None):
    return _new(like, dtype) if t is None else _same(t, name, like, dtype)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _view(t):
    """The retention_view_t of a tensor of two to four dimensions: [B, H, N, d], or without the H, the N or both. The
    strides of the dimensions that are missing are those of sizes of 1, which are not read."""
    if t is None:
        return None
    s = t.stride()
    return _lib.View(t.data_ptr(), s[0], s[1], s[-2])


def _call(name, like, *args):
    """Calls the entry point with ``like``'s device current, on its current stream."""
    fn, device = getattr(_lib.load(), name), like.get_device()
    stream = _stream(like) if _raw_stream is None else _raw_stream(device)
    if device == _current_device():
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream)
    if rc:
        raise RetentionError(name, rc)


def _workspace(workspace, nbytes, device):
    if workspace is None:
        return (torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None), nbytes
    _require_workspace(workspace, "workspace", nbytes, device)
    return workspace, workspace.numel() * workspace.element_size()


# ---------------------------------------------------------------------------
# Gated recurrence


def _form(form):
    if form not in FORMS:
        raise ValueError(f"form must be one of {sorted(FORMS)}, not {form!r}")
    return FORMS[form]


def _sequences(t, cu_seqlens, max_len):
    """((B, H, N, d), state shape, sequences, max_len) of the activations ``t``."""
    B, N, d = t.size(0), t.size(-2), t.size(-1)
    H = t.size(1) if t.dim() == 4 else 1
    if cu_seqlens is None:
        if max_len is not None:
            raise ValueError("max_len needs cu_seqlens")
        S, max_len = B, N
    else:
        if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be a tensor of at least two offsets")
        _require(cu_seqlens, "cu_seqlens", (cu_seqlens.numel(),), torch.int32, t.device)
        if B != 1:
            raise ValueError("packed sequences (cu_seqlens) need a batch of one row")
        S, max_len = cu_seqlens.numel() - 1, N if max_len is None else min(int(max_len), N)
        if max_len <= 0:
            raise ValueError("max_len must be positive")
    return _ints(B, H, N, d), ((S, H, d) if t.dim() == 4 else (S, d)), S, max_len


def _state_to_fill(t, name, shape, device):
    if t is True:
        return torch.empty(shape, dtype=torch.float32, device=device)
    if t is False or t is None:
        return None
    return _f32(t, name, shape, device)


def gated_recurrence_workspace_bytes(sequences, H, N, d, dtype=torch.bfloat16, max_len=None) -> int:
    """Workspace bytes of gated_recurrence and its backward: for ``sequences`` rows of N tokens or, with ``max_len``,
    as many packed sequences of at most that length in one row of N tokens."""
    code = _lib.RET_BF16 if dtype == torch.bfloat16 else _lib.RET_F32
    return _scan_bytes(sequences, (1, H, N, d), N if max_len is None else max_len, max_len is not None, code)


def _scan_bytes(S, dims, max_len, packed, code):
    return int(_lib.load().retention_gated_recurrence_workspace_bytes(S, dims[1], dims[2], max_len, packed, dims[3],
                                                                      code))


def gated_recurrence(x, gate, form: str = "sigmoid", state_in=None, state_out: Union[bool, torch.Tensor] = False,
                     cu_seqlens=None, max_len: Optional[int] = None, out=None, workspace=None):
    """Gated linear recurrence over sequences, per channel. Returns (h, state_out or None).

    ``form`` "sigmoid": a = sigmoid(gate), h_t = a_t h_{t-1} + (1 - a_t) x_t;
    "log": a = exp(gate), h_t = a_t h_{t-1} + x_t (gate <= 0 for a decay; -inf
    starts the state anew; above 0 only while the products of 256 tokens' decays
    stay in fp32's range). x and gate are [B, N, D] or [B, H, N, d]; states
    are fp32 [B, D] or [B, H, d]. ``state_out``: False (not produced), True
    (allocate) or a tensor to fill (it may be ``state_in`` itself).

    Packed sequences: with ``cu_seqlens`` (device int32 [S + 1]) B is 1 and
    sequence s holds tokens cu_seqlens[s] up to cu_seqlens[s + 1]; states are
    [S, ...] and ``max_len`` (default N) bounds a sequence's length. Tokens
    outside every sequence, or beyond max_len of one, are not written, so in
    an output allocated here they are undefined.
    """
    dt = _activations(x, "x", (3, 4))
    _same(gate, "gate", x)
    code = _form(form)
    dims, states, S, max_len = _sequences(x, cu_seqlens, max_len)
    dev = x.device
    out = _output(out, "out", x)
    if state_in is not None:
        _f32(state_in, "state_in", states, dev)
    state_out = _state_to_fill(state_out, "state_out", states, dev)
    nbytes = _scan_bytes(S, dims, max_len, cu_seqlens is not None, dt)
    workspace, have = _workspace(workspace, nbytes, dev)
    _call("retention_gated_recurrence", x, _view(x), _view(gate), _view(out), *dims, code, dt, _ptr(state_in),
          _ptr(state_out), _ptr(cu_seqlens), S, max_len, _ptr(workspace), have)
    return out, state_out


def gated_recurrence_backward(grad_h, x, gate, h, form: str = "sigmoid", state_in=None, grad_state_out=None,
                              grad_state_in: Union[bool, torch.Tensor] = False, cu_seqlens=None,
                              max_len: Optional[int] = None, grads=None, workspace=None):
    """Gradients of gated_recurrence for dL/dh = grad_h. Returns (grad_x, grad_gate, grad_state_in or None).

    ``h`` is the forward call's output and ``state_in`` its starting state;
    x may be None in the "log" form, which does not read it. ``grad_state_out``
    is dL/d(final state) (fp32, None = 0); ``grad_state_in``: False (not
    produced), True (allocate) or a tensor to fill. ``grads``: optional
    preallocated (grad_x, grad_gate). Sequences as in the forward call. A
    gradient of a broadcast input comes in the input's full shape.
    """
    code = _form(form)
    dt = _activations(gate, "gate", (3, 4))
    _same(grad_h, "grad_h", gate)
    _same(h, "h", gate)
    if x is not None:
        _same(x, "x", gate)
    elif code == 0:
        raise ValueError("the sigmoid form needs x")
    dims, states, S, max_len = _sequences(gate, cu_seqlens, max_len)
    dev = gate.device
    if grads is None:
        grads = (_new(gate), _new(gate))
    if len(grads) != 2:
        raise ValueError("grads must be (grad_x, grad_gate)")
    for name, t in zip(("grad_x", "grad_gate"), grads):
        _same(t, name, gate)
    for name, t in (("state_in", state_in), ("grad_state_out", grad_state_out)):
        if t is not None:
            _f32(t, name, states, dev)
    grad_state_in = _state_to_fill(grad_state_in, "grad_state_in", states, dev)
    nbytes = _scan_bytes(S, dims, max_len, cu_seqlens is not None, dt)
    workspace, have = _workspace(workspace, nbytes, dev)
    _call("retention_gated_recurrence_backward", gate, _view(grad_h), _view(x), _view(gate), _view(h),
          _view(grads[0]), _view(grads[1]), *dims, code, dt, _ptr(state_in), _ptr(grad_state_out),
          _ptr(grad_state_in), _ptr(cu_seqlens), S, max_len, _ptr(workspace), have)
    return grads[0], grads[1], grad_state_in


def _step_dims(x, states):
    shape = x.shape
    return _ints(shape[0], shape[1] if len(shape) == 3 else 1, shape[-1], states)


def gated_recurrence_step(x, gate, state, form: str = "sigmoid", slots=None, out=None):
    """One token of gated_recurrence per row, the states updated in place. Returns h.

    x and gate are [B, D] or [B, H, d]; state is fp32 [B, D] or [B, H, d], or
    with ``slots`` (device int32 [B]) a pool of states [P, ...] in which row b
    has slots[b]. A row whose slot is negative or not below P is idle: its
    output is not written. Rows naming the same slot take effect one after
    another in row order.
    """
    dt = _activations(x, "x", (2, 3))
    _same(gate, "gate", x)
    code, dev, shape = _form(form), x.device, x.shape
    if not isinstance(state, torch.Tensor) or state.dim() != len(shape):
        raise ValueError(f"state must be a tensor with {len(shape)} dimensions")
    P = shape[0] if slots is None else state.size(0)
    _f32(state, "state", (P, *shape[1:]), dev)
    if slots is not None:
        _require(slots, "slots", shape[:1], torch.int32, dev)
    B, H, d, P = _step_dims(x, P)
    out = _output(out, "out", x)
    _call("retention_gated_recurrence_step", x, _view(x), _view(gate), _view(out), B, H, d, code, dt,
          state.data_ptr(), P, _ptr(slots))
    return out


# ---------------------------------------------------------------------------
# Norms


def _norm_struct(norm, n, device):
    """The retention_norm_t of ``norm`` with n weights and biases; its tensors stay alive in the caller's ``norm``."""
    if not isinstance(norm, (Norm, GroupNorm)):
        raise ValueError("norm must be a Norm or a GroupNorm")
    weight, bias = norm.weight, norm.bias
    if weight is not None:
        weight = _f32(weight, "the norm's weight", (n,), device).data_ptr()
    if bias is not None:
        bias = _f32(bias, "the norm's bias", (n,), device).data_ptr()
    return _lib.NormStruct(norm.eps, getattr(norm, "rms", False), weight, bias)


def _head_dims(t):
    return _ints(t.size(0), t.size(1), t.size(2) if t.dim() == 4 else 1, t.size(-1))


def gated_norm(o, gate=None, norm: NormLike = GroupNorm(), out=None):
    """The norm and swish gate after the mixer, per head and token:
    (norm(o) * weight + bias) * swish(gate).

    o, gate (optional) and the output are [B, H, N, d], or [B, H, d] for one
    token; the norm's weight and bias hold H*d values. With a GroupNorm and
    contiguous tensors this is the ``gn``/``gate`` epilogue of ``chunkwise``
    as an operator of its own, for training, where the backward needs o.
    """
    dt = _activations(o, "o", (3, 4))
    if gate is not None:
        _same(gate, "gate", o)
    dims = _head_dims(o)
    n = _norm_struct(norm, dims[1] * dims[3], o.device)
    out = _output(out, "out", o)
    _call("retention_gated_norm", o, _view(o), _view(gate), _view(out), *dims, dt, n)
    return out


def gated_norm_backward_workspace_bytes(B, H, N, d, dtype=torch.bfloat16, with_params: bool = True) -> int:
    code = _lib.RET_BF16 if dtype == torch.bfloat16 else _lib.RET_F32
    return int(_lib.load().retention_gated_norm_backward_workspace_bytes(B, H, N, d, code, int(with_params)))


def gated_norm_backward(grad_y, o, gate=None, norm: NormLike = GroupNorm(), grads=None, workspace=None):
    """Gradients of gated_norm for dL/dy = grad_y. Returns (grad_o, grad_gate, grad_weight, grad_bias): grad_gate is
    None without a gate, grad_weight and grad_bias (fp32 [H*d]) where the norm has no weight or bias. ``grads``:
    optional preallocated (grad_o, grad_gate). grad_o is what chunkwise_backward takes as grad_o."""
    dt = _activations(o, "o", (3, 4))
    _same(grad_y, "grad_y", o)
    if gate is not None:
        _same(gate, "gate", o)
    dims, dev = _head_dims(o), o.device
    n = _norm_struct(norm, dims[1] * dims[3], dev)
    if grads is None:
        grads = (_new(o), None if gate is None else _new(o))
    if len(grads) != 2 or (grads[1] is None) != (gate is None):
        raise ValueError("grads must be (grad_o, grad_gate), grad_gate None without a gate")
    _same(grads[0], "grad_o", o)
    if gate is not None:
        _same(grads[1], "grad_gate", o)
    dw = None if norm.weight is None else torch.empty_like(norm.weight)
    db = None if norm.bias is None else torch.empty_like(norm.bias)
    params = dw is not None or db is not None
    nbytes = _lib.load().retention_gated_norm_backward_workspace_bytes(*dims, dt, params) if params else 0
    workspace, have = _workspace(workspace, nbytes, dev)
    _call("retention_gated_norm_backward", o, _view(grad_y), _view(o), _view(gate), _view(grads[0]), _view(grads[1]),
          *dims, dt, n, _ptr(dw), _ptr(db), _ptr(workspace), have)
    return grads[0], grads[1], dw, db


def _rows_view(t):
    """Rows of the last dimension: [B, N, D] or [R, D] with any strides, one, or those of a contiguous tensor of more
    dimensions, which lie D apart (the stride of a dimension of one element says nothing)."""
    if t is None or 2 <= t.dim() <= 3:
        return _view(t)
    return _lib.View(t.data_ptr(), 0, 0, t.size(-1))


def _row_dims(t):
    if t.dim() == 3:
        return _ints(*t.shape)
    return _ints(1, math.prod(t.shape[:-1]), t.size(-1))


def _rows(t, name):
    dt = _activations(t, name, range(1, 65))
    _rows_layout(t, name)
    return dt


def _rows_layout(t, name):
    if t.dim() > 3 and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous when it has more than three dimensions")
    return t


def _stream_dtype(t, name, dtype):
    if not isinstance(t, torch.Tensor) or t.dtype not in (dtype, torch.float32):
        raise ValueError(f"{name} must be a tensor of {dtype} or torch.float32")
    return t.dtype


def residual_norm(x, residual, norm: NormLike, scale=None, alpha: float = 1.0, out=None, residual_out=None):
    """The residual and the norm before the next block. Returns (y, r):
    r = alpha * residual + scale * x, y = norm(r) * weight + bias.

    x and residual are [..., D]; the residual stream (residual and r) has x's
    dtype or float32, y has x's. ``scale`` (fp32 [D], default 1) weighs the
    branch per channel.
    """
    dt, dev, dims = _rows(x, "x"), x.device, _row_dims(x)
    D = dims[-1]
    stream = _stream_dtype(residual, "residual", x.dtype)
    n = _norm_struct(norm, D, dev)
    if scale is not None:
        _f32(scale, "scale", (D,), dev)
    out, residual_out = _output(out, "out", x), _output(residual_out, "residual_out", x, stream)
    _same(residual, "residual", x, stream)
    if x.dim() > 3:
        for name, t in (("residual", residual), ("out", out), ("residual_out", residual_out)):
            _rows_layout(t, name)
    _call("retention_residual_norm", x, _rows_view(x), _rows_view(residual), _rows_view(out), _rows_view(residual_out),
          *dims, dt, _CODES[stream], n, _ptr(scale), float(alpha))
    return out, residual_out


def residual_norm_backward_workspace_bytes(B, N, D, dtype=torch.bfloat16, with_params: bool = True) -> int:
    code = _lib.RET_BF16 if dtype == torch.bfloat16 else _lib.RET_F32
    return int(_lib.load().retention_residual_norm_backward_workspace_bytes(B, N, D, code, int(with_params)))


def residual_norm_backward(grad_y, r, norm: NormLike, grad_r=None, x=None, scale=None, alpha: float = 1.0,
                           residual=None, grads=None, workspace=None):
    """Gradients of residual_norm for dL/dy = grad_y and dL/dr = grad_r (None = 0).

    Returns (grad_x, grad_residual, grad_scale, grad_weight, grad_bias):
    grad_scale (fp32 [D]) is formed when ``x`` and ``scale`` are given, the
    norm's gradients where it has a weight or bias. ``r`` is the forward call's
    output. In a bf16 stream it carries bf16's rounding, which grad_weight and
    grad_scale then show; with ``residual`` and ``x`` given the row is formed
    again from them in fp32 and r is not read (it may be None). Without a
    scale, with alpha 1 and one dtype, the two activation gradients are equal
    and grad_x is grad_residual, the same tensor. ``grads``: optional
    preallocated (grad_x, grad_residual), two tensors.
    """
    dt, dev, dims = _rows(grad_y, "grad_y"), grad_y.device, _row_dims(grad_y)
    D = dims[-1]
    if residual is not None and x is None:
        raise ValueError("residual needs x")
    row, name = (r, "r") if residual is None else (residual, "residual")
    stream = _stream_dtype(row, name, grad_y.dtype)
    n = _norm_struct(norm, D, dev)
    if scale is not None:
        _f32(scale, "scale", (D,), dev)
    if grads is None:
        d_res = _new(grad_y, stream)
        shared = scale is None and float(alpha) == 1.0 and stream == grad_y.dtype
        grads = (d_res if shared else _new(grad_y), d_res)
    else:
        shared = False
        if len(grads) != 2:
            raise ValueError("grads must be (grad_x, grad_residual)")
    _same(grads[0], "grad_x", grad_y)
    for what, t in ((name, row), ("grad_r", grad_r), ("grad_residual", grads[1])):
        if t is not None:
            _rows_layout(_same(t, what, grad_y, stream), what)
    if x is not None:
        _rows_layout(_same(x, "x", grad_y), "x")
    _rows_layout(grads[0], "grad_x")
    d_scale = torch.empty_like(scale) if scale is not None and x is not None else None
    dw = None if norm.weight is None else torch.empty_like(norm.weight)
    db = None if norm.bias is None else torch.empty_like(norm.bias)
    params = any(t is not None for t in (d_scale, dw, db))
    nbytes = _lib.load().retention_residual_norm_backward_workspace_bytes(*dims, dt, params) if params else 0
    workspace, have = _workspace(workspace, nbytes, dev)
    _call("retention_residual_norm_backward", grad_y, _rows_view(grad_y), _rows_view(grad_r),
          None if residual is not None else _rows_view(r),
          _rows_view(x if d_scale is not None or residual is not None else None), _rows_view(residual),
          None if shared else _rows_view(grads[0]), _rows_view(grads[1]), *dims, dt,
          _CODES[stream], n, _ptr(scale), float(alpha), _ptr(d_scale), _ptr(dw), _ptr(db), _ptr(workspace), have)
    return grads[0], grads[1], d_scale, dw, db
