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


class _Like:
    """What the tensors of a call share with the first of them: its shape, dtype and device, asked for once. ``flat``:
    taken as rows of a contiguous tensor."""

    __slots__ = ("t", "shape", "dtype", "device", "flat")

    def __init__(self, t, flat=False):
        self.t, self.shape, self.dtype, self.device, self.flat = t, t.shape, t.dtype, t.device, flat

    def view(self, t, name, dtype=None):
        """The retention_view_t of ``t``, after the checks of _same()."""
        dtype = dtype or self.dtype
        if (self.flat or not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != self.shape
                or t.device != self.device):
            return (_flat_view(_same(t, name, self.t, dtype), name) if self.flat else
                    _view(_same(t, name, self.t, dtype)))
        s = t.stride()
        if s[-1] != 1:
            _last_contiguous(t, name)
        return _lib.View(t.data_ptr(), s[0], s[1], s[-2])

    def output(self, t, name, dtype=None):
        """(tensor, view) of an output, allocated if None."""
        if t is not None:
            return t, self.view(t, name, dtype)
        t = _new(self.t, dtype)
        return t, (_flat_view(t, name) if self.flat else _view(t))


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
    if dtype is None or dtype is like.dtype:
        if like.is_contiguous():
            return torch.empty_like(like)
        return torch.empty_like(like, memory_format=torch.contiguous_format)
    return torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format)


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


def _h_dtype(given, name, dtype):
    """The dtype of h from a tensor, a dtype or None (the inputs' dtype): the inputs' or float32."""
    if isinstance(given, torch.Tensor):
        given = given.dtype
    h = dtype if given is None else given
    if h not in (dtype, torch.float32):
        raise ValueError(f"{name} must be {dtype} or torch.float32, not {h}")
    return h


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
                     cu_seqlens=None, max_len: Optional[int] = None, out=None, workspace=None, out_dtype=None):
    """Gated linear recurrence over sequences, per channel. Returns (h, state_out or None).

    ``form`` "sigmoid": a = sigmoid(gate), h_t = a_t h_{t-1} + (1 - a_t) x_t;
    "log": a = exp(gate), h_t = a_t h_{t-1} + x_t (gate <= 0 for a decay; above
    0 only while the products of 256 tokens' decays stay in fp32's range). A
    gate of -inf starts the state anew, whatever it holds, and one of +inf in
    the sigmoid form keeps it, whatever x holds. x and gate are [B, N, D] or [B, H, N, d]; states
    are fp32 [B, D] or [B, H, d]. ``state_out``: False (not produced), True
    (allocate) or a tensor to fill (it may be ``state_in`` itself). h has x's
    dtype, or float32 where ``out_dtype`` (or ``out``) is: the backward reads
    h, and a bfloat16 one brings its rounding into grad_gate.

    Packed sequences: with ``cu_seqlens`` (device int32 [S + 1]) B is 1 and
    sequence s holds tokens cu_seqlens[s] up to cu_seqlens[s + 1]; states are
    [S, ...] and ``max_len`` (default N) bounds a sequence's length. Tokens
    outside every sequence, or beyond max_len of one, are not written, so in
    an output allocated here they are undefined.

    ``workspace``: at least gated_recurrence_workspace_bytes, of this call alone
    while it runs. If its first four bytes (where any are needed) are 0
    afterwards, a wait between parts of a sequence was given up after about a
    second and the results behind it are NaN; they are all ones otherwise.
    """
    dt = _activations(x, "x", (3, 4))
    like = _Like(x)
    gate_view, code = like.view(gate, "gate"), _form(form)
    dims, states, S, max_len = _sequences(x, cu_seqlens, max_len)
    dev = like.device
    h_dtype = _h_dtype(out if out_dtype is None else out_dtype, "out", like.dtype)
    out, out_view = like.output(out, "out", h_dtype)
    if state_in is not None:
        _f32(state_in, "state_in", states, dev)
    state_out = _state_to_fill(state_out, "state_out", states, dev)
    nbytes = _scan_bytes(S, dims, max_len, cu_seqlens is not None, dt)
    workspace, have = _workspace(workspace, nbytes, dev)
    _call("retention_gated_recurrence", x, _view(x), gate_view, out_view, *dims, code,
          dt if h_dtype is like.dtype else dt | _lib.H_F32, _ptr(state_in),
          _ptr(state_out), _ptr(cu_seqlens), S, max_len, _ptr(workspace), have)
    return out, state_out


def gated_recurrence_backward(grad_h, x, gate, h, form: str = "sigmoid", state_in=None, grad_state_out=None,
                              grad_state_in: Union[bool, torch.Tensor] = False, cu_seqlens=None,
                              max_len: Optional[int] = None, grads=None, workspace=None):
    """Gradients of gated_recurrence for dL/dh = grad_h. Returns (grad_x, grad_gate, grad_state_in or None).

    ``h`` is the forward call's output (in the inputs' dtype or float32) and
    ``state_in`` its starting state; x may be None in the "log" form, which does not read it. ``grad_state_out``
    is dL/d(final state) (fp32, None = 0); ``grad_state_in``: False (not
    produced), True (allocate) or a tensor to fill. ``grads``: optional
    preallocated (grad_x, grad_gate). Sequences as in the forward call. A
    gradient of a broadcast input comes in the input's full shape.
    """
    code = _form(form)
    dt = _activations(gate, "gate", (3, 4))
    like = _Like(gate)
    if x is None and code == 0:
        raise ValueError("the sigmoid form needs x")
    h_dtype = _h_dtype(h, "h", like.dtype)
    inputs = (like.view(grad_h, "grad_h"), None if x is None else like.view(x, "x"), _view(gate),
              like.view(h, "h", h_dtype))
    dims, states, S, max_len = _sequences(gate, cu_seqlens, max_len)
    dev = like.device
    if grads is None:
        grads = None, None
    elif len(grads) != 2 or any(t is None for t in grads):
        raise ValueError("grads must be (grad_x, grad_gate)")
    (grad_x, dx_view), (grad_gate, dg_view) = like.output(grads[0], "grad_x"), like.output(grads[1], "grad_gate")
    for name, t in (("state_in", state_in), ("grad_state_out", grad_state_out)):
        if t is not None:
            _f32(t, name, states, dev)
    grad_state_in = _state_to_fill(grad_state_in, "grad_state_in", states, dev)
    nbytes = _scan_bytes(S, dims, max_len, cu_seqlens is not None, dt)
    workspace, have = _workspace(workspace, nbytes, dev)
    _call("retention_gated_recurrence_backward", gate, *inputs, dx_view, dg_view, *dims, code,
          dt if h_dtype is like.dtype else dt | _lib.H_F32,
          _ptr(state_in), _ptr(grad_state_out), _ptr(grad_state_in), _ptr(cu_seqlens), S, max_len, _ptr(workspace),
          have)
    return grad_x, grad_gate, grad_state_in


def _step_dims(shape, states):
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
    like = _Like(x)
    gate_view, code, dev, shape = like.view(gate, "gate"), _form(form), like.device, like.shape
    if not isinstance(state, torch.Tensor) or state.dim() != len(shape):
        raise ValueError(f"state must be a tensor with {len(shape)} dimensions")
    P = shape[0] if slots is None else state.size(0)
    _f32(state, "state", (P, *shape[1:]), dev)
    if slots is not None:
        _require(slots, "slots", shape[:1], torch.int32, dev)
    B, H, d, P = _step_dims(shape, P)
    out, out_view = like.output(out, "out")
    _call("retention_gated_recurrence_step", x, _view(x), gate_view, out_view, B, H, d, code, dt,
          state.data_ptr(), P, _ptr(slots))
    return out


# ---------------------------------------------------------------------------
# Norms

_ROWS = range(1, 65)  # dimensions of a tensor of rows


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


def _head_dims(shape):
    return _ints(shape[0], shape[1], shape[2] if len(shape) == 4 else 1, shape[-1])


def gated_norm(o, gate=None, norm: NormLike = GroupNorm(), out=None):
    """The norm and swish gate after the mixer, per head and token:
    (norm(o) * weight + bias) * swish(gate).

    o, gate (optional) and the output are [B, H, N, d], or [B, H, d] for one
    token; the norm's weight and bias hold H*d values. With a GroupNorm and
    contiguous tensors this is the ``gn``/``gate`` epilogue of ``chunkwise``
    as an operator of its own, for training, where the backward needs o.
    """
    dt = _activations(o, "o", (3, 4))
    like = _Like(o)
    gate_view = None if gate is None else like.view(gate, "gate")
    dims = _head_dims(like.shape)
    n = _norm_struct(norm, dims[1] * dims[3], like.device)
    out, out_view = like.output(out, "out")
    _call("retention_gated_norm", o, _view(o), gate_view, out_view, *dims, dt, n)
    return out


def gated_norm_backward_workspace_bytes(B, H, N, d, dtype=torch.bfloat16, with_params: bool = True) -> int:
    code = _lib.RET_BF16 if dtype == torch.bfloat16 else _lib.RET_F32
    return int(_lib.load().retention_gated_norm_backward_workspace_bytes(B, H, N, d, code, int(with_params)))


def gated_norm_backward(grad_y, o, gate=None, norm: NormLike = GroupNorm(), grads=None, workspace=None):
    """Gradients of gated_norm for dL/dy = grad_y. Returns (grad_o, grad_gate, grad_weight, grad_bias): grad_gate is
    None without a gate, grad_weight and grad_bias (fp32 [H*d]) where the norm has no weight or bias. ``grads``:
    optional preallocated (grad_o, grad_gate). grad_o is what chunkwise_backward takes as grad_o."""
    dt = _activations(o, "o", (3, 4))
    like = _Like(o)
    inputs = like.view(grad_y, "grad_y"), _view(o), None if gate is None else like.view(gate, "gate")
    dims, dev = _head_dims(like.shape), like.device
    n = _norm_struct(norm, dims[1] * dims[3], dev)
    if grads is None:
        grads = None, None
    elif len(grads) != 2 or grads[0] is None or (grads[1] is None) != (gate is None):
        raise ValueError("grads must be (grad_o, grad_gate), grad_gate None without a gate")
    grad_o, do_view = like.output(grads[0], "grad_o")
    grad_gate, dg_view = (None, None) if gate is None else like.output(grads[1], "grad_gate")
    dw = None if norm.weight is None else torch.empty_like(norm.weight)
    db = None if norm.bias is None else torch.empty_like(norm.bias)
    params = dw is not None or db is not None
    nbytes = _lib.load().retention_gated_norm_backward_workspace_bytes(*dims, dt, params) if params else 0
    workspace, have = _workspace(workspace, nbytes, dev)
    _call("retention_gated_norm_backward", o, *inputs, do_view, dg_view, *dims, dt, n, _ptr(dw), _ptr(db),
          _ptr(workspace), have)
    return grad_o, grad_gate, dw, db


def _rows_like(t):
    """_Like() of rows of the last dimension: [B, N, D] or [R, D] with any strides, one row, or those of a contiguous
    tensor of more dimensions."""
    return _Like(t, not 2 <= t.dim() <= 3)


def _flat_view(t, name):
    """The rows of a contiguous tensor, which lie D apart (the stride of a dimension of one element says nothing)."""
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous when it has more than three dimensions")
    return _lib.View(t.data_ptr(), 0, 0, t.size(-1))


def _row_dims(shape):
    if len(shape) == 3:
        return _ints(*shape)
    return _ints(1, math.prod(shape[:-1]), shape[-1])


def _stream_dtype(t, name, dtype):
    if not isinstance(t, torch.Tensor) or t.dtype not in (dtype, torch.float32):
        raise ValueError(f"{name} must be a tensor of {dtype} or torch.float32")
    return t.dtype


def residual_norm(x, residual, norm: NormLike, scale=None, alpha: float = 1.0, out=None, residual_out=None):
    """The residual and the norm before the next block. Returns (y, r):
    r = alpha * residual + scale * x, y = norm(r) * weight + bias.

    x and residual are [..., D]; the residual stream (residual and r) has x's
    dtype or float32, y has x's. ``scale`` (fp32 [D], default 1) weighs the
    branch per channel. ``residual_out`` may be ``residual`` itself.
    """
    dt, like = _activations(x, "x", _ROWS), _rows_like(x)
    dims, dev = _row_dims(like.shape), like.device
    D = dims[-1]
    stream = _stream_dtype(residual, "residual", like.dtype)
    n = _norm_struct(norm, D, dev)
    if scale is not None:
        _f32(scale, "scale", (D,), dev)
    inputs = like.view(x, "x"), like.view(residual, "residual", stream)
    out, out_view = like.output(out, "out")
    residual_out, r_view = like.output(residual_out, "residual_out", stream)
    _call("retention_residual_norm", x, *inputs, out_view, r_view, *dims, dt, _CODES[stream], n, _ptr(scale),
          float(alpha))
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
    dt, like = _activations(grad_y, "grad_y", _ROWS), _rows_like(grad_y)
    dims, dev = _row_dims(like.shape), like.device
    D = dims[-1]
    if residual is not None and x is None:
        raise ValueError("residual needs x")
    row, name = (r, "r") if residual is None else (residual, "residual")
    stream = _stream_dtype(row, name, like.dtype)
    n = _norm_struct(norm, D, dev)
    if scale is not None:
        _f32(scale, "scale", (D,), dev)
    shared = grads is None and scale is None and float(alpha) == 1.0 and stream == like.dtype
    if grads is None:
        grads = None, None
    elif len(grads) != 2 or any(t is None for t in grads):
        raise ValueError("grads must be (grad_x, grad_residual)")
    grad_residual, d_res_view = like.output(grads[1], "grad_residual", stream)
    grad_x, dx_view = (grad_residual, None) if shared else like.output(grads[0], "grad_x")
    row_view, x_view = like.view(row, name, stream), None if x is None else like.view(x, "x")
    views = (like.view(grad_y, "grad_y"), None if grad_r is None else like.view(grad_r, "grad_r", stream),
             row_view if residual is None else None, x_view if scale is not None or residual is not None else None,
             None if residual is None else row_view, dx_view, d_res_view)
    d_scale = torch.empty_like(scale) if scale is not None and x is not None else None
    dw = None if norm.weight is None else torch.empty_like(norm.weight)
    db = None if norm.bias is None else torch.empty_like(norm.bias)
    params = any(t is not None for t in (d_scale, dw, db))
    nbytes = _lib.load().retention_residual_norm_backward_workspace_bytes(*dims, dt, params) if params else 0
    workspace, have = _workspace(workspace, nbytes, dev)
    _call("retention_residual_norm_backward", grad_y, *views, *dims, dt, _CODES[stream], n, _ptr(scale), float(alpha),
          _ptr(d_scale), _ptr(dw), _ptr(db), _ptr(workspace), have)
    return grad_x, grad_residual, d_scale, dw, db
