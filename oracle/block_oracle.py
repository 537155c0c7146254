"""fp64 NumPy oracle of the operators around retention in a gated block.

Test infrastructure only; shares no code with the HIP path. Inputs (NumPy
arrays or torch tensors, bf16 values widened exactly) are taken as given and
everything is computed in float64, token by token for the recurrence.

  gated recurrence   a = 1/(1+e^-g), h_t = a_t h_{t-1} + (1 - a_t) x_t  (sigmoid)
                     a = e^g,        h_t = a_t h_{t-1} + x_t            (log)
  gated norm         (norm(o) w + b) * g / (1 + e^-g), norm over the last axis
  residual norm      r = alpha residual + scale x, y = norm(r) w + b

``*_error`` functions give the fp32 rounding that each operator's arithmetic can accumulate, from its formula: a count
of roundings, each of at most half a step, times the magnitudes that are rounded.
"""

from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24  # half a step of float32, relative


def f64(t):
    if t is None:
        return None
    if hasattr(t, "detach"):
        t = t.detach().cpu().double().numpy()
    return np.asarray(t, dtype=np.float64)


def decay(gate, form):
    """(a, weight of the input)."""
    g = f64(gate)
    if form == "sigmoid":
        e = np.exp(-np.abs(g))
        small, large = e / (1 + e), 1 / (1 + e)
        return np.where(g >= 0, large, small), np.where(g >= 0, small, large)
    return np.exp(g), np.ones_like(g)


def recurrence(x, gate, form, state=None):
    """x, gate [..., N, d] -> (h [..., N, d], final state [..., d])."""
    x = f64(x)
    a, c = decay(gate, form)
    now = np.zeros_like(x[..., 0, :]) if state is None else f64(state).copy()
    h = np.empty_like(x)
    for t in range(x.shape[-2]):
        now = a[..., t, :] * now + c[..., t, :] * x[..., t, :]
        h[..., t, :] = now
    return h, now


def recurrence_error(x, gate, form, state=None):
    """Bound of the fp32 error of h [..., N, d] and of the final state.

    A decay carries a relative error of (|g| + 8) U32: the exponent's product is rounded relative to |g|, and exp2, the
    reciprocal, the sums and products after it add a few steps (|g| beyond 88 has a = 0). Each token adds that times the
    magnitude M_t = a M_{t-1} + |b_t| carried through it; joining pieces of the sequence adds 32 more roundings.
    """
    x = f64(x)
    a, c = decay(gate, form)
    per = (np.minimum(np.abs(f64(gate)), 88.0) + 8.0) * U32
    m = np.zeros_like(x[..., 0, :]) if state is None else np.abs(f64(state))
    err = np.zeros_like(m)
    out = np.empty_like(x)
    for t in range(x.shape[-2]):
        m = a[..., t, :] * m + c[..., t, :] * np.abs(x[..., t, :])
        err = a[..., t, :] * err + per[..., t, :] * m
        out[..., t, :] = err + 32 * U32 * m
    return out, (out[..., -1, :] if x.shape[-2] else err)


def recurrence_backward(grad_h, x, gate, h, form, state=None, grad_state=None):
    """(grad_x, grad_gate, grad_state_in) for a given forward output h."""
    dh, g, h = f64(grad_h), f64(gate), f64(h)
    a, c = decay(g, form)
    before = np.concatenate((np.zeros_like(h[..., :1, :]) if state is None else f64(state)[..., None, :], h[..., :-1, :]), -2)
    w = np.zeros_like(dh[..., 0, :]) if grad_state is None else f64(grad_state).copy()
    u = np.empty_like(dh)
    for t in range(dh.shape[-2] - 1, -1, -1):
        u[..., t, :] = dh[..., t, :] + w
        w = a[..., t, :] * u[..., t, :]
    if form == "sigmoid":
        return c * u, a * c * (before - f64(x)) * u, w
    return u, a * before * u, w


def recurrence_backward_error(grad_h, x, gate, h, form, state=None, grad_state=None):
    """Bounds of the fp32 errors of the three gradients: those of the reverse recurrence of magnitudes (see
    recurrence_error), then the products with the decay's factors, (|g| + 8) U32 each, and the difference h - x."""
    dh, g, h = np.abs(f64(grad_h)), f64(gate), f64(h)
    a, c = decay(g, form)
    per = (np.minimum(np.abs(g), 88.0) + 8.0) * U32
    before = np.concatenate((np.zeros_like(h[..., :1, :]) if state is None else f64(state)[..., None, :], h[..., :-1, :]), -2)
    m = np.zeros_like(dh[..., 0, :]) if grad_state is None else np.abs(f64(grad_state))
    err = np.zeros_like(m)
    mu, eu = np.empty_like(dh), np.empty_like(dh)
    for t in range(dh.shape[-2] - 1, -1, -1):
        mu[..., t, :] = dh[..., t, :] + m
        eu[..., t, :] = err + 40 * U32 * mu[..., t, :]
        err = a[..., t, :] * err + per[..., t, :] * a[..., t, :] * mu[..., t, :]
        m = a[..., t, :] * mu[..., t, :]
    end = err + 40 * U32 * m
    if form == "sigmoid":
        size = np.abs(before) + np.abs(f64(x))
        return c * (eu + per * mu), a * c * size * (eu + 3 * per * mu), end
    return eu, a * np.abs(before) * (eu + 3 * per * mu), end


def norm_rows(v, eps, rms):
    """(xhat, 1 / deviation) over the last axis."""
    d = v if rms else v - v.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    return d * rstd, rstd


def swish(g):
    g = f64(g)
    return g * decay(g, "sigmoid")[0]


def swish_slope(g):
    g = f64(g)
    s, less = decay(g, "sigmoid")
    return s * (1 + g * less)


def _heads(p, H, d, none):
    return np.full((1, 1, 1), none) if p is None else f64(p).reshape(H, 1, d)


def gated_norm(o, gate, weight, bias, eps, rms):
    """o, gate [B, H, N, d]; weight, bias [H d]."""
    o = f64(o)
    H, d = o.shape[1], o.shape[3]
    z = norm_rows(o, eps, rms)[0] * _heads(weight, H, d, 1.0) + _heads(bias, H, d, 0.0)
    return z if gate is None else z * swish(gate)


# Roundings of a row's arithmetic: sums of up to 16384 values in runs of at most 64 and then in pairs (64 + 8), the
# deviation's square root and reciprocal, and the few products and sums of an element.
ROW = 96 * U32


def gated_norm_error(o, gate, weight, bias, eps, rms):
    """ROW times the magnitudes that enter: the largest value of the row over its deviation (what the mean's and the
    deviation's errors scale with), times |w|, plus |b|; the gate's factor adds (|g| + 8) U32 of the result."""
    o = f64(o)
    H, d = o.shape[1], o.shape[3]
    xhat, rstd = norm_rows(o, eps, rms)
    size = np.abs(o).max(-1, keepdims=True) * rstd
    z = (size + np.abs(xhat)) * np.abs(_heads(weight, H, d, 1.0)) + np.abs(_heads(bias, H, d, 0.0))
    if gate is None:
        return ROW * z
    return (ROW + (np.minimum(np.abs(f64(gate)), 88.0) + 8) * U32) * z * np.abs(swish(gate))


def gated_norm_backward(grad_y, o, gate, weight, bias, eps, rms):
    """(grad_o, grad_gate or None, grad_weight [H d], grad_bias [H d])."""
    dy, o = f64(grad_y), f64(o)
    H, d = o.shape[1], o.shape[3]
    w = _heads(weight, H, d, 1.0)
    xhat, rstd = norm_rows(o, eps, rms)
    dz, dg = dy, None
    if gate is not None:
        dz = dy * swish(gate)
        dg = dy * (xhat * w + _heads(bias, H, d, 0.0)) * swish_slope(gate)
    q = dz * w
    do = norm_rows_backward(q, xhat, rstd, rms)
    return do, dg, (dz * xhat).sum((0, 2)).reshape(-1), dz.sum((0, 2)).reshape(-1)


def norm_rows_backward(q, xhat, rstd, rms):
    t = q - xhat * (q * xhat).mean(-1, keepdims=True)
    return rstd * (t if rms else t - q.mean(-1, keepdims=True))


def norm_rows_backward_error(q, v, xhat, rstd):
    """ROW times the magnitudes of the gradient's terms, with xhat's own error (the row's largest value over its
    deviation) in each."""
    size = 1 + np.abs(v).max(-1, keepdims=True) * rstd
    mean = np.abs(q).mean(-1, keepdims=True)
    return ROW * rstd * size * (np.abs(q) + mean + (size + np.abs(xhat)) * (np.abs(q) * (size + np.abs(xhat))).mean(-1, keepdims=True))


def gated_norm_backward_error(grad_y, o, gate, weight, bias, eps, rms):
    """Bounds of the four gradients' fp32 errors; a parameter's sum over R rows adds R roundings of the summed
    magnitudes at most."""
    dy, o = f64(grad_y), f64(o)
    H, d = o.shape[1], o.shape[3]
    w = _heads(weight, H, d, 1.0)
    xhat, rstd = norm_rows(o, eps, rms)
    size = np.abs(o).max(-1, keepdims=True) * rstd
    dz, dg, steps = np.abs(dy), None, ROW
    if gate is not None:
        steps = ROW + (np.minimum(np.abs(f64(gate)), 88.0) + 8) * U32
        dz = np.abs(dy * swish(gate))
        g = f64(gate)
        s, less = decay(g, "sigmoid")
        dg = steps * np.abs(dy) * ((size + np.abs(xhat)) * np.abs(w) + np.abs(_heads(bias, H, d, 0.0))) * s * (1 + np.abs(g) * less)
    do = np.max(steps / ROW) * norm_rows_backward_error(dz * np.abs(w), o, xhat, rstd)
    rows = o.shape[0] * o.shape[2]
    per = (rows + np.max(steps / U32)) * U32
    return (do, dg, per * (dz * (size + np.abs(xhat))).sum((0, 2)).reshape(-1), per * dz.sum((0, 2)).reshape(-1))


def residual_norm(x, residual, weight, bias, eps, rms, scale=None, alpha=1.0):
    """(y, r); x, residual [..., D]."""
    r = alpha * f64(residual) + f64(x) * (1.0 if scale is None else f64(scale))
    y = norm_rows(r, eps, rms)[0]
    return y * (1.0 if weight is None else f64(weight)) + (0.0 if bias is None else f64(bias)), r


def residual_norm_error(x, residual, weight, bias, eps, rms, scale=None, alpha=1.0):
    terms = np.abs(alpha * f64(residual)) + np.abs(f64(x) * (1.0 if scale is None else f64(scale)))
    _, r = residual_norm(x, residual, weight, bias, eps, rms, scale, alpha)
    xhat, rstd = norm_rows(r, eps, rms)
    size = (terms.max(-1, keepdims=True) + terms) * rstd + np.abs(xhat)
    y = ROW * (size * (1.0 if weight is None else np.abs(f64(weight))) + (0.0 if bias is None else np.abs(f64(bias))))
    return y, 4 * U32 * terms


def residual_norm_backward(grad_y, grad_r, r, weight, eps, rms, x=None, scale=None, alpha=1.0):
    """(grad_x, grad_residual, grad_scale or None, grad_weight, grad_bias)."""
    dy, r = f64(grad_y), f64(r)
    xhat, rstd = norm_rows(r, eps, rms)
    t = norm_rows_backward(dy * (1.0 if weight is None else f64(weight)), xhat, rstd, rms)
    t = t if grad_r is None else t + f64(grad_r)
    lead = tuple(range(dy.ndim - 1))
    dscale = (t * f64(x)).sum(lead) if x is not None and scale is not None else None
    return (t * (1.0 if scale is None else f64(scale)), alpha * t, dscale, (dy * xhat).sum(lead), dy.sum(lead))


def residual_norm_backward_error(grad_y, grad_r, r, weight, eps, rms, x=None, scale=None, alpha=1.0):
    dy, r = f64(grad_y), f64(r)
    xhat, rstd = norm_rows(r, eps, rms)
    size = np.abs(r).max(-1, keepdims=True) * rstd + np.abs(xhat)
    e = norm_rows_backward_error(dy * (1.0 if weight is None else f64(weight)), r, xhat, rstd)
    t = norm_rows_backward(np.abs(dy) * (1.0 if weight is None else np.abs(f64(weight))), xhat, rstd, True)
    if grad_r is not None:
        t, e = np.abs(t) + np.abs(f64(grad_r)), e + 4 * U32 * np.abs(f64(grad_r))
    lead = tuple(range(dy.ndim - 1))
    rows = int(np.prod(dy.shape[:-1]))
    per = (rows + 96) * U32
    dscale = None
    if x is not None and scale is not None:
        dscale = (np.abs(f64(x)) * (e + per * np.abs(t))).sum(lead)
    return (e * (1.0 if scale is None else np.abs(f64(scale))), abs(alpha) * e, dscale,
            per * (np.abs(dy) * size).sum(lead), per * np.abs(dy).sum(lead))
