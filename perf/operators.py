"""Timing cases of the operators around retention in a gated recurrent block.

The gated recurrence (over sequences, its backward, one token per request) and
the two norms of the block (per head with the swish gate after the mixer,
residual and norm before the next block) with their backward passes. Each case
runs either in plain torch operations (``own`` false) or through the public
functions of retnet_retention_msr_amd (``own`` true); ``exact`` states what
each operator computes in 64 bits.

Formulas. Recurrence, per channel, with a gate value g per token:
  form "sigmoid": a = 1/(1 + e^-g), h_t = a_t h_{t-1} + (1 - a_t) x_t
  form "log":     a = e^g,          h_t = a_t h_{t-1} + x_t
Gated norm over the d outputs of a head: y = (norm(o) w + b) * g/(1 + e^-g).
Residual norm: r = alpha residual + scale x, y = norm(r) w + b. norm is the
layer form (mean and biased variance) or the root-mean-square form.
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-5
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # One decode step of the recurrence for a batch of eight requests at model width: latency.
        dict(name="step_b8", op="step", B=8, D=4096, slots=0, form="sigmoid", dtype="bf16"),
        # A full serving batch whose states live in a larger pool, picked by slot.
        dict(name="step_pool_b512", op="step", B=512, D=8192, slots=1024, form="log", dtype="bf16"),
        # Prefill of batch 8, 8k tokens, model width 4096 (16 heads of 256), final state out; x and gate are
        # the two halves of one projection's output.
        dict(name="scan_prefill", op="scan", B=8, H=0, N=8192, D=4096, form="sigmoid", dtype="bf16", fused=True, S=0),
        # One long sequence in the head layout of Q and K: few rows, so the time axis has to be split.
        dict(name="scan_long_heads", op="scan", B=1, H=16, N=65536, D=128, form="log", dtype="bf16", fused=False, S=0),
        # Ragged requests packed end to end (some empty), each with its own state in and out, odd width, fp32.
        dict(name="scan_packed", op="scan", B=1, H=0, N=30011, D=1001, form="sigmoid", dtype="f32", fused=False, S=37),
        # A training step (forward and backward) of batch 2, 2k tokens, width 2048 (8 heads of 256).
        dict(name="scan_train_mid", op="scan_train", B=2, H=0, N=2048, D=2048, form="sigmoid", dtype="bf16", fused=True),
        # A training step at model width over 8k tokens in the log form.
        dict(name="scan_train_large", op="scan_train", B=4, H=0, N=8192, D=4096, form="log", dtype="bf16", fused=False),
        # The norm and gate after the mixer at the prefill shape: 16 heads of 512, 8 x 8k tokens.
        dict(name="gnorm_prefill", op="gnorm", B=8, H=16, N=8192, D=512, rms=False, gate=True, affine=True, dtype="bf16"),
        # The same with its gradients in a training step of 8 heads, 2 x 2k tokens.
        dict(name="gnorm_train", op="gnorm_train", B=2, H=8, N=2048, D=512, rms=False, gate=True, affine=True, dtype="bf16"),
        # Heads of an odd width in fp32, root-mean-square form.
        dict(name="gnorm_train_odd", op="gnorm_train", B=3, H=5, N=777, D=97, rms=True, gate=True, affine=True, dtype="f32"),
        # Residual and norm before a block for the eight tokens of a decode step: latency.
        dict(name="rnorm_decode", op="rnorm", B=8, N=1, D=4096, rms=True, scale=False, alpha=1.0, stream="bf16", dtype="bf16"),
        # Residual and norm of a training step, forward and backward, with a per-channel branch scale and the
        # residual stream kept in fp32.
        dict(name="rnorm_train", op="rnorm_train", B=8, N=2048, D=4096, rms=False, scale=True, alpha=1.0, stream="f32", dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "scan", "scan", "scan_train", "gnorm", "gnorm_train", "rnorm", "rnorm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    form = rng.choice(["sigmoid", "log"])
    if op == "step":
        B = _spread(rng, 1, 512)
        return dict(op=op, B=B, D=_width(rng, 64, 8192), slots=rng.choice([0, B + _spread(rng, 1, 512)]), form=form, dtype=dtype)
    if op in ("scan", "scan_train"):
        most = 1 << (27 if op == "scan" else 26)  # values of x
        H = rng.choice([0, 0, _spread(rng, 1, 16)])
        D = _width(rng, 16, 256) if H else _width(rng, 64, 8192)
        N = min(_spread(rng, 1, 65536), most // (max(H, 1) * D))
        B = min(_spread(rng, 1, 64), max(1, most // (N * max(H, 1) * D)))
        fused = H == 0 and rng.random() < 0.5
        c = dict(op=op, B=B, H=H, N=N, D=D, form=form, dtype=dtype, fused=fused)
        if op == "scan":
            c["S"] = _spread(rng, 1, 64) if rng.random() < 0.4 else 0
            if c["S"]:
                c["B"] = 1
        return c
    rms = rng.random() < 0.5
    if op in ("gnorm", "gnorm_train"):
        most = 1 << (28 if op == "gnorm" else 26)
        H, D = _spread(rng, 1, 64), _width(rng, 16, 1024)
        N = min(_spread(rng, 1, 16384), max(1, most // (H * D)))
        B = min(_spread(rng, 1, 64), max(1, most // (N * H * D)))
        return dict(op=op, B=B, H=H, N=N, D=D, rms=rms, gate=rng.random() < 0.8, affine=rng.random() < 0.8, dtype=dtype)
    most = 1 << (27 if op == "rnorm" else 26)
    D = _width(rng, 64, 8192)
    N = min(_spread(rng, 1, 8192), max(1, most // D))
    B = min(_spread(rng, 1, 64), max(1, most // (N * D)))
    return dict(op=op, B=B, N=N, D=D, rms=rms, scale=rng.random() < 0.5, alpha=rng.choice([1.0, 1.0, 1.75]),
                stream=rng.choice([dtype, "f32"]), dtype=dtype)


def _width(rng, lo, hi):
    """A width: mostly a multiple of eight, sometimes odd."""
    d = _spread(rng, lo, hi)
    return d | 1 if rng.random() < 0.2 else max(8, d // 8 * 8)


# ---------------------------------------------------------------------------
# Inputs


def _offsets(S, T):
    """S lengths that add up to T, some of them zero, as S + 1 offsets; the same for every seed."""
    r = np.random.RandomState(S * 7919 + T)
    share = r.exponential(size=S) * (r.random(S) > 0.1) + 1e-9
    cu = np.floor(np.cumsum(share) / share.sum() * T).astype(np.int64)
    cu[-1] = T
    return np.concatenate([[0], cu])


def _gates(case, shape, gen):
    """Gate values: pre-activations that keep 0.88 to 0.99 of the state, or decays whose memory is 2 to 500 tokens."""
    if case["form"] == "sigmoid":
        return torch.randn(shape, generator=gen, device=DEV) + 3.0
    return -torch.exp(torch.rand(shape, generator=gen, device=DEV) * 5.5 - 6.2)


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    T = TYPES[case["dtype"]]

    def randn(*shape, dtype=T):
        return torch.randn(shape, generator=gen, device=DEV).to(dtype)

    s = dict(case=case)
    op, D = case["op"], case["D"]
    if op == "step":
        B = case["B"]
        P = case["slots"] or B
        s["x"], s["gate"] = randn(B, D), _gates(case, (B, D), gen).to(T)
        s["state"] = randn(P, D, dtype=torch.float32)
        s["slots"] = torch.randperm(P, generator=gen, device=DEV)[:B].to(torch.int32) if case["slots"] else None
        return s
    if op in ("scan", "scan_train"):
        B, H, N = case["B"], case["H"], case["N"]
        lead = (B, H) if H else (B,)
        if case["fused"]:
            both = torch.empty(*lead, N, 2 * D, dtype=T, device=DEV)
            s["x"], s["gate"] = both[..., :D], both[..., D:]
            s["x"].copy_(torch.randn(*lead, N, D, generator=gen, device=DEV))
            s["gate"].copy_(_gates(case, (*lead, N, D), gen))
        else:
            s["x"], s["gate"] = randn(*lead, N, D), _gates(case, (*lead, N, D), gen).to(T)
        S = case.get("S", 0)
        states = (S or B, H, D) if H else (S or B, D)
        s["state_in"] = randn(*states, dtype=torch.float32) if S else None
        if S:
            cu = _offsets(S, N)
            s["cu"] = torch.from_numpy(cu.astype(np.int32)).to(DEV)
            s["max_len"] = int((cu[1:] - cu[:-1]).max())
        if op == "scan_train":
            s["dh"] = randn(*lead, N, D)
            s["dstate"] = randn(*states, dtype=torch.float32)
        return s
    if op in ("gnorm", "gnorm_train"):
        B, H, N = case["B"], case["H"], case["N"]
        s["o"] = randn(B, H, N, D)
        s["gate"] = (2 * torch.randn(B, H, N, D, generator=gen, device=DEV)).to(T) if case["gate"] else None
        s["w"] = 1 + 0.25 * randn(H * D, dtype=torch.float32) if case["affine"] else None
        s["b"] = 0.1 * randn(H * D, dtype=torch.float32) if case["affine"] else None
        if op == "gnorm_train":
            s["dy"] = randn(B, H, N, D)
        return s
    B, N = case["B"], case["N"]
    stream = TYPES[case["stream"]]
    s["x"], s["res"] = randn(B, N, D), randn(B, N, D, dtype=stream)
    s["w"], s["b"] = 1 + 0.25 * randn(D, dtype=torch.float32), 0.1 * randn(D, dtype=torch.float32)
    s["scale"] = 0.5 + 0.1 * randn(D, dtype=torch.float32) if case["scale"] else None
    if op == "rnorm_train":
        s["dy"], s["dr"] = randn(B, N, D), randn(B, N, D, dtype=stream)
    return s


# ---------------------------------------------------------------------------
# The plain form: torch operations in 32 bits, rounded once at the end


def _keep(g, form):
    """(a, what x is multiplied by) of the gate values."""
    if form == "sigmoid":
        return torch.sigmoid(g), torch.sigmoid(-g)
    return torch.exp(g), None


def _scan(a, b):
    """y_t = a_t y_{t-1} + b_t along the last axis but one, y_{-1} = 0, by doubling steps."""
    k, n = 1, a.shape[-2]
    while k < n:
        b = torch.cat((b[..., :k, :], b[..., k:, :] + a[..., k:, :] * b[..., :-k, :]), -2)
        a = torch.cat((a[..., :k, :], a[..., k:, :] * a[..., :-k, :]), -2)
        k *= 2
    return b


def _plain_step(s):
    form, T = s["case"]["form"], s["x"].dtype
    a, c = _keep(s["gate"].float(), form)
    x = s["x"].float()
    x = x if c is None else c * x
    if s["slots"] is None:
        s["state"].mul_(a).add_(x)
        return s["state"].to(T), s["state"]
    at = s["slots"].long()
    h = a * s["state"][at] + x
    s["state"][at] = h
    return h.to(T), s["state"]


def _plain_scan(s):
    """(h in 32 bits, final states)."""
    a, c = _keep(s["gate"].float(), s["case"]["form"])
    b = s["x"].float()
    b = b if c is None else c * b
    if s["state_in"] is None:
        h = _scan(a, b)
        return h, h[..., -1, :].clone()
    cu = s["cu"].long()
    some = (cu[1:] > cu[:-1]).nonzero()[:, 0]  # the sequences that hold a token
    first = cu[:-1][some]
    start = s["state_in"][some].movedim(0, -2)  # [(H,) sequences, D]
    b[0, ..., first, :] += a[0, ..., first, :] * start
    a[0, ..., first, :] = 0
    h = _scan(a, b)
    last = (cu[1:] - 1).clamp(min=0)
    ends = h[0, ..., last, :].movedim(-2, 0)
    empty = (cu[1:] == cu[:-1]).reshape(-1, *[1] * (ends.dim() - 1))
    return h, torch.where(empty, s["state_in"], ends)


def _plain_scan_backward(s, h):
    a, c = _keep(s["gate"].float(), s["case"]["form"])
    dh = s["dh"].float()
    start = torch.zeros_like(h[..., :1, :])
    b = a * dh
    b[..., -1, :] += a[..., -1, :] * s["dstate"]
    w = _scan(a.flip(-2), b.flip(-2)).flip(-2)
    u = dh + torch.cat((w[..., 1:, :], s["dstate"].unsqueeze(-2)), -2)
    before = torch.cat((start, h[..., :-1, :]), -2)
    T = s["x"].dtype
    if c is None:
        return u.to(T), (u * before * a).to(T), w[..., 0, :]
    return (u * c).to(T), (u * (before - s["x"].float()) * a * c).to(T), w[..., 0, :]


def _plain_norm(r, rms):
    """(the normalised rows, 1 over their deviation)."""
    mean = 0 if rms else r.mean(-1, keepdim=True)
    d = r - mean
    rstd = (d.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return d * rstd, rstd


def _plain_norm_back(g, xhat, rstd, rms):
    t = g - xhat * (g * xhat).mean(-1, keepdim=True)
    return rstd * (t if rms else t - g.mean(-1, keepdim=True))


def _by_head(s, key):
    c = s["case"]
    return None if s[key] is None else s[key].view(c["H"], 1, c["D"])


def _plain_gnorm(s):
    xhat, _ = _plain_norm(s["o"].float(), s["case"]["rms"])
    if s["w"] is not None:
        xhat = xhat * _by_head(s, "w") + _by_head(s, "b")
    if s["gate"] is not None:
        g = s["gate"].float()
        xhat = xhat * (g * torch.sigmoid(g))
    return xhat.to(s["o"].dtype)


def _plain_gnorm_backward(s):
    T, rms = s["o"].dtype, s["case"]["rms"]
    xhat, rstd = _plain_norm(s["o"].float(), rms)
    dz, dgate, dw, db = s["dy"].float(), None, None, None
    z = xhat if s["w"] is None else xhat * _by_head(s, "w") + _by_head(s, "b")
    if s["gate"] is not None:
        g = s["gate"].float()
        sg = torch.sigmoid(g)
        dgate = (dz * z * (sg * (1 + g * (1 - sg)))).to(T)
        dz = dz * (g * sg)
    if s["w"] is not None:
        dw, db = (dz * xhat).sum((0, 2)).reshape(-1), dz.sum((0, 2)).reshape(-1)
        dz = dz * _by_head(s, "w")
    return _plain_norm_back(dz, xhat, rstd, rms).to(T), dgate, dw, db


def _plain_rnorm(s):
    x, res = s["x"].float(), s["res"].float()
    r = s["case"]["alpha"] * res + (x if s["scale"] is None else s["scale"] * x)
    xhat, _ = _plain_norm(r, s["case"]["rms"])
    return (xhat * s["w"] + s["b"]).to(s["x"].dtype), r


def _plain_rnorm_backward(s, r):
    rms, T = s["case"]["rms"], s["x"].dtype
    xhat, rstd = _plain_norm(r, rms)
    dy = s["dy"].float()
    t = s["dr"].float() + _plain_norm_back(dy * s["w"], xhat, rstd, rms)
    dscale = None if s["scale"] is None else (t * s["x"].float()).sum((0, 1))
    dx = t if s["scale"] is None else t * s["scale"]
    return dx.to(T), (s["case"]["alpha"] * t).to(s["res"].dtype), dscale, (dy * xhat).sum((0, 1)), dy.sum((0, 1))


def _run_plain(s):
    op = s["case"]["op"]
    if op == "step":
        return _plain_step(s)
    if op == "scan":
        h, state = _plain_scan(s)
        return h.to(s["x"].dtype), state
    if op == "scan_train":
        h, state = _plain_scan(s)
        return (h.to(s["x"].dtype), state, *_plain_scan_backward(s, h))
    if op == "gnorm":
        return _plain_gnorm(s)
    if op == "gnorm_train":
        return (_plain_gnorm(s), *_plain_gnorm_backward(s))
    y, r = _plain_rnorm(s)
    if op == "rnorm":
        return y, r.to(s["res"].dtype)
    return (y, r.to(s["res"].dtype), *_plain_rnorm_backward(s, r))


# ---------------------------------------------------------------------------
# The framework's operators


def _run_own(s):
    import retnet_retention_msr_amd as ret

    c = s["case"]
    op = c["op"]
    if op == "step":
        return ret.gated_recurrence_step(s["x"], s["gate"], s["state"], form=c["form"], slots=s["slots"]), s["state"]
    if op == "scan":
        return ret.gated_recurrence(s["x"], s["gate"], form=c["form"], state_in=s["state_in"], state_out=True,
                                    cu_seqlens=s.get("cu"), max_len=s.get("max_len"))
    if op == "scan_train":
        h, state = ret.gated_recurrence(s["x"], s["gate"], form=c["form"], state_out=True)
        return (h, state, *ret.gated_recurrence_backward(s["dh"], s["x"], s["gate"], h, form=c["form"],
                                                         grad_state_out=s["dstate"], grad_state_in=True))
    norm = ret.Norm(EPS, s["w"], s["b"], rms=c["rms"])
    if op == "gnorm":
        return ret.gated_norm(s["o"], s["gate"], norm)
    if op == "gnorm_train":
        return (ret.gated_norm(s["o"], s["gate"], norm), *ret.gated_norm_backward(s["dy"], s["o"], s["gate"], norm))
    y, r = ret.residual_norm(s["x"], s["res"], norm, scale=s["scale"], alpha=c["alpha"])
    if op == "rnorm":
        return y, r
    # A bf16 r carries its rounding into the parameters' fp32 gradients; x and the residual give them exactly.
    residual = s["res"] if s["res"].dtype != torch.float32 else None
    return (y, r, *ret.residual_norm_backward(s["dy"], r, norm, grad_r=s["dr"], x=s["x"], scale=s["scale"],
                                              alpha=c["alpha"], residual=residual))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without


def work(case):
    op, e, D = case["op"], SIZE[case["dtype"]], case["D"]
    if op == "step":
        n = case["B"] * D
        return {"bytes": n * (3 * e + 8) + (4 * case["B"] if case["slots"] else 0), "flops": 7 * n}
    if op in ("scan", "scan_train"):
        heads = max(case["H"], 1)
        n = case["B"] * heads * case["N"] * D
        S = case.get("S", 0)
        state = (S or case["B"]) * heads * D * 4
        if op == "scan":
            return {"bytes": 3 * e * n + (2 * state + 4 * (S + 1) if S else state), "flops": 8 * n}
        back = 6 if case["form"] == "sigmoid" else 5
        return {"bytes": (3 + back) * e * n + 3 * state, "flops": 22 * n}
    if op in ("gnorm", "gnorm_train"):
        n = case["B"] * case["H"] * case["N"] * D
        gate, par = int(case["gate"]), 8 * case["H"] * D * int(case["affine"])
        fwd = (2 + gate) * e * n + par
        if op == "gnorm":
            return {"bytes": fwd, "flops": 14 * n}
        return {"bytes": fwd + (3 + 2 * gate) * e * n + 2 * par, "flops": 45 * n}
    n, er = case["B"] * case["N"] * D, SIZE[case["stream"]]
    fwd = (2 * e + 2 * er) * n + 8 * D + 4 * D * int(case["scale"])
    if op == "rnorm":
        return {"bytes": fwd, "flops": 10 * n}
    return {"bytes": fwd + (2 * e + 3 * er + e * int(case["scale"])) * n + 16 * D + 8 * D * int(case["scale"]), "flops": 35 * n}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, token by token and through autograd


def exact(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
         for k, v in prepare(case, seed).items()}
    op = case["op"]
    if op in ("step", "scan", "scan_train"):
        a = 1 / (1 + torch.exp(-s["gate"])) if case["form"] == "sigmoid" else torch.exp(s["gate"])
        one_less = 1 / (1 + torch.exp(s["gate"])) if case["form"] == "sigmoid" else torch.ones_like(a)
        del s["gate"]
    if op == "step":
        at = s["slots"].long() if s["slots"] is not None else torch.arange(case["B"], device=DEV)
        h = a * s["state"][at] + one_less * s["x"]
        state = s["state"].clone()
        state[at] = h
        return h, state
    if op in ("scan", "scan_train"):
        return _exact_scan(case, s, a, one_less)
    if op in ("gnorm", "gnorm_train"):
        leaves = [s[k].requires_grad_(op == "gnorm_train") for k in ("o", "gate", "w", "b") if s[k] is not None]
        z = _exact_norm(s["o"], case["rms"])
        if case["affine"]:
            z = z * s["w"].view(case["H"], 1, -1) + s["b"].view(case["H"], 1, -1)
        y = z * s["gate"] / (1 + torch.exp(-s["gate"])) if case["gate"] else z
        if op == "gnorm":
            return y
        grads = list(torch.autograd.grad(y, leaves, s["dy"]))
        return (y.detach(), grads.pop(0), grads.pop(0) if case["gate"] else None, *(grads or (None, None)))
    leaves = [s[k].requires_grad_(op == "rnorm_train") for k in ("x", "res", "scale", "w", "b") if s[k] is not None]
    r = case["alpha"] * s["res"] + (s["x"] * s["scale"] if case["scale"] else s["x"])
    y = _exact_norm(r, case["rms"]) * s["w"] + s["b"]
    if op == "rnorm":
        return y, r
    grads = list(torch.autograd.grad([y, r], leaves, [s["dy"], s["dr"]]))
    return (y.detach(), r.detach(), grads[0], grads[1], grads[2] if case["scale"] else None, *grads[-2:])


def _exact_norm(r, rms):
    if rms:
        return r / torch.sqrt((r * r).mean(-1, keepdim=True) + EPS)
    return (r - r.mean(-1, keepdim=True)) / torch.sqrt(r.var(-1, unbiased=False, keepdim=True) + EPS)


def _exact_scan(case, s, a, one_less):
    x, N = s["x"], case["N"]
    h = torch.empty_like(x)
    S = case.get("S", 0)
    if S:
        cu = [int(c) for c in _offsets(S, N)]
        ends = s["state_in"].clone()
        for i in range(S):
            for t in range(cu[i], cu[i + 1]):
                ends[i] = a[0, ..., t, :] * ends[i] + one_less[0, ..., t, :] * x[0, ..., t, :]
                h[0, ..., t, :] = ends[i]
        return h, ends
    b = one_less * x
    at, now = a.movedim(-2, 0), torch.zeros_like(x[..., 0, :])
    for t, (at_t, b_t) in enumerate(zip(at.unbind(0), b.movedim(-2, 0).unbind(0))):
        now = torch.addcmul(b_t, at_t, now)
        h[..., t, :] = now
    if case["op"] == "scan":
        return h, now
    u = torch.empty_like(x)
    carried = s["dstate"]
    for t in range(N - 1, -1, -1):
        u[..., t, :] = s["dh"][..., t, :] + carried
        carried = at[t] * u[..., t, :]
    before = torch.cat((torch.zeros_like(h[..., :1, :]), h[..., :-1, :]), -2)
    if case["form"] == "log":
        return h, now, u, u * a * before, carried
    return h, now, u * one_less, u * a * one_less * (before - x), carried
