"""GPU parity of the block operators (gated recurrence, gated norm, residual norm and their gradients) with the fp64 oracle.

Tolerance of an element: half a step of the output's type relative to the value (bf16 2^-8, fp32 2^-24), plus the bound
that the oracle's ``*_error`` functions derive for the operator's fp32 arithmetic, plus 2^-120 for what underflows.
"""

import numpy as np
import pytest
import torch

import retnet_retention_msr_amd as ret
from oracle import block_oracle as orc
from oracle import retention_oracle as rorc
from retnet_retention_msr_amd import synthetic

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def _announce(msg):
    print(f"[case] {msg}", flush=True)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(shape, seed, dtype=F32, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=_gen(seed)) * std + mean).to(dtype)


def _gate(shape, seed, dtype, form):
    """Pre-activations around 2 or log decays with memories from a token to a few hundred; a few -inf (a = 0) and, in the
    sigmoid form, +inf (a = 1)."""
    g = _randn(shape, seed, F32, 2.0, 2.0) if form == "sigmoid" else -torch.exp(_randn(shape, seed, F32, 2.0, -3.0))
    flat = g.view(-1)
    flat[:: 97] = -float("inf")
    if form == "sigmoid":
        flat[5:: 131] = float("inf")
    return g.to(dtype)


def _check(got, ref, err, what):
    half = torch.finfo(got.dtype).eps / 2
    g, err = orc.f64(got), np.broadcast_to(err, ref.shape)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert np.all(np.isfinite(g)), (what, "not finite")
    if not g.size:
        return
    over = np.abs(g - ref) - (half * (np.abs(ref) + err) + err + 2.0 ** -120)
    i = np.unravel_index(np.argmax(over), over.shape)
    assert over[i] <= 0, f"{what} at {i}: {g[i]!r}, not {ref[i]!r} (allowed {err[i] + half * abs(ref[i]):.3e})"


def _strided(t, seed):
    """The same values as columns of a wider tensor, starting at an odd column."""
    wide = torch.full((*t.shape[:-1], 2 * t.shape[-1] + 3), float("nan"), dtype=t.dtype, device=DEV)
    view = wide[..., 3: 3 + t.shape[-1]]
    view.copy_(t)
    return view


# ---------------------------------------------------------------------------
# Gated recurrence

# Lengths around the pieces that a sequence is cut into (waves of 8, 16 or 32 tokens, workgroups of up to 256), widths
# around the 64 channels of a workgroup and the vector widths.
SHAPES = [
    ((1, 1, 1), "sigmoid", BF16), ((1, 1, 1), "log", F32), ((3, 2, 8), "log", BF16), ((2, 31, 64), "sigmoid", BF16),
    ((1, 32, 72), "log", F32), ((1, 33, 65), "sigmoid", F32), ((2, 63, 3), "log", BF16), ((1, 64, 64), "sigmoid", BF16),
    ((2, 65, 40), "sigmoid", F32), ((1, 127, 96), "log", BF16), ((1, 255, 24), "sigmoid", BF16),
    ((2, 256, 128), "log", F32), ((1, 257, 64), "log", BF16), ((1, 511, 33), "sigmoid", BF16),
    ((1, 513, 16), "sigmoid", F32), ((3, 1000, 200), "sigmoid", BF16), ((1, 2049, 70), "log", BF16),
    ((1, 5000, 64), "sigmoid", BF16), ((1, 4097, 8), "log", F32), ((2, 3, 77, 24), "sigmoid", BF16),
    ((1, 16, 700, 64), "log", BF16), ((2, 5, 300, 7), "sigmoid", F32), ((1, 700, 5), "log", BF16), ((2, 500, 3), "sigmoid", F32),
    ((260, 270, 64), "sigmoid", BF16), ((87, 3, 400, 24), "log", F32),
]


def _states(shape):
    return (*shape[:-2], shape[-1])


@pytest.mark.parametrize("shape, form, dtype", SHAPES)
@pytest.mark.parametrize("strided", [False, True])
def test_recurrence_matches_the_oracle(shape, form, dtype, strided):
    _announce(f"recurrence {shape} {form} {dtype} strided={strided}")
    x, g = _randn(shape, 1, dtype), _gate(shape, 2, dtype, form)
    s0 = _randn(_states(shape), 3) if strided else None
    place = (lambda t: _strided(t, 0)) if strided else (lambda t: t.to(DEV))
    h, s1 = ret.gated_recurrence(place(x), place(g), form, state_in=None if s0 is None else s0.to(DEV), state_out=True)
    torch.cuda.synchronize()
    ref, end = orc.recurrence(x, g, form, s0)
    e, e_end = orc.recurrence_error(x, g, form, s0)
    _check(h, ref, e, "h")
    _check(s1, end, e_end, "state")


@pytest.mark.parametrize("shape, form, dtype", SHAPES)
@pytest.mark.parametrize("strided", [False, True])
def test_recurrence_backward_matches_the_oracle(shape, form, dtype, strided):
    _announce(f"recurrence backward {shape} {form} {dtype} strided={strided}")
    x, g, dh = _randn(shape, 1, dtype), _gate(shape, 2, dtype, form), _randn(shape, 4, dtype)
    s0, ds = (_randn(_states(shape), 3), _randn(_states(shape), 5)) if strided else (None, None)
    h = torch.from_numpy(orc.recurrence(x, g, form, s0)[0]).to(dtype)
    place = (lambda t: _strided(t, 0)) if strided else (lambda t: t.to(DEV))
    dev = [None if t is None else t.to(DEV) for t in (s0, ds)]
    dx, dg, ds0 = ret.gated_recurrence_backward(place(dh), place(x), place(g), place(h), form, state_in=dev[0],
                                                grad_state_out=dev[1], grad_state_in=True)
    torch.cuda.synchronize()
    refs = orc.recurrence_backward(dh, x, g, h, form, s0, ds)
    errs = orc.recurrence_backward_error(dh, x, g, h, form, s0, ds)
    for got, ref, e, what in zip((dx, dg, ds0), refs, errs, ("grad_x", "grad_gate", "grad_state_in")):
        _check(got, ref, e, what)


def test_the_gradients_are_those_of_differences_of_the_forward():
    """In fp32, a step along a random direction changes the kernel's own outputs by what its gradients say."""
    shape, form = (1, 300, 64), "sigmoid"
    _announce("recurrence gradients against differences")
    x, g, dh = (_randn(shape, s).to(DEV) for s in (11, 12, 13))
    s0, ds = _randn((1, 64), 14).to(DEV), _randn((1, 64), 15).to(DEV)
    dirs = [_randn(shape, 16).to(DEV), _randn(shape, 17).to(DEV), _randn((1, 64), 18).to(DEV)]
    h, _ = ret.gated_recurrence(x, g, form, state_in=s0)
    grads = ret.gated_recurrence_backward(dh, x, g, h, form, state_in=s0, grad_state_out=ds, grad_state_in=True)

    def loss(k, eps):
        at = [x, g, s0]
        at[k] = at[k] + eps * dirs[k]
        y, end = ret.gated_recurrence(at[0], at[1], form, state_in=at[2], state_out=True)
        return ((y.double() * dh).sum() + (end.double() * ds).sum()).item()

    # Central differences of step e err by O(e^2) of the third derivative and by the outputs' fp32 roundings over e:
    # 2^-24 * sqrt(19200 terms) * a few / 2e = 3e-3 at e = 2^-8, against directional derivatives of order 100.
    for k in range(3):
        e = 2.0 ** -8
        slope = (loss(k, e) - loss(k, -e)) / (2 * e)
        want = (grads[k].double() * dirs[k]).sum().item()
        assert abs(slope - want) <= 2e-2 + 1e-3 * abs(want), (k, slope, want)


@pytest.mark.parametrize("dtype, form, d, heads", [(BF16, "sigmoid", 72, 0), (F32, "log", 33, 0), (BF16, "log", 64, 3)])
def test_packed_sequences(dtype, form, d, heads):
    """Ragged sequences, some empty, in one row with rows before, behind and (past max_len) between them that stay as
    they were; against each sequence on its own."""
    _announce(f"packed {dtype} {form} d={d} heads={heads}")
    lens = [5, 0, 700, 1, 64, 0, 300, 2, 0]
    cu = np.concatenate([[3], 3 + np.cumsum(lens)])
    T, max_len = int(cu[-1]) + 9, 520  # the sequence of 700 is cut at 520
    lead = (1, heads) if heads else (1,)
    shape = (*lead, T, d)
    x, g, dh = _randn(shape, 1, dtype), _gate(shape, 2, dtype, form), _randn(shape, 3, dtype)
    S = len(lens)
    states = (S, heads, d) if heads else (S, d)
    s0, ds = _randn(states, 4), _randn(states, 5)
    mark = 7.5
    out = torch.full(shape, mark, dtype=dtype, device=DEV)
    grads = [torch.full(shape, mark, dtype=dtype, device=DEV) for _ in range(2)]
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    dev = [t.to(DEV) for t in (x, g, s0, dh, ds)]
    _, s1 = ret.gated_recurrence(dev[0], dev[1], form, state_in=dev[2], state_out=True, cu_seqlens=cud, max_len=max_len, out=out)
    _, _, ds0 = ret.gated_recurrence_backward(dev[3], dev[0], dev[1], out, form, state_in=dev[2], grad_state_out=dev[4],
                                              grad_state_in=True, cu_seqlens=cud, max_len=max_len, grads=grads)
    torch.cuda.synchronize()
    left = torch.ones(T, dtype=torch.bool)
    for i in range(S):
        a, b = int(cu[i]), int(cu[i]) + min(lens[i], max_len)
        left[a:b] = False
        at = (0, Ellipsis, slice(a, b), slice(None))
        args = (x[at], g[at], form, s0[i])
        ref, end = orc.recurrence(*args)
        e, e_end = orc.recurrence_error(*args)
        _check(s1[i], end, e_end, f"state {i}")
        h = out[at].cpu()
        _check(h, ref, e, f"h {i}")
        bargs = (dh[at], x[at], g[at], h, form, s0[i], ds[i])
        for got, r, e, what in zip((grads[0][at], grads[1][at], ds0[i]), orc.recurrence_backward(*bargs),
                                   orc.recurrence_backward_error(*bargs), ("grad_x", "grad_gate", "grad_state_in")):
            _check(got, r, e, f"{what} {i}")
    for t in (out, *grads):
        assert bool((t.cpu()[..., left, :] == mark).all())


@pytest.mark.parametrize("S, longest", [(70, 900), (300, 300), (4200, 9)])
def test_many_packed_sequences(S, longest):
    """More sequences than a wave has lanes (and than its square), a few longer than a tile: the result is that of the
    rows padded to one length."""
    _announce(f"{S} packed sequences")
    d, rng = 24, np.random.default_rng(S)
    lens = rng.integers(0, 6, S)
    lens[rng.integers(0, S, 5)] = longest
    cu = np.concatenate([[0], np.cumsum(lens)])
    T, most = int(cu[-1]), int(lens.max())
    x, g, dh = _randn((1, T, d), 1), _gate((1, T, d), 2, F32, "log"), _randn((1, T, d), 3)
    s0, ds = _randn((S, d), 4).to(DEV), _randn((S, d), 5).to(DEV)
    pad = np.full((S, most), T)
    for i in range(S):
        pad[i, :lens[i]] = np.arange(cu[i], cu[i + 1])
    at = torch.from_numpy(pad)
    rows = [torch.cat((t[0], torch.zeros(1, d)))[at].to(DEV) for t in (x, g, dh)]  # padding: a = 1, x = 0 keep the state
    h_pad, s_pad = ret.gated_recurrence(rows[0], rows[1], "log", state_in=s0, state_out=True)
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    dev = [t.to(DEV) for t in (x, g, dh)]
    h, s1 = ret.gated_recurrence(dev[0], dev[1], "log", state_in=s0, state_out=True, cu_seqlens=cud)
    dx, dg, ds0 = ret.gated_recurrence_backward(dev[2], dev[0], dev[1], h, "log", state_in=s0, grad_state_out=ds,
                                                grad_state_in=True, cu_seqlens=cud, max_len=most)
    back = ret.gated_recurrence_backward(rows[2], rows[0], rows[1], h_pad, "log", state_in=s0, grad_state_out=ds, grad_state_in=True)
    torch.cuda.synchronize()
    live = at < T
    # Both are the same recurrences in another tiling: twice the bound of one.
    e, e_end = orc.recurrence_error(rows[0].cpu(), rows[1].cpu(), "log", s0.cpu())
    _check(h[0], orc.f64(h_pad)[live.numpy()], 2 * e[live.numpy()], "h")
    _check(s1, orc.f64(s_pad), 2 * e_end, "state")
    errs = orc.recurrence_backward_error(rows[2].cpu(), rows[0].cpu(), rows[1].cpu(), h_pad.cpu(), "log", s0.cpu(), ds.cpu())
    # grad_gate also takes the h of its own call, which differs by up to 2 e.
    dh_err = 2 * np.concatenate((np.zeros((S, 1, d)), e[:, :-1]), 1) * np.abs(orc.f64(back[0])) * orc.decay(rows[1].cpu(), "log")[0]
    _check(dx[0], orc.f64(back[0])[live.numpy()], 2 * errs[0][live.numpy()], "grad_x")
    _check(dg[0], orc.f64(back[1])[live.numpy()], (2 * errs[1] + dh_err)[live.numpy()], "grad_gate")
    _check(ds0, orc.f64(back[2]), 2 * errs[2], "grad_state_in")


def test_offsets_out_of_range_are_clamped():
    _announce("offsets out of range")
    T, d = 40, 16
    x, g = _randn((1, T, d), 1).to(DEV), _gate((1, T, d), 2, F32, "log").to(DEV)
    cu = torch.tensor([-5, 10, 25, 1000], dtype=torch.int32, device=DEV)
    right = torch.tensor([0, 10, 25, 40], dtype=torch.int32, device=DEV)
    h, s = ret.gated_recurrence(x, g, "log", state_out=True, cu_seqlens=cu)
    h2, s2 = ret.gated_recurrence(x, g, "log", state_out=True, cu_seqlens=right)
    assert torch.equal(h, h2) and torch.equal(s, s2)


def test_gates_of_every_size():
    """Gates from -95 to 95, through those whose e^-g or whose decay leaves fp32's normal numbers (a product with such a
    decay may be 0: off by less than 2^-126 times its other factors, here below 8), in the recurrence, its backward, its
    step and the norm's gate."""
    _announce("gates of every size")
    g = torch.linspace(-95, 95, 1901).view(1, 1, -1)
    x, dh, s0 = _randn(g.shape, 1), _randn(g.shape, 2), _randn((1, 1901), 3)
    dev = [t.to(DEV) for t in (x, g, dh, s0)]
    tiny = 2.0 ** -123
    for form, gate in (("sigmoid", g), ("log", -g.abs())):
        gd = gate.to(DEV)
        h, s1 = ret.gated_recurrence(dev[0], gd, form, state_in=dev[3], state_out=True)
        (ref, _), (e, _) = orc.recurrence(x, gate, form, s0), orc.recurrence_error(x, gate, form, s0)
        _check(h, ref, e + tiny, "h")
        state = dev[3].clone()
        step = ret.gated_recurrence_step(dev[0][0], gd[0], state, form)
        _check(step[None], ref, e + tiny, "step")
        assert torch.equal(state, step) and torch.equal(s1, h[:, 0])
        got = ret.gated_recurrence_backward(dev[2], dev[0], gd, h, form, state_in=dev[3], grad_state_in=True)
        refs = orc.recurrence_backward(dh, x, gate, h.cpu(), form, s0, None)
        errs = orc.recurrence_backward_error(dh, x, gate, h.cpu(), form, s0, None)
        for t, r, e, what in zip(got, refs, errs, ("grad_x", "grad_gate", "grad_state_in")):
            _check(t, r, e + tiny, what)
    # The norm's gate multiplies such a decay by the gate itself (below 2^6.5) and by factors below 2^6 together.
    tiny = 2.0 ** -113
    shape = (1, 2, 1, 950)
    gate, o, dy = g.reshape(-1)[:1900].view(shape), _randn(shape, 4), _randn(shape, 5)
    norm = ret.Norm(EPS)
    args = (o, gate, None, None, EPS, False)
    _check(ret.gated_norm(o.to(DEV), gate.to(DEV), norm), orc.gated_norm(*args), orc.gated_norm_error(*args) + tiny, "y")
    got = ret.gated_norm_backward(dy.to(DEV), o.to(DEV), gate.to(DEV), norm)
    refs, errs = orc.gated_norm_backward(dy, *args), orc.gated_norm_backward_error(dy, *args)
    for t, r, e, what in zip(got[:2], refs, errs, ("grad_o", "grad_gate")):
        _check(t, r, e + tiny, what)


def test_states_in_place_and_fused_gradient_buffers():
    """state_out may be state_in, grad_state_in grad_state_out, and the gradients two halves of one tensor."""
    _announce("states in place")
    shape, form = (2, 1500, 64), "sigmoid"
    x, g, dh = _randn(shape, 1, BF16).to(DEV), _gate(shape, 2, BF16, form).to(DEV), _randn(shape, 3, BF16).to(DEV)
    s0, ds = _randn((2, 64), 4).to(DEV), _randn((2, 64), 5).to(DEV)
    h, s1 = ret.gated_recurrence(x, g, form, state_in=s0, state_out=True)
    again = s0.clone()
    h2, _ = ret.gated_recurrence(x, g, form, state_in=again, state_out=again)
    assert torch.equal(h, h2) and torch.equal(again, s1)
    dx, dg, ds0 = ret.gated_recurrence_backward(dh, x, g, h, form, state_in=s0, grad_state_out=ds, grad_state_in=True)
    both, same = torch.empty(2, 1500, 128, dtype=BF16, device=DEV), ds.clone()
    ret.gated_recurrence_backward(dh, x, g, h, form, state_in=s0, grad_state_out=same, grad_state_in=same,
                                  grads=(both[..., :64], both[..., 64:]))
    assert torch.equal(both[..., :64], dx) and torch.equal(both[..., 64:], dg) and torch.equal(same, ds0)


def test_broadcast_gate():
    """One gate for all rows of the batch (stride 0): the full gradient's sum over the rows is the gate's."""
    _announce("broadcast gate")
    shape = (3, 90, 64)
    x, dh = _randn(shape, 1).to(DEV), _randn(shape, 2).to(DEV)
    g1 = _gate((1, 90, 64), 3, F32, "sigmoid").to(DEV)
    h, _ = ret.gated_recurrence(x, g1.expand(shape), "sigmoid")
    want, _ = ret.gated_recurrence(x, g1.expand(shape).contiguous(), "sigmoid")
    assert torch.equal(h, want)
    _, dg, _ = ret.gated_recurrence_backward(dh, x, g1.expand(shape), h, "sigmoid")
    _, ref, _ = ret.gated_recurrence_backward(dh, x, g1.expand(shape).contiguous(), h, "sigmoid")
    assert dg.shape == shape and torch.equal(dg, ref)


def test_nan_stays_with_its_channel_sequence_and_later_tokens():
    """A NaN input reaches the tokens from its own on in its own channel, however they are cut into pieces, and nothing
    else; its bits do not matter (all ones is what the library's own words hold before they are written)."""
    _announce("nan")
    B, N, D = 2, 3000, 72
    x, g = _randn((B, N, D), 1), _gate((B, N, D), 2, F32, "log").clamp_(min=-5)
    want, s_want = ret.gated_recurrence(x.to(DEV), g.to(DEV), "log", state_out=True)
    bad = x.clone()
    bad[1, 1000, 7] = torch.tensor(-1, dtype=torch.int32).view(F32)
    h, s = ret.gated_recurrence(bad.to(DEV), g.to(DEV), "log", state_out=True)
    hit = torch.zeros(B, N, D, dtype=torch.bool)
    hit[1, 1000:, 7] = True
    assert torch.equal(h.isnan().cpu(), hit) and torch.equal(h[~hit], want[~hit])
    assert s.isnan().nonzero().tolist() == [[1, 7]]
    dh = torch.zeros(B, N, D)
    dh[1, 1000, 7] = float("nan")
    dx, dg, ds = ret.gated_recurrence_backward(dh.to(DEV), x.to(DEV), g.to(DEV), want, "log", grad_state_in=True)
    assert dx.isnan().nonzero().shape[0] == 1001 and bool(dx[1, :1001, 7].isnan().all())
    assert ds.isnan().nonzero().tolist() == [[1, 7]] and bool((dx[0] == 0).all())


def test_a_workspace_serves_any_contents_and_both_directions():
    _announce("workspace")
    for shape, form in (((1, 3000, 64), "sigmoid"), ((260, 300, 64), "log")):
        x, g, dh = _randn(shape, 1).to(DEV), _gate(shape, 2, F32, form).to(DEV), _randn(shape, 3).to(DEV)
        want = ret.gated_recurrence(x, g, form, state_out=True)
        back = ret.gated_recurrence_backward(dh, x, g, want[0], form, grad_state_in=True)
        n = ret.gated_recurrence_workspace_bytes(shape[0], 1, shape[1], shape[2], F32)
        assert n > 0
        for fill in (0, 255, 66):
            ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
            for _ in range(2):  # the second call finds what the first one left
                h, s = ret.gated_recurrence(x, g, form, state_out=True, workspace=ws)
                assert torch.equal(h, want[0]) and torch.equal(s, want[1])
                got = ret.gated_recurrence_backward(dh, x, g, h, form, grad_state_in=True, workspace=ws)
                assert all(torch.equal(a, b) for a, b in zip(got, back))
    with pytest.raises(ValueError, match="bytes are needed|are needed"):
        ret.gated_recurrence(x, g, form, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))


def test_refusals_reach_python_as_errors():
    """What only the C ABI can tell comes back as RetentionError, and nothing is launched."""
    _announce("refusals")
    x = _randn((2, 40, 64), 1).to(DEV)
    mark = x.clone()
    with pytest.raises(ret.RetentionError, match="invalid argument"):
        ret.gated_recurrence(x, mark, out=x)
    with pytest.raises(ret.RetentionError, match="invalid argument"):
        ret.gated_norm(x.view(2, 4, 10, 64), out=x.view(2, 4, 10, 64))
    with pytest.raises(ret.RetentionError, match="invalid argument"):
        ret.gated_recurrence(x, mark, out=torch.zeros(1, 40, 64, device=DEV).expand(2, 40, 64))
    with pytest.raises(ret.RetentionError, match="invalid argument"):
        ret.gated_recurrence_step(x[:, 0], x[:, 1], mark.view(-1)[:128].view(2, 64), out=mark.view(-1)[64:192].view(2, 64))
    with pytest.raises(ret.RetentionError, match="unsupported"):
        ret.gated_norm(torch.zeros(1, 1, 1, 2048, device=DEV))
    with pytest.raises(ret.RetentionError, match="invalid argument"):
        ret.residual_norm(x, x, ret.Norm(eps=float("nan")))
    with pytest.raises(ret.RetentionError, match="invalid argument"):
        ret.gated_recurrence(x[:, :0], x[:, :0])
    torch.cuda.synchronize()
    assert torch.equal(x, mark)


def test_log_form_needs_no_x():
    _announce("log form without x")
    shape = (1, 70, 40)
    g, dh, h = _gate(shape, 1, BF16, "log").to(DEV), _randn(shape, 2, BF16).to(DEV), _randn(shape, 3, BF16).to(DEV)
    a = ret.gated_recurrence_backward(dh, None, g, h, "log")
    b = ret.gated_recurrence_backward(dh, h, g, h, "log")
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("shape, dtype", [((1, 20000, 64), BF16), ((1, 16, 6000, 64), BF16), ((2, 3001, 200), F32)])
def test_repeated_calls_are_bit_identical(shape, dtype):
    _announce(f"repeated {shape} {dtype}")
    x, g, dh = _randn(shape, 1, dtype).to(DEV), _gate(shape, 2, dtype, "sigmoid").to(DEV), _randn(shape, 3, dtype).to(DEV)
    first = None
    for _ in range(30):
        h, s = ret.gated_recurrence(x, g, state_out=True)
        dx, dg, ds = ret.gated_recurrence_backward(dh, x, g, h, grad_state_in=True)
        got = [t.clone() for t in (h, s, dx, dg, ds)]
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_two_streams_at_once():
    """Two calls that overlap on two streams, each with its own workspace and tensors, give what each gives alone."""
    _announce("two streams")
    shapes = [(1, 30000, 256), (2, 9000, 320)]
    args = [(_randn(s, 1, BF16).to(DEV), _gate(s, 2, BF16, "sigmoid").to(DEV)) for s in shapes]
    want = [ret.gated_recurrence(*a, state_out=True) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    for _ in range(5):
        got = []
        for st, a in zip(streams, args):
            with torch.cuda.stream(st):
                got.append(ret.gated_recurrence(*a, state_out=True))
        torch.cuda.synchronize()
        for (h, s), (h0, s0) in zip(got, want):
            assert torch.equal(h, h0) and torch.equal(s, s0)


# ---------------------------------------------------------------------------
# One token

@pytest.mark.parametrize("B, lead, d, dtype, form", [
    (1, (), 1, F32, "sigmoid"), (1, (), 64, BF16, "log"), (5, (), 333, BF16, "sigmoid"), (8, (4,), 72, F32, "log"),
    (300, (2,), 40, BF16, "sigmoid"), (3, (), 4096, BF16, "log"), (7, (), 2048, F32, "sigmoid")])
@pytest.mark.parametrize("strided", [False, True])
def test_step_matches_the_oracle(B, lead, d, dtype, form, strided):
    _announce(f"step {B} {lead} {d} {dtype} {form} strided={strided}")
    shape = (B, *lead, d)
    x, g, s0 = _randn(shape, 1, dtype), _gate(shape, 2, dtype, form), _randn(shape, 3)
    place = (lambda t: _strided(t, 0)) if strided else (lambda t: t.to(DEV))
    state = s0.to(DEV)
    h = ret.gated_recurrence_step(place(x), place(g), state, form)
    torch.cuda.synchronize()
    tok = [t.unsqueeze(-2) for t in (x, g)]
    ref, end = orc.recurrence(*tok, form, s0)
    e, _ = orc.recurrence_error(*tok, form, s0)
    _check(h, ref[..., 0, :], e[..., 0, :], "h")
    _check(state, end, e[..., 0, :], "state")


@pytest.mark.parametrize("dtype, d", [(BF16, 96), (F32, 35)])
def test_step_with_slots(dtype, d):
    """Rows pick states of a pool; idle rows (slots below 0 or beyond the pool) and unnamed states stay as they were; rows
    of one slot take effect in row order."""
    _announce(f"slots {dtype} {d}")
    P, slots = 12, [3, -1, 7, 3, 11, 12, 0, 3, 7, -2147483648, 2147483647]
    B = len(slots)
    x, g, pool = _randn((B, d), 1, dtype), _gate((B, d), 2, dtype, "sigmoid"), _randn((P, d), 3)
    out = torch.full((B, d), 9.0, dtype=dtype, device=DEV)
    state = pool.to(DEV)
    ret.gated_recurrence_step(x.to(DEV), g.to(DEV), state, "sigmoid", slots=torch.tensor(slots, dtype=torch.int32, device=DEV), out=out)
    torch.cuda.synchronize()
    for s in range(P):
        rows = [i for i, v in enumerate(slots) if v == s]
        if not rows:
            assert torch.equal(state[s].cpu(), pool[s])
            continue
        ref, end = orc.recurrence(x[rows], g[rows], "sigmoid", pool[s])
        e, e_end = orc.recurrence_error(x[rows], g[rows], "sigmoid", pool[s])
        _check(out[rows], ref, e, f"h of slot {s}")
        _check(state[s], end, e_end, f"state {s}")
    idle = [i for i, v in enumerate(slots) if not 0 <= v < P]
    assert bool((out[idle] == 9.0).all())


def test_prefill_then_steps_is_the_whole_sequence():
    _announce("prefill and steps")
    B, N, D, k = 2, 400, 128, 5
    x, g = _randn((B, N, D), 1, BF16), _gate((B, N, D), 2, BF16, "sigmoid")
    xd, gd = x.to(DEV), g.to(DEV)
    _, state = ret.gated_recurrence(xd[:, :N - k], gd[:, :N - k], state_out=True)
    h = [ret.gated_recurrence_step(xd[:, t], gd[:, t], state) for t in range(N - k, N)]
    torch.cuda.synchronize()
    ref, end = orc.recurrence(x, g, "sigmoid")
    e, e_end = orc.recurrence_error(x, g, "sigmoid")
    _check(torch.stack(h, 1), ref[:, N - k:], e[:, N - k:], "h")
    _check(state, end, e_end, "state")


# ---------------------------------------------------------------------------
# Norms

HEADS = [
    (1, 1, 1, 1, BF16), (1, 2, 3, 8, F32), (2, 3, 5, 64, BF16), (1, 4, 7, 65, F32), (2, 2, 33, 96, BF16),
    (1, 3, 50, 127, BF16), (3, 5, 21, 97, F32), (2, 8, 40, 256, BF16), (1, 4, 60, 320, F32), (2, 4, 130, 512, BF16),
    (1, 2, 30, 513, BF16), (2, 3, 17, 1024, BF16), (1, 2, 9, 1024, F32), (1, 2, 11, 1023, F32), (4, 16, 1, 512, BF16),
]


def _norm_params(n, seed, which):
    w = _randn((n,), seed, F32, 0.25, 1.0) if "w" in which else None
    b = _randn((n,), seed + 1, F32, 0.1) if "b" in which else None
    return w, b, dict(weight=None if w is None else w.to(DEV), bias=None if b is None else b.to(DEV))


@pytest.mark.parametrize("B, H, N, d, dtype", HEADS)
@pytest.mark.parametrize("rms, gated, which, strided", [(False, True, "wb", False), (True, True, "w", True),
                                                         (False, False, "", True), (True, False, "b", False)])
def test_gated_norm_matches_the_oracle(B, H, N, d, dtype, rms, gated, which, strided):
    _announce(f"gated norm {B, H, N, d} {dtype} rms={rms} gate={gated} {which} strided={strided}")
    shape = (B, H, N, d)
    o, dy = _randn(shape, 1, dtype, 2.0, 0.5), _randn(shape, 2, dtype)
    gate = _randn(shape, 3, dtype, 3.0) if gated else None
    w, b, params = _norm_params(H * d, 4, which)
    norm = ret.Norm(EPS, rms=rms, **params)
    place = (lambda t: None if t is None else _strided(t, 0)) if strided else (lambda t: None if t is None else t.to(DEV))
    od, gd = place(o), place(gate)
    y = ret.gated_norm(od, gd, norm)
    got = ret.gated_norm_backward(place(dy), od, gd, norm)
    torch.cuda.synchronize()
    args = (o, gate, w, b, EPS, rms)
    _check(y, orc.gated_norm(*args), orc.gated_norm_error(*args), "y")
    refs, errs = orc.gated_norm_backward(dy, *args), orc.gated_norm_backward_error(dy, *args)
    for t, ref, e, what, wanted in zip(got, refs, errs, ("grad_o", "grad_gate", "grad_weight", "grad_bias"),
                                       (True, gated, "w" in which, "b" in which)):
        assert (t is not None) == wanted, what
        if wanted:
            _check(t, ref, e, what)


def test_gated_norm_is_the_chunkwise_epilogue():
    """On one token's and a sequence's worth of the retention's raw output, token-major output included."""
    _announce("gated norm as the epilogue")
    B, H, N, dk, dv, C = 2, 4, 200, 64, 128, 64
    q, k, v = (t.to(DEV) for t in synthetic.make_qkv(B, H, N, dk, dv, dtype=F32, seed=3))
    g = synthetic.head_gammas(H)
    w, b = (t.to(DEV) for t in synthetic.make_gn_affine(H, dv, seed=4))
    gate = synthetic.make_gate((B, H, N, dv), F32, seed=5).to(DEV)
    gn = ret.GroupNorm(EPS, w, b)
    raw, _ = ret.chunkwise(q, k, v, g, C)
    fused, _ = ret.chunkwise(q, k, v, g, C, gn=gn, gate=gate)
    y = ret.gated_norm(raw, gate, gn)
    # Both norm the same fp32 values; each is within the operator's bound of the exact result.
    args = (raw, gate, w, b, EPS, False)
    _check(fused, orc.gated_norm(*args), orc.gated_norm_error(*args), "epilogue")
    _check(y, orc.gated_norm(*args), orc.gated_norm_error(*args), "operator")
    token_major = torch.empty(B, N, H, dv, device=DEV)
    ret.gated_norm(raw, gate, gn, out=token_major.transpose(1, 2))
    assert torch.equal(token_major.transpose(1, 2), y)
    one = ret.gated_norm(raw[:, :, 7], gate[:, :, 7], gn)
    assert torch.equal(one, y[:, :, 7])


def test_msr_training_step():
    """The gated MSR block's gradient chain: gated_norm_backward, then chunkwise_backward on what it gives, against the
    oracle's."""
    _announce("norm backward into retention backward")
    B, H, N, dk, dv, C = 1, 3, 150, 32, 64, 64
    q, k, v = synthetic.make_qkv(B, H, N, dk, dv, dtype=F32, seed=6)
    g = synthetic.head_gammas(H)
    gate, dy = synthetic.make_gate((B, H, N, dv), F32, seed=7), _randn((B, H, N, dv), 8)
    w, b = synthetic.make_gn_affine(H, dv, seed=9)
    dev = [t.to(DEV) for t in (q, k, v, gate, dy, w, b)]
    gn = ret.GroupNorm(EPS, dev[5], dev[6])
    o, _ = ret.chunkwise(*dev[:3], g, C)
    do, dgate, dw, db = ret.gated_norm_backward(dev[4], o, dev[3], gn)
    grads = ret.chunkwise_backward(*dev[:3], do, g, C)[:3]
    torch.cuda.synchronize()
    o_ref, _ = rorc.chunkwise(q, k, v, g, C)
    refs = orc.gated_norm_backward(dy, o_ref, gate, w, b, EPS, False)
    back = rorc.backward(q, k, v, g, refs[0])[:3]
    # fp32 chunkwise results are held to 1e-4 of the head's largest value; the norm multiplies the relative error of
    # its input by at most a few tens (values up to about five deviations, squared).
    for got, ref in zip((do, dgate, dw, db, *grads), (*refs, *back)):
        np.testing.assert_allclose(orc.f64(got), ref, rtol=0, atol=2e-3 * np.abs(ref).max())


ROWS = [
    ((1, 1), BF16, BF16), ((3, 8), F32, F32), ((5, 65), BF16, F32), ((2, 7, 64), BF16, BF16), ((2, 3, 5, 96), F32, F32),
    ((130, 1000), BF16, F32), ((33, 1023), BF16, BF16), ((9, 1024), F32, F32), ((40, 2048), BF16, F32),
    ((7, 2049), F32, F32), ((70, 4096), BF16, BF16), ((3, 5000), BF16, F32), ((5, 8192), F32, F32), ((4, 8192), BF16, F32),
    ((3, 16384), BF16, BF16), ((2, 16384), F32, F32), ((2, 16383), BF16, F32), ((4096,), BF16, BF16),
    ((600, 9001), BF16, F32), ((300, 16384), F32, F32), ((600, 5000), BF16, BF16),
]


@pytest.mark.parametrize("shape, dtype, stream", ROWS)
@pytest.mark.parametrize("rms, scaled, alpha, which, strided", [(False, True, 1.75, "wb", False), (True, False, 1.0, "w", True),
                                                                (True, True, 1.0, "", False), (False, False, 0.5, "b", True)])
def test_residual_norm_matches_the_oracle(shape, dtype, stream, rms, scaled, alpha, which, strided):
    _announce(f"residual norm {shape} {dtype} {stream} rms={rms} scale={scaled} alpha={alpha} {which} strided={strided}")
    D = shape[-1]
    x, res = _randn(shape, 1, dtype), _randn(shape, 2, stream, 2.0, 0.5)
    dy, dr = _randn(shape, 3, dtype), _randn(shape, 4, stream)
    scale = _randn((D,), 5, F32, 0.2, 0.7) if scaled else None
    w, b, params = _norm_params(D, 6, which)
    norm = ret.Norm(EPS, rms=rms, **params)
    place = (lambda t: _strided(t, 0)) if strided and len(shape) in (2, 3) else (lambda t: t.to(DEV))
    xd, sd = place(x), None if scale is None else scale.to(DEV)
    y, r = ret.residual_norm(xd, place(res), norm, scale=sd, alpha=alpha)
    with_dr = alpha != 0.5  # one of the four takes no gradient from the stream
    got = ret.residual_norm_backward(place(dy), r, norm, grad_r=place(dr) if with_dr else None, x=xd, scale=sd, alpha=alpha)
    torch.cuda.synchronize()
    args = (x, res, w, b, EPS, rms, scale, alpha)
    y_ref, r_ref = orc.residual_norm(*args)
    e_y, e_r = orc.residual_norm_error(*args)
    _check(y, y_ref, e_y, "y")
    _check(r, r_ref, e_r, "r")
    bargs = (dy, dr if with_dr else None, r.cpu(), w, EPS, rms, x, scale, alpha)
    refs, errs = orc.residual_norm_backward(*bargs), orc.residual_norm_backward_error(*bargs)
    for t, ref, e, what, wanted in zip(got, refs, errs, ("grad_x", "grad_residual", "grad_scale", "grad_weight", "grad_bias"),
                                       (True, True, scaled, "w" in which, "b" in which)):
        assert (t is not None) == wanted, what
        if wanted:
            _check(t, ref, e, what)
    shared = not scaled and alpha == 1.0 and dtype == stream
    assert (got[0] is got[1]) == shared
    # From x and the residual instead of r: the gradients at the row before its rounding. What forming it rounds (4 steps
    # of its terms, e_r) changes the normed row like a change of the row itself: by at most three times that over the
    # deviation, within ROW of the magnitudes already counted.
    got = ret.residual_norm_backward(place(dy), None, norm, grad_r=place(dr) if with_dr else None, x=xd, scale=sd, alpha=alpha,
                                     residual=place(res))
    torch.cuda.synchronize()
    bargs = (dy, dr if with_dr else None, r_ref, w, EPS, rms, x, scale, alpha)
    terms = np.abs(alpha * orc.f64(res)) + np.abs(orc.f64(x) * (1.0 if scale is None else orc.f64(scale)))
    grow = 1 + float((terms.max(-1) / np.abs(r_ref).max(-1)).max())
    refs, errs = orc.residual_norm_backward(*bargs), orc.residual_norm_backward_error(*bargs)
    for t, ref, e, what, wanted in zip(got, refs, errs, ("grad_x", "grad_residual", "grad_scale", "grad_weight", "grad_bias"),
                                       (True, True, scaled, "w" in which, "b" in which)):
        if wanted:
            _check(t, ref, grow * e, what + " from the residual")


def test_constant_rows_and_huge_values():
    """A row of one value has no deviation: the layer form gives the bias. Values near the top of bf16's exponents that
    still square in fp32, and rows of zeros in the rms form, stay finite."""
    _announce("constant rows")
    x = torch.full((2, 3, 4, 64), 3.0, dtype=BF16, device=DEV)
    b = _randn((192,), 1).to(DEV)
    y = ret.gated_norm(x, None, ret.Norm(EPS, None, b))
    assert torch.equal(y, b.view(3, 1, 64).expand(2, 3, 4, 64).to(BF16))
    assert bool((ret.gated_norm(torch.zeros_like(x), None, ret.Norm(EPS, rms=True)) == 0).all())
    big = torch.full((1, 1, 1, 64), 1e17, dtype=BF16, device=DEV)
    assert bool((ret.gated_norm(big, None, ret.Norm(EPS, rms=True)) == 1).all())
    gate = torch.tensor([-1e4, 1e4] * 32, dtype=BF16, device=DEV).view(1, 1, 1, 64)
    dy = torch.ones_like(big)
    y = ret.gated_norm(big, gate, ret.Norm(EPS, rms=True)).view(-1)
    assert bool((y[::2] == 0).all()) and bool((y[1::2] == gate.view(-1)[1]).all())
    dgate = ret.gated_norm_backward(dy, big, gate, ret.Norm(EPS, rms=True))[1].view(-1)
    assert bool((dgate[::2] == 0).all()) and bool((dgate[1::2] == 1).all())


def test_residual_norm_of_many_dimensions():
    """Rows in five dimensions, one of them of one element with a stride of its own, are those of the flat tensor."""
    _announce("residual norm in five dimensions")
    norm = ret.Norm(EPS, _randn((64,), 1).to(DEV), rms=True)
    x, res, dy = (_randn((2, 3, 1, 4, 64), i, BF16).to(DEV).transpose(2, 3) for i in (2, 3, 4))
    assert x.is_contiguous() and x.stride(-2) != 64
    flat = [t.reshape(24, 64) for t in (x, res, dy)]
    for got, ref in zip(ret.residual_norm(x, res, norm), ret.residual_norm(flat[0], flat[1], norm)):
        assert got.shape == x.shape and torch.equal(got.reshape(24, 64), ref)
    for got, ref in zip(ret.residual_norm_backward(dy, res, norm), ret.residual_norm_backward(flat[2], flat[1], norm)):
        assert got is ref is None or torch.equal(got.reshape(ref.shape), ref)


# ---------------------------------------------------------------------------
# Together


def _torch_block(x, res, gate, wg, scale, w1, w2, b2, form):
    """The block in float64: residual and norm, gated recurrence, norm and gate, residual and norm."""
    def norm(v, rms):
        d = v if rms else v - v.mean(-1, keepdim=True)
        return d / torch.sqrt((d * d).mean(-1, keepdim=True) + EPS)

    B, N, D = x.shape
    r1 = res + x
    y1 = norm(r1, True) * w1
    a = torch.sigmoid(gate)
    now, hs = torch.zeros(B, D, dtype=torch.float64), []
    for t in range(N):
        now = a[:, t] * now + (1 - a[:, t]) * y1[:, t]
        hs.append(now)
    h = torch.stack(hs, 1)
    H = 4
    m = norm(h.view(B, N, H, D // H), False).view(B, N, D) * w2 + b2
    m = m * torch.nn.functional.silu(wg)
    r2 = r1 + scale * m
    return norm(r2, True) * w1, r2


def test_a_block_forward_and_backward():
    """residual_norm, gated_recurrence, gated_norm, residual_norm in fp32 and back, against torch autograd in float64.
    Every operator is within 1e-5 of its largest value (the per-operator bounds above); four of them in a row, with
    norms that pass relative errors on, stay within 1e-4."""
    _announce("block forward and backward")
    B, N, D, H = 2, 90, 256, 4
    names = ("x", "res", "gate", "wg", "scale", "w1", "w2", "b2")
    shapes = ((B, N, D),) * 4 + ((D,),) * 4
    leaves = {n: _randn(s, 20 + i, F32, 0.3 if len(s) == 1 else 1.0, 1.0 if n in ("gate", "w1", "w2", "scale") else 0.0)
              for i, (n, s) in enumerate(zip(names, shapes))}
    dy, dr = _randn((B, N, D), 40), _randn((B, N, D), 41)
    t64 = {n: v.double().requires_grad_() for n, v in leaves.items()}
    y, r2 = _torch_block(*[t64[n] for n in names], "sigmoid")
    want = dict(zip(names, torch.autograd.grad([y, r2], [t64[n] for n in names], [dy.double(), dr.double()])))

    p = {n: v.to(DEV) for n, v in leaves.items()}
    n1, n2 = ret.Norm(EPS, p["w1"], rms=True), ret.GroupNorm(EPS, p["w2"], p["b2"])
    heads = lambda t: t.view(B, N, H, D // H).transpose(1, 2)  # noqa: E731
    y1, r1 = ret.residual_norm(p["x"], p["res"], n1)
    h, _ = ret.gated_recurrence(y1, p["gate"])
    m = torch.empty_like(h)
    ret.gated_norm(heads(h), heads(p["wg"]), n2, out=heads(m))
    y2, r = ret.residual_norm(m, r1, n1, scale=p["scale"])
    dm, dr1, dscale, dw1b, _ = ret.residual_norm_backward(dy.to(DEV), r, n1, grad_r=dr.to(DEV), x=m, scale=p["scale"])
    dh, dwg = torch.empty_like(h), torch.empty_like(h)
    _, _, dw2, db2 = ret.gated_norm_backward(heads(dm), heads(h), heads(p["wg"]), n2, grads=(heads(dh), heads(dwg)))
    dy1, dgate, _ = ret.gated_recurrence_backward(dh, y1, p["gate"], h)
    dx, dres, _, dw1a, _ = ret.residual_norm_backward(dy1, r1, n1, grad_r=dr1)
    torch.cuda.synchronize()
    got = dict(x=dx, res=dres, gate=dgate, wg=dwg, scale=dscale, w1=dw1a + dw1b, w2=dw2, b2=db2)
    for name, ref in (("y", y), ("r", r2)):
        val = orc.f64(y2 if name == "y" else r)
        np.testing.assert_allclose(val, ref.detach().numpy(), rtol=0, atol=1e-4 * ref.abs().max().item(), err_msg=name)
    for name in names:
        ref = want[name].numpy()
        np.testing.assert_allclose(orc.f64(got[name]), ref, rtol=0, atol=1e-4 * np.abs(ref).max(), err_msg=name)


def test_captured_and_replayed():
    """A block's forward and backward in one graph with its own workspaces, replayed on new inputs between eager calls of
    the same operators: every replay gives the eager results bit for bit."""
    _announce("graph")
    B, N, D = 1, 3000, 128
    x, g, dh = _randn((B, N, D), 1, BF16).to(DEV), _gate((B, N, D), 2, BF16, "sigmoid").to(DEV), _randn((B, N, D), 3, BF16).to(DEV)
    w = torch.ones(D, device=DEV)
    norm = ret.Norm(EPS, w, rms=True)

    def block():
        h, s = ret.gated_recurrence(x, g, state_out=True)
        y, r = ret.residual_norm(h, x, norm)
        back = ret.residual_norm_backward(dh, r, norm, grad_r=x)
        dx, dg, _ = ret.gated_recurrence_backward(back[0], x, g, h, grad_state_out=s)
        step = ret.gated_recurrence_step(x[:, 0], g[:, 0], s)
        return [h, s, y, r, back[0], back[3], dx, dg, step]

    block()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = block()
    for i in range(4):
        x.copy_(_randn((B, N, D), 50 + i, BF16))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = block()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (i, k)


def test_outputs_past_two_to_the_31_elements():
    """A tensor of 2.2e9 values: the last rows of the outputs, against the oracle from the state the rows before leave
    (the running mean of 0.5, to a rounding of fp32, which the oracle's bound counts per token) and against the same rows
    on their own."""
    _announce("2.2e9 values")
    N, D, k = 34000, 65536, 40
    x = torch.empty(1, N, D, dtype=BF16, device=DEV)
    x.view(-1)[:].fill_(0.5)
    x[:, -k:] = _randn((1, k, D), 1, BF16).to(DEV)
    g = torch.zeros(1, 1, D, dtype=BF16, device=DEV).expand(1, N, D)
    assert x.numel() > 2 ** 31
    h, s = ret.gated_recurrence(x, g, state_out=True)
    start = h[:, -k - 1].float()
    assert bool((start == 0.5).all())
    args = (x[:, -k:], g[:, -k:], "sigmoid", start)
    (ref, end), (e, e_end) = orc.recurrence(*args), orc.recurrence_error(*args)
    _check(h[:, -k:], ref, e, "h")
    _check(s, end, e_end, "state")
    y, _ = ret.residual_norm(x.view(-1, 16384), h.view(-1, 16384), ret.Norm(EPS, rms=True))
    y2, _ = ret.residual_norm(x.view(-1, 16384)[-k:], h.view(-1, 16384)[-k:], ret.Norm(EPS, rms=True))
    assert torch.equal(y[-k:], y2)


@pytest.mark.parametrize("shape, pitch, form, dtype", [
    ((1, 17600, 1001), 1001, "sigmoid", F32), ((3, 12000, 1003), 1010, "log", BF16), ((300, 130, 1000), 1004, "sigmoid", BF16)])
def test_wide_results_in_rows_that_begin_anywhere(shape, pitch, form, dtype):
    """Results too large to leave the inputs in the caches, in rows that do not begin on cache lines: some channels
    (the recurrence is per channel) of a few rows against the oracle, and nothing written beside the rows."""
    _announce(f"wide results {shape} pitch {pitch} {form} {dtype}")
    B, N, D = shape
    at = [*range(10), *range(60, 70), *range(D - 70, D - 60), *range(D - 9, D)]
    x, g = _randn(shape, 1, dtype), _gate(shape, 2, dtype, form)
    s0 = _randn((B, D), 3)
    wide = torch.full((B, N, pitch), float("nan"), dtype=dtype, device=DEV)
    h, s1 = ret.gated_recurrence(x.to(DEV), g.to(DEV), form, state_in=s0.to(DEV), state_out=True, out=wide[..., :D])
    rows = [0, B - 1]
    args = (x[rows][..., at], g[rows][..., at], form, s0[rows][..., at])
    (ref, end), (e, e_end) = orc.recurrence(*args), orc.recurrence_error(*args)
    _check(h[rows][..., at], ref, e, "h")
    _check(s1[rows][..., at], end, e_end, "state")
    assert bool(torch.isnan(wide[..., D:]).all()) and not bool(torch.isnan(h).any())


def test_large_offsets():
    """Rows whose element offsets pass 2^31: the last rows of a tall strided tensor, checked on their own."""
    _announce("offsets past 2^31")
    N, D, pitch = 1100, 64, 2_000_000
    wide = torch.empty(N, pitch, dtype=BF16, device=DEV)
    x = wide[:, :D].unsqueeze(0)
    assert (N - 1) * pitch > 2 ** 31
    vals, g = _randn((1, N, D), 1, BF16), _gate((1, N, D), 2, BF16, "sigmoid")
    x.copy_(vals)
    h, _ = ret.gated_recurrence(x, g.to(DEV))
    ref, e = orc.recurrence(vals, g, "sigmoid")[0], orc.recurrence_error(vals, g, "sigmoid")[0]
    _check(h, ref, e, "h")
    y, _ = ret.residual_norm(x, h, ret.Norm(EPS))
    y2, _ = ret.residual_norm(x.contiguous(), h, ret.Norm(EPS))
    assert torch.equal(y, y2)


# ---------------------------------------------------------------------------
# h in fp32 beside bf16 activations


@pytest.mark.parametrize("shape, form", [((1, 1, 1), "sigmoid"), ((2, 31, 64), "sigmoid"), ((1, 33, 65), "log"), ((2, 63, 3), "log"),
                                         ((3, 1000, 200), "sigmoid"), ((1, 2049, 70), "log"), ((2, 3, 77, 24), "sigmoid"),
                                         ((260, 270, 64), "log")])
@pytest.mark.parametrize("strided", [False, True])
def test_a_float32_h_keeps_its_rounding_out_of_the_gradients(shape, form, strided):
    """h of bf16 inputs in fp32, to fp32's bound, and the gradients of the formula itself, whose h is exact: what is left
    of the fp32 h's own error enters grad_gate as |a c u| (log: |a u|) times it."""
    _announce(f"fp32 h {shape} {form} strided={strided}")
    x, g, dh = _randn(shape, 1, BF16), _gate(shape, 2, BF16, form), _randn(shape, 4, BF16)
    s0, ds = (_randn(_states(shape), 3), _randn(_states(shape), 5)) if strided else (None, None)
    place = (lambda t: _strided(t, 0)) if strided else (lambda t: t.to(DEV))
    s0d, dsd = (None if t is None else t.to(DEV) for t in (s0, ds))
    out = _strided(torch.zeros(shape), 0) if strided else None
    h, s1 = ret.gated_recurrence(place(x), place(g), form, state_in=s0d, state_out=True, out=out, out_dtype=F32)
    h16, s16 = ret.gated_recurrence(place(x), place(g), form, state_in=s0d, state_out=True)
    dx, dg, ds0 = ret.gated_recurrence_backward(place(dh), place(x), place(g), h, form, state_in=s0d, grad_state_out=dsd,
                                                grad_state_in=True)
    torch.cuda.synchronize()
    assert h.dtype is F32 and dx.dtype is dg.dtype is BF16
    assert torch.equal(h.to(BF16), h16) and torch.equal(s1, s16)
    ref, e = orc.recurrence(x, g, form, s0)[0], orc.recurrence_error(x, g, form, s0)[0]
    _check(h, ref, e, "h")
    args = (dh, x, g, ref, form, s0, ds)
    refs, errs = orc.recurrence_backward(*args), orc.recurrence_backward_error(*args)
    a, c = orc.decay(g, form)
    u = np.abs(refs[0]) if form == "log" else np.abs(np.divide(refs[0], c, out=np.zeros_like(refs[0]), where=c > 0))
    off = np.concatenate((np.zeros_like(e[..., :1, :]), (e + 2.0 ** -24 * np.abs(ref))[..., :-1, :]), -2)
    extra = (0.0, 2 * a * c * u * off, 0.0)
    for got, r, err, more, what in zip((dx, dg, ds0), refs, errs, extra, ("grad_x", "grad_gate", "grad_state_in")):
        _check(got, r, err + more, what)


def test_a_bf16_h_rounds_grad_gate_twice():
    """Against the formula's gradient in 64 bits, memories of 2 to 500 tokens. A rounding to bf16 is even within half a
    step, 2^-8 / m of a value of mantissa m in [1, 2): 2^-8 / sqrt(3) / m in the 2-norm, 1.13e-3 to 2.26e-3. A float32 h
    leaves grad_gate that alone; a bf16 h adds another one, so that the error grows by sqrt(1 + (1.13 / 2.26)^2) = 1.118
    at least."""
    _announce("h in bf16 and in fp32")
    shape = (2, 3000, 64)
    x, dh = _randn(shape, 1, BF16), _randn(shape, 2, BF16)
    g = -torch.exp(torch.rand(shape, generator=_gen(3)) * 5.5 - 6.2).to(BF16)
    ref = orc.recurrence_backward(dh, x, g, orc.recurrence(x, g, "log")[0], "log")[1]

    def off(h):
        dg = ret.gated_recurrence_backward(dh.to(DEV), None, g.to(DEV), h, "log")[1]
        return np.linalg.norm(orc.f64(dg) - ref) / np.linalg.norm(ref)

    narrow = off(ret.gated_recurrence(x.to(DEV), g.to(DEV), "log")[0])
    wide = off(ret.gated_recurrence(x.to(DEV), g.to(DEV), "log", out_dtype=F32)[0])
    assert 1.13e-3 < wide < 2.26e-3 and narrow > 1.118 * wide


# ---------------------------------------------------------------------------
# Decays near 1

# A rounding of the state per tile (of 64 tokens at least, in the backward of 32768 tokens 512 of them, 2^-24 each:
# 3.1e-5), the decays' and the weights' own errors, (|g| + 8) 2^-24 of their distance from 1 (1.4e-6 at 16), and some 32
# roundings within a tile (1.9e-6).
LONG = 5e-5


@pytest.mark.parametrize("B, N, D", [(1, 32768, 65), (256, 8192, 64)])
def test_long_memories_of_the_sigmoid_form(B, N, D):
    """Constant gates up to 16 (memories of 3000 to 9 million tokens) and a constant input, against the closed form
    x (1 - a^t): the weights of the state and of the input add up to 1 however many tokens there are."""
    _announce(f"long memories {B, N, D}")
    t = np.arange(1, N + 1)
    x = torch.full((1, 1, D), 0.7, device=DEV).expand(B, N, D)
    v = float(x[0, 0, 0])
    for g in (8.0, 10.0, 12.0, 14.0, 15.0, 16.0):
        gate = torch.full((1, 1, D), g, device=DEV).expand(B, N, D)
        rise = -np.expm1(-np.log1p(np.exp(-g)) * t)  # 1 - a^t
        h, s = ret.gated_recurrence(x, gate, state_out=True)
        dx, dg, ds = ret.gated_recurrence_backward(x, x, gate, h, grad_state_in=True)
        assert bool((h == h[:1, :, :1]).all()) and bool((dx == dx[:1, :, :1]).all())
        np.testing.assert_allclose(orc.f64(h[0, :, 0]), v * rise, rtol=LONG)
        np.testing.assert_allclose(orc.f64(s[0, 0]), v * rise[-1], rtol=LONG)
        np.testing.assert_allclose(orc.f64(dx[0, :, 0]), v * rise[::-1], rtol=LONG)
        c = 1 / (1 + np.exp(g))
        before = v * np.concatenate(([0.0], rise[:-1]))
        np.testing.assert_allclose(orc.f64(dg[0, :, 0]), (1 - c) * (before - v) * v * rise[::-1], rtol=0, atol=3 * LONG * v * v)
        np.testing.assert_allclose(orc.f64(ds[0, 0]), v * rise[-1] * (1 - c) / c, rtol=LONG)


def test_steps_keep_a_state_that_equals_the_input():
    """Gates from 0 up: a state that is the input stays it to the bit, however many steps are taken."""
    _announce("steps at a fixed point")
    g = torch.linspace(0, 24, 333, device=DEV).expand(2, 333).contiguous()
    x = torch.stack((torch.full((333,), 0.7), torch.linspace(-3, 5, 333))).to(DEV)
    state = x.clone()
    for _ in range(2000):
        h = ret.gated_recurrence_step(x, g, state)
    assert torch.equal(state, x) and torch.equal(h, x)


@pytest.mark.parametrize("shape", [(2, 1, 65), (1, 40, 3), (3, 129, 64), (1, 5000, 72), (260, 300, 64)])
def test_the_last_h_is_the_final_state(shape):
    _announce(f"last h {shape}")
    x, s0 = _randn(shape, 1).to(DEV), _randn(_states(shape), 2).to(DEV)
    for form in ("sigmoid", "log"):
        h, s1 = ret.gated_recurrence(x, _gate(shape, 3, F32, form).to(DEV), form, state_in=s0, state_out=True)
        assert torch.equal(h[:, -1], s1)


@pytest.mark.parametrize("B, N, D", [(1, 32768, 65), (256, 8192, 64)])
def test_long_memories_of_the_log_form(B, N, D):
    """Constant gates down to -1e-6 and a constant input, against the closed form x (1 - a^t) / (1 - a)."""
    _announce(f"long memories, log form {B, N, D}")
    t = np.arange(1, N + 1)
    x = torch.full((1, 1, D), 0.7, device=DEV).expand(B, N, D)
    v = float(x[0, 0, 0])
    for g in (-0.1, -1e-2, -1e-3, -1e-4, -1e-5, -1e-6):
        gate = torch.full((1, 1, D), g, device=DEV).expand(B, N, D)
        g = float(gate[0, 0, 0])
        want = v * np.expm1(g * t) / np.expm1(g)
        h, s = ret.gated_recurrence(x, gate, "log", state_out=True)
        dx, dg, ds = ret.gated_recurrence_backward(x, x, gate, h, "log", grad_state_in=True)
        assert bool((h == h[:1, :, :1]).all()) and bool((dx == dx[:1, :, :1]).all())
        np.testing.assert_allclose(orc.f64(h[0, :, 0]), want, rtol=LONG)
        np.testing.assert_allclose(orc.f64(s[0, 0]), want[-1], rtol=LONG)
        np.testing.assert_allclose(orc.f64(dx[0, :, 0]), want[::-1], rtol=LONG)
        before = np.concatenate(([0.0], want[:-1]))
        np.testing.assert_allclose(orc.f64(dg[0, :, 0]), np.exp(g) * before * want[::-1], rtol=3 * LONG)
        np.testing.assert_allclose(orc.f64(ds[0, 0]), np.exp(g) * want[-1], rtol=LONG)


def test_log_steps_keep_a_state_that_the_input_sustains():
    """Where x is (1 - a) times the state, the state stays: what x's rounding and 1 - a's leave, a few 2^-24 of x, is
    below half a step of a state 16 times as large or more."""
    _announce("log steps at a fixed point")
    g = -torch.logspace(-7, -1.5, 333, device=DEV).expand(2, 333).contiguous()
    state = torch.stack((torch.full((333,), 0.7), torch.linspace(-3, 5, 333))).to(DEV)
    x = (-torch.expm1(g.double()) * state.double()).float()
    keep = state.clone()
    for _ in range(2000):
        h = ret.gated_recurrence_step(x, g, state, "log")
    assert torch.equal(state, keep) and torch.equal(h, keep)


# ---------------------------------------------------------------------------
# Values that are not finite, and decays of 0 and 1


def _bad_values():
    return (float("inf"), -float("inf"), float("nan"))


def _mixed(shape, form, seed):
    """Gates between a memory of a few tokens and decays whose products over a tile leave fp32's range."""
    if form == "sigmoid":
        return _randn(shape, seed, F32, 4.0, 1.0)
    return -torch.exp(_randn(shape, seed, F32, 2.0, -1.0))


@pytest.mark.parametrize("form", ["sigmoid", "log"])
@pytest.mark.parametrize("B, N, D", [(1, 3000, 72), (260, 300, 64), (2, 200, 3), (1, 20, 9)])
def test_a_reset_forgets_whatever_the_state_holds(B, N, D, form):
    """A gate of -inf starts anew: behind it everything is as if the tokens and the state before it had been finite, to
    the bit. From the bad value to the reset h is not finite; other channels and rows are untouched."""
    _announce(f"reset {B, N, D} {form}")
    x, g, s0, dh = _randn((B, N, D), 1), _mixed((B, N, D), form, 2), _randn((B, D), 3), _randn((B, N, D), 4)
    dev = [t.to(DEV) for t in (x, g, s0, dh)]
    for bad in _bad_values():
        for at, reset in ((N // 3, N // 2), (N // 3, N // 3 + 1), (-1, 0), (-1, N - 1), (N - 2, N - 1)):  # -1: the state itself
            gr = dev[1].clone()
            gr[-1, reset, 1] = -float("inf")
            clean = ret.gated_recurrence(dev[0], gr, form, state_in=dev[2], state_out=True)
            xb, sb = dev[0].clone(), dev[2].clone()
            if at >= 0:
                xb[-1, at, 1] = bad
            else:
                sb[-1, 1] = bad
            h, s1 = ret.gated_recurrence(xb, gr, form, state_in=sb, state_out=True)
            hit = torch.zeros(B, N, D, dtype=torch.bool, device=DEV)
            hit[-1, max(at, 0):reset, 1] = True
            assert torch.equal(~h.isfinite(), hit), (bad, at, reset)
            assert torch.equal(h[~hit], clean[0][~hit]) and torch.equal(s1, clean[1])
            # The gradients of what lies behind the reset, and nothing that is not finite where the decay is 0.
            want = ret.gated_recurrence_backward(dev[3], dev[0], gr, clean[0], form, state_in=dev[2], grad_state_in=True)
            got = ret.gated_recurrence_backward(dev[3], xb, gr, h, form, state_in=sb, grad_state_in=True)
            assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
            bad_dg = torch.zeros_like(hit)
            bad_dg[-1, max(at, 0):reset, 1] = True
            assert torch.equal(got[1][~bad_dg], want[1][~bad_dg]) and float(got[1][-1, reset, 1]) == 0.0


@pytest.mark.parametrize("form", ["sigmoid", "log"])
@pytest.mark.parametrize("B, N, D", [(1, 3000, 72), (260, 300, 64), (2, 200, 3)])
def test_what_is_not_finite_stays_so_without_a_reset(B, N, D, form):
    """Whatever the decays' products do, h does not turn finite again by itself; the gradient carried back likewise, and a
    reset keeps it from the tokens before."""
    _announce(f"not finite {B, N, D} {form}")
    x, g, dh = (t.to(DEV) for t in (_randn((B, N, D), 1), _mixed((B, N, D), form, 2), _randn((B, N, D), 4)))
    g[-1, :, 1].clamp_(min=-30.0)
    want, end = ret.gated_recurrence(x, g, form, state_out=True)
    back = ret.gated_recurrence_backward(dh, x, g, want, form, grad_state_in=True)
    for bad in _bad_values():
        xb = x.clone()
        xb[-1, N // 3, 1] = bad
        h, s = ret.gated_recurrence(xb, g, form, state_out=True)
        hit = torch.zeros(B, N, D, dtype=torch.bool, device=DEV)
        hit[-1, N // 3:, 1] = True
        assert torch.equal(~h.isfinite(), hit) and torch.equal(h[~hit], want[~hit])
        assert (~s.isfinite()).nonzero().tolist() == [[B - 1, 1]]
        db = dh.clone()
        db[-1, N // 2, 1] = bad
        for reset in (None, N // 4):
            gr = g.clone()
            if reset is not None:
                gr[-1, reset, 1] = -float("inf")
            hr = want if reset is None else ret.gated_recurrence(x, gr, form)[0]
            ref = back if reset is None else ret.gated_recurrence_backward(dh, x, gr, hr, form, grad_state_in=True)
            dx, dg, ds = ret.gated_recurrence_backward(db, x, gr, hr, form, grad_state_in=True)
            hit = torch.zeros(B, N, D, dtype=torch.bool, device=DEV)
            hit[-1, reset or 0:N // 2 + 1, 1] = True
            assert torch.equal(dx[~hit], ref[0][~hit]) and torch.equal(dg[~hit], ref[1][~hit])
            assert not bool(dx[hit].isfinite().any())
            if reset is not None:
                assert float(dg[-1, reset, 1]) == 0.0 and torch.equal(ds, ref[2])
            else:
                assert (~ds.isfinite()).nonzero().tolist() == [[B - 1, 1]]


def test_a_decay_of_one_passes_over_whatever_x_holds():
    """A gate of +inf in the sigmoid form keeps the state: padding whose x is anything, in the recurrence, its gradients
    and its step."""
    _announce("gates of +inf")
    B, N, D = 2, 700, 72
    x, dh, s0 = _randn((B, N, D), 1).to(DEV), _randn((B, N, D), 2).to(DEV), _randn((B, D), 3).to(DEV)
    g = _gate((B, N, D), 4, F32, "sigmoid").to(DEV)
    keep = torch.rand(B, N, 1, generator=_gen(5)).to(DEV) < 0.3
    g = torch.where(keep, float("inf"), g)
    want = ret.gated_recurrence(x, g, state_in=s0, state_out=True)
    back = ret.gated_recurrence_backward(dh, x, g, want[0], state_in=s0, grad_state_in=True)
    for bad in _bad_values():
        xb = torch.where(keep, bad, x)
        got = ret.gated_recurrence(xb, g, state_in=s0, state_out=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        got = ret.gated_recurrence_backward(dh, xb, g, got[0], state_in=s0, grad_state_in=True)
        assert all(torch.equal(a, b) for a, b in zip(got, back))
        state = s0.clone()
        h = ret.gated_recurrence_step(torch.full_like(s0, bad), torch.full_like(s0, float("inf")), state)
        assert torch.equal(state, s0) and torch.equal(h, s0)


@pytest.mark.parametrize("dtype", [F32, torch.bfloat16])
@pytest.mark.parametrize("B,N,D", [(2, 1, 64), (1, 20, 70), (2, 317, 200), (300, 33, 64)])
def test_a_sequence_that_is_passed_over_hands_on_what_is_infinite(B, N, D, dtype):
    """Gates of +inf throughout: the state and its gradient go through as they are, at lengths that fill no tile."""
    _announce(f"gates of +inf throughout {B} x {N} x {D} {dtype}")
    x, dh = _randn((B, N, D), 1, dtype).to(DEV), torch.zeros(B, N, D, dtype=dtype, device=DEV)
    g = torch.full_like(x, float("inf"))
    s0, ds = _randn((B, D), 2).to(DEV), _randn((B, D), 3).to(DEV)
    for t in (s0, ds):
        t[0, ::3], t[-1, 1::3] = float("inf"), -float("inf")
    h, state = ret.gated_recurrence(x, g, state_in=s0, state_out=True)
    assert torch.equal(state, s0) and torch.equal(h, s0[:, None].to(dtype).expand(B, N, D))
    dx, dg, ds0 = ret.gated_recurrence_backward(dh, x, g, h, state_in=s0, grad_state_out=ds, grad_state_in=True)
    assert torch.equal(ds0, ds) and not bool(dx.any()) and not bool(dg.any())


@pytest.mark.parametrize("form", ["sigmoid", "log"])
def test_a_step_resets_a_slot_of_any_contents(form):
    _announce(f"step resets {form}")
    x = _randn((3, 70), 1).to(DEV)
    pool = torch.stack([torch.full((70,), b) for b in _bad_values()]).to(DEV)
    slots = torch.tensor([2, 0, 1], dtype=torch.int32, device=DEV)
    h = ret.gated_recurrence_step(x, torch.full_like(x, -float("inf")), pool, form, slots=slots)
    assert torch.equal(h, x) and torch.equal(pool[slots.long()], x)
    pool = torch.full((1, 70), float("inf"), device=DEV)
    for _ in range(3):
        h = ret.gated_recurrence_step(x[:1], torch.full_like(x[:1], -1e-3 if form == "log" else 5.0), pool, form)
        assert not bool(h.isfinite().any())


@pytest.mark.parametrize("form", ["sigmoid", "log"])
def test_a_reset_ends_a_gate_of_nan(form):
    _announce(f"gate of nan {form}")
    B, N, D = 2, 1500, 40
    x, s0 = _randn((B, N, D), 1).to(DEV), _randn((B, D), 2).to(DEV)
    g = _mixed((B, N, D), form, 3).to(DEV)
    for at, reset in ((0, 1), (100, 103), (100, 900), (0, N - 1)):
        gr = g.clone()
        gr[1, reset, 7] = -float("inf")
        want = ret.gated_recurrence(x, gr, form, state_in=s0, state_out=True)
        gr[1, at, 7] = float("nan")
        h, s = ret.gated_recurrence(x, gr, form, state_in=s0, state_out=True)
        hit = torch.zeros(B, N, D, dtype=torch.bool, device=DEV)
        hit[1, at:reset, 7] = True
        assert torch.equal(h.isnan(), hit) and torch.equal(h[~hit], want[0][~hit]) and torch.equal(s, want[1])


# ---------------------------------------------------------------------------
# Norms whose workgroups take several turns


def _turns(rows, at_once, parts):
    return -(-rows // (at_once * parts))


def _head_plan(H, rows, d, dtype):
    """(turns of the forward, turns of the backward) of the gated norm, by the launches' rules."""
    V = 4 if dtype == F32 else 8
    at_once = 256 // (8 if d <= 8 * V else 16 if d <= 16 * V else 32 if d <= 32 * V else 64)
    want = -(-rows // at_once)
    back = max(512, min(4096, H * want // 8))
    return (_turns(rows, at_once, min(want, -(-4096 // H))), _turns(rows, at_once, min(want, -(-back // H))))


def _row_plan(rows, D):
    """The same of the residual norm."""
    at_once = 4 if D <= 1024 else 1
    want = -(-rows // at_once)
    back = 1024 if D <= 2048 else 512 if D <= 4096 else 256
    return _turns(rows, at_once, min(want, 4096)), _turns(rows, at_once, min(want, back))


@pytest.mark.parametrize("rms, gated, which", [(False, True, "wb"), (True, False, "w")])
@pytest.mark.parametrize("d, dtype", [(64, BF16), (33, BF16), (5, BF16), (128, BF16), (97, BF16), (256, BF16), (200, BF16), (512, BF16),
                                      (505, BF16), (1024, BF16), (1000, BF16), (32, F32), (61, F32), (128, F32), (97, F32), (256, F32),
                                      (512, F32), (1024, F32), (1001, F32)])
def test_gated_norm_backward_over_several_turns(d, dtype, rms, gated, which):
    """Two workgroups a head, four turns each, the last one partly past the rows; the batch's rows end inside a turn."""
    V = 4 if dtype == F32 else 8
    at_once = 256 // (8 if d <= 8 * V else 16 if d <= 16 * V else 32 if d <= 32 * V else 64)
    B, H, N = 2, 256, (7 * at_once - 2) // 2
    _announce(f"gated norm backward, turns {B, H, N, d} {dtype} rms={rms}")
    assert _head_plan(H, B * N, d, dtype)[1] >= 3 and N % (2 * at_once) and B * N % at_once
    shape = (B, H, N, d)
    o, dy = _randn(shape, 1, dtype, 2.0, 0.5), _randn(shape, 2, dtype)
    gate = _randn(shape, 3, dtype, 3.0) if gated else None
    w, b, params = _norm_params(H * d, 4, which)
    got = ret.gated_norm_backward(dy.to(DEV), o.to(DEV), None if gate is None else gate.to(DEV), ret.Norm(EPS, rms=rms, **params))
    args = (o, gate, w, b, EPS, rms)
    refs, errs = orc.gated_norm_backward(dy, *args), orc.gated_norm_backward_error(dy, *args)
    for t, ref, e, what in zip(got, refs, errs, ("grad_o", "grad_gate", "grad_weight", "grad_bias")):
        if t is not None:
            _check(t, ref, e, what)


@pytest.mark.parametrize("d, dtype", [(64, BF16), (33, BF16), (5, BF16), (128, BF16), (97, BF16), (256, BF16), (200, BF16), (512, BF16),
                                      (505, BF16), (1024, BF16), (1000, BF16), (32, F32), (61, F32), (128, F32), (97, F32), (256, F32),
                                      (512, F32), (1024, F32), (1001, F32)])
def test_gated_norm_over_several_turns(d, dtype):
    """256 heads, 16 workgroups each, four turns; some heads (rows do not meet) against the oracle."""
    V = 4 if dtype == F32 else 8
    at_once = 256 // (8 if d <= 8 * V else 16 if d <= 16 * V else 32 if d <= 32 * V else 64)
    B, H, N = 3, 256, 17 * at_once - 1
    _announce(f"gated norm, turns {B, H, N, d} {dtype}")
    assert _head_plan(H, B * N, d, dtype)[0] >= 4 and N % (16 * at_once) and B * N % at_once
    shape, heads = (B, H, N, d), [0, 1, 130, 255]
    gen = torch.Generator(DEV).manual_seed(d)
    o = (2 * torch.randn(shape, generator=gen, device=DEV) + 0.5).to(dtype)
    gate = (3 * torch.randn(shape, generator=gen, device=DEV)).to(dtype)
    w, b, params = _norm_params(H * d, 4, "wb")
    y = ret.gated_norm(o, gate, ret.Norm(EPS, **params))
    at = lambda p: p.view(H, d)[heads].reshape(-1)  # noqa: E731
    args = (o[:, heads].cpu(), gate[:, heads].cpu(), at(w), at(b), EPS, False)
    _check(y[:, heads], orc.gated_norm(*args), orc.gated_norm_error(*args), "y")
    assert not bool(y.isnan().any())


@pytest.mark.parametrize("B, N, D, dtype, stream", [
    (3, 4111, 7, BF16, F32), (2, 6163, 64, BF16, BF16), (3, 4111, 128, BF16, F32), (5, 2467, 97, F32, F32), (2, 6163, 500, BF16, BF16),
    (3, 4111, 512, BF16, F32), (2, 6163, 1000, BF16, BF16), (3, 1033, 1100, BF16, F32), (2, 1549, 2048, BF16, BF16), (3, 1033, 2048, F32, F32),
    (3, 517, 2100, BF16, BF16), (3, 517, 4096, BF16, F32), (5, 311, 4095, F32, F32)])
@pytest.mark.parametrize("rms, scaled, residual", [(False, True, False), (True, False, True)])
def test_residual_norm_backward_over_several_turns(B, N, D, dtype, stream, rms, scaled, residual):
    """Four turns a workgroup, the last one partly past the rows, and batches whose rows end inside a turn."""
    _announce(f"residual norm backward, turns {B, N, D} {dtype} {stream} rms={rms}")
    assert _row_plan(B * N, D)[1] >= 4
    shape = (B, N, D)
    x, res = _randn(shape, 1, dtype), _randn(shape, 2, stream, 2.0, 0.5)
    dy, dr = _randn(shape, 3, dtype), _randn(shape, 4, stream)
    scale = _randn((D,), 5, F32, 0.2, 0.7) if scaled else None
    w, b, params = _norm_params(D, 6, "wb")
    norm, alpha = ret.Norm(EPS, rms=rms, **params), 1.75 if scaled else 1.0
    sd = None if scale is None else scale.to(DEV)
    _, r = ret.residual_norm(x.to(DEV), res.to(DEV), norm, scale=sd, alpha=alpha)
    got = ret.residual_norm_backward(dy.to(DEV), None if residual else r, norm, grad_r=dr.to(DEV), x=x.to(DEV), scale=sd, alpha=alpha,
                                     residual=res.to(DEV) if residual else None)
    row = orc.residual_norm(x, res, w, b, EPS, rms, scale, alpha)[1] if residual else r.cpu()
    args = (dy, dr, row, w, EPS, rms, x, scale, alpha)
    refs, errs = orc.residual_norm_backward(*args), orc.residual_norm_backward_error(*args)
    grow = 1.0
    if residual:  # the row formed again: 4 steps of its terms, as in test_residual_norm_matches_the_oracle
        terms = np.abs(alpha * orc.f64(res)) + np.abs(orc.f64(x) * (1.0 if scale is None else orc.f64(scale)))
        grow = 1 + float((terms.max(-1) / np.abs(row).max(-1)).max())
    for t, ref, e, what in zip(got, refs, errs, ("grad_x", "grad_residual", "grad_scale", "grad_weight", "grad_bias")):
        if t is not None:
            _check(t, ref, grow * e, what)


@pytest.mark.parametrize("B, N, D, dtype, stream", [
    (3, 16411, 7, BF16, F32), (2, 24593, 64, BF16, BF16), (3, 16411, 97, F32, F32), (3, 16411, 500, BF16, F32), (2, 24593, 1000, BF16, BF16),
    (3, 4111, 1100, BF16, F32), (2, 6163, 2048, BF16, BF16), (3, 4111, 2100, F32, F32), (2, 6163, 4096, BF16, F32), (3, 4111, 5000, BF16, BF16)])
def test_residual_norm_over_several_turns(B, N, D, dtype, stream):
    """Four turns a workgroup: rows of every turn against the oracle, the rest against the same rows on their own."""
    _announce(f"residual norm, turns {B, N, D} {dtype} {stream}")
    assert _row_plan(B * N, D)[0] >= 4
    gen = torch.Generator(DEV).manual_seed(D)
    x = torch.randn((B, N, D), generator=gen, device=DEV).to(dtype)
    res = (2 * torch.randn((B, N, D), generator=gen, device=DEV) + 0.5).to(stream)
    w, b, params = _norm_params(D, 6, "wb")
    scale = _randn((D,), 5, F32, 0.2, 0.7)
    norm = ret.Norm(EPS, **params)
    y, r = ret.residual_norm(x, res, norm, scale=scale.to(DEV), alpha=1.75)
    rows = sorted({*range(0, B * N, 997), N - 1, N, B * N - 2, B * N - 1})
    args = (x.view(-1, D)[rows].cpu(), res.view(-1, D)[rows].cpu(), w, b, EPS, False, scale, 1.75)
    refs, errs = orc.residual_norm(*args), orc.residual_norm_error(*args)
    _check(y.view(-1, D)[rows], refs[0], errs[0], "y")
    _check(r.view(-1, D)[rows], refs[1], errs[1], "r")
    step = 4000  # at most one turn
    for at in range(0, B * N, step):
        some = slice(at, at + step)
        y1, r1 = ret.residual_norm(x.view(-1, D)[some], res.view(-1, D)[some], norm, scale=scale.to(DEV), alpha=1.75)
        assert torch.equal(y.view(-1, D)[some], y1) and torch.equal(r.view(-1, D)[some], r1)


# ---------------------------------------------------------------------------
# Layouts together


@pytest.mark.parametrize("dtype, form", [(BF16, "sigmoid"), (F32, "log"), (BF16, "log"), (F32, "sigmoid")])
@pytest.mark.parametrize("d, heads", [(72, 0), (33, 0), (24, 3), (7, 5), (200, 2)])
def test_packed_sequences_in_any_layout(d, heads, dtype, form):
    """Ragged sequences in slices of a fused projection, in token-major heads and in gradients side by side: to the bit
    those of contiguous tensors, and nothing beside them is written."""
    _announce(f"packed layouts {d} {heads} {dtype} {form}")
    lens = [300, 0, 1, 700, 65, 0, 2, 129]
    cu = torch.tensor(np.concatenate([[2], 2 + np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    T, S = int(cu[-1]) + 5, len(lens)
    lead, states = ((1, heads), (S, heads, d)) if heads else ((1,), (S, d))
    shape = (*lead, T, d)
    x, g, dh = (t.to(DEV) for t in (_randn(shape, 1, dtype), _gate(shape, 2, dtype, form), _randn(shape, 3, dtype)))
    s0, ds = _randn(states, 4).to(DEV), _randn(states, 5).to(DEV)
    zeros = lambda: torch.zeros(shape, dtype=dtype, device=DEV)  # noqa: E731
    want = ret.gated_recurrence(x, g, form, state_in=s0, state_out=True, cu_seqlens=cu, out=zeros())
    back = ret.gated_recurrence_backward(dh, x, g, want[0], form, state_in=s0, grad_state_out=ds, grad_state_in=True, cu_seqlens=cu,
                                         grads=(zeros(), zeros()))

    def fused(n):  # n tensors of this shape as columns of one [1, T, ...], heads token-major
        width = max(heads, 1) * d
        both = torch.full((1, T, n * width + 3), 5.0, dtype=dtype, device=DEV)
        cut = [both[..., 3 + i * width: 3 + (i + 1) * width] for i in range(n)]
        return both, [c.unflatten(-1, (heads, d)).transpose(1, 2) if heads else c for c in cut]

    _, (xf, gf, hf, dhf) = fused(4)
    for to, t in ((xf, x), (gf, g), (dhf, dh)):
        to.copy_(t)
    hf.zero_()
    _, s1 = ret.gated_recurrence(xf, gf, form, state_in=s0, state_out=True, cu_seqlens=cu, out=hf)
    assert torch.equal(hf, want[0]) and torch.equal(s1, want[1])
    whole, (dxf, dgf) = fused(2)
    dxf.zero_(), dgf.zero_()
    got = ret.gated_recurrence_backward(dhf, xf, gf, hf, form, state_in=s0, grad_state_out=ds, grad_state_in=True, cu_seqlens=cu,
                                        grads=(dxf, dgf))
    assert all(torch.equal(a, b) for a, b in zip(got, back))
    assert bool((whole[..., :3] == 5).all()) and bool((hf[..., :2, :] == 0).all()) and bool((dxf[..., T - 5:, :] == 0).all())


@pytest.mark.parametrize("shape, pitch, form, dtype", [
    ((1, 17600, 1001), 1001, "sigmoid", F32), ((3, 12000, 1003), 1010, "log", BF16), ((300, 130, 1000), 1004, "sigmoid", BF16),
    ((1, 17600, 1000), 1024, "log", F32), ((2, 12000, 2000), 2048, "sigmoid", BF16)])
def test_wide_gradients_in_rows_that_begin_anywhere(shape, pitch, form, dtype):
    """Gradients too large for the caches, in rows on cache lines and off them: some channels of a few rows against the
    oracle, and nothing written beside the rows."""
    _announce(f"wide gradients {shape} pitch {pitch} {form} {dtype}")
    B, N, D = shape
    at = [*range(10), *range(60, 70), *range(D - 70, D - 60), *range(D - 9, D)]
    x, g, dh, s0, ds = _randn(shape, 1, dtype), _gate(shape, 2, dtype, form), _randn(shape, 3, dtype), _randn((B, D), 4), _randn((B, D), 5)
    rows = [0, B - 1]
    some = [t[rows][..., at] for t in (dh, x, g)]
    s0s, dss = s0[rows][..., at], ds[rows][..., at]
    dev = [t.to(DEV) for t in (dh, x, g, s0, ds)]
    h = ret.gated_recurrence(dev[1], dev[2], form, state_in=dev[3])[0]
    wide = torch.full((2, B, N, pitch), float("nan"), dtype=dtype, device=DEV)
    dx, dg, ds0 = ret.gated_recurrence_backward(*dev[:3], h, form, state_in=dev[3], grad_state_out=dev[4], grad_state_in=True,
                                                grads=(wide[0, ..., :D], wide[1, ..., :D]))
    args = (*some, h[rows][..., at].cpu(), form, s0s, dss)
    refs, errs = orc.recurrence_backward(*args), orc.recurrence_backward_error(*args)
    for got, ref, e, what in zip((dx, dg, ds0), refs, errs, ("grad_x", "grad_gate", "grad_state_in")):
        _check(got[rows][..., at], ref, e, what)
    assert bool(torch.isnan(wide[..., D:]).all()) and not bool(torch.isnan(wide[..., :D]).any())


@pytest.mark.parametrize("shape, cu", [((1, 20000, 64), None), ((260, 300, 64), None), ((1, 4000, 40), [0, 3000, 3000, 3999])])
def test_the_status_word_says_that_every_wait_was_met(shape, cu):
    _announce(f"status word {shape}")
    x, g = _randn(shape, 1).to(DEV), _gate(shape, 2, F32, "log").to(DEV)
    cu = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    S = shape[0] if cu is None else cu.numel() - 1
    n = ret.gated_recurrence_workspace_bytes(S, 1, shape[1], shape[2], F32, max_len=None if cu is None else shape[1])
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    h, _ = ret.gated_recurrence(x, g, "log", workspace=ws, cu_seqlens=cu)
    assert ws[:4].tolist() == [255] * 4
    ws.zero_()
    ret.gated_recurrence_backward(x, None, g, h, "log", workspace=ws, cu_seqlens=cu)
    assert ws[:4].tolist() == [255] * 4


@pytest.mark.parametrize("shape, dtype, stream", [((1, 1), BF16, BF16), ((3, 65), BF16, F32), ((8, 4096), BF16, BF16), ((700, 1001), F32, F32),
                                                  ((5, 9001), BF16, F32), ((2, 9000, 1100), BF16, BF16), ((3, 17000, 97), BF16, F32),
                                                  ((4, 16383), BF16, BF16), ((4, 16384), F32, F32)])
@pytest.mark.parametrize("strided", [False, True])
def test_the_residual_stream_in_place(shape, dtype, stream, strided):
    """residual_out=residual gives what a tensor of its own gives, to the bit, odd widths (threads that read beside their
    own channels) and several turns a workgroup included."""
    _announce(f"residual in place {shape} {dtype} {stream} strided={strided}")
    gen = torch.Generator(DEV).manual_seed(len(shape))
    x = torch.randn(shape, generator=gen, device=DEV).to(dtype)
    res = torch.randn(shape, generator=gen, device=DEV).to(stream)
    norm = ret.Norm(EPS, _randn((shape[-1],), 1).to(DEV), rms=True)
    scale = _randn((shape[-1],), 2).to(DEV)
    want = ret.residual_norm(x, res, norm, scale=scale, alpha=1.25)
    place = _strided(res, 0) if strided else res.clone()
    y, r = ret.residual_norm(x, place, norm, scale=scale, alpha=1.25, residual_out=place)
    assert r is place and torch.equal(y, want[0]) and torch.equal(place, want[1])
