"""Pins of the block operators' fp64 oracle (CPU only): hand-worked values, closed forms, torch's own operators, central
differences and torch autograd through the definitions, and planted mistakes that the pins catch."""

import numpy as np
import pytest
import torch

from oracle import block_oracle as orc

RNG = np.random.default_rng(5)


def test_hand_worked_recurrence():
    # sigmoid(0) = 1/2: each token halves the distance to its input.
    h, end = orc.recurrence([[8.0], [4.0], [-2.0]], [[0.0], [0.0], [0.0]], "sigmoid")
    assert h[:, 0].tolist() == [4.0, 4.0, 1.0] and end.tolist() == [1.0]
    # log form, a = 1/2 from a starting state of 16.
    g = np.full((3, 1), -np.log(2.0))
    h, end = orc.recurrence([[0.0], [1.0], [0.0]], g, "log", [16.0])
    np.testing.assert_allclose(h[:, 0], [8.0, 5.0, 2.5], rtol=1e-15)
    # a gate of -inf starts the state anew.
    h, _ = orc.recurrence([[3.0], [5.0]], [[-np.inf], [-np.inf]], "sigmoid", [100.0])
    assert h[:, 0].tolist() == [3.0, 5.0]
    h, _ = orc.recurrence([[3.0], [5.0]], [[0.0], [-np.inf]], "log", [100.0])
    assert h[:, 0].tolist() == [103.0, 5.0]


def test_a_constant_gate_gives_the_geometric_series():
    a, n = 0.75, 40
    h, _ = orc.recurrence(np.ones((n, 1)), np.full((n, 1), np.log(a)), "log")
    np.testing.assert_allclose(h[:, 0], [(1 - a ** (t + 1)) / (1 - a) for t in range(n)], rtol=1e-13)
    h, _ = orc.recurrence(np.ones((n, 1)), np.full((n, 1), np.log(a / (1 - a))), "sigmoid")
    np.testing.assert_allclose(h[:, 0], [1 - a ** (t + 1) for t in range(n)], rtol=1e-13)


def test_decay_keeps_its_digits_on_both_sides():
    a, c = orc.decay(np.array([40.0, -40.0]), "sigmoid")
    np.testing.assert_allclose(c[0], np.exp(-40.0), rtol=1e-12)
    np.testing.assert_allclose(a[1], np.exp(-40.0), rtol=1e-12)
    np.testing.assert_allclose(a + c, 1.0, rtol=1e-15)


def _definition(x, g, form, s):
    a = torch.sigmoid(g) if form == "sigmoid" else torch.exp(g)
    now, out = s, []
    for t in range(x.shape[0]):
        now = a[t] * now + ((1 - a[t]) if form == "sigmoid" else 1.0) * x[t]
        out.append(now)
    return torch.stack(out), now


@pytest.mark.parametrize("form", ["sigmoid", "log"])
def test_recurrence_gradients_are_autograds_and_central_differences(form):
    n, d = 7, 3
    x, s = RNG.normal(size=(n, d)), RNG.normal(size=d)
    g = RNG.normal(size=(n, d)) if form == "sigmoid" else -RNG.exponential(size=(n, d))
    dh, ds = RNG.normal(size=(n, d)), RNG.normal(size=d)
    h, _ = orc.recurrence(x, g, form, s)
    dx, dg, dstate = orc.recurrence_backward(dh, x, g, h, form, s, ds)
    leaves = [torch.tensor(v, requires_grad=True) for v in (x, g, s)]
    th, tend = _definition(leaves[0], leaves[1], form, leaves[2])
    np.testing.assert_allclose(h, th.detach().numpy(), rtol=1e-12, atol=1e-13)
    want = torch.autograd.grad([th, tend], leaves, [torch.tensor(dh), torch.tensor(ds)])
    for got, w in zip((dx, dg, dstate), want):
        np.testing.assert_allclose(got, w.numpy(), rtol=1e-11, atol=1e-12)

    def loss(x, g, s):
        h, end = orc.recurrence(x, g, form, s)
        return (h * dh).sum() + (end * ds).sum()

    eps = 1e-6
    for at, got in ((0, dx), (1, dg), (2, dstate)):
        args = [x, g, s]
        for i in np.ndindex(*args[at].shape):
            up, down = [v.copy() for v in args], [v.copy() for v in args]
            up[at][i] += eps
            down[at][i] -= eps
            assert abs((loss(*up) - loss(*down)) / (2 * eps) - got[i]) < 1e-7


def test_norms_are_torchs():
    o, w, b = RNG.normal(size=(2, 3, 4, 10)), RNG.normal(size=30), RNG.normal(size=30)
    got = orc.gated_norm(o, None, w, b, 1e-5, False)
    want = torch.nn.functional.group_norm(torch.tensor(o).permute(0, 2, 1, 3).reshape(8, 30), 3, torch.tensor(w),
                                          torch.tensor(b), 1e-5)
    np.testing.assert_allclose(got, want.reshape(2, 4, 3, 10).permute(0, 2, 1, 3).numpy(), rtol=1e-11, atol=1e-12)
    got = orc.gated_norm(o[:, :1], None, w[:10], None, 1e-5, True)
    want = torch.nn.functional.rms_norm(torch.tensor(o[:, :1]), (10,), torch.tensor(w[:10]), 1e-5)
    np.testing.assert_allclose(got, want.numpy(), rtol=1e-11)
    np.testing.assert_allclose(orc.swish(o), torch.nn.functional.silu(torch.tensor(o)).numpy(), rtol=1e-13)
    y, r = orc.residual_norm(o, 2 * o, None, None, 1e-5, False, scale=np.full(10, 0.5), alpha=3.0)
    np.testing.assert_allclose(r, 6.5 * o)
    np.testing.assert_allclose(y, torch.nn.functional.layer_norm(torch.tensor(6.5 * o), (10,)).numpy(), rtol=1e-10, atol=1e-11)


def _torch_norm(v, rms):
    d = v if rms else v - v.mean(-1, keepdim=True)
    return d / torch.sqrt((d * d).mean(-1, keepdim=True) + 1e-5)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_gated_norm_gradients_are_autograds(rms, gated):
    B, H, N, d = 2, 3, 4, 5
    arrays = [RNG.normal(size=s) for s in ((B, H, N, d), (B, H, N, d), (H * d,), (H * d,))]
    dy = RNG.normal(size=(B, H, N, d))
    o, g, w, b = [torch.tensor(a, requires_grad=True) for a in arrays]
    y = _torch_norm(o, rms) * w.view(H, 1, d) + b.view(H, 1, d)
    if gated:
        y = y * torch.nn.functional.silu(g)
    want = torch.autograd.grad(y, [o, w, b] + ([g] if gated else []), torch.tensor(dy))
    gate = arrays[1] if gated else None
    np.testing.assert_allclose(orc.gated_norm(arrays[0], gate, arrays[2], arrays[3], 1e-5, rms), y.detach().numpy(), rtol=1e-11, atol=1e-12)
    do, dg, dw, db = orc.gated_norm_backward(dy, arrays[0], gate, arrays[2], arrays[3], 1e-5, rms)
    for got, ref in zip((do, dw, db, dg), want):
        np.testing.assert_allclose(got, ref.numpy(), rtol=1e-9, atol=1e-11)
    assert (dg is None) == (not gated)


@pytest.mark.parametrize("rms", [False, True])
def test_residual_norm_gradients_are_autograds(rms):
    shape, D = (2, 3, 6), 6
    x, res, scale, w, b = [torch.tensor(RNG.normal(size=s), requires_grad=True) for s in (shape, shape, (D,), (D,), (D,))]
    dy, dr = RNG.normal(size=shape), RNG.normal(size=shape)
    r = 1.75 * res + scale * x
    y = _torch_norm(r, rms) * w + b
    want = torch.autograd.grad([y, r], [x, res, scale, w, b], [torch.tensor(dy), torch.tensor(dr)])
    got = orc.residual_norm_backward(dy, dr, r, w, 1e-5, rms, x=x, scale=scale, alpha=1.75)
    for g, ref in zip(got, want):
        np.testing.assert_allclose(g, ref.numpy(), rtol=1e-9, atol=1e-11)


def test_planted_mistakes_are_seen():
    """The pins tell the formulas from near ones: a decay taken from the next token, the gate's factor a left out of its
    gradient, the h of the token itself for the one before it."""
    n, d = 6, 2
    x, g, dh = RNG.normal(size=(n, d)), RNG.normal(size=(n, d)), RNG.normal(size=(n, d))
    h, _ = orc.recurrence(x, g, "sigmoid")
    dx, dg, _ = orc.recurrence_backward(dh, x, g, h, "sigmoid")
    a, c = orc.decay(g, "sigmoid")
    shifted, _ = orc.recurrence(x, np.roll(g, -1, 0), "sigmoid")
    assert np.abs(shifted - h).max() > 1e-2
    u = dx / c
    assert np.abs(c * (np.vstack((np.zeros((1, d)), h[:-1])) - x) * u - dg).max() > 1e-2
    assert np.abs(a * c * (h - x) * u - dg).max() > 1e-2
