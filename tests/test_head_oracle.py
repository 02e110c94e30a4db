"""Pins of the head losses' fp64 oracle: torch's own float64 losses and their
autograd on the CPU, closed forms, and differences."""

import numpy as np
import pytest
import torch

from oracle import head_oracle as ho

RNG = np.random.default_rng


def _problem(seed, t=7, d=5, v=11):
    r = RNG(seed)
    return r.standard_normal((t, d)), r.standard_normal((v, d)), r.integers(0, v, t), r.standard_normal(t)


def test_cross_entropy_matches_torch_float64():
    h, w, y, g = _problem(1)
    y[2] = y[5] = -100
    H, W = torch.tensor(h, requires_grad=True), torch.tensor(w, requires_grad=True)
    s = H @ W.T
    losses = torch.nn.functional.cross_entropy(s, torch.tensor(y), ignore_index=-100, reduction="none")
    live = torch.tensor(y != -100)
    lse = torch.logsumexp(s, 1) * live
    gl = np.linspace(-1, 1, 7)
    ((losses * torch.tensor(g)).sum() + (lse * torch.tensor(gl)).sum()).backward()
    o = ho.cross_entropy(h, w, y, -100, g, gl)
    np.testing.assert_allclose(o["losses"], losses.detach().numpy(), rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(o["lse"], lse.detach().numpy(), rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(o["dh"], H.grad.numpy(), rtol=1e-11, atol=1e-13)
    np.testing.assert_allclose(o["dw"], W.grad.numpy(), rtol=1e-11, atol=1e-13)


@pytest.mark.parametrize("tau", [1.0, 2.0, 0.7])
def test_distill_matches_torch_float64(tau):
    h, w, _, g = _problem(2)
    r = RNG(3)
    ids = np.stack([r.permutation(11)[:4] for _ in range(7)])
    ids[1, 2:] = -1
    ids[3] = -1
    ids[4, 1] = ids[4, 0]  # an id held twice
    z = r.standard_normal((7, 4)) * 2
    H, W = torch.tensor(h, requires_grad=True), torch.tensor(w, requires_grad=True)
    logp = torch.log_softmax(H @ W.T / tau, 1)
    total, losses = 0.0, []
    for t in range(7):
        sel = ids[t] >= 0
        if not sel.any():
            losses.append(0.0)
            continue
        q = torch.softmax(torch.tensor(z[t][sel]) / tau, 0)
        loss = tau ** 2 * (q * (torch.log(q) - logp[t][torch.tensor(ids[t][sel])])).sum()
        losses.append(loss.item())
        total = total + g[t] * loss
    total.backward()
    o = ho.distill(h, w, ids, z, tau, g)
    np.testing.assert_allclose(o["losses"], losses, rtol=1e-11, atol=1e-13)
    np.testing.assert_allclose(o["dh"], H.grad.numpy(), rtol=1e-10, atol=1e-13)
    np.testing.assert_allclose(o["dw"], W.grad.numpy(), rtol=1e-10, atol=1e-13)


def test_gradients_against_differences():
    h, w, y, g = _problem(4)
    ids, z = np.array([[0, 3, 5]] * 7), RNG(5).standard_normal((7, 3))
    e = RNG(6).standard_normal(w.shape)
    step = 1e-5
    for f in (lambda x: ho.cross_entropy(h, x, y, -100, g), lambda x: ho.distill(h, x, ids, z, 1.7, g)):
        diff = ((f(w + step * e)["losses"] - f(w - step * e)["losses"]) @ g) / (2 * step)
        # the third derivatives are of order 10: step^2 of them, and 1e-16 / step of rounding
        assert abs(diff - (f(w)["dw"] * e).sum()) < 1e-7 * max(1.0, abs(diff))


def test_closed_forms():
    # equal logits: lse = log v, loss = log v; a teacher equal to the student loses nothing
    h, w = np.zeros((3, 4)), np.ones((8, 4))
    o = ho.cross_entropy(h, w, np.array([0, 7, -100]))
    np.testing.assert_allclose(o["losses"], [np.log(8), np.log(8), 0.0])
    ids = np.tile(np.arange(8), (3, 1))
    h = RNG(7).standard_normal((3, 4))
    w = RNG(8).standard_normal((8, 4))
    o = ho.distill(h, w, ids, h @ w.T, 3.0, np.ones(3))
    np.testing.assert_allclose(o["losses"], 0.0, atol=1e-13)
    np.testing.assert_allclose(o["dw"], 0.0, atol=1e-13)
