"""The log probabilities' oracle against direct sums and against differences."""

import numpy as np
import pytest

from oracle.logprobs_oracle import log_probs


def problem(t=5, d=4, v=9, seed=0):
    rng = np.random.default_rng(seed)
    h, w = rng.standard_normal((t, d)), rng.standard_normal((v, d))
    y = rng.integers(0, v, t)
    y[1] = -100
    return h, w, y, rng.standard_normal(t), rng.standard_normal(t)


@pytest.mark.parametrize("tau", [1.0, 0.6, 3.0])
def test_direct_sums(tau):
    h, w, y, _, _ = problem()
    o = log_probs(h, w, y, temperature=tau, top_k=4)
    for t in range(5):
        p = np.exp(h[t] @ w.T / tau)
        p /= p.sum()
        if t == 1:
            assert o["logprobs"][t] == o["entropy"][t] == o["lse"][t] == 0.0 and (o["top_ids"][t] == -1).all()
            continue
        assert abs(o["logprobs"][t] - np.log(p[y[t]])) < 1e-12
        assert abs(o["entropy"][t] + (p * np.log(p)).sum()) < 1e-12
        order = sorted(range(9), key=lambda i: (-p[i], i))[:4]
        assert list(o["top_ids"][t]) == order and np.allclose(o["top_logprobs"][t], np.log(p[order]), atol=1e-12)


def test_equal_logits_by_the_lower_id():
    o = log_probs(np.zeros((1, 3)), np.ones((7, 3)), top_k=3)
    assert list(o["top_ids"][0]) == [0, 1, 2] and abs(o["entropy"][0] - np.log(7)) < 1e-12


@pytest.mark.parametrize("tau", [1.0, 0.7])
def test_gradients_against_differences(tau):
    h, w, y, g, e = problem(seed=3)
    o = log_probs(h, w, y, temperature=tau, grad_logprobs=g, grad_entropy=e)

    def value(h, w):
        r = log_probs(h, w, y, temperature=tau)
        return (g * r["logprobs"]).sum() + (e * r["entropy"]).sum()

    for x, grad in ((h, o["dh"]), (w, o["dw"])):
        for i in np.ndindex(*x.shape):
            keep, step = x[i], 1e-5
            x[i] = keep + step
            up = value(h, w)
            x[i] = keep - step
            down = value(h, w)
            x[i] = keep
            assert abs((up - down) / (2 * step) - grad[i]) < 1e-8 * (1 + abs(grad[i])) + 1e-9, i
