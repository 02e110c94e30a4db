"""The device checks of the log probabilities on the CPU: they accept outputs that are
right to fp32 and refuse ones that are not."""

import pytest
import torch

import probs_device as pd
from oracle.logprobs_oracle import log_probs

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="runs on the CPU")


def case(dtype, seed=1, t=30, d=24, v=300):
    h, w, y, g, e = pd.inputs(t, d, v, dtype, seed, dead=0.2)
    return h, w, dict(y=y, k=5, tau=0.8, g=g, e=e)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_accepts_what_is_right(dtype):
    h, w, kw = case(dtype)
    got = pd.plain(h, w, **kw)
    pd.check("plain", got, h, w, **kw)
    # the same numbers as the oracle's
    o = log_probs(h.double().numpy(), w.double().numpy(), kw["y"].numpy(), temperature=0.8, top_k=5,
                  grad_logprobs=kw["g"].double().numpy(), grad_entropy=kw["e"].double().numpy())
    for n, m in (("lse", "lse"), ("entropy", "entropy"), ("logprobs", "logprobs"), ("top_logprobs", "top_logprobs")):
        assert torch.allclose(got[n].double(), torch.from_numpy(o[m]), atol=1e-5), n
    assert (got["top_ids"].numpy() == o["top_ids"]).all()
    tol = 1e-6 if dtype == torch.float32 else 1e-2
    for n in ("dh", "dw"):
        ref = torch.from_numpy(o[n])
        assert float((got[n].double() - ref).norm()) <= tol * float(ref.norm()), n


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", ["lse", "entropy", "logprobs", "top_logprobs", "top_ids", "dh", "dw"])
def test_refuses_what_is_wrong(dtype, name):
    h, w, kw = case(dtype)
    got = pd.plain(h, w, **kw)
    live = int((kw["y"] != pd.IGN).nonzero()[0])
    if name == "top_ids":  # another id, an id twice, two that are exchanged
        for change in (lambda x: x[live].add_(1).remainder_(300), lambda x: x[live, 1:2].copy_(x[live, :1]),
                       lambda x: x[live].copy_(x[live].flip(0))):
            bad = {**got, name: got[name].clone()}
            change(bad[name])
            with pytest.raises(AssertionError):
                pd.check("bad", bad, h, w, **kw)
        return
    bad = {**got, name: got[name].clone()}
    bad[name].view(-1)[0 if name == "dw" else live * (bad[name].numel() // len(h))] += 0.05 * float(got[name].abs().max())
    with pytest.raises(AssertionError):
        pd.check("bad", bad, h, w, **kw)


def test_refuses_a_lost_entropy_gradient():
    h, w, kw = case(torch.float32)
    got = pd.plain(h, w, **{**kw, "e": None})
    with pytest.raises(AssertionError):
        pd.check("bad", got, h, w, **kw)


def test_grid_logits_are_exact():
    h, w, y = pd.grid_inputs(20, 100, 400, torch.float32, 3)
    s = h @ w.t()
    assert torch.equal(s.double(), h.double() @ w.double().t())
    assert torch.equal(s, sum(h[:, i:i + 1] * w[:, i] for i in range(100)))
    assert len(s[0].unique()) < 400  # some are equal
