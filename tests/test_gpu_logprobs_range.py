"""Words that a mask pushes to the end of the range by finite weights (fp32: of magnitude up
to 3e38): logits may still be -inf, and gradients are those of the words left."""

import math
import sys

import pytest
import torch

import probs_device as pd
from probs_device import BF16, F32

pytestmark = pytest.mark.gpu


def masked(t, v, first, last, dd):
    """One column carries the logits: h is `first` there, and words 100 .. 399 hold -3e38."""
    w = torch.zeros(v, dd, device="cuda")
    w[:, 0] = (torch.arange(v, device="cuda") % 7 - 3.0) / first
    w[100:400, 0] = -3e38
    h = torch.zeros(t, dd, device="cuda")
    h[:, 0] = first
    y = torch.full((t,), 3, device="cuda")
    y[-1] = last
    return h, w, y


@pytest.mark.parametrize("t", [1, 70, 300, 600])
@pytest.mark.parametrize("first", [1.0, 2.0])
def test_masked_words_fp32(t, first):
    """Logits of -3e38, or of -inf by overflow: probability 0, no NaN in the sums.  (300 and 600 tokens: the
    logits' two fp16 parts, formed again in three because of the rows' range.)"""
    print("masked", t, first, flush=True)
    sys.stdout.flush()
    v, dd, k = 500, 40, 125
    h, w, y = masked(t, v, first, 250, dd)
    g = torch.full((t,), 1.0 / t, device="cuda")
    got = pd.run(h, w, y, k, 1.0)
    open_ = torch.cat([w[:100, 0], w[400:, 0]]).double() * first
    logp = torch.log_softmax(open_, 0)
    ent = float(-(logp.exp() * logp).sum())
    # sums of 200 terms of one size and logits exact: a few roundings of values below 8
    assert torch.allclose(got["entropy"], torch.full((t,), ent, device="cuda"), rtol=1e-5)
    assert torch.allclose(got["logprobs"][:-1], torch.full((t - 1,), float(logp[3]), device="cuda"), rtol=1e-5)
    assert float(got["logprobs"][-1]) <= -1e38
    # the 125 best of the 200 words that are not masked
    want = torch.sort((w[:, 0].double() * first).float(), descending=True, stable=True).indices[:k]
    assert torch.equal(got["top_ids"], want.expand(t, k))
    # fewer words above -inf than alternatives
    w[4:, 0] = -3e38
    got = pd.run(h, w, None, 9, 1.0)
    ids = [3, 2, 1, 0] + ([-1] * 5 if first == 2.0 else [4, 5, 6, 7, 8])
    assert torch.equal(got["top_ids"], torch.tensor(ids, device="cuda").expand(t, 9))
    assert bool(got["top_logprobs"][:, :4].isfinite().all()) and bool((got["top_logprobs"][:, 4:] <= -1e38).all())
    assert first == 1.0 or bool((got["top_logprobs"][:, 4:] == -math.inf).all())
    # gradients of the words that are open, as if there were no others
    y = torch.zeros(t, dtype=torch.int64, device="cuda")
    got = pd.run(h, w, y, 0, 1.0, g, None)
    p = torch.softmax(w[:4, 0].double() * first, 0)
    want = torch.zeros(v, dtype=torch.float64, device="cuda")
    want[:4] = -p
    want[0] += 1.0
    assert bool((got["dw"][4:] == 0).all())
    assert torch.allclose(got["dw"][:, 0].double(), want * float(g.double().sum()) * first, rtol=1e-5, atol=1e-9)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t", [1, 70, 300, 1100])
@pytest.mark.parametrize("first", [1.0, 2.0])
def test_gradients_of_masked_words(t, first, dtype):
    """dH and dW with and without entropy's gradient, against a head of the open words alone."""
    print("masked gradients", t, first, dtype, flush=True)
    v, dd = 700, 64
    gen = torch.Generator("cuda").manual_seed(t)
    low = torch.finfo(BF16).min if dtype == BF16 else -3e38
    w = torch.randn(v, dd, device="cuda", generator=gen).mul_(0.2).to(dtype)
    h = torch.randn(t, dd, device="cuda", generator=gen).to(dtype)
    h[:, 0] = first
    mask = torch.rand(v, device="cuda", generator=gen) < 0.3
    mask[:300] = False
    w[mask] = 0
    w[mask, 0] = low
    y = torch.randint(0, 300, (t,), device="cuda", generator=gen)
    g = torch.randn(t, device="cuda", generator=gen) / t
    e = torch.randn(t, device="cuda", generator=gen) * 0.1 / t
    left = w[~mask].contiguous()
    new = torch.cumsum(~mask, 0) - 1
    for up in ((g, None), (None, e), (g, e)):
        got = pd.run(h, w, y, 0, 1.0, *up)
        of_left = {n: x if n != "dw" else x[~mask] for n, x in got.items()}
        pd.check(f"{t} masked", of_left, h, left, new[y], 0, 1.0, *up)
        assert bool((got["dw"][mask] == 0).all())
