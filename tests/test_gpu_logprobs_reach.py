"""Log probabilities at sizes that reach what is decided by sizes: chunks of tokens of
which the last takes other tiles, and dH's splits chosen on the device by the rows that
take part.  (tests/test_probs_layout.py holds that they do.)"""

import sys

import pytest
import torch

import probs_device as pd
from matrix_optimizer_02_amd import dmuon_logprobs as lp
from probs_device import BF16, F32

pytestmark = pytest.mark.gpu

# tokens, hidden, vocab, K: two chunks, the last of 20 tokens
CHUNKED = [(3348, 64, 600000, 5)]
ONE_CHUNK = [(3328, 64, 600000, 5)]
# tokens, hidden, vocab: one and two pieces of the vocabulary, the last one short
LIVE = [(2049, 2048, 8200), (2300, 1024, 20011), (3000, 700, 50257)]
DEAD = [0.0, 0.3, 0.7, 0.95, 0.9995]


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,dd,v,k", CHUNKED)
def test_a_last_chunk_of_other_tiles(t, dd, v, k, dtype):
    """The last rows with alternatives and without: other tiles (fp32: other parts of the operands too), both
    within the bounds."""
    say("last chunk", t, dd, v, k, dtype)
    h, w, y, _, _ = pd.inputs(t, dd, v, dtype, 5)
    for kk in (k, 0):
        got = pd.run(h, w, y, kk, 0.9)
        # rows on both sides of the boundary, and the first ones
        for rows in (slice(0, 40), slice(t - 60, t)):
            pd.check(f"K {kk} rows {rows}", {n: x[rows] for n, x in got.items()}, h[rows], w, y[rows], kk, 0.9, block=64)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,dd,v,k", ONE_CHUNK)
def test_statistics_do_not_depend_on_k_in_one_chunk(t, dd, v, k, dtype):
    say("one chunk", t, dd, v, k, dtype)
    h, w, y, _, _ = pd.inputs(t, dd, v, dtype, 6)
    a, b = pd.run(h, w, y, k), pd.run(h, w, y, 0)
    for n in ("lse", "entropy", "logprobs"):
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dead", DEAD)
@pytest.mark.parametrize("t,dd,v", LIVE)
def test_splits_by_the_rows_that_take_part(t, dd, v, dead):
    say("dead", t, dd, v, dead)
    h, w, y, g, e = pd.inputs(t, dd, v, BF16, t, dead)
    y[5], h[5], g[5], e[5] = 1, 0.5, 0.01, 0.01  # (one at least does)
    got = pd.run(h, w, y, 0, 1.0, g, e)
    pd.check(f"{t}x{dd}x{v}, {dead}", got, h, w, y, 0, 1.0, g, e, block=256)
    # and the same bits from call to call
    again = pd.run(h, w, y, 0, 1.0, g, e)
    for n in got:
        assert torch.equal(got[n], again[n]), n


@pytest.mark.parametrize("t,dd,v", [LIVE[0], LIVE[2]])
def test_replayed_with_other_splits(t, dd, v):
    """A captured training step whose rows that take part, and so dH's splits, change from replay to replay."""
    say("replayed", t, dd, v)
    h, w, y, g, e = pd.inputs(t, dd, v, BF16, 3)
    ws = pd.workspace(t, dd, v, BF16)
    f = lambda *s, dt=F32: torch.empty(s, dtype=dt, device="cuda")
    o = dict(lse=f(t), logprobs=f(t), entropy=f(t), dh=f(t, dd, dt=BF16), dw=f(v, dd, dt=BF16))

    def step():
        lp.head_log_probs_forward(h, w, y, o["logprobs"], o["entropy"], o["lse"], workspace=ws)
        lp.head_log_probs_backward(h, w, y, o["lse"], o["entropy"], g, e, o["dh"], o["dw"], workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    first, at = y.clone(), torch.rand(t, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    for dead in (0.0, 0.7, 0.3, 0.9995, 0.95, 1.0, 0.0):
        y.copy_(torch.where(at < dead, pd.IGN, first))
        graph.replay()
        torch.cuda.synchronize()
        got = {n: x.clone() for n, x in o.items()}
        for x in o.values():
            x.fill_(float("nan"))
        step()
        torch.cuda.synchronize()
        for n in o:
            assert torch.equal(got[n], o[n]), (dead, n)
        if dead in (0.7, 0.95):
            pd.check(f"{dead} dead", got, h, w, y, 0, 1.0, g, e, block=256)
