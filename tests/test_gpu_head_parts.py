"""fp32 operands of the output-head losses keep their bits: outputs that are one
product each (every other product of their sums is an exact 0), so that no
allowance for additions hides a part that was left out.

With u = 2^-24.  Three bf16 parts (rounded to nearest) leave less than 2^-26 of an
operand, two leave up to 2^-18.  The six products kept leave out 3 x 2^-27 of a
product; they are added smallest first, so two additions at most are of the whole's
size, 2 u each, the others of 2^-8 of it.

  * dW, dH at a target, where ds = g (p - 1) with p = 1 / V: dividing by the
    largest weight 2 u, the difference u, the parts 2 u, the products and their
    additions 5 u, the scale again 2 u, p's own error (2^-18 of p) below u for
    V >= 300.  13 u; held to 16 u = 2^-20.  Two parts miss it (2^-18 = 64 u, and a
    test below holds that they do).
  * logits from three bf16 parts: 6 u, held to 8 u; from two fp16 parts: 2^-22 = 4 u
    of each operand, 4 u of the dropped product, 4 u of additions: 16 u, held to
    20 u, and an element below 2^-17 of its row's largest 2^-39 of that.
  * p where two large logits share the mass: (logit's bound, twice: its own and
    lse's) |s| + lse's rounding and statistics + 8 u (1 + |x|), relative.
"""

import numpy as np
import pytest
import torch

import head_device as dev

gpu = pytest.mark.gpu
F32 = torch.float32
U = 2.0 ** -24

# (tokens, hidden, vocab): the tiles of dH and dW, in splits and not, from streamed and packed W
SHAPES = [(200, 96, 700), (1100, 96, 700), (2049, 200, 300), (400, 64, 40000), (300, 136, 3000), (250, 264, 100100), (600, 512, 30000), (1300, 1000, 20001), (1500, 1024, 40003),
          (3000, 256, 15001), (8192, 256, 30001), (2050, 1096, 33000)]


def _values(n, seed):
    """n fp32 numbers of full 24-bit mantissas, magnitudes in [1, 8)."""
    r = np.random.default_rng(seed)
    x = (1.0 + r.random(n)) * 2.0 ** r.integers(0, 3, n) * r.choice([-1.0, 1.0], n)
    return torch.from_numpy(x.astype(np.float32))


def _close(name, got, ref, rel, absolute=0.0):
    err = (got.double().cpu() - ref).abs()
    bound = rel * ref.abs() + absolute
    assert bool((err <= bound).all()), (name, float((err / ref.abs()).max() / U), "u; outside:", int((err > bound).sum()))


@gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_dw_is_one_product(shape):
    # W 0: every logit 0.  Column c of H is zero but for one token's element.
    print(f"case one product, dW {shape}", flush=True)
    t, d, v = shape
    n = min(t, d)
    at = torch.arange(n) * t // n
    h = torch.zeros(t, d)
    h[at, torch.arange(n)] = _values(n, 1)
    up = _values(t, 2) / t
    y = torch.from_numpy(np.random.default_rng(3).permutation(v)[torch.arange(t).numpy() % v]).long()
    y[0], y[at[-1]] = v - 1, 0
    got = dev.run(h.cuda(), torch.zeros(v, d, device="cuda"), up.cuda(), y=y.cuda())
    x, g = h[at, torch.arange(n)].double(), up[at].double()
    dw = got["dw"].cpu()
    _close("dW at targets", dw[y[at], torch.arange(n)], g * (1.0 / v - 1.0) * x, 16 * U)
    # the other words: p = 1 / V, whose lse is rounded: 2 u |lse|, the statistics, the exponential
    other = (y[at] + 1) % v
    p = (2 * 12 + 2 * (64 + v / 512 + 24) + 8 * 13) * U
    _close("dW elsewhere", dw[other, torch.arange(n)], g * x / v, p + 16 * U)


@gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_dh_is_one_product(shape):
    # H 0: every logit 0.  Column c of W is zero but for one word's element; a token's target is such a word.
    print(f"case one product, dH {shape}", flush=True)
    t, d, v = shape
    n = min(d, v)
    word = torch.arange(n) * v // n
    word[-1] = v - 1
    w = torch.zeros(v, d)
    w[word, torch.arange(n)] = _values(n, 4)
    up = _values(t, 5) / t
    c = torch.arange(t) % n
    got = dev.run(torch.zeros(t, d, device="cuda"), w.cuda(), up.cuda(), y=word[c].cuda())
    x = w[word, torch.arange(n)].double()
    _close("dH at targets", got["dh"].cpu()[torch.arange(t), c], up.double() * (1.0 / v - 1.0) * x[c], 16 * U)


# (tokens, hidden, vocab): logits kept by the call itself, from each tile of three and of two parts
KEPT = [(50, 128, 700), (40, 1024, 40000), (200, 512, 20000), (128, 512, 2500), (300, 512, 900), (300, 512, 20000), (1100, 640, 5000),
        (2100, 1024, 7000)]


@gpu
@pytest.mark.parametrize("shape", KEPT, ids=str)
def test_logits_are_one_product(shape):
    # one element a row of H; the logits come back as the student's
    print(f"case one product, logits {shape}", flush=True)
    t, d, v = shape
    k = 256
    h = torch.zeros(t, d)
    c = torch.arange(t) % d
    h[torch.arange(t), c] = _values(t, 6) / 4
    w = (_values(v * d, 7) / 8).view(v, d)
    ids = torch.from_numpy(np.random.default_rng(8).integers(0, v, (t, k)))
    ids[:, 0], ids[:, 1] = v - 1, 0
    got = dev.run(h.cuda(), w.cuda(), torch.ones(t, device="cuda"), ids=ids.cuda(), z=torch.zeros(t, k, device="cuda"))
    ref = h[torch.arange(t), c].double()[:, None] * w.double()[ids, c[:, None]]
    if t <= 256:
        _close("logits", got["student"], ref, 8 * U)
    else:
        rowmax = w.double().abs().max(1).values[ids] * h[torch.arange(t), c].double().abs()[:, None]
        _close("logits", got["student"], ref, 20 * U, 2.0 ** -39 * rowmax)


@gpu
@pytest.mark.parametrize("size", [20.0, 200.0])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_probabilities_from_large_logits(shape, size):
    # two words near s = size share the mass of the tokens that have an element; the target is a third one
    print(f"case large logits {shape} {size}", flush=True)
    t, d, v = shape
    n = min(t, d)
    at, cols = torch.arange(n) * t // n, torch.arange(n)
    r = np.random.default_rng(9)
    h = torch.zeros(t, d)
    h[at, cols] = torch.from_numpy((8.0 + 8.0 * r.random(n)).astype(np.float32))
    w = torch.zeros(v, d)
    pair = (1, v - 1)
    near = (size + r.random(n)) / h[at, cols].double().numpy()
    w[pair[0], cols] = torch.from_numpy(near.astype(np.float32))
    w[pair[1], cols] = torch.from_numpy((near * (1 + 0.01 * (r.random(n) - 0.5))).astype(np.float32))
    up = _values(t, 10) / t
    y = torch.full((t,), 2, dtype=torch.int64)
    got = dev.run(h.cuda(), w.cuda(), up.cuda(), y=y.cuda())
    x = h[at, cols].double()
    s = torch.stack([w[q, cols].double() * x for q in pair])
    lse = torch.logsumexp(torch.cat([s, torch.full((1, n), float(np.log(v - 2)), dtype=torch.float64)]), 0)  # the others: 0
    _close("lse", got["lse"].cpu()[at], lse, 0.0, (20 * s.max(0).values + 2 * lse + 2 * (64 + v / 512 + 24)) * U + 4 * U * size)
    parts = 40 if t > 256 else 16
    for i, q in enumerate(pair):
        arg = (s[i] - lse).abs()
        rel = (parts * s[i] + 2 * lse + 2 * (64 + v / 512 + 24) + 4 * size + 8 * (1 + arg) + 16) * U
        ref = up[at].double() * (s[i] - lse).exp() * x
        err = (got["dw"].cpu()[q, cols].double() - ref).abs()
        assert bool((err <= rel * ref.abs()).all()), (q, float((err / (rel * ref.abs())).max()))


def _parts(x, n):
    out = []
    for _ in range(n):
        b = x.bfloat16().float()
        out.append(b)
        x = x - b
    return [b.double() for b in out]


def test_two_parts_or_a_lost_product_miss_the_bounds():
    """The products as the kernels form them, on the CPU: all six of three parts lie
    within the bounds above, without any one of them, or with two parts, some do not."""
    x, y = _values(4000, 11), _values(4000, 12)
    ref = x.double() * y.double()
    a, b = _parts(x, 3), _parts(y, 3)
    kept = [(0, 0), (0, 1), (1, 0), (1, 1), (0, 2), (2, 0)]

    def worst(pairs):
        return float(((sum(a[i] * b[j] for i, j in pairs) - ref).abs() / ref.abs()).max() / U)

    assert worst(kept) < 1
    assert worst([(0, 0), (0, 1), (1, 0), (1, 1)]) > 32
    for lost in kept:
        assert worst([q for q in kept if q != lost]) > 32, lost
