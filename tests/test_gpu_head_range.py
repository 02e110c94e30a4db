"""fp32 rows of wide range: one element far larger than the others, against a zero
of the other operand, so that it takes no part in any logit.

Batches above the few-token forms multiply logits as two fp16 parts of rows scaled
by their largest element: such rows leave the others no bits.  The bounds are
test_gpu_head.py's, of the magnitudes that do meet; for rows whose range the two
parts are taken to hold, 2^-22 T more (include/dmuon_head.h).
"""

import numpy as np
import pytest
import torch

import head_device as dev

pytestmark = pytest.mark.gpu

# tokens, hidden, vocab: few-token form, 64 x 64, 256 x 256 and 256 x 128 tiles of two fp16 parts, pieces
SHAPES = [(200, 96, 700), (300, 96, 700), (1100, 130, 1001), (1300, 1000, 20001), (2100, 512, 20000)]


def _problem(t, d, v, seed, side, big):
    h, w, y, up = dev.inputs(t, d, v, torch.float32, seed, (0, v - 1))
    c = d // 3
    if side == "hidden":  # a channel that no word reads; its rows' other elements are ordinary
        w[:, c] = 0.0
        h[1::7, c] = big
    else:
        h[:, c] = 0.0
        w[2::11, c] = big
    return h, w, y, up


@pytest.mark.parametrize("side", ["hidden", "weight"])
@pytest.mark.parametrize("big", [2.0 ** 24, -2.0 ** 32, 2.0 ** 40, 1e30], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rows_of_wide_range(shape, big, side):
    print(f"case wide range {shape} {big} {side}", flush=True)
    t, d, v = shape
    h, w, y, up = _problem(t, d, v, t, side, big)
    gl = torch.full((t,), 0.3 / t, device="cuda")
    dev.check("ce", dev.run(h, w, up, y=y, gl=gl), h, w, up, y=y, gl=gl)


@pytest.mark.parametrize("side", ["hidden", "weight"])
@pytest.mark.parametrize("shape", SHAPES[1:], ids=str)
def test_rows_of_wide_range_distill(shape, side):
    print(f"case wide range, distillation {shape} {side}", flush=True)
    t, d, v = shape
    h, w, _, up = _problem(t, d, v, t + 1, side, 2.0 ** 36)
    # (many entries: small vocabularies then take the logits from the product itself)
    for k in (5, 200):
        ids, z = dev.teacher(t, k, v, 3, (0, v - 1))
        dev.check("kd", dev.run(h, w, up, ids=ids, z=z, tau=2.0), h, w, up, ids=ids, z=z, tau=2.0)


def test_ignored_rows_do_not_count():
    # a wide row without a loss: the call's results are those without it, bit for bit
    print("case ignored wide row", flush=True)
    t, d, v = 400, 128, 900
    h, w, y, up = dev.inputs(t, d, v, torch.float32, 8)
    y[5] = dev.IGN
    a = dev.run(h, w, up, y=y)
    h2 = h.clone()
    h2[5, 3] = 1e30
    b = dev.run(h2, w, up, y=y)
    assert all(torch.equal(a[n], b[n]) for n in ("losses", "lse", "dh", "dw"))


def test_wide_rows_of_one_piece_and_a_changing_range():
    # several pieces of W, the wide rows in the last one only; then the same call without them
    print("case one wide piece", flush=True)
    t, d, v = 2100, 512, 20000
    h, w, y, up = dev.inputs(t, d, v, torch.float32, 12, (0, v - 1))
    h[:, 7] = 0.0
    for big in (2.0 ** 40, 0.0, 2.0 ** 40):
        w[19990:, 7] = big
        dev.check(f"big {big}", dev.run(h, w, up, y=y), h, w, up, y=y)


@pytest.mark.parametrize("temperature", [1.0, 0.05])
def test_ranges_that_two_parts_hold(temperature):
    # 2^10 beside ordinary elements: within 2^-22 of s / T of the bound of ordinary rows.  One word: lse is s / T.
    print(f"case moderate range {temperature}", flush=True)
    t, d = 300, 64
    r = np.random.default_rng(3)
    h = r.standard_normal((t, d)).astype(np.float32)
    w = r.standard_normal((1, d)).astype(np.float32)
    w[:, 5] = 0.0
    h[:, 5] = 2.0 ** 10
    H, W = torch.from_numpy(h).cuda(), torch.from_numpy(w).cuda()
    ids, z = torch.zeros((t, 1), dtype=torch.int64, device="cuda"), torch.zeros((t, 1), device="cuda")
    got = dev.run(H, W, torch.ones(t, device="cuda"), ids=ids, z=z, tau=temperature)["lse"].cpu().double().numpy()
    ref = (h.astype(np.float64) @ w.astype(np.float64).T)[:, 0] / temperature
    mag = (np.abs(h).astype(np.float64) @ np.abs(w).astype(np.float64).T)[:, 0] / temperature
    # 6 x 64 products added up, 8 u32 of each left out, one rounding of lse; and 2^-22
    assert (np.abs(got - ref) <= (2 * 6 * 64 + 16) * 2.0 ** -24 * mag + 2.0 ** -22).all()


def test_captured_calls_follow_the_range():
    # one graph of forward and backward; its inputs' range changes between replays
    print("case graph, changing range", flush=True)
    t, d, v = 400, 96, 900
    h, w, y, up = dev.inputs(t, d, v, torch.float32, 20)
    w[:, 7] = 0.0
    ws = {n: dev.workspace(t, d, v, torch.float32) for n in ("graph", "eager")}

    def outs():
        f = lambda *s: torch.zeros(s, device="cuda")
        return [f(t), f(t), f(t, d), f(v, d)]

    def call(o, n):
        dev.hd.head_cross_entropy_forward(h, w, y, o[0], o[1], workspace=ws[n])
        dev.hd.head_cross_entropy_backward(h, w, y, o[1], up, o[2], o[3], workspace=ws[n])

    captured, eager = outs(), outs()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph):
            call(captured, "graph")
    torch.cuda.current_stream().wait_stream(side)
    for turn, big in enumerate((1.0, 2.0 ** 40, 1.0, -2.0 ** 30, 2.0 ** 40)):
        h[:, 7] = big
        call(eager, "eager")
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager)), turn
        got = dict(zip(("losses", "lse", "dh", "dw"), captured))
        dev.check(f"replay {turn}", got, h, w, up, y=y)
