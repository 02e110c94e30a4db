"""GPU parity of the output-head losses (through the C ABI) against the fp64
oracle, element by element, with bounds derived from the arithmetic.

With A = |H| |W|^T and u32 = 2^-24, u16 = 2^-8 (half a step of bf16):
  * a logit is a sum of D exact products in fp32, every addition off by at most
    2 u32 of the running sum of magnitudes.  fp32 operands are multiplied in parts:
    6 D products of three bf16 parts, which leave out at most 3 x 2^-24 = 3 u32 of
    each, or 3 D products of two fp16 parts (the row scaled so that its largest
    element is near 2^14), which leave out 2^-21 = 8 u32 of each and, where a low
    part is a subnormal of fp16, 2^-39 of the row's largest element.  The second
    form is charged 6 D additions too, which is far more than it leaves out:
        es = (2 D' + 8) u32 A,  D' = D (bf16) or 6 D (fp32), padded to slabs
  * lse: the largest es of the row over T, the sum over the vocabulary in chains
    of at most 64 + 2 parts/16 + 16 additions and exponentials good to 4 u32 with
    arguments x rounded by 2 u32 |x|:
        el = max es / T + (chain + 8) 2 u32 + 4 u32 xmax + 2 u32 |lse|
  * p = exp(s / T - lse): ep = p (es / T + el + 8 u32 (1 + |x|)), ds = cp p - ct q:
        ed = cp ep + 8 u32 (cp p + ct q) + ur |ds|,
    ur the rounding of ds as an operand: u16 (bf16), 2^-15 (bf16 of at most 128
    tokens: two parts leave u16^2), 2^-22 (fp32, three parts);
    below 2^-126 the device's exponentials and products may be 0, so p, cp p and
    ds are each also off by up to 2^-126: (cp + 2) 2^-126 more
  * dH = ds W:  ed |W| + (2 V' + 64) u32 |ds| |W| + out |dH|,  V' terms as D';
    dW the same over the tokens; out = u16 (bf16) or 2 u32.
"""

import sys

import numpy as np
import pytest
import torch

from matrix_optimizer_02_amd import dmuon_head as hd
from matrix_optimizer_02_amd import dmuon_ns as dn
from oracle import adamw_step, head_oracle as ho

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8
IGN = -100
BF16, F32 = torch.bfloat16, torch.float32


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


class Guarded:
    """A device tensor inside a larger one whose rest must stay untouched."""

    def __init__(self, shape, dtype):
        n = int(np.prod(shape)) if len(shape) else 1
        self.pad = 64
        self.all = torch.full((n + 2 * self.pad,), 7.0, dtype=dtype, device="cuda")
        self.t = self.all[self.pad:self.pad + n].view(shape)
        self.t.fill_(float("nan"))

    def check(self, what):
        n = self.all.numel()
        assert bool((self.all[:self.pad] == 7.0).all()) and bool((self.all[n - self.pad:] == 7.0).all()), what


def workspace(t, d, v, dtype, k=0, extra=0):
    ws = hd.workspace_for(t + extra, d, v, dtype, top_k=k)
    ws.fill_(0xFF)  # NaN patterns: what a call reads it must have written
    return ws


def within(name, got, ref, bound):
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(np.isnan(err), np.inf, err / np.maximum(bound, 1e-300))), err.shape)
        raise AssertionError(f"{name}{i}: gpu {got[i]!r} ref {ref[i]!r} err {err[i]:.3e} bound {bound[i]:.3e}; "
                             f"{bad.sum()} of {bad.size} outside")


def bounds(o, h, w, tau, dtype, losses_extra=0.0):
    live = o["live"]
    H = np.where(live[:, None], np.abs(h), 0.0)
    A = H @ np.abs(w).T
    d, v = w.shape[1], w.shape[0]
    mul = 1 if dtype == BF16 else 6
    pad = lambda x: max(128, (x + 255) // 256 * 256)
    es = (2 * mul * pad(d) + 8) * U32 * A
    x = o["s"] / tau - o["lse"][:, None]
    chain = 64 + 2 * (v / 64 / 16 + 1) + 16
    el = es.max(axis=1) / tau + (chain + 8) * 2 * U32 + 4 * U32 * np.abs(x).max(axis=1) + 2 * U32 * np.abs(o["lse"])
    el = np.where(live, el, 0.0)
    b = {"es": es, "lse": el}
    if "ds" in o:
        ur = 2.0 ** -22 if dtype == F32 else U16 if len(h) > 128 else 2.0 ** -15
        ep = o["p"] * (es / tau + el[:, None] + 8 * U32 * (1 + np.abs(x)))
        # a temperature scales s inside p only: ds carries it in cp and ct already
        ed = o["cp"] * ep + 8 * U32 * (o["cp"] * o["p"] + o["ct"] * o["hot"])
        ed = np.where(live[:, None], ed + ur * (np.abs(o["ds"]) + ed) + (o["cp"] + 2) * 2.0 ** -126, 0.0)
        out = U16 if dtype == BF16 else 2 * U32
        mag = np.abs(o["ds"]) + ed
        b["dh"] = (ed @ np.abs(w) + (2 * mul * pad(v) + 64) * U32 * (mag @ np.abs(w))) * (1 + out) + out * np.abs(o["dh"])
        b["dw"] = (ed.T @ H + (2 * mul * pad(len(h)) + 64) * U32 * (mag.T @ H)) * (1 + out) + out * np.abs(o["dw"])
        b["ed"] = ed
    return b


def make(t, d, v, dtype, seed, live=None):
    r = np.random.default_rng(seed)
    w = torch.from_numpy((r.standard_normal((v, d)) * 1.3 / np.sqrt(d)).astype(np.float32)).to(dtype)
    y = torch.from_numpy(r.integers(0, v, t))
    h = r.standard_normal((t, d)).astype(np.float32) + (r.random((t, 1)) * 6).astype(np.float32) * f64(w)[f64(y).astype(int)]
    h = torch.from_numpy(h.astype(np.float32)).to(dtype)
    g = torch.from_numpy((r.standard_normal(t) / max(t, 1)).astype(np.float32))
    if live is not None:
        y[~torch.from_numpy(live)] = IGN
        h[~torch.from_numpy(live)] = float("nan")  # nothing of these rows may be used
        g[~torch.from_numpy(live)] = float("nan")
    return h, w, y, g


def run_ce(h, w, y, g, gl=None, ws=None, stream=None):
    t, d, v, dtype = h.shape[0], h.shape[1], w.shape[0], h.dtype
    ws = workspace(t, d, v, dtype) if ws is None else ws
    H, W, Y, G = h.cuda(), w.cuda(), y.cuda(), g.cuda()
    GL = None if gl is None else gl.cuda()
    o = {n: Guarded(s, dt) for n, s, dt in (("losses", (t,), F32), ("lse", (t,), F32), ("dh", (t, d), dtype),
                                            ("dw", (v, d), dtype))}
    hd.head_cross_entropy_forward(H, W, Y, o["losses"].t, o["lse"].t, ignore_index=IGN, workspace=ws)
    hd.head_cross_entropy_backward(H, W, Y, o["lse"].t, G, o["dh"].t, o["dw"].t, grad_lse=GL, ignore_index=IGN,
                                   workspace=ws)
    torch.cuda.synchronize()
    for n, x in o.items():
        x.check(n)
    return {n: x.t for n, x in o.items()}


def check_ce(h, w, y, g, gl, got, what):
    hh, ww = f64(h), f64(w)
    o = ho.cross_entropy(hh, ww, y.numpy(), IGN, f64(g), None if gl is None else f64(gl))
    b = bounds(o, hh, ww, 1.0, h.dtype)
    rows = np.arange(len(y))
    at = np.where(o["live"], y.numpy(), 0)
    within(what + " lse", f64(got["lse"]), o["lse"], b["lse"])
    within(what + " losses", f64(got["losses"]), o["losses"],
           np.where(o["live"], b["lse"] + b["es"][rows, at] + 2 * U32 * np.abs(o["losses"]), 0.0))
    within(what + " dh", f64(got["dh"]), o["dh"], b["dh"])
    within(what + " dw", f64(got["dw"]), o["dw"], b["dw"])


# tokens, hidden, vocab: one of each, odd widths (packed rows), tile and slab edges, several pieces of the vocabulary
SHAPES = [(1, 64, 1), (1, 128, 257), (2, 5, 3), (3, 1, 300), (63, 192, 256), (64, 128, 1000), (65, 130, 1001),
          (127, 256, 255), (128, 64, 256), (129, 72, 513), (200, 448, 300), (256, 320, 512), (257, 129, 300),
          (300, 512, 777), (40, 128, 20000), (300, 128, 9000), (70, 100, 17000)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_cross_entropy_parity(shape, dtype):
    t, d, v = shape
    say(f"case cross entropy {shape} {dtype}")
    h, w, y, g = make(t, d, v, dtype, 100 + t)
    check_ce(h, w, y, g, None, run_ce(h, w, y, g), str(shape))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("mask", ["none", "all", "one", "last", "alternate", "prompt"])
@pytest.mark.parametrize("t", [1, 50, 300])
def test_cross_entropy_masked_rows_hold_nan(mask, t, dtype):
    live = {"none": np.ones(t, bool), "all": np.zeros(t, bool), "one": np.arange(t) == 0,
            "last": np.arange(t) == t - 1, "alternate": np.arange(t) % 2 == 1, "prompt": np.arange(t) >= t // 3}[mask]
    say(f"case masked {mask} t {t} {dtype}")
    h, w, y, g = make(t, 136, 700, dtype, 7 + t, live)
    gl = torch.from_numpy(np.random.default_rng(t).standard_normal(t).astype(np.float32) / t)
    got = run_ce(h, w, y, g, gl)
    clean = torch.where(torch.from_numpy(live)[:, None], h.float(), torch.zeros(())).to(dtype)
    check_ce(clean, w, y, torch.nan_to_num(g), gl, got, mask)
    dead = ~torch.from_numpy(live)
    assert not got["dh"].cpu()[dead].float().any() and not got["losses"].cpu()[dead].any()
    assert not got["lse"].cpu()[dead].any()


def teacher(t, k, v, seed, kind):
    r = np.random.default_rng(seed)
    ids = np.stack([r.permutation(v)[:k] if v >= k else r.integers(0, v, k) for _ in range(t)]).astype(np.int64)
    z = (r.standard_normal((t, k)) * 2 + 5).astype(np.float32)
    if kind == "ragged":
        held = r.integers(0, k + 1, (t, 1))
        ids = np.where(np.arange(k) < held, ids, -1 - np.arange(k))
        z = np.where(ids >= 0, z, np.float32("nan"))  # absent entries' logits are not used
    elif kind == "repeated":
        ids[:, k // 2:] = ids[:, :k - k // 2]
    elif kind == "masked":
        z[:, ::2] = -np.inf
        z[0] = -np.inf
        z[-1, :] = np.finfo(np.float32).min  # the lowest value: equal entries, not absent ones
    elif kind == "empty":
        ids[:] = -1
    return torch.from_numpy(ids), torch.from_numpy(z)


def run_kd(h, w, ids, z, g, tau, ws=None):
    t, d, v, k, dtype = h.shape[0], h.shape[1], w.shape[0], ids.shape[1], h.dtype
    ws = workspace(t, d, v, dtype, k) if ws is None else ws
    H, W, I, Z, G = h.cuda(), w.cuda(), ids.cuda(), z.cuda(), g.cuda()
    o = {n: Guarded(s, dt) for n, s, dt in (("losses", (t,), F32), ("lse", (t,), F32), ("student", (t, k), F32),
                                            ("dh", (t, d), dtype), ("dw", (v, d), dtype))}
    hd.head_distill_forward(H, W, I, Z, o["losses"].t, o["lse"].t, o["student"].t, temperature=tau, workspace=ws)
    hd.head_distill_backward(H, W, I, Z, o["lse"].t, o["student"].t, G, o["dh"].t, o["dw"].t, temperature=tau,
                             workspace=ws)
    torch.cuda.synchronize()
    for n, x in o.items():
        x.check(n)
    return {n: x.t for n, x in o.items()}


def check_kd(h, w, ids, z, g, tau, got, what):
    hh, ww, ii = f64(h), f64(w), ids.numpy()
    o = ho.distill(hh, ww, ii, f64(z), tau, f64(g))
    b = bounds(o, hh, ww, tau, h.dtype)
    es_k = np.take_along_axis(b["es"], np.maximum(ii, 0), axis=1)
    es_k = np.where((ii >= 0) & o["live"][:, None], es_k, 0.0)
    within(what + " lse", f64(got["lse"]), o["lse"], b["lse"])
    within(what + " student", f64(got["student"]), o["student"], es_k)
    # per entry: q off by 16 u32 (1 + |z/T|), the bracket by es / T, lse's error and a few roundings
    zt = np.where(o["q"] > 0, np.abs(np.nan_to_num(f64(z), posinf=0.0, neginf=0.0)) / tau, 0.0)
    zt = np.minimum(zt, 1e3)  # (the lowest value: exact differences)
    logq = np.where(o["q"] > 0, np.log(np.maximum(o["q"], 1e-300)), 0.0)
    bracket = np.abs(logq) + np.abs(o["student"]) / tau + np.abs(o["lse"])[:, None]
    k = ii.shape[1]
    lb = tau ** 2 * (o["q"] * (es_k / tau + b["lse"][:, None] + (16 * (1 + zt) + k + 8) * U32 * (1 + bracket))).sum(1)
    within(what + " losses", f64(got["losses"]), o["losses"], np.where(o["live"], lb * 2 + 1e-30, 0.0))
    # q's own rounding in ds: at most (16 (1 + |z/T|) + K) u32 q
    dq = np.zeros_like(o["ds"])
    for t in range(len(ii)):
        sel = o["q"][t] > 0
        np.add.at(dq[t], ii[t][sel], ((16 * (1 + zt[t]) + k) * U32 * o["q"][t])[sel])
    dq *= o["ct"]
    within(what + " dh", f64(got["dh"]), o["dh"], b["dh"] + 2 * dq @ np.abs(ww))
    H = np.where(o["live"][:, None], np.abs(hh), 0.0)
    within(what + " dw", f64(got["dw"]), o["dw"], b["dw"] + 2 * dq.T @ H)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape,k,kind,tau", [
    ((1, 64, 1), 1, "full", 1.0), ((1, 130, 257), 3, "full", 2.0), ((2, 5, 3), 3, "repeated", 0.5),
    ((64, 128, 1000), 8, "ragged", 1.0), ((65, 130, 1001), 65, "ragged", 2.0), ((129, 72, 513), 20, "repeated", 1.5),
    ((200, 448, 300), 300, "full", 4.0), ((300, 512, 777), 50, "ragged", 1.0), ((257, 129, 300), 7, "masked", 2.0),
    ((30, 64, 100), 4, "empty", 1.0), ((40, 128, 20000), 64, "ragged", 2.0), ((300, 128, 9000), 33, "full", 1.0),
    ((3, 64, 2000), 1024, "ragged", 3.0)], ids=str)
def test_distill_parity(shape, k, kind, tau, dtype):
    t, d, v = shape
    say(f"case distill {shape} k {k} {kind} tau {tau} {dtype}")
    h, w, _, g = make(t, d, v, dtype, 200 + t)
    ids, z = teacher(t, k, v, 300 + t, kind)
    dead = ~(((ids >= 0) & ~(z == -np.inf)).any(1))
    h[dead] = float("nan")
    got = run_kd(h, w, ids, z, g, tau)
    h[dead] = 0.0
    check_kd(h, w, ids, z, g, tau, got, f"{shape} {kind}")
    assert not got["dh"].cpu()[dead].float().any() and not got["losses"].cpu()[dead].any()


# More than 1024 tokens: rows found and packed by two launches.  fp32: packed weights, products in three parts, several
# pieces of the vocabulary.  bf16 rows of odd width that are packed; sums over the tokens in several splits.
MANY = [(400, 130, 1001), (500, 128, 9000), (1030, 33, 129), (1100, 96, 700), (2100, 64, 300), (2049, 200, 70)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", MANY, ids=str)
def test_cross_entropy_parity_many_tokens(shape, dtype):
    t, d, v = shape
    say(f"case cross entropy, many tokens {shape} {dtype}")
    live = np.random.default_rng(t).random(t) < 0.8
    h, w, y, g = make(t, d, v, dtype, 500 + t, live)
    got = run_ce(h, w, y, g)
    clean = torch.where(torch.from_numpy(live)[:, None], h.float(), torch.zeros(())).to(dtype)
    check_ce(clean, w, y, torch.nan_to_num(g), None, got, str(shape))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape,k,kind,tau", [
    ((400, 130, 1001), 20, "ragged", 2.0), ((500, 128, 9000), 9, "repeated", 1.0), ((1100, 96, 700), 33, "ragged", 1.5),
    ((2100, 64, 300), 5, "masked", 3.0)], ids=str)
def test_distill_parity_many_tokens(shape, k, kind, tau, dtype):
    t, d, v = shape
    say(f"case distill, many tokens {shape} k {k} {kind} tau {tau} {dtype}")
    h, w, _, g = make(t, d, v, dtype, 600 + t)
    ids, z = teacher(t, k, v, 700 + t, kind)
    dead = ~(((ids >= 0) & ~(z == -np.inf)).any(1))
    h[dead] = float("nan")
    got = run_kd(h, w, ids, z, g, tau)
    h[dead] = 0.0
    check_kd(h, w, ids, z, g, tau, got, f"{shape} {kind}")
    assert not got["dh"].cpu()[dead].float().any() and not got["losses"].cpu()[dead].any()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("t", [5, 1100])
def test_distill_teacher_logits_at_the_types_limits(t, dtype):
    # equal entries at the lowest value at a temperature whose inverse is no power of two; the lowest beside an
    # ordinary and beside a large one, whose difference overflows: no mass
    v, k, lo = 40, 4, float(np.finfo(np.float32).min)
    say(f"case teacher at the limits {t} {dtype}")
    h, w, _, g = make(t, 64, v, dtype, 31)
    ids, z = teacher(t, k, v, 32, "full")
    z[0] = lo
    z[1] = torch.tensor([lo, 2.0, lo, 1.0])
    z[2] = torch.tensor([lo, 1e38, 1e38, -3.0])
    z[t - 1] = torch.tensor([lo, lo, -np.inf, -np.inf])
    check_kd(h, w, ids, z, g, 3.0, run_kd(h, w, ids, z, g, 3.0), "limits")
    check_kd(h, w, ids, z, g, 0.7, run_kd(h, w, ids, z, g, 0.7), "limits, T < 1")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("t", [9, 1030])
def test_gradient_weights_of_any_size(t, dtype):
    # subnormal weights give nothing beyond the underflow that the bounds count, large ones no overflow on the way
    for size in (1e-40, 1e-30, 1e30):
        say(f"case weights {size} t {t} {dtype}")
        h, w, y, g = make(t, 64, 130, dtype, 41)
        g = (g.double() / g.abs().max() * size).float()
        got = run_ce(h, w, y, g)
        check_ce(h, w, y, g, None, got, f"weights {size}")
    g[0] = float("inf")  # its row's gradients and dW are not finite; the other rows' are right
    got = run_ce(h, w, y, g)
    g0 = g.clone()
    g0[0] = 0.0
    o = ho.cross_entropy(f64(h), f64(w), y.numpy(), IGN, f64(g0), None)
    b = bounds(o, f64(h), f64(w), 1.0, dtype)
    within("others' dh", f64(got["dh"])[1:], o["dh"][1:], b["dh"][1:])
    assert not bool(got["dh"][0].isfinite().any())


def test_a_mask_that_differs_from_call_to_call_leaves_nothing_behind():
    # one workspace: all rows, few, none, all again
    t, d, v = 1100, 72, 500
    ws = workspace(t, d, v, BF16)
    for kept in (1.0, 0.01, 0.0, 1.0):
        live = np.random.default_rng(3).random(t) < kept
        say(f"case changing mask {kept}")
        h, w, y, g = make(t, d, v, BF16, 17, live)
        got = run_ce(h, w, y, g, ws=ws)
        clean = torch.where(torch.from_numpy(live)[:, None], h.float(), torch.zeros(())).to(BF16)
        check_ce(clean, w, y, torch.nan_to_num(g), None, got, f"kept {kept}")


def test_fp32_products_keep_24_bits():
    # one word, one non-zero product a row: lse is the logit itself.  Three bf16 parts leave out at most
    # 2 x 2^-8 2^-16 + 2^-32 of it, two fp16 parts 2^-22 (the low parts' roundings, 2^-23 each, and the
    # product of the two low parts, 2^-22), six additions add 6 x 2^-23, lse one rounding: below 2^-20
    r = np.random.default_rng(5)
    t, d = 300, 130
    h = np.zeros((t, d), np.float32)
    h[np.arange(t), np.arange(t) % d] = r.standard_normal(t)
    w = r.standard_normal((1, d)).astype(np.float32)
    say("case fp32 products")
    got = run_ce(torch.from_numpy(h), torch.from_numpy(w), torch.zeros(t, dtype=torch.int64), torch.ones(t))
    ref = h.astype(np.float64) @ w.astype(np.float64).T
    within("lse", f64(got["lse"]), ref[:, 0], 2.0 ** -20 * np.abs(ref[:, 0]))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_targets_outside_the_vocabulary_are_nan(dtype):
    say(f"case bad targets {dtype}")
    h, w, y, g = make(70, 64, 300, dtype, 1)
    y[3], y[40], y[69] = 300, -1, 2 ** 40
    got = run_ce(h, w, y, g)
    bad = torch.zeros(70, dtype=torch.bool)
    bad[[3, 40, 69]] = True
    assert torch.isnan(got["losses"].cpu()[bad]).all() and not torch.isnan(got["losses"].cpu()[~bad]).any()
    assert torch.isnan(got["dh"].cpu()[bad].float()).all() and not torch.isnan(got["dh"].cpu()[~bad].float()).any()
    assert torch.isnan(got["dw"].cpu().float()).all()
    ids, z = teacher(70, 4, 300, 2, "full")
    ids[3, 2], ids[69, 0] = 300, 2 ** 40
    bad[40] = False
    got = run_kd(h, w, ids, z, g, 1.0)
    assert torch.isnan(got["losses"].cpu()[bad]).all() and not torch.isnan(got["losses"].cpu()[~bad]).any()
    assert torch.isnan(got["dh"].cpu()[bad].float()).all() and not torch.isnan(got["dh"].cpu()[~bad].float()).any()


def test_large_logits_and_nan_inputs():
    # logits of +-1000: the running maximum keeps every exponential in range
    say("case large logits")
    r = np.random.default_rng(9)
    t, d, v = 100, 128, 600
    h = torch.from_numpy(r.standard_normal((t, d)).astype(np.float32) * 30).bfloat16()
    w = torch.from_numpy(r.standard_normal((v, d)).astype(np.float32) * 3).bfloat16()
    y, g = torch.from_numpy(r.integers(0, v, t)), torch.ones(t)
    check_ce(h, w, y, g, None, run_ce(h, w, y, g), "large")
    h2 = h.clone()
    h2[5, 3] = float("nan")
    h2[6, 0] = float("inf")
    got = run_ce(h2, w, y, g)
    bad = torch.zeros(t, dtype=torch.bool)
    bad[[5, 6]] = True
    assert not torch.isfinite(got["losses"].cpu()[bad]).any() and torch.isfinite(got["losses"].cpu()[~bad]).all()
    assert torch.isfinite(got["dh"].cpu()[~bad].float()).all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_one_gradient_at_a_time_and_no_tokens(dtype):
    say(f"case partial gradients {dtype}")
    h, w, y, g = make(90, 128, 500, dtype, 3)
    got = run_ce(h, w, y, g)
    H, W, Y, G = h.cuda(), w.cuda(), y.cuda(), g.cuda()
    ws = workspace(90, 128, 500, dtype)
    dh, dw = torch.empty_like(H), torch.empty_like(W)
    hd.head_cross_entropy_backward(H, W, Y, got["lse"], G, dh, None, ignore_index=IGN, workspace=ws)
    hd.head_cross_entropy_backward(H, W, Y, got["lse"], G, None, dw, ignore_index=IGN, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(dh, got["dh"]) and torch.equal(dw, got["dw"])
    # a batch of no tokens: no gradient of the weight
    e, f = H[:0], G[:0]
    dw.fill_(float("nan"))
    hd.head_cross_entropy_forward(e, W, Y[:0], f, f.clone(), workspace=ws)
    hd.head_cross_entropy_backward(e, W, Y[:0], f, f, None, dw, workspace=ws)
    torch.cuda.synchronize()
    assert not dw.float().any()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_repeats_share_a_workspace_and_agree_bit_for_bit(dtype):
    # lengths of every kind through one workspace sized for the longest, twice
    say(f"case repeats {dtype}")
    ws = workspace(600, 192, 9000, dtype, extra=37)
    first = {}
    for turn in range(2):
        for t in (600, 1, 64, 65, 300):
            h, w, y, g = make(t, 192, 9000, dtype, 11)
            got = run_ce(h, w, y, g, ws=ws)
            if turn == 0:
                first[t] = {n: x.clone() for n, x in got.items()}
            else:
                for n, x in got.items():
                    assert torch.equal(x, first[t][n]), (t, n)


def test_captured_calls_replay():
    # forward and backward of both losses in one graph; inputs change between replays
    say("case graph")
    t, d, v, k = 150, 192, 1500, 6
    h, w, y, g = (x.cuda() for x in make(t, d, v, BF16, 21))
    ids, z = (x.cuda() for x in teacher(t, k, v, 22, "ragged"))
    ws_g, ws_e = workspace(t, d, v, BF16, k), workspace(t, d, v, BF16, k)

    def call(o, ws):
        hd.head_cross_entropy_forward(h, w, y, o[0], o[1], ignore_index=IGN, workspace=ws)
        hd.head_cross_entropy_backward(h, w, y, o[1], g, o[2], o[3], ignore_index=IGN, workspace=ws)
        hd.head_distill_forward(h, w, ids, z, o[4], o[5], o[6], temperature=2.0, workspace=ws)
        hd.head_distill_backward(h, w, ids, z, o[5], o[6], g, o[7], o[8], temperature=2.0, workspace=ws)

    def outs():
        f = lambda *s: torch.zeros(s, device="cuda")
        b = lambda *s: torch.zeros(s, device="cuda", dtype=BF16)
        return [f(t), f(t), b(t, d), b(v, d), f(t), f(t), f(t, k), b(t, d), b(v, d)]

    captured, eager = outs(), outs()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph):
            call(captured, ws_g)
    torch.cuda.current_stream().wait_stream(side)
    for turn in range(4):
        h2, _, y2, _ = make(t, d, v, BF16, 30 + turn, np.arange(t) % (turn + 2) != 1)
        h.copy_(torch.nan_to_num(h2))
        y.copy_(y2)
        g.copy_(torch.full((t,), 1.0 / t))
        call(eager, ws_e)
        graph.replay()
        assert torch.isfinite(torch.randn(1 << 16, device="cuda").sum())
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(captured, eager)):
            assert torch.equal(a, b), (turn, i)


def test_two_streams_with_their_own_workspaces():
    say("case streams")
    sets = []
    for s in range(2):
        t, d, v = (200, 256, 3000) if s == 0 else (30, 100, 5000)
        h, w, y, g = make(t, d, v, BF16, 40 + s)
        alone = run_ce(h, w, y, g)
        sets.append((tuple(x.cuda() for x in (h, w, y, g)), alone, workspace(t, d, v, BF16),
                     {n: torch.empty_like(x) for n, x in alone.items()}, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        for (h, w, y, g), _, ws, o, st in sets:
            hd.head_cross_entropy_forward(h, w, y, o["losses"], o["lse"], ignore_index=IGN, workspace=ws, stream=st)
            hd.head_cross_entropy_backward(h, w, y, o["lse"], g, o["dh"], o["dw"], ignore_index=IGN, workspace=ws,
                                           stream=st)
    torch.cuda.synchronize()
    for _, alone, _, o, _ in sets:
        for n in o:
            assert torch.equal(o[n], alone[n]), n


def test_gradient_against_differences():
    # fp32: (L(W + e D) - L(W - e D)) / 2 e against <dW, D>.  L ~ 7 with 3e-7 of rounding: 1e-6 / e;
    # the third derivative along D (logits move by about 1 per unit) is of order 1: e^2
    say("case differences")
    t, d, v = 100, 128, 800
    h, w, y, _ = make(t, d, v, F32, 50)
    ids, z = teacher(t, 5, v, 51, "ragged")
    g = torch.full((t,), 1.0 / t)
    D = torch.from_numpy((np.random.default_rng(52).standard_normal((v, d)) / np.sqrt(d)).astype(np.float32))
    e = 2.0 ** -7
    for run in (lambda x: run_ce(h, x, y, g), lambda x: run_kd(h, x, ids, z, g, 2.0)):
        hi, lo = (f64(run(w + s * e * D)["losses"]).sum() / t for s in (1.0, -1.0))
        slope = float((f64(run(w)["dw"]) * f64(D)).sum())
        assert abs((hi - lo) / (2 * e) - slope) <= e * e * 4 + 4e-6 / e, ((hi - lo) / (2 * e), slope)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_training_steps_with_adamw(dtype):
    """The head's training step as it is used: loss, gradients, AdamW on the head
    (cross entropy and distillation added up), each step checked from the state
    the GPU held before it."""
    say(f"case training steps {dtype}")
    t, d, v, k, tau = 180, 128, 1200, 8, 2.0
    h, w, y, _ = make(t, d, v, dtype, 60, np.arange(t) % 5 != 0)
    h = torch.nan_to_num(h)
    ids, z = teacher(t, k, v, 61, "ragged")
    W = w.cuda()
    m, s2 = torch.zeros(v, d, device="cuda"), torch.zeros(v, d, device="cuda")
    g = torch.where(y != IGN, 0.5 / t, 0.0).float()
    for step in range(1, 4):
        ce, kd = run_ce(h, W.cpu(), y, g), run_kd(h, W.cpu(), ids, z, g, tau)
        check_ce(h, W.cpu(), y, g, None, ce, f"step {step}")
        check_kd(h, W.cpu(), ids, z, g, tau, kd, f"step {step}")
        grad = (ce["dw"].float() + kd["dw"].float()).to(dtype)
        p0, m0, v0 = f64(W), f64(m), f64(s2)
        dn.adamw_step_batched([W], [grad], [m], [s2], step=step, lr=1e-2)
        torch.cuda.synchronize()
        pr, _, _ = adamw_step(p0, f64(grad), m0, v0, step, lr=1e-2)
        # the step is at most about lr / sqrt(1 - beta2) wide; its rounding 1e-5 of that, and the parameter's own
        out = U16 if dtype == BF16 else 2 * U32
        within("W", f64(W), pr, out * np.abs(pr) + 1e-2 * 32 * 1e-5 + 16 * U32 * np.abs(p0))
