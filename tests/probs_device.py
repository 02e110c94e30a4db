"""Device-side checks of the output head's log probabilities: the definitions in
fp64 on the GPU (a block of tokens at a time) and error bounds.

Bounds, with u32 = 2^-24 and u16 = 2^-8 (half a step of fp32 and bf16), x = s / T
and y = x - lse = log p:
    es = (2 D' + 8) u32 |H| |W|^T      a logit; D' = D (bf16) or 6 D (fp32), padded
    dx = max over the row of es / T, twice: a logit's and the largest one's
    c  = V / 64 + 128                  additions in a row, a softmax sum
    el = dx + (c + 8) 2 u32 + 4 u32 max |y| + 2 u32 |lse|      lse
    log probability: el + es / T + 4 u32 |y|
    entropy: a shift of the logits by dx moves it by at most dx sum p |y + H|; the
        sums: (c + 8) 2 u32 (1 + H); an exponential of z = x - max x is off by
        (2 |z| + 8) u32 relative, and so is its share of sum p z:
        2 u32 sum p (1 + |z|) (2 |z| + 8)
    ds: p (cp + ce y) - ct at the target with cp = -(g + e H) / T, ce = -e / T, ct =
        -g / T; p is off by rp = es / T + el + 8 u32 (1 + |y|) relative, y by dy = es / T
        + el + 4 u32 |y|, H by its own bound; ur is the rounding of ds (2^-8 bf16, 2^-15
        where it is held in two parts, 2^-22 fp32) of a value of at most its own size
    dH: ed |W| + (2 V' + 64) u32 |ds| |W| + out |dH|, dW the same over the tokens
Alternatives: each value is the log probability of its own id, within that bound; the
ids are different, no word left out has a logit above the last one's by more than both
logits' es, and none is followed by one that is larger by more than that.
"""

import torch

from head_device import BF16, BLOCK, DEVICE, F32, F64, IGN, U16, U32, guarded, pad, untouched, within
from matrix_optimizer_02_amd import dmuon_logprobs as lp


def workspace(t, d, v, dtype, k=0, backward=True):
    ws = lp.workspace_for(t, d, v, dtype, top_k=k, backward=backward)
    ws.fill_(0xFF)  # NaN patterns: what a call reads it must have written
    return ws


def run(h, w, y=None, k=0, tau=1.0, g=None, e=None, entropy=True, stream=None, ws=None):
    """Forward and, with upstream gradients, backward."""
    t, d, v = h.shape[0], h.shape[1], w.shape[0]
    back = g is not None or e is not None
    ws = workspace(t, d, v, h.dtype, k, back) if ws is None else ws
    shapes = [("lse", (t,), F32)]
    shapes += [("logprobs", (t,), F32)] if y is not None else []
    shapes += [("entropy", (t,), F32)] if entropy else []
    shapes += [("top_ids", (t, k), torch.int64), ("top_logprobs", (t, k), F32)] if k else []
    shapes += [("dh", (t, d), h.dtype), ("dw", (v, d), h.dtype)] if back else []
    full, r = {}, {}
    for n, s, dt in shapes:
        full[n], r[n] = guarded(s, dt) if dt != torch.int64 else guarded_ids(s)
    lp.head_log_probs_forward(h, w, y, r.get("logprobs"), r.get("entropy"), r["lse"], r.get("top_ids"),
                              r.get("top_logprobs"), temperature=tau, ignore_index=IGN, workspace=ws, stream=stream)
    if back:
        lp.head_log_probs_backward(h, w, y, r["lse"], r.get("entropy"), g, e, r["dh"], r["dw"], temperature=tau,
                                   ignore_index=IGN, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    for n, x in full.items():
        untouched(x, n)
    return r


def guarded_ids(shape):
    full = torch.full((shape[0] * shape[1] + 128,), 7, dtype=torch.int64, device=DEVICE)
    view = full[64:64 + shape[0] * shape[1]].view(shape)
    view.fill_(-7)
    return full, view


def check(what, got, h, w, y=None, k=0, tau=1.0, g=None, e=None, exact_ids=False, block=BLOCK):
    """Every element of every output against the definitions in fp64."""
    t, d, v, dtype = h.shape[0], h.shape[1], w.shape[0], h.dtype
    mul = 1 if dtype == BF16 else 6
    out = U16 if dtype == BF16 else 2 * U32
    ur = 2.0 ** -22 if dtype == F32 else U16 if t > 128 else 2.0 ** -15
    c = v / 64 + 128
    W = w.to(F64)
    Wt, aW = W.t(), W.abs()
    aWt = aW.t()
    back = g is not None or e is not None
    dw, bdw, mdw = (torch.zeros_like(W) if back else None for _ in range(3))
    for r0 in range(0, t, block):
        rows = slice(r0, min(t, r0 + block))
        n = rows.stop - r0
        live = torch.ones(n, dtype=torch.bool, device=h.device) if y is None else y[rows] != IGN
        L = live[:, None]
        H = torch.where(L, h[rows].to(F64), 0.0)
        s = H @ Wt
        es = (2 * mul * pad(d) + 8) * U32 * (H.abs() @ aWt)
        x = s / tau
        lse = torch.logsumexp(x, 1)
        ly = x - lse[:, None]
        p = ly.exp()
        z = x - x.max(1, keepdim=True).values
        ent = -(p * ly).sum(1)
        dx = 2 * es.max(1).values / tau
        el = dx + (c + 8) * 2 * U32 + 4 * U32 * ly.abs().max(1).values + 2 * U32 * lse.abs()
        eh = (dx * (p * (ly + ent[:, None]).abs()).sum(1) + (c + 8) * 2 * U32 * (1 + ent) +
              2 * U32 * (p * (1 + z.abs()) * (2 * z.abs() + 8)).sum(1) + 4 * U32 * ent)
        if y is not None or not back or "lse" in got:
            within(f"{what} lse from row {r0}", got["lse"][rows], torch.where(live, lse, 0.0),
                   torch.where(live, el, 0.0))
        if "entropy" in got:
            within(f"{what} entropy from row {r0}", got["entropy"][rows], torch.where(live, ent, 0.0),
                   torch.where(live, eh, 0.0))
        el_p = (el[:, None] + es / tau + 4 * U32 * ly.abs())
        if y is not None:
            col = torch.where(live, y[rows], 0)[:, None]
            within(f"{what} logprobs from row {r0}", got["logprobs"][rows],
                   torch.where(live, ly.gather(1, col)[:, 0], 0.0),
                   torch.where(live, el_p.gather(1, col)[:, 0], 0.0))
        if k:
            ids, val = got["top_ids"][rows], got["top_logprobs"][rows]
            assert bool((ids[~live] == -1).all()) and bool((val[~live] == 0).all()), what
            i, s_, es_, lr = ids[live], s[live], es[live], live.nonzero()[:, 0]
            if len(lr):
                assert bool(((i >= 0) & (i < v)).all()), what
                assert bool((i.sort(1).values.diff(dim=1) > 0).all()), f"{what}: an id twice"
                within(f"{what} alternatives from row {r0}", val[live], ly[live].gather(1, i), el_p[live].gather(1, i))
                if exact_ids:
                    want = torch.sort(s_, dim=1, descending=True, stable=True).indices[:, :k]
                    assert torch.equal(i, want), f"{what}: ids of row {r0 + int(lr[(i != want).any(1)][0])}"
                else:
                    at, ea = s_.gather(1, i), es_.gather(1, i)
                    assert bool((at[:, 1:] - at[:, :-1] <= ea[:, 1:] + ea[:, :-1]).all()), f"{what}: order"
                    left = (s_ - es_).scatter(1, i, -torch.inf)
                    assert bool((left.max(1).values <= (at + ea)[:, -1]).all()), f"{what}: a larger one left out"
        if back:
            zero = torch.zeros(n, dtype=F64, device=h.device)
            G = torch.where(live, zero if g is None else g[rows].to(F64), 0.0)[:, None] / tau
            E = torch.where(live, zero if e is None else e[rows].to(F64), 0.0)[:, None] / tau
            hot = torch.zeros_like(s)
            if y is not None:
                hot.scatter_(1, torch.where(live, y[rows], 0)[:, None], live.to(F64)[:, None])
            cp, ce = -(G + E * ent[:, None]), -E
            f = cp + ce * ly
            ds = p * f + G * hot
            ey = es / tau + el[:, None]
            ed = (p * f.abs() * (ey + 8 * U32 * (1 + ly.abs())) +
                  p * (ce.abs() * (ey + 4 * U32 * ly.abs() + eh[:, None]) + 8 * U32 * (cp.abs() + (ce * ly).abs())) +
                  8 * U32 * (p * f.abs() + G.abs() * hot))
            big = torch.maximum(torch.maximum(cp.abs(), ce.abs()), G.abs())
            ed = torch.where(L, ed + ur * (ds.abs() + ed) + (big + 2) * 2.0 ** -126, 0.0)
            mag = ds.abs() + ed
            ref = ds @ W
            b = (ed @ aW + (2 * mul * pad(v) + 64) * U32 * (mag @ aW)) * (1 + out) + out * ref.abs()
            within(f"{what} dh from row {r0}", got["dh"][rows], ref, b)
            dw += ds.t() @ H
            bdw += ed.t() @ H.abs()
            mdw += mag.t() @ H.abs()
    if back:
        b = (bdw + (2 * mul * pad(t) + 64) * U32 * mdw) * (1 + out) + out * dw.abs()
        within(f"{what} dw", got["dw"], dw, b)


def inputs(t, d, v, dtype, seed, dead=0.0):
    """hidden, weight, targets and two upstream gradients.  Rows lean towards a word by 0 to 12 times its own
    row of W, half of them towards their target.  Rows without a target hold NaN."""
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=gen, device=DEVICE)
    word = lambda: torch.randint(0, v, (t,), generator=gen, device=DEVICE)
    w = (rand(v, d) * (1.3 / d ** 0.5)).to(dtype)
    y = word()
    lean = torch.where(torch.rand(t, generator=gen, device=DEVICE) < 0.5, y, word())
    h = (rand(t, d) + torch.rand((t, 1), generator=gen, device=DEVICE) * 12 * w[lean].float()).to(dtype)
    g, e = rand(t) / t, rand(t) * 0.1 / t
    if dead:
        off = torch.rand(t, generator=gen, device=DEVICE) < dead
        y[off] = IGN
        h[off] = float("nan")
        g[off] = float("nan")
        e[off] = float("nan")
    return h, w, y, g, e


def grid_inputs(t, d, v, dtype, seed, dead=0.0):
    """As inputs(), on a grid of small integers: every logit is exact in fp32 in any order of summation, and
    many are equal."""
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    w = torch.randn((v, d), generator=gen, device=DEVICE).mul_(2.5).round_().clamp_(-8, 8)
    h = torch.randn((t, d), generator=gen, device=DEVICE).mul_(2.0).round_().clamp_(-15, 15)
    y = torch.randint(0, v, (t,), generator=gen, device=DEVICE)
    h, w = h.to(dtype), (w * 2.0 ** round(-2.0 - torch.log2(torch.tensor(float(d))).item() / 2)).to(dtype)
    if dead:
        off = torch.rand(t, generator=gen, device=DEVICE) < dead
        y[off] = IGN
        h[off] = float("nan")
    return h, w, y


def plain(h, w, y=None, k=0, tau=1.0, g=None, e=None):
    """The outputs by fp32 torch operations, results rounded once: what check() has to accept."""
    live = torch.ones(len(h), dtype=torch.bool, device=h.device) if y is None else y != IGN
    hf, wf = torch.where(live[:, None], h.float(), 0.0), w.float()
    s = hf @ wf.t()
    ly = torch.log_softmax(s / tau, 1)
    p = ly.exp()
    ent = -(p * ly).sum(1)
    r = {"lse": torch.where(live, torch.logsumexp(s / tau, 1), 0.0), "entropy": torch.where(live, ent, 0.0)}
    if y is not None:
        col = torch.where(live, y, 0)[:, None]
        r["logprobs"] = torch.where(live, ly.gather(1, col)[:, 0], 0.0)
    if k:
        ids = torch.sort(s, dim=1, descending=True, stable=True).indices[:, :k]
        r["top_ids"] = torch.where(live[:, None], ids, -1)
        r["top_logprobs"] = torch.where(live[:, None], ly.gather(1, ids), 0.0)
    if g is not None or e is not None:
        zero = torch.zeros(len(h), device=h.device)
        G = torch.where(live, zero if g is None else g, 0.0)[:, None]
        E = torch.where(live, zero if e is None else e, 0.0)[:, None]
        hot = torch.zeros_like(s)
        if y is not None:
            hot.scatter_(1, col, live.float()[:, None])
        ds = (G * (hot - p) - E * p * (ly + ent[:, None])) / tau
        r["dh"], r["dw"] = (ds @ wf).to(h.dtype), (ds.t() @ hf).to(h.dtype)
    return r
