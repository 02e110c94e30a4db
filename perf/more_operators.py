"""Workloads of the token log probabilities over the output head, with entropy
and the top alternatives, of their gradients, and of the global gradient norm
with clipping.

With hidden states H (tokens x hidden), the head W (vocab x hidden) and a
temperature T:

  s = H W^T;  x = s / T;  lse_t = log sum_v exp x_tv
  logprob_t = x_t,target - lse_t;  entropy_t = lse_t - sum_v p_tv x_tv,  p = exp(x - lse)
  alternatives: the K largest logits of a row, equal ones by the lower id, as x - lse
  gradient of sum(g logprob) + sum(e entropy):
      dx_tv = g_t ([v = target] - p_tv) - e_t p_tv (x_tv - lse_t + entropy_t),  dH = dx W / T,  dW = dx^T H / T

  norm = sqrt(sum of the squares of all elements of all tensors)
  clipped = g min(1, max_norm / (norm + eps))

A "forward" case is scoring (log probabilities, entropy, alternatives), a "train"
case the forward call and then the gradients; "norm" and "clip" run over a
list of gradients that lie in one buffer per type.

``own`` selects the framework's kernels; where it is false the same results are
computed in elementary torch operations in 32 bits.
"""

import random

import torch

own = False

IGNORE = -100
EPS = 1e-6

# rows x columns of the projections of one layer
LAYER = [(4096, 4096), (1024, 4096), (1024, 4096), (4096, 4096), (14336, 4096), (14336, 4096), (4096, 14336)]
SMALL = [(128, 128), (128, 512), (512, 128)]


def _head(name, mode, dtype, tokens, hidden, vocab, **kw):
    c = {"name": name, "op": "logprobs", "mode": mode, "dtype": dtype, "tokens": tokens, "hidden": hidden,
         "vocab": vocab, "top_k": 0, "ignored": 0.0, "temperature": 1.0}
    c.update(kw)
    return c


def _grads(name, op, dtype, layout, count, typical, **kw):
    c = {"name": name, "op": op, "dtype": dtype, "layout": layout, "count": count, "typical": typical, "spread": 0.0,
         "packed": False, "ratio": 0.35}
    c.update(kw)
    return c


def listed():
    return [
        # one new token of one request: its probability and five alternatives; the head is read once
        _head("lp_decode_1", "forward", "bf16", 1, 4096, 128256, top_k=5),
        # a serving batch's new tokens with twenty alternatives each, at a sampling temperature
        _head("lp_serve_40", "forward", "bf16", 40, 3584, 152064, top_k=20, temperature=0.7),
        # scoring a prompt with alternatives
        _head("lp_prompt_2048", "forward", "bf16", 2048, 4096, 128256, top_k=5),
        # a teacher's pass over a batch: what distillation stores, padding left out
        _head("lp_teacher_4096", "forward", "bf16", 4096, 4096, 128256, top_k=64, ignored=0.1),
        # a small full precision teacher
        _head("lp_teacher_f32", "forward", "f32", 700, 1000, 32000, top_k=32),
        # a policy-gradient step on packed sequences: prompts carry no loss
        _head("pg_train_8192", "train", "bf16", 8192, 4096, 128256, ignored=0.3),
        # a short last micro-batch, odd vocabulary, trained at the sampling temperature
        _head("pg_train_odd", "train", "bf16", 1531, 1536, 50257, ignored=0.07, temperature=0.8),
        # full precision policy gradient of a small model
        _head("pg_train_f32", "train", "f32", 300, 1000, 32000, ignored=0.2),
        # the gradient norm of one owner's share of an 8B model: 28 matrices
        _grads("norm_share", "norm", "bf16", "layers", 28, 0),
        # many small matrices: call latency
        _grads("norm_small_96", "norm", "bf16", "small", 96, 0),
        # the same share clipped
        _grads("clip_share", "clip", "bf16", "layers", 28, 0),
        # a whole small model's parameters of any size, both types, packed without padding
        _grads("clip_ragged", "clip", "mixed", "ragged", 290, 60000, spread=3.0, packed=True, ratio=0.1),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    if rng.random() < 0.3:
        op = rng.choice(["norm", "clip"])
        count = _log_uniform(rng, 1, 600)
        typical = _log_uniform(rng, 200, min(50_000_000, 600_000_000 // count))
        c = _grads("", op, rng.choice(["bf16", "f32", "mixed"]), "ragged", count, typical,
                   spread=round(2.0 * rng.random(), 2), packed=rng.random() < 0.5,
                   ratio=rng.choice([0.1, 0.35, 0.9, 3.0]))
        del c["name"]
        return c
    limit = 8192 * 4096 * 128256
    while True:
        dtype = rng.choice(["bf16", "bf16", "f32"])
        mode = rng.choice(["train", "forward"])
        tokens = _log_uniform(rng, 1, 8192)
        hidden = _log_uniform(rng, 64, 5120)
        vocab = _log_uniform(rng, 200, 152064)
        if rng.random() < 0.6:  # most models' widths are multiples of 64; the others stay odd
            hidden = max(64, hidden // 64 * 64)
        if rng.random() < 0.4:
            vocab = max(256, vocab // 128 * 128)
        if tokens * hidden * vocab * (6 if dtype == "f32" else 1) <= limit:
            break
    kw = {"temperature": rng.choice([1.0, 1.0, round(0.5 + rng.random(), 2)]),
          "ignored": rng.choice([0.0, round(rng.random() * 0.6, 3)])}
    if mode == "forward" and tokens * vocab <= 4096 * 128256:
        kw["top_k"] = rng.choice([0, 1, 5, 20, _log_uniform(rng, 1, 128)])
    c = _head("", mode, dtype, tokens, hidden, vocab, **kw)
    del c["name"]
    return c


def _ignored(case):
    return int(case["tokens"] * case["ignored"])


# ---- gradient lists ----------------------------------------------------------------


def _sizes(case):
    """(type, elements) of each tensor."""
    if case["layout"] == "layers":
        return [(case["dtype"], r * c) for r, c in (LAYER * case["count"])[:case["count"]]]
    if case["layout"] == "small":
        return [(case["dtype"], r * c) for r, c in (SMALL * case["count"])[:case["count"]]]
    rng = random.Random(case["count"] * 7919 + case["typical"])
    types = ["bf16", "bf16", "f32"] if case["dtype"] == "mixed" else [case["dtype"]]
    most = 2 * case["typical"] * max(1.0, case["spread"])  # a few large ones among many small
    return [(rng.choice(types), 1 + int(min(most, case["typical"] * 2.718281828 ** rng.gauss(0.0, case["spread"]))))
            for _ in range(case["count"])]


def _elements(case, dtype):
    return sum(n for t, n in _sizes(case) if t == dtype)


def _work_grads(case):
    n = _elements(case, "bf16") + _elements(case, "f32")
    nbytes = 2 * _elements(case, "bf16") + 4 * _elements(case, "f32")
    if case["op"] == "norm":
        return {"bytes": nbytes + 4, "flops": 2 * n}
    return {"bytes": 2 * nbytes + 4, "flops": 3 * n}


def _flat(case, dtype, g):
    """One type's gradients in one buffer: (buffer, [(first, elements)], expected sum of squares)."""
    sizes = [n for t, n in _sizes(case) if t == dtype]
    if not sizes:
        return None, [], 0.0
    step = 1 if case["packed"] else 128  # elements that a tensor's place is a multiple of
    held = torch.tensor([(n + step - 1) // step * step for n in sizes])
    first = (torch.cumsum(held, 0) - held).tolist()
    std = 1e-3 * torch.exp(torch.randn(len(sizes), generator=g, device="cuda"))  # tensors differ in scale
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    total = int(held.sum())
    flat = torch.randn(total, generator=g, device="cuda").mul_(torch.repeat_interleave(std, held.cuda())).to(dt)
    if not case["packed"]:
        at = torch.arange(int(max(held - torch.tensor(sizes))), device="cuda")
        pos = torch.tensor([f + n for f, n in zip(first, sizes)], device="cuda")[:, None] + at
        end = torch.tensor([f + int(h) for f, h in zip(first, held.tolist())], device="cuda")[:, None]
        flat[pos[pos < end]] = 0.0  # the padding between tensors
    counts = torch.tensor(sizes, dtype=torch.float64)
    return flat, list(zip(first, sizes)), float((counts * std.double().cpu() ** 2).sum())


def _inputs_grads(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed((seed * 1000003 + case["count"] * 7919 + case["typical"] * 31) & 0x7FFFFFFFFFFF)
    parts = [(t, *_flat(case, t, gen)) for t in ("bf16", "f32")]
    parts = [p for p in parts if p[1] is not None]
    expected = sum(p[3] for p in parts) ** 0.5
    return {"case": dict(case), "flats": [p[1] for p in parts], "places": [p[2] for p in parts],
            "max_norm": case["ratio"] * expected}


def _views(flats, places):
    return [f[a:a + n] for f, place in zip(flats, places) for a, n in place]


def _norm_plain(s):
    return torch.sqrt(sum((f.float() * f.float()).sum(dtype=torch.float64) for f in s["flats"])).float()


def _run_grads_plain(s):
    norm = _norm_plain(s)
    if s["case"]["op"] == "norm":
        return [norm]
    factor = torch.clamp(s["max_norm"] / (norm + EPS), max=1.0)
    return [norm] + [(f.float() * factor).to(f.dtype) for f in s["flats"]]


def _run_grads_own(s):
    s["batch"].norm(s["norm"])
    if s["case"]["op"] == "norm":
        return [s["norm"]]
    s["batch"].clip(s["norm"], s["max_norm"], eps=EPS)
    return [s["norm"]] + s["outs"]


def _exact_grads(case, seed):
    s = _inputs_grads(case, seed)
    norm = torch.sqrt(sum(f.double().square().sum() for f in s["flats"]))
    if case["op"] == "norm":
        return [norm]
    factor = min(1.0, s["max_norm"] / (float(norm) + EPS))
    return [norm] + [f.double() * factor for f in s["flats"]]


# ---- log probabilities ---------------------------------------------------------------


def work(case):
    if case["op"] != "logprobs":
        return _work_grads(case)
    t, d, v, k = case["tokens"], case["hidden"], case["vocab"], case["top_k"]
    e = 2 if case["dtype"] == "bf16" else 4
    counted = t - _ignored(case)
    nbytes = counted * d * e + v * d * e + 8 * t + 12 * t + 12 * t * k  # targets; logprob, entropy, lse; alternatives
    flops = 2 * counted * d * v
    if case["mode"] == "train":
        nbytes += 8 * t + t * d * e + v * d * e
        flops += 4 * counted * d * v
    return {"bytes": nbytes, "flops": flops}


def _on_grid(x, most):
    return torch.round(x).clamp_(-most, most)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed((seed * 1000003 + case["tokens"] * 7919 + case["vocab"] * 31 + case["hidden"]) & 0x7FFFFFFFFFFF)
    t, d, v, k = case["tokens"], case["hidden"], case["vocab"], case["top_k"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    weight = torch.randn((v, d), generator=g, device="cuda")
    hidden = torch.randn((t, d), generator=g, device="cuda")
    targets = torch.randint(0, v, (t,), generator=g, device="cuda")
    lean = torch.rand((t, 1), generator=g, device="cuda") * 10.0  # nats by which a row leans to its token
    if k:
        # Alternatives are ids, whole numbers that have to be the same in any order of
        # summation: weights and states lie on a grid of small integers, as of a quantised
        # checkpoint, where every logit is an exact fp32 sum (and some are equal).
        step = 2.0 ** round(torch.log2(torch.tensor(1.3 / (5.0 * d ** 0.5))).item())
        weight = _on_grid(weight.mul_(2.5), 8)
        hidden = _on_grid(hidden.mul_(2.0) + lean / (6.25 * d * step) * weight[targets], 15)
        weight.mul_(step)
    else:
        # a head whose logits of a normed hidden state have a standard deviation near 1.3
        weight.mul_(1.3 / d ** 0.5)
        hidden = hidden + lean / 1.69 * weight[targets].to(dt).float()
    n = _ignored(case)
    if n:
        # runs of ignored tokens: the prompts (or the padding) of the packed sequences
        run = max(1, t // 8)
        pos = torch.arange(t, device="cuda")
        key = ((pos // run).float() * 0.37 + (pos % run).float() / run * 3.0) % 2.0
        targets[torch.argsort(key, stable=True)[:n]] = IGNORE
    state = {"case": dict(case), "weight": weight.to(dt), "hidden": hidden.to(dt), "targets": targets}
    if case["mode"] == "train":
        # advantages over the tokens that count, and an entropy bonus
        live = (targets != IGNORE).float() / max(1, t - n)
        state["grad_logprobs"] = -torch.randn(t, generator=g, device="cuda") * live
        state["grad_entropy"] = -0.01 * live
    return state


def prepare(case, seed):
    if case["op"] != "logprobs":
        state = _inputs_grads(case, seed)
        if own:
            from matrix_optimizer_02_amd import dmuon_clip

            state["norm"] = torch.zeros((), dtype=torch.float32, device="cuda")
            state["outs"] = [torch.zeros_like(f) for f in state["flats"]] if case["op"] == "clip" else []
            outs = _views(state["outs"], state["places"]) if case["op"] == "clip" else None
            state["batch"] = dmuon_clip.GradBatch(_views(state["flats"], state["places"]), outs)
        return state
    state = _inputs(case, seed)
    if own:
        from matrix_optimizer_02_amd import dmuon_logprobs

        t, d, v, k = case["tokens"], case["hidden"], case["vocab"], case["top_k"]
        train = case["mode"] == "train"
        state["workspace"] = dmuon_logprobs.workspace_for(t, d, v, state["weight"].dtype, top_k=k, backward=train)
        for name in ("logprobs", "entropy", "lse"):
            state[name] = torch.empty(t, dtype=torch.float32, device="cuda")
        if k:
            state["top_ids"] = torch.empty((t, k), dtype=torch.int64, device="cuda")
            state["top_logprobs"] = torch.empty((t, k), dtype=torch.float32, device="cuda")
        if train:
            state["grad_hidden"] = torch.empty_like(state["hidden"])
            state["grad_weight"] = torch.empty_like(state["weight"])
    return state


def _run_own(s):
    from matrix_optimizer_02_amd import dmuon_logprobs as lp

    c = s["case"]
    how = {"temperature": c["temperature"], "ignore_index": IGNORE, "workspace": s["workspace"]}
    lp.head_log_probs_forward(s["hidden"], s["weight"], s["targets"], s["logprobs"], s["entropy"], s["lse"],
                              s.get("top_ids"), s.get("top_logprobs"), **how)
    out = [s["logprobs"], s["entropy"], s["lse"]]
    if c["top_k"]:
        out += [s["top_ids"], s["top_logprobs"]]
    if c["mode"] == "train":
        lp.head_log_probs_backward(s["hidden"], s["weight"], s["targets"], s["lse"], s["entropy"], s["grad_logprobs"],
                                   s["grad_entropy"], s["grad_hidden"], s["grad_weight"], **how)
        out += [s["grad_hidden"], s["grad_weight"]]
    return out


def _top_plain(logits, k):
    """The k largest of each row, equal ones by the lower id: ids and logits."""
    bits = (logits + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()  # the floats' own order, as integers
    key = (order << 32) | (0xFFFFFFFF - torch.arange(logits.shape[1], device=logits.device))
    ids = 0xFFFFFFFF - (torch.topk(key, k, dim=1, sorted=True).values & 0xFFFFFFFF)
    return ids, logits.gather(1, ids)


def _run_plain(s):
    c = s["case"]
    dt = s["weight"].dtype
    tau = c["temperature"]
    counts = s["targets"] != IGNORE
    zero = torch.zeros(c["tokens"], device="cuda")
    hf, wf = s["hidden"].float(), s["weight"].float()
    logits = hf @ wf.t()
    x = logits / tau if tau != 1.0 else logits
    top = x.max(dim=1, keepdim=True).values
    ex = torch.exp(x - top)
    total = ex.sum(dim=1, keepdim=True)
    log_total = torch.log(total)
    # distances from the row's largest logit: no part of the sums is of the logits' own size
    entropy = (log_total - (ex * (x - top)).sum(dim=1, keepdim=True) / total).squeeze(1)
    lse = (top + log_total).squeeze(1)
    col = torch.where(counts, s["targets"], torch.zeros_like(s["targets"])).unsqueeze(1)
    logprobs = (x.gather(1, col) - top - log_total).squeeze(1)
    out = [torch.where(counts, y, zero) for y in (logprobs, entropy, lse)]
    if c["top_k"]:
        ids, z = _top_plain(logits, c["top_k"])
        live = counts.unsqueeze(1)
        out += [torch.where(live, ids, torch.full_like(ids, -1)),
                torch.where(live, z / tau - top - log_total, torch.zeros_like(z))]
    if c["mode"] == "train":
        g = torch.where(counts, s["grad_logprobs"], zero).unsqueeze(1)
        e = torch.where(counts, s["grad_entropy"], zero).unsqueeze(1)
        p = ex.div_(total)
        grad = -p * (g + e * (x - top - log_total + entropy.unsqueeze(1)))
        grad.scatter_add_(1, col, g)
        grad.div_(tau)
        out += [(grad @ wf).to(dt), (grad.t() @ hf).to(dt)]
    return out


def run(state):
    if state["case"]["op"] != "logprobs":
        return _run_grads_own(state) if own else _run_grads_plain(state)
    return _run_own(state) if own else _run_plain(state)


def exact(case, seed):
    """The definitions in 64 bits, a block of tokens at a time."""
    if case["op"] != "logprobs":
        return _exact_grads(case, seed)
    s = _inputs(case, seed)
    t, k, v = case["tokens"], case["top_k"], case["vocab"]
    tau = case["temperature"]
    w = s["weight"].double()
    train = case["mode"] == "train"
    out = [torch.zeros(t, dtype=torch.float64, device="cuda") for _ in range(3)]
    if k:
        out += [torch.full((t, k), -1, dtype=torch.int64, device="cuda"),
                torch.zeros((t, k), dtype=torch.float64, device="cuda")]
    if train:
        out += [torch.zeros((t, case["hidden"]), dtype=torch.float64, device="cuda"), torch.zeros_like(w)]
    for t0 in range(0, t, 1024):
        rows = torch.arange(t0, min(t, t0 + 1024), device="cuda")
        rows = rows[s["targets"][rows] != IGNORE]
        if not len(rows):
            continue
        h = s["hidden"][rows].double()
        logits = h @ w.t()
        logp = torch.log_softmax(logits / tau, dim=1)
        prob = torch.exp(logp)
        entropy = -(prob * logp).sum(dim=1)
        y = s["targets"][rows]
        out[0][rows] = logp.gather(1, y.unsqueeze(1)).squeeze(1)
        out[1][rows] = entropy
        out[2][rows] = torch.logsumexp(logits / tau, dim=1)
        if k:
            ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
            out[3][rows] = ids
            out[4][rows] = logp.gather(1, ids)
        if train:
            g, e = (s[n][rows].double().unsqueeze(1) for n in ("grad_logprobs", "grad_entropy"))
            hot = torch.zeros_like(logits).scatter_(1, y.unsqueeze(1), 1.0)
            ds = (g * (hot - prob) - e * prob * (logp + entropy.unsqueeze(1))) / tau
            out[-2][rows] = ds @ w
            out[-1] += ds.t() @ h
    return out
