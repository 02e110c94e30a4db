"""Workloads of the output-head losses: softmax cross entropy and distillation
from a teacher's top logits, both over the product of hidden states with the
head's weight, and their gradients.

With hidden states H (tokens x hidden) and the head W (vocab x hidden):

  cross entropy   s = H W^T;  lse_t = log sum_v exp s_tv;  loss_t = lse_t - s_t,target
  distillation    s as above, temperature T;  lse_t = log sum_v exp(s_tv / T);
                  q_t = softmax over the row's K teacher entries of z_t / T;
                  loss_t = T^2 sum_k q_tk (log q_tk - s_t,id_k / T + lse_t)

A "forward" case is the losses alone (evaluation, scoring), a "train" case the
forward call and then the backward call with the loss of every token weighted
by 1 / (tokens that count): what the optimizer's step consumes next.

``own`` selects the framework's kernels; where it is false the same results are
computed in elementary torch operations in 32 bits.
"""

import torch

own = False

IGNORE = -100


def _case(name, op, mode, dtype, tokens, hidden, vocab, **kw):
    c = {"name": name, "op": op, "mode": mode, "dtype": dtype, "tokens": tokens, "hidden": hidden, "vocab": vocab,
         "ignored": 0.0, "top_k": 0, "ragged": False, "temperature": 1.0, "z_loss": 0.0}
    c.update(kw)
    return c


def listed():
    return [
        # scoring the one new token of a request over the full vocabulary: the head is read once
        _case("ce_score_1", "ce", "forward", "bf16", 1, 4096, 128256),
        # a unit-test sized model's training step: call latency
        _case("ce_train_tiny_f32", "ce", "train", "f32", 96, 256, 1000),
        # held-out perplexity of a batch with its padding left out
        _case("ce_eval_4096", "ce", "forward", "bf16", 4096, 3584, 128256, ignored=0.1),
        # one micro-batch of pretraining: every token counts
        _case("ce_train_8192", "ce", "train", "bf16", 8192, 4096, 128256),
        # instruction tuning: the prompts' tokens carry no loss
        _case("ce_train_sft_2048", "ce", "train", "bf16", 2048, 4096, 128256, ignored=0.5),
        # a short last micro-batch, odd vocabulary, with the z loss on the normaliser
        _case("ce_train_odd", "ce", "train", "bf16", 1531, 1536, 50257, ignored=0.07, z_loss=1e-4),
        # full precision training of a small model
        _case("ce_train_f32", "ce", "train", "f32", 1024, 1536, 32000, ignored=0.2),
        # scoring a few tokens against a cached teacher
        _case("kd_score_37", "kd", "forward", "bf16", 37, 512, 10007, top_k=8, temperature=2.0),
        # distillation's evaluation on held-out text, full precision
        _case("kd_eval_f32", "kd", "forward", "f32", 700, 1000, 32000, top_k=20, ragged=True),
        # distillation from 64 stored teacher logits a token
        _case("kd_train_4096", "kd", "train", "bf16", 4096, 4096, 128256, top_k=64, temperature=2.0),
        # teachers that stored a nucleus of varying size; some rows hold none
        _case("kd_train_odd", "kd", "train", "bf16", 777, 1536, 50257, top_k=50, ragged=True, temperature=1.5),
        # full precision distillation of a small model
        _case("kd_train_f32", "kd", "train", "f32", 512, 1024, 32000, top_k=32),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    limit = 8192 * 4096 * 128256
    while True:
        dtype = rng.choice(["bf16", "bf16", "f32"])
        tokens = _log_uniform(rng, 1, 8192)
        hidden = _log_uniform(rng, 64, 5120)
        vocab = _log_uniform(rng, 100, 152064)
        if rng.random() < 0.6:  # most models' widths are multiples of 64; the others stay odd
            hidden = max(64, hidden // 64 * 64)
        if rng.random() < 0.4:
            vocab = max(128, vocab // 128 * 128)
        if tokens * hidden * vocab * (6 if dtype == "f32" else 1) <= limit:
            break
    op = rng.choice(["ce", "kd"])
    mode = rng.choice(["train", "train", "forward"])
    kw = {}
    if op == "ce":
        kw["ignored"] = rng.choice([0.0, round(rng.random() * 0.6, 3)])
        kw["z_loss"] = rng.choice([0.0, 1e-4])
    else:
        kw["top_k"] = min(_log_uniform(rng, 1, 200), vocab)
        kw["ragged"] = rng.random() < 0.5
        kw["temperature"] = rng.choice([1.0, 2.0, round(0.5 + 3 * rng.random(), 2)])
    c = _case("", op, mode, dtype, tokens, hidden, vocab, **kw)
    del c["name"]
    return c


def _ignored(case):
    return int(case["tokens"] * case["ignored"])


def work(case):
    t, d, v, k = case["tokens"], case["hidden"], case["vocab"], case["top_k"]
    e = 2 if case["dtype"] == "bf16" else 4
    counted = t - _ignored(case)
    train = case["mode"] == "train"
    nbytes = counted * d * e + v * d * e + 8 * t  # hidden, weight; losses and lse
    nbytes += 8 * t if case["op"] == "ce" else t * k * (8 + 4 + 4)  # targets, or ids, teacher and student logits
    flops = 2 * counted * d * v
    if train:
        nbytes += 4 * t + t * d * e + v * d * e
        flops += 4 * counted * d * v
    return {"bytes": nbytes, "flops": flops}


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed((seed * 1000003 + case["tokens"] * 7919 + case["vocab"] * 31 + case["hidden"]) & 0x7FFFFFFFFFFF)
    t, d, v, k = case["tokens"], case["hidden"], case["vocab"], case["top_k"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    dev = "cuda"
    # a head whose logits of a normed hidden state have a standard deviation near 1.3
    weight = (torch.randn((v, d), generator=g, device=dev) * (1.3 / d ** 0.5)).to(dt)
    hidden = torch.randn((t, d), generator=g, device=dev)
    state = {"case": dict(case), "weight": weight}
    if case["op"] == "ce":
        targets = torch.randint(0, v, (t,), generator=g, device=dev)
        liked = targets
        n = _ignored(case)
        if n:
            # runs of ignored tokens: the prompts (or the padding) of the packed sequences
            run = max(1, t // 8)
            pos = torch.arange(t, device=dev)
            key = ((pos // run).float() * 0.37 + (pos % run).float() / run * 3.0) % 2.0
            targets = targets.clone()
            targets[torch.argsort(key, stable=True)[:n]] = IGNORE
        counts = (targets != IGNORE)
        state["targets"] = targets
        state["grad_lse"] = None
        weights = counts.float() / max(1, t - n)
    else:
        # K distinct ids a row, the most likely first
        start = torch.randint(0, v, (t, 1), generator=g, device=dev)
        step = torch.randint(1, max(2, v // k), (t, 1), generator=g, device=dev)
        ids = (start + torch.arange(k, device=dev) * step) % v
        z = torch.sort(torch.randn((t, k), generator=g, device=dev) * 2.0 + 8.0, dim=1, descending=True).values
        liked = ids[:, 0].clone()
        if case["ragged"]:
            held = torch.randint(0, k + 1, (t, 1), generator=g, device=dev)
            ids = torch.where(torch.arange(k, device=dev) < held, ids, torch.full_like(ids, -1))
        state["teacher_ids"] = ids.contiguous()
        state["teacher_logits"] = z.contiguous()
        weights = (ids >= 0).any(dim=1).float()
        weights = weights / weights.sum().clamp(min=1.0)
    # the model already leans towards its target, by 0 to 10 nats
    lean = torch.rand((t, 1), generator=g, device=dev) * 10.0 / 1.69
    hidden = hidden + lean * weight[liked].float()
    state["hidden"] = hidden.to(dt)
    state["grad_losses"] = weights
    return state


def prepare(case, seed):
    state = _inputs(case, seed)
    if own:
        from matrix_optimizer_02_amd import dmuon_head

        t, d, v, k = case["tokens"], case["hidden"], case["vocab"], case["top_k"]
        w = state["weight"]
        state["workspace"] = dmuon_head.workspace_for(t, d, v, w.dtype, top_k=k, backward=case["mode"] == "train")
        state["losses"] = torch.empty(t, dtype=torch.float32, device="cuda")
        state["lse"] = torch.empty(t, dtype=torch.float32, device="cuda")
        if case["op"] == "kd":
            state["student_logits"] = torch.empty((t, k), dtype=torch.float32, device="cuda")
        if case["mode"] == "train":
            state["grad_hidden"] = torch.empty_like(state["hidden"])
            state["grad_weight"] = torch.empty_like(w)
    return state


def _run_own(s):
    from matrix_optimizer_02_amd import dmuon_head as h

    c = s["case"]
    ws = s["workspace"]
    if c["op"] == "ce":
        h.head_cross_entropy_forward(s["hidden"], s["weight"], s["targets"], s["losses"], s["lse"],
                                     ignore_index=IGNORE, workspace=ws)
        out = [s["losses"], s["lse"]]
        if c["mode"] == "train":
            grad_lse = 2.0 * c["z_loss"] * s["grad_losses"] * s["lse"] if c["z_loss"] else None
            h.head_cross_entropy_backward(s["hidden"], s["weight"], s["targets"], s["lse"], s["grad_losses"],
                                          s["grad_hidden"], s["grad_weight"], grad_lse=grad_lse,
                                          ignore_index=IGNORE, workspace=ws)
            out += [s["grad_hidden"], s["grad_weight"]]
    else:
        h.head_distill_forward(s["hidden"], s["weight"], s["teacher_ids"], s["teacher_logits"], s["losses"], s["lse"],
                               s["student_logits"], temperature=c["temperature"], workspace=ws)
        out = [s["losses"], s["lse"], s["student_logits"]]
        if c["mode"] == "train":
            h.head_distill_backward(s["hidden"], s["weight"], s["teacher_ids"], s["teacher_logits"], s["lse"],
                                    s["student_logits"], s["grad_losses"], s["grad_hidden"], s["grad_weight"],
                                    temperature=c["temperature"], workspace=ws)
            out += [s["grad_hidden"], s["grad_weight"]]
    return out


def _run_plain(s):
    c = s["case"]
    dt = s["weight"].dtype
    hf, wf = s["hidden"].float(), s["weight"].float()
    tau = c["temperature"]
    logits = hf @ wf.t()
    scaled = logits / tau if tau != 1.0 else logits
    top = scaled.max(dim=1, keepdim=True).values
    ex = torch.exp(scaled - top)
    total = ex.sum(dim=1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(1)
    if c["op"] == "ce":
        counts = s["targets"] != IGNORE
        col = torch.where(counts, s["targets"], torch.zeros_like(s["targets"])).unsqueeze(1)
        lse = torch.where(counts, lse, torch.zeros_like(lse))
        losses = torch.where(counts, lse - logits.gather(1, col).squeeze(1), torch.zeros_like(lse))
        out = [losses, lse]
        if c["mode"] == "train":
            up = torch.where(counts, s["grad_losses"], torch.zeros_like(lse)).unsqueeze(1)
            norm = up + 2.0 * c["z_loss"] * up * lse.unsqueeze(1)
            grad = ex.mul_(norm / total)
            grad.scatter_add_(1, col, -up)
            out += [(grad @ wf).to(dt), (grad.t() @ hf).to(dt)]
        return out
    held = s["teacher_ids"] >= 0
    ids = torch.where(held, s["teacher_ids"], torch.zeros_like(s["teacher_ids"]))
    any_held = held.any(dim=1)
    z = torch.where(held, s["teacher_logits"] / tau, torch.full_like(s["teacher_logits"], float("-inf")))
    zmax = torch.where(any_held, z.max(dim=1).values, torch.zeros_like(lse)).unsqueeze(1)
    qe = torch.exp(z - zmax)
    qsum = torch.where(any_held, qe.sum(dim=1), torch.ones_like(lse)).unsqueeze(1)
    q = qe / qsum
    student = logits.gather(1, ids)
    logq = torch.where(held, z - zmax - torch.log(qsum), torch.zeros_like(z))
    lse = torch.where(any_held, lse, torch.zeros_like(lse))
    losses = tau * tau * (q * (logq - student / tau + lse.unsqueeze(1))).sum(dim=1)
    out = [losses, lse, torch.where(held, student, torch.zeros_like(student))]
    if c["mode"] == "train":
        up = torch.where(any_held, s["grad_losses"], torch.zeros_like(lse)).unsqueeze(1) * tau
        grad = ex.mul_(up / total)
        grad.scatter_add_(1, ids, -up * q)
        out += [(grad @ wf).to(dt), (grad.t() @ hf).to(dt)]
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


def exact(case, seed):
    """The definitions in 64 bits, a block of tokens at a time."""
    s = _inputs(case, seed)
    t, k = case["tokens"], case["top_k"]
    tau = case["temperature"]
    w = s["weight"].double()
    train = case["mode"] == "train"
    losses = torch.zeros(t, dtype=torch.float64, device="cuda")
    lses = torch.zeros_like(losses)
    student = torch.zeros((t, k), dtype=torch.float64, device="cuda") if k else None
    dh = torch.zeros((t, case["hidden"]), dtype=torch.float64, device="cuda") if train else None
    dw = torch.zeros_like(w) if train else None
    for t0 in range(0, t, 1024):
        rows = slice(t0, min(t, t0 + 1024))
        h = s["hidden"][rows].double()
        n = h.shape[0]
        x = h @ w.t()
        lse = torch.logsumexp(x / tau, dim=1)
        mass = torch.zeros_like(x)  # the target distribution over the vocabulary
        if case["op"] == "ce":
            live = s["targets"][rows] != IGNORE
            mass[torch.arange(n, device="cuda")[live], s["targets"][rows][live]] = 1.0
            losses[rows] = torch.where(live, lse - (mass * x).sum(dim=1), 0.0)
        else:
            ids, z = s["teacher_ids"][rows], s["teacher_logits"][rows].double() / tau
            live = (ids >= 0).any(dim=1)
            z = z.masked_fill(ids < 0, float("-inf"))
            z[~live] = 0.0
            mass.scatter_add_(1, ids.clamp(min=0), torch.softmax(z, dim=1).masked_fill(ids < 0, 0.0))
            entropy = torch.where(mass > 0, mass * torch.log(mass.clamp(min=1e-300)), 0.0).sum(dim=1)
            cross = (mass * (x / tau - lse.unsqueeze(1))).sum(dim=1)
            losses[rows] = torch.where(live, tau * tau * (entropy - cross), 0.0)
            student[rows] = torch.where(ids >= 0, x.gather(1, ids.clamp(min=0)), 0.0)
        lses[rows] = torch.where(live, lse, 0.0)
        if train:
            up = s["grad_losses"][rows].double().unsqueeze(1) * live.unsqueeze(1)
            prob = torch.exp(x / tau - lse.unsqueeze(1))
            coef = up * (1.0 + 2.0 * case["z_loss"] * lse.unsqueeze(1)) if case["op"] == "ce" else up
            gx = tau * (coef * prob - up * mass)
            dh[rows] = gx @ w
            dw += gx.t() @ h
    out = [losses, lses]
    if case["op"] == "kd":
        out.append(student)
    if train:
        out += [dh, dw]
    return out
