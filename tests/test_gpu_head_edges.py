"""Edges of the output-head losses on the GPU: masked teacher entries with ids out
of range, +inf and NaN teacher logits, inputs that require gradients."""

import pytest
import torch

import head_device as dev

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("t", [70, 300, 1100])
@pytest.mark.parametrize("k", [4, 200])  # (200: the logits are kept and gathered)
def test_masked_teacher_entries_may_hold_any_id(t, k, dtype):
    print(f"case masked entries out of range {t} {k} {dtype}", flush=True)
    d, v = 128, 300
    h, w, _, up = dev.inputs(t, d, v, dtype, 70 + t)
    ids, z = dev.teacher(t, k, v, 71)
    ids = torch.where(ids < 0, 5, ids)
    z = torch.nan_to_num(z, nan=1.0)
    off = torch.arange(k, device="cuda") % 3 == 1
    absent, wild = torch.where(off, -1, ids), torch.where(off, 2 ** 40 + ids, ids)
    wild[:, 1] = v
    inf = torch.where(off, float("-inf"), z)
    a = dev.run(h, w, up, ids=absent, z=z, tau=1.5)
    dev.check("absent", a, h, w, up, ids=absent, z=z, tau=1.5)
    b = dev.run(h, w, up, ids=wild, z=inf, tau=1.5)
    for n in ("losses", "lse", "student", "dh", "dw"):
        assert torch.equal(a[n], b[n]), n
    # rows with nothing else carry no loss
    wild[3] = v
    inf[3] = float("-inf")
    c = dev.run(h, w, up, ids=wild, z=inf, tau=1.5)
    assert float(c["losses"][3]) == 0.0 and float(c["lse"][3]) == 0.0 and not bool(c["dh"][3].float().any())
    keep = torch.arange(t, device="cuda") != 3
    assert torch.equal(c["losses"][keep], b["losses"][keep])


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_teacher_logits_without_a_softmax_make_their_rows_nan(value):
    print(f"case teacher {value}", flush=True)
    t, d, v, k = 70, 64, 300, 4
    h, w, _, up = dev.inputs(t, d, v, F32, 80)
    ids, z = dev.teacher(t, k, v, 81)
    ids, z = torch.where(ids < 0, 5, ids), torch.nan_to_num(z, nan=1.0)
    z[9, 2] = value
    got = dev.run(h, w, up, ids=ids, z=z)
    rows = torch.arange(t, device="cuda") == 9
    assert bool(torch.isnan(got["losses"][rows]).all()) and bool(torch.isfinite(got["losses"][~rows]).all())
    assert bool(torch.isfinite(got["dh"][~rows]).all()) and bool(torch.isnan(got["dh"][rows]).any())


def test_inputs_that_require_gradients():
    print("case requires grad", flush=True)
    h, w, y, up = dev.inputs(90, 64, 500, F32, 90)
    plain = dev.run(h, w, up, y=y)
    got = dev.run(h.clone().requires_grad_(), w.clone().requires_grad_(), up, y=y)
    for n in ("losses", "lse", "dh", "dw"):
        assert torch.equal(got[n], plain[n]) and got[n].grad_fn is None


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("t", [5, 300, 1100])
def test_losses_of_large_logits_keep_their_bits(t, dtype):
    # s = 32768 + x, x a multiple of 1/16: exact in every form, 2^-9 to 2^-4 of its rounding.  A loss is a matter of
    # the differences.  u = 2^-24: the sum of at most 2 (the largest logit's 1 and the rest) in chains of at most
    # 64 + 24 additions, 2 u each, exponentials of |x| <= 16 good to (4 + 2 |x|) u: 400 u; its logarithm and the
    # loss's own additions 8 u (1 + loss).  The teacher's part: q good to (16 (1 + |z|) + K) u as ever.
    print(f"case losses of large logits {t} {dtype}", flush=True)
    u, v, d, k = 2.0 ** -24, 300, 64, 4
    g = torch.Generator(device="cuda")
    g.manual_seed(100 + t)
    h, w = torch.zeros(t, d, device="cuda"), torch.zeros(v, d, device="cuda")
    h[:, 0] = 1.0
    w[:, 0] = 32768.0
    c = 1 + torch.arange(t, device="cuda") % (d - 1)
    h[torch.arange(t, device="cuda"), c] = 1.0
    w[:, 1:] = torch.randint(0, 33, (v, d - 1), generator=g, device="cuda") / 16.0
    y = torch.randint(0, v, (t,), generator=g, device="cuda")
    best = torch.randint(0, v, (d,), generator=g, device="cuda")
    w[best[1:], torch.arange(1, d, device="cuda")] = 12.0
    y = torch.where(torch.arange(t, device="cuda") % 3 == 0, best[c], y)  # small losses and large ones
    h, w, up = h.to(dtype), w.to(dtype), torch.full((t,), 1.0 / t, device="cuda")
    x = w.double()[:, c].t()  # less the common 32768
    lse = torch.logsumexp(x, 1)
    got = dev.run(h, w, up, y=y)
    ref = lse - x.gather(1, y[:, None])[:, 0]
    dev.within("ce", got["losses"], ref, 400 * u + 8 * u * (1 + ref))
    ids = torch.stack([y, best[c], (y + 1) % v, (y + 7) % v], 1)
    z = torch.randn((t, k), generator=g, device="cuda")
    q = torch.softmax(z.double(), 1)
    parts = torch.log_softmax(z.double(), 1) - x.gather(1, ids) + lse[:, None]
    got = dev.run(h, w, up, ids=ids, z=z)
    bound = (q * (400 * u + 8 * u * (1 + parts.abs()) + 2 * (16 * (1 + z.double().abs()) + k) * u * (1 + parts.abs()))).sum(1)
    dev.within("kd", got["losses"], (q * parts).sum(1), bound)
