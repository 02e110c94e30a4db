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
