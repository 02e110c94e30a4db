"""The checks that the large GPU cases use (tests/head_device.py), on the CPU:
outputs from the definitions pass, outputs with a planted mistake do not."""

import pytest
import torch

import head_device as dev

cpu_only = pytest.mark.skipif(dev.DEVICE != "cpu", reason="host test of the checks")
T, D, V, K = 200, 32, 700, 6


def _outputs(h, w, up, y=None, ids=None, z=None, tau=1.0, gl=None, skip=None):
    """The definitions in fp64, rounded once; without the vocabulary rows `skip` in dH."""
    W, live = w.double(), (y != dev.IGN) if ids is None else (ids >= 0).any(1)
    H = torch.where(live[:, None], h.double(), 0.0)
    s = H @ W.t()
    lse = torch.logsumexp(s / tau, 1)
    p = (s / tau - lse[:, None]).exp()
    mass = torch.zeros_like(s)
    out = {}
    if ids is None:
        at = torch.where(live, y, 0)[:, None]
        mass.scatter_(1, at, live.double()[:, None])
        losses = lse - s.gather(1, at)[:, 0]
    else:
        at = ids.clamp(min=0)
        zt = torch.where(ids >= 0, z.double() / tau, float("-inf"))
        zt[~live] = 0.0
        q = torch.where(ids >= 0, torch.softmax(zt, 1), 0.0)
        mass.scatter_add_(1, at, q)
        student = torch.where((ids >= 0) & live[:, None], s.gather(1, at), 0.0)
        out["student"] = student.float()
        logq = torch.where(ids >= 0, torch.log_softmax(zt, 1), 0.0)
        losses = tau ** 2 * (q * (logq - student / tau + lse[:, None])).sum(1)
    g = torch.where(live, up.double(), 0.0)[:, None] * tau
    n = 0.0 if gl is None else torch.where(live, gl.double(), 0.0)[:, None]
    ds = (g + n) * p - g * mass
    cut = ds.clone()
    if skip is not None:
        cut[:, skip] = 0.0
    out.update(losses=torch.where(live, losses, 0.0).float(), lse=torch.where(live, lse, 0.0).float(),
               dh=(cut @ W).to(h.dtype), dw=(ds.t() @ H).to(h.dtype))
    return out


def _problem(kind, dtype):
    h, w, y, up = dev.inputs(T, D, V, dtype, 5, (255, 256, V - 1), dead=0.1 if kind == "ce" else 0.0)
    if kind == "ce":
        return h, w, up, dict(y=y, gl=torch.full((T,), 0.3 / T))
    ids, z = dev.teacher(T, K, V, 6, (255, 256, V - 1))
    return h, w, up, dict(ids=ids, z=z, tau=2.0)


@cpu_only
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["ce", "kd"])
def test_definitions_pass_and_planted_mistakes_fail(kind, dtype):
    h, w, up, args = _problem(kind, dtype)
    good = _outputs(h, w, up, **args)
    dev.check("good", good, h, w, up, **args)
    # a part of the vocabulary lost from dH: the first two tiles, the last partial one
    for skip in (slice(0, 256), slice(512, V)):
        with pytest.raises(AssertionError, match="dh"):
            dev.check("lost", _outputs(h, w, up, skip=skip, **args), h, w, up, **args)
    for name, where, match in (("dw", V - 1, "dw"), ("losses", T - 1, "losses"), ("lse", 3, "lse")):
        bad = {n: x.clone() for n, x in good.items()}
        bad[name][where] = bad[name][where] * 1.1 + (1 if name != "dw" else 0)
        with pytest.raises(AssertionError, match=match):
            dev.check("off", bad, h, w, up, **args)
    bad = {n: x.clone() for n, x in good.items()}
    bad["dw"][7, 0] = float("nan")
    with pytest.raises(AssertionError, match="dw"):
        dev.check("nan", bad, h, w, up, **args)
