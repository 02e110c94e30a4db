"""The output head's log probabilities on the host: exports, the header as plain C,
workspace sizes, and argument errors that come back before any device work (no GPU
is touched by these tests)."""

import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

from matrix_optimizer_02_amd import build as build_mod
from matrix_optimizer_02_amd import dmuon_head as h
from matrix_optimizer_02_amd import dmuon_logprobs as lp
from matrix_optimizer_02_amd import dmuon_ns as d

LIB = d._lib
host_only = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="fake device addresses: host-only validation test")
OK, E_ARG, E_UNS, E_WS = d.DMUON_OK, d.DMUON_ERR_INVALID_ARG, d.DMUON_ERR_UNSUPPORTED, d.DMUON_ERR_WORKSPACE
BF16, F32 = d.DMUON_BF16, d.DMUON_F32


def test_exports_and_header():
    names = build_mod.exported_symbols("dmuon_logprobs.h")
    assert set(names) == {"head_log_probs_workspace_bytes", "head_log_probs_forward", "head_log_probs_backward"}
    raw = ctypes.CDLL(d.library_path())
    for n in names:
        assert hasattr(raw, n), n
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    with tempfile.TemporaryDirectory() as td:
        src = os.path.join(td, "t.c")
        with open(src, "w") as f:
            f.write('#include "dmuon_logprobs.h"\nint main(void){ dmuon_head_desc x; (void)x; return 0; }\n')
        r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", f"-I{inc}", src, "-o", os.path.join(td, "t")],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr


def need(t, dd, v, k, dt, back):
    n = ctypes.c_size_t()
    st = LIB.head_log_probs_workspace_bytes(ctypes.byref(h.HeadDesc(t, dd, v, k, dt)), back, ctypes.byref(n))
    return st, n.value


def test_workspace_sizes():
    for dt in (BF16, F32):
        for back in (0, 1):
            for dd, v in ((64, 1000), (1000, 50257), (4096, 128256)):
                for k in (0,) if back else (0, 1, 20, 128):
                    last = 0
                    for t in (0, 1, 63, 64, 65, 255, 256, 257, 1000, 2048, 8192, 8193, 20000):
                        st, n = need(t, dd, v, k, dt, back)
                        assert st == OK and n >= last and n % 256 == 0, (dt, back, dd, v, k, t)
                        last = n
    # alternatives of any number of tokens take a chunk at a time
    for dt in (BF16, F32):
        assert need(1 << 20, 4096, 128256, 20, dt, 0)[1] < (8 << 30)
    assert lp.workspace_bytes(100, 64, 1000, torch.bfloat16, top_k=5) == max(need(100, 64, 1000, 5, BF16, 0)[1],
                                                                           need(100, 64, 1000, 0, BF16, 1)[1])


@pytest.mark.parametrize("args,want", [
    ((-1, 64, 10, 0, BF16), E_ARG), ((1, 0, 10, 0, BF16), E_ARG), ((1, 64, 0, 0, BF16), E_ARG),
    ((1, 64, 10, -1, BF16), E_ARG), ((1, 64, 10, 0, 7), E_ARG), ((1 << 24, 64, 10, 0, BF16), E_UNS),
    ((1, 65537, 10, 0, BF16), E_UNS), ((1, 64, 1 << 27, 0, BF16), E_UNS),
    ((1 << 20, 64, (1 << 22) + 1, 0, BF16), E_UNS), ((0, 1, 1, 0, F32), OK)])
def test_sizes_checked(args, want):
    for back in (0, 1):
        assert need(*args, back)[0] == want
    assert LIB.head_log_probs_workspace_bytes(None, 0, ctypes.byref(ctypes.c_size_t())) == E_ARG
    assert LIB.head_log_probs_workspace_bytes(ctypes.byref(h.HeadDesc(1, 64, 10, 0, BF16)), 0, None) == E_ARG


def test_alternatives_checked():
    assert need(5, 64, 10, 10, BF16, 0)[0] == OK and need(5, 64, 10, 11, BF16, 0)[0] == E_ARG
    assert need(5, 64, 1000, 128, BF16, 0)[0] == OK and need(5, 64, 1000, 129, BF16, 0)[0] == E_UNS
    assert need(5, 64, 10, 1, BF16, 1)[0] == E_ARG


# fake, disjoint, aligned addresses
A = {n: 0x10000000 * (i + 1) for i, n in enumerate(
    ["hidden", "weight", "targets", "logprobs", "entropy", "lse", "ids", "top", "ws", "g", "e", "dh", "dw"])}
BIG = 1 << 40


def fwd(desc=(64, 128, 1000, 4, BF16), ws_bytes=BIG, tau=1.0, **kw):
    a = {**A, **kw}
    return LIB.head_log_probs_forward(ctypes.byref(h.HeadDesc(*desc)) if desc else None, a["hidden"], a["weight"],
                                      a["targets"], -100, tau, a["logprobs"], a["entropy"], a["lse"], a["ids"],
                                      a["top"], a["ws"], ws_bytes, None)


def bwd(desc=(64, 128, 1000, 0, BF16), ws_bytes=BIG, tau=1.0, **kw):
    a = {**A, **kw}
    return LIB.head_log_probs_backward(ctypes.byref(h.HeadDesc(*desc)) if desc else None, a["hidden"], a["weight"],
                                       a["targets"], -100, tau, a["lse"], a["entropy"], a["g"], a["e"], a["dh"],
                                       a["dw"], a["ws"], ws_bytes, None)


READ = {fwd: ["hidden", "weight", "targets"], bwd: ["hidden", "weight", "targets", "lse", "entropy", "g", "e"]}
WRITTEN = {fwd: ["logprobs", "entropy", "lse", "ids", "top"], bwd: ["dh", "dw"]}


@host_only
@pytest.mark.parametrize("f", [fwd, bwd])
def test_argument_errors_before_device_work(f):
    assert f(desc=None) == E_ARG
    for name in READ[f] + WRITTEN[f]:
        assert f(**{name: A[name] + 8}) == E_ARG, name
    for w in WRITTEN[f]:  # a written buffer over anything else
        for other in READ[f] + WRITTEN[f]:
            if other != w:
                assert f(**{w: A[other]}) == E_ARG, (w, other)
        assert f(**{w: A["ws"] + 256}) == E_ARG
    assert f(ws=None) == E_WS and f(ws=A["ws"] + 128) == E_WS and f(ws_bytes=0) == E_WS
    k = 4 if f is fwd else 0
    size = need(64, 128, 1000, k, BF16, f is bwd)[1]
    assert size > 256 and f(ws_bytes=255) == E_WS
    assert f(desc=(64, 128, 1000, k, 3)) == E_ARG
    assert f(desc=(64, 128, 1 << 27, k, BF16)) == E_UNS
    assert f(desc=(64, 128, 1000, 129, BF16)) in (E_UNS, E_ARG)
    for tau in (0.0, -1.0, float("inf"), float("nan"), 1e-39, 1.1e-38 / 2, 3e38):
        assert f(tau=tau) == E_ARG, tau


@host_only
def test_what_goes_together():
    for name in ("hidden", "weight", "lse", "ids", "top"):
        assert fwd(**{name: None}) == E_ARG, name
    assert fwd(targets=None) == E_ARG and fwd(logprobs=None) == E_ARG
    assert fwd(desc=(64, 128, 1000, 0, BF16)) == E_ARG  # buffers for alternatives that are not asked for
    assert fwd(desc=(64, 128, 3, 4, BF16)) == E_ARG     # more alternatives than words
    for name in ("hidden", "weight", "lse"):
        assert bwd(**{name: None}) == E_ARG, name
    assert bwd(g=None, e=None) == E_ARG and bwd(dh=None, dw=None) == E_ARG
    assert bwd(targets=None) == E_ARG   # upstream of the log probabilities of no token
    assert bwd(entropy=None) == E_ARG   # needed by the entropy's gradient
    assert bwd(desc=(64, 128, 1000, 4, BF16)) == E_ARG


@host_only
def test_no_tokens_enqueue_nothing():
    none = {n: None for n in A}
    assert fwd(desc=(0, 128, 1000, 4, BF16), ws_bytes=0, **{**none, "weight": A["weight"]}) == OK
    assert bwd(desc=(0, 128, 1000, 0, BF16), ws_bytes=0, **{**none, "weight": A["weight"]}) == OK


def test_binding_checks(monkeypatch):
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    f, y = torch.zeros(4), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="device tensor"):
        lp.head_log_probs_forward(x, x, y, f, f, f, workspace=f)
    with pytest.raises(d.DMuonError):
        lp.workspace_bytes(1, 64, 5, torch.float32, top_k=6)
    monkeypatch.setattr(h, "_on_current_device", lambda t, what: None)
    ws = torch.zeros(16, dtype=torch.uint8)
    ids, top = torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2)
    good = dict(hidden=x, weight=x, targets=y, logprobs=f, entropy=f.clone(), lse=f.clone(), top_ids=ids,
                top_logprobs=top, workspace=ws)
    for kw in (dict(targets=None), dict(logprobs=None), dict(top_ids=None), dict(top_logprobs=None),
               dict(top_ids=ids[0]), dict(top_ids=ids.int()), dict(top_logprobs=top[:, :1]), dict(targets=y.int()),
               dict(lse=f[:3]), dict(entropy=f.double()), dict(logprobs=torch.zeros(8)[::2]), dict(workspace=None),
               dict(weight=x.float())):
        with pytest.raises(ValueError):
            lp.head_log_probs_forward(**{**good, **kw})
    good = dict(hidden=x, weight=x, targets=y, lse=f, entropy=f, grad_logprobs=f, grad_entropy=f, grad_hidden=x,
                grad_weight=x, workspace=ws)
    for kw in (dict(lse=f[:3]), dict(grad_logprobs=f.double()), dict(grad_entropy=f[:2]), dict(grad_hidden=x[:2]),
               dict(grad_weight=x.float()), dict(workspace=None)):
        with pytest.raises(ValueError):
            lp.head_log_probs_backward(**{**good, **kw})
