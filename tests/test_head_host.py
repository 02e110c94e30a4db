"""The output-head losses on the host: exports, the header as plain C, the
workspace sizes, and argument errors that come back before any device work (no
GPU is touched by these tests)."""

import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

from matrix_optimizer_02_amd import build as build_mod
from matrix_optimizer_02_amd import dmuon_head as h
from matrix_optimizer_02_amd import dmuon_ns as d

LIB = d._lib
host_only = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="fake device addresses: host-only validation test")
E_ARG, E_UNS, E_WS = d.DMUON_ERR_INVALID_ARG, d.DMUON_ERR_UNSUPPORTED, d.DMUON_ERR_WORKSPACE
BF16, F32 = d.DMUON_BF16, d.DMUON_F32


def test_exports_and_header():
    names = build_mod.exported_symbols("dmuon_head.h")
    assert set(names) == {"head_loss_workspace_bytes", "head_cross_entropy_forward", "head_cross_entropy_backward",
                          "head_distill_forward", "head_distill_backward"}
    raw = ctypes.CDLL(d.library_path())
    for n in names:
        assert hasattr(raw, n), n
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    with tempfile.TemporaryDirectory() as td:
        src = os.path.join(td, "t.c")
        with open(src, "w") as f:
            f.write('#include "dmuon_head.h"\nint main(void){ dmuon_head_desc x; (void)x; return 0; }\n')
        r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", f"-I{inc}", src, "-o", os.path.join(td, "t")],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
    assert ctypes.sizeof(h.HeadDesc) == 32


def _bytes(t, dd, v, k, dt, back):
    n = ctypes.c_size_t()
    st = LIB.head_loss_workspace_bytes(ctypes.byref(h.HeadDesc(t, dd, v, k, dt)), back, ctypes.byref(n))
    return st, n.value


def test_workspace_sizes():
    for dt in (BF16, F32):
        for back in (0, 1):
            for dd, v in ((64, 1000), (1000, 50257), (4096, 128256)):
                last = 0
                for t in (0, 1, 63, 64, 65, 255, 256, 257, 1000, 2048, 8192, 8193, 20000):
                    st, n = _bytes(t, dd, v, 0, dt, back)
                    assert st == d.DMUON_OK and n >= last and n % 256 == 0, (dt, back, dd, v, t)
                    last = n
    # the logits of 8192 tokens over 128256 words would be 2.1 GB in bf16: a piece of them is held
    st, n = _bytes(8192, 4096, 128256, 0, BF16, 1)
    assert n < (640 << 20)
    st, n = _bytes(8192, 4096, 128256, 0, BF16, 0)
    assert n < (160 << 20)
    assert h.workspace_bytes(100, 64, 1000, torch.bfloat16) == max(_bytes(100, 64, 1000, 0, BF16, 0)[1],
                                                                  _bytes(100, 64, 1000, 0, BF16, 1)[1])


@pytest.mark.parametrize("args,want", [
    ((-1, 64, 10, 0, BF16), E_ARG), ((1, 0, 10, 0, BF16), E_ARG), ((1, 64, 0, 0, BF16), E_ARG),
    ((1, 64, 10, -1, BF16), E_ARG), ((1, 64, 10, 0, 7), E_ARG), ((1 << 24, 64, 10, 0, BF16), E_UNS),
    ((1, 65537, 10, 0, BF16), E_UNS), ((1, 64, 1 << 27, 0, BF16), E_UNS), ((1, 64, 10, 1025, BF16), E_UNS),
    ((1 << 20, 64, (1 << 22) + 1, 0, BF16), E_UNS), ((1 << 20, 64, 1 << 22, 0, BF16), d.DMUON_OK),
    ((0, 1, 1, 0, F32), d.DMUON_OK), (((1 << 24) - 1, 1, 1, 1024, F32), d.DMUON_OK)])
def test_sizes_checked(args, want):
    t, dd, v, k, dt = args
    for back in (0, 1):
        assert _bytes(t, dd, v, k, dt, back)[0] == want
    assert LIB.head_loss_workspace_bytes(None, 0, ctypes.byref(ctypes.c_size_t())) == E_ARG
    assert LIB.head_loss_workspace_bytes(ctypes.byref(h.HeadDesc(1, 64, 10, 0, BF16)), 0, None) == E_ARG


# fake, disjoint, aligned addresses
A = {n: 0x10000000 * (i + 1) for i, n in enumerate(
    ["hidden", "weight", "targets", "losses", "lse", "ws", "g", "gl", "dh", "dw", "ids", "z", "student"])}
BIG = 1 << 40


def _ce_fwd(desc=(64, 128, 1000, 0, BF16), ws_bytes=BIG, **kw):
    a = {**A, **kw}
    return LIB.head_cross_entropy_forward(ctypes.byref(h.HeadDesc(*desc)) if desc else None, a["hidden"], a["weight"],
                                          a["targets"], -100, a["losses"], a["lse"], a["ws"], ws_bytes, None)


def _ce_bwd(desc=(64, 128, 1000, 0, BF16), ws_bytes=BIG, **kw):
    a = {**A, **kw}
    return LIB.head_cross_entropy_backward(ctypes.byref(h.HeadDesc(*desc)) if desc else None, a["hidden"],
                                           a["weight"], a["targets"], -100, a["lse"], a["g"], a["gl"], a["dh"],
                                           a["dw"], a["ws"], ws_bytes, None)


def _kd_fwd(desc=(64, 128, 1000, 4, BF16), ws_bytes=BIG, tau=1.0, **kw):
    a = {**A, **kw}
    return LIB.head_distill_forward(ctypes.byref(h.HeadDesc(*desc)) if desc else None, a["hidden"], a["weight"],
                                    a["ids"], a["z"], tau, a["losses"], a["lse"], a["student"], a["ws"], ws_bytes,
                                    None)


def _kd_bwd(desc=(64, 128, 1000, 4, BF16), ws_bytes=BIG, tau=1.0, **kw):
    a = {**A, **kw}
    return LIB.head_distill_backward(ctypes.byref(h.HeadDesc(*desc)) if desc else None, a["hidden"], a["weight"],
                                     a["ids"], a["z"], tau, a["lse"], a["student"], a["g"], a["dh"], a["dw"],
                                     a["ws"], ws_bytes, None)


READ = {_ce_fwd: ["hidden", "weight", "targets"], _ce_bwd: ["hidden", "weight", "targets", "lse", "g"],
        _kd_fwd: ["hidden", "weight", "ids", "z"],
        _kd_bwd: ["hidden", "weight", "ids", "z", "lse", "student", "g"]}
WRITTEN = {_ce_fwd: ["losses", "lse"], _ce_bwd: ["dh", "dw"], _kd_fwd: ["losses", "lse", "student"],
           _kd_bwd: ["dh", "dw"]}


@host_only
@pytest.mark.parametrize("f", [_ce_fwd, _ce_bwd, _kd_fwd, _kd_bwd])
def test_argument_errors_before_device_work(f):
    k = 4 if f in (_kd_fwd, _kd_bwd) else 0
    assert f(desc=None) == E_ARG
    for name in READ[f] + WRITTEN[f]:
        if name in ("dh", "dw"):  # one of the two may be absent (and the call then goes on)
            assert f(**{name: A[name] + 4}) == E_ARG
            continue
        assert f(**{name: None}) == E_ARG, name
        assert f(**{name: A[name] + 8}) == E_ARG, name
    if f in (_ce_bwd, _kd_bwd):
        assert f(dh=None, dw=None) == E_ARG
    # a written buffer over anything else
    for w in WRITTEN[f]:
        for other in READ[f] + WRITTEN[f]:
            if other != w:
                assert f(**{w: A[other]}) == E_ARG, (w, other)
        assert f(**{w: A["ws"] + 256}) == E_ARG
    assert f(ws=None) == E_WS
    assert f(ws=A["ws"] + 128) == E_WS
    need = _bytes(64, 128, 1000, k, BF16, 1 if f in (_ce_bwd, _kd_bwd) else 0)[1]
    assert f(ws_bytes=0) == E_WS
    assert need > 256 and f(desc=(64, 128, 1000, k, BF16), ws_bytes=255) == E_WS
    assert f(desc=(64, 128, 1000, k, 3)) == E_ARG
    assert f(desc=(64, 128, 1 << 27, k, BF16)) == E_UNS
    assert f(desc=(64, 128, 1000, 1 if k == 0 else 0, BF16)) == E_ARG


@host_only
def test_temperature_checked():
    for f in (_kd_fwd, _kd_bwd):
        for tau in (0.0, -1.0, float("inf"), float("nan"), 1e-39):
            assert f(tau=tau) == E_ARG, tau


@host_only
def test_no_tokens_enqueue_nothing():
    for f, k in ((_ce_fwd, 0), (_kd_fwd, 4)):
        assert f(desc=(0, 128, 1000, k, BF16), hidden=None, targets=None, ids=None, z=None, losses=None, lse=None,
                 student=None, ws=None, ws_bytes=0) == d.DMUON_OK
    for f, k in ((_ce_bwd, 0), (_kd_bwd, 4)):
        assert f(desc=(0, 128, 1000, k, BF16), hidden=None, targets=None, ids=None, z=None, lse=None, student=None,
                 g=None, gl=None, dh=None, dw=None, ws=None, ws_bytes=0) == d.DMUON_OK


def test_binding_checks_tensors():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        h.head_cross_entropy_forward(x, x, torch.zeros(4, dtype=torch.int64), torch.zeros(4), torch.zeros(4),
                                     workspace=torch.zeros(8))
    with pytest.raises(ValueError, match="2-D"):
        h.head_cross_entropy_forward(x[0], x, None, None, None, workspace=None)
    with pytest.raises(ValueError, match="equal columns"):
        h.head_cross_entropy_forward(x, torch.zeros(4, 9, dtype=torch.bfloat16), None, None, None)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        h.head_cross_entropy_forward(x.half(), x.half(), None, None, None)
    with pytest.raises(d.DMuonError):
        h.workspace_bytes(1, 0, 5, torch.float32)


def test_binding_checks_shapes(monkeypatch):
    # with the device check out of the way: shapes, dtypes and strides
    monkeypatch.setattr(h, "_on_current_device", lambda t, what: None)
    x, w = torch.zeros(4, 8), torch.zeros(5, 8)
    y, f = torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    ws = torch.zeros(16, dtype=torch.uint8)
    bad = [dict(targets=y.int()), dict(targets=y[:3]), dict(losses=f.double()), dict(lse=torch.zeros(8)[::2]),
           dict(hidden=torch.zeros(4, 16)[:, ::2]), dict(weight=w.bfloat16()), dict(workspace=None)]
    for kw in bad:
        a = dict(hidden=x, weight=w, targets=y, losses=f, lse=torch.zeros(4), workspace=ws)
        a.update(kw)
        with pytest.raises(ValueError):
            h.head_cross_entropy_forward(a["hidden"], a["weight"], a["targets"], a["losses"], a["lse"],
                                         workspace=a["workspace"])
    ids, z = torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2)
    for i, zz, s in ((ids.int(), z, z), (ids[0], z, z), (ids, z[:, :1], z), (ids, z, torch.zeros(4, 3)),
                     (ids, z.double(), z)):
        with pytest.raises(ValueError):
            h.head_distill_forward(x, w, i, zz, f, torch.zeros(4), s, workspace=ws)
    with pytest.raises(ValueError):
        h.head_cross_entropy_backward(x, w, y, f, f, torch.zeros(4, 7), None, workspace=ws)
    with pytest.raises(ValueError):
        h.head_cross_entropy_backward(x, w, y, f, f, None, w, grad_lse=torch.zeros(3), workspace=ws)
