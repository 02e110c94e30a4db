"""How calls of the output-head losses are cut (csrc/head_layout.cpp, compiled
with g++): the GPU tests' shapes reach every kernel and tile that large calls
use, and the layouts are consistent."""

import os
import random
import subprocess

import pytest

import test_gpu_head_large as large
import test_gpu_head_parts as parts

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "matrix_optimizer_02_amd", "csrc")
BF16, F32 = 1, 0


@pytest.fixture(scope="module")
def layouts(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("layout") / "head_layout_print")
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I" + CSRC,
                        os.path.join(ROOT, "tests", "head_layout_print.cpp"),
                        os.path.join(CSRC, "head_layout.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def of(calls):
        text = "".join(" ".join(str(x) for x in c) + "\n" for c in calls)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=60)
        assert r.returncode == 0
        out = [{k: int(x) for k, x in (f.split("=") for f in line.split())} for line in r.stdout.splitlines()]
        assert len(out) == len(calls)
        return out

    return of


def up(a, b):
    return -(-a // b)


def launches(t, d, v, k, dtype, fwd, back):
    """(kernel, product, tile, several tiles a workgroup, later pieces too) of a
    forward and a backward call."""
    got = set()

    def add(kernel, mode, L, which, tiles, later):
        got.add((kernel, mode, (L[which + "_tp"], L[which + "_tq"]), tiles > L[which + "_slots"], later))

    logits = "stream" if fwd["stream"] else "gemm"
    ty = "bf16" if dtype == BF16 else "f32"
    later = fwd["pack"] == 1 and fwd["pieces"] > 1  # (read in place, one launch covers the vocabulary)
    rows = min(fwd["piece"], v) if fwd["pack"] else v
    add(f"{logits} {ty}", "statistics", fwd, "s", up(rows, fwd["s_tp"]) * up(t, fwd["s_tq"]), later)
    logits = "stream" if back["stream"] else "gemm"
    later = back["pieces"] > 1
    rows = min(back["piece"], v)
    add(f"{logits} {ty}", "ds", back, "s", up(rows, back["s_tp"]) * up(t, back["s_tq"]), later)
    grads = "gemm bf16" if dtype == BF16 else "x3 f32"
    add(f"stream {ty}" if back["stream"] else grads, "dH", back, "dh",
        up(d, back["dh_tp"]) * up(t, back["dh_tq"]) * back["splits"], later)
    add(grads, "dW in splits" if back["dw_splits"] > 1 else "dW", back, "dw",
        up(d, back["dw_tp"]) * up(rows, back["dw_tq"]) * back["dw_splits"], later)
    return got


def test_large_cases_reach_every_wide_tile(layouts):
    reached, partial_tail = set(), 0
    for t, d, v, k in large.CASES.values():
        for dtype in (BF16, F32):
            fwd, back = layouts([(t, d, v, k, dtype, 0), (t, d, v, k, dtype, 1)])
            reached |= launches(t, d, v, k, dtype, fwd, back)
            partial_tail += back["pieces"] > 1 and v % 256 != 0
    have = lambda *want: any(all(w is None or w == g for w, g in zip(want, got)) for got in reached)
    W, M, N = (256, 256), (256, 128), (64, 64)
    for kernel in ("gemm bf16", "gemm f32"):
        for mode in ("statistics", "ds"):
            for tile in (W, M):
                assert have(kernel, mode, tile, True), (kernel, mode, tile)
        assert have(kernel, "ds", None, None, True), kernel
    assert have("gemm f32", "statistics", None, None, True)  # a packed forward's later pieces
    assert have("gemm bf16", "statistics", None, None, True)
    for kernel in ("gemm bf16", "x3 f32"):
        for mode, tiles in (("dH", (W, M)), ("dW", (W, M)), ("dW in splits", (W, M))):
            for tile in tiles:
                assert have(kernel, mode, tile), (kernel, mode, tile)
        assert have(kernel, "dH", W, None, True) and have(kernel, "dH", None, True)
        assert have(kernel, "dW", W, True, True)
    for kernel in ("stream bf16", "stream f32"):
        assert have(kernel, "statistics", M, True) and have(kernel, "ds", M) and have(kernel, "dH", None, None, True)
    assert have("stream f32", "dH", M) and have("stream f32", "ds", M, True, True)
    assert partial_tail >= 8


def test_single_product_cases_reach_every_fp32_tile(layouts):
    reached = set()
    for t, d, v in parts.SHAPES:
        fwd, back = layouts([(t, d, v, 0, F32, 0), (t, d, v, 0, F32, 1)])
        reached |= {r[:3] for r in launches(t, d, v, 0, F32, fwd, back)}
    W, M, N = (256, 256), (256, 128), (64, 64)
    for tile in (W, M, N):
        for what in (("x3 f32", "dH"), ("x3 f32", "dW"), ("x3 f32", "dW in splits"), ("gemm f32", "ds")):
            assert (*what, tile) in reached, (what, tile)
    for tile in (M, N):
        assert ("stream f32", "dH", tile) in reached and ("stream f32", "ds", tile) in reached
    kept = set()
    for t, d, v in parts.KEPT:
        L, = layouts([(t, d, v, 256, F32, 0)])
        assert L["keep"]
        kept.add((L["stream"], L["s_tp"], L["s_tq"]))
    assert kept >= {(1, 64, 64), (1, 256, 64), (1, 256, 128), (0, 64, 64), (0, 256, 128), (0, 256, 256)}


def test_layouts_are_consistent(layouts):
    r = random.Random(1)
    calls = []
    for _ in range(4000):
        t, d = int(2 ** r.uniform(0, 15)), int(2 ** r.uniform(0, 13))
        calls.append((t, d, int(2 ** r.uniform(0, 18)), r.choice([0, 0, 1, 8, 300]), r.choice([BF16, F32]), r.choice([0, 1])))
    for (t, d, v, k, dtype, back), L in zip(calls, layouts(calls)):
        assert not L["refused"]
        assert L["piece"] % 256 == 0 and (L["pieces"] - 1) * L["piece"] < v <= L["pieces"] * L["piece"]
        assert L["t_pad"] % 256 == 0 and L["t_pad"] >= t
        assert not (L["pack"] and L["stream"])
        if L["stream"] or L["low"]:  # kernels of few tokens: no 256-row tiles of them
            assert L["s_tq"] <= 128 and L["dh_tq"] <= 128
        if L["low"]:
            assert 2 * max(64, up(t, 64) * 64) <= L["t_pad"] and dtype == BF16 and back
        assert L["splits"] >= 1 and L["dw_splits"] >= 1 and L["dw_splits"] <= max(1, up(2 * t if L["low"] else t, 64)) + 1
