"""How calls of the log probabilities are cut (csrc/head_layout.cpp, compiled with g++):
the GPU tests' sizes reach what they are for, and the layouts are consistent."""

import os
import random
import subprocess

import pytest

import test_gpu_head_narrow as narrow
import test_gpu_logprobs_reach as reach

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "matrix_optimizer_02_amd", "csrc")
BF16, F32 = 1, 0
MOST_SPLITS, SUM_SLABS = 16, 20


@pytest.fixture(scope="module")
def layouts(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("layout") / "probs_layout_print")
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I" + CSRC,
                        os.path.join(ROOT, "tests", "probs_layout_print.cpp"),
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


def forward(t, d, v, k, dtype):
    return t, d, v, k, dtype, 0, t


def backward(t, d, v, live, dtype=BF16):
    return t, d, v, 0, dtype, 1, live


def test_chunked_sizes_end_in_a_chunk_of_other_tiles(layouts):
    for c in reach.CHUNKED:
        (b,), (f,) = layouts([forward(*c, BF16)]), layouts([forward(*c, F32)])
        for L in (b, f):
            assert L["chunk"] < c[0] and L["last"] < L["chunk"]
            assert (L["s_tp"], L["s_tq"]) != (L["last_s_tp"], L["last_s_tq"])
        assert f["stream"] == 0 and f["last_stream"] == 1  # two fp16 parts, then three of bf16
    for c in reach.ONE_CHUNK:
        L, = layouts([forward(*c, BF16)])
        assert L["chunk"] == c[0]
    for t, v, k in ((14400, 152064, 3), (33100, 8000, 128)):  # (test_more_tokens_than_a_chunk)
        L, = layouts([forward(t, 64, v, k, BF16)])
        assert L["chunk"] < t


def test_live_sizes_leave_the_splits_to_the_device(layouts):
    pieces = set()
    for t, d, v in reach.LIVE:
        rows = [max(1, round(t * (1 - dead))) for dead in reach.DEAD]
        Ls = layouts([backward(t, d, v, n) for n in rows])
        assert all(L["room"] > 0 and L["dh_tq"] == 256 for L in Ls)
        assert len({L["live_splits"] for L in Ls}) >= 3, (t, d, v)
        pieces.add(Ls[0]["pieces"])
        assert Ls[0]["pieces"] == 1 or v % Ls[0]["piece"] != 0
    assert 1 in pieces and max(pieces) > 1
    L, = layouts([backward(4200, 320, 70001, 4200)])  # (of test_rows_that_take_no_part)
    assert L["room"] > 0


def test_splits_fit_their_room(layouts):
    r = random.Random(2)
    calls = []
    for _ in range(4000):
        t = int(2 ** r.uniform(7, 15))
        calls.append(backward(t, int(2 ** r.uniform(5, 13)), int(2 ** r.uniform(8, 18)), r.randint(1, t)))
    up = lambda a, b: -(-a // b)
    seen = 0
    for (t, d, v, _, _, _, live), L in zip(calls, layouts(calls)):
        if L["room"] == 0:
            continue
        seen += 1
        slabs = up(min(L["piece"], v), 64)
        tiles = up(d, 256) * up(live, 256)
        s = L["live_splits"]
        assert 1 <= s <= min(MOST_SPLITS, slabs) and s * tiles <= L["room"]
        # the definition: the fewest rounds of 256 slots, a round's sums counted as slabs
        cost = lambda n: up(n * tiles, 256) * (up(slabs, n) + SUM_SLABS)
        assert cost(s) == min(cost(n) for n in range(1, MOST_SPLITS + 1) if n <= slabs and n * tiles <= L["room"])
    assert seen > 100


def test_where_ds_stays_in_the_caches(layouts):
    """dH in 64 x 64 tiles reads ds at the memory's rate: there ds is written through the last-level cache, as
    long as it stays in it."""
    sizes = [(*c, True) for c in narrow.CACHED] + [(*c, False) for c in narrow.PAST]
    sizes += [(2048, 128, 50257, True), (4096, 128, 50257, True), (4096, 64, 30000, True), (4096, 64, 32700, False),
              (8192, 4096, 128256, False), (8192, 128, 128256, False)]
    for (t, d, v, cached), L in zip(sizes, layouts([backward(t, d, v, t) for t, d, v, _ in sizes])):
        assert (L["s_tp"], L["s_tq"]) == (256, 256), (t, d, v)  # (whose kernel it is for)
        assert L["cached"] == cached == (L["dh_tp"] == 64 and 2 * L["t_pad"] * L["piece"] <= 240 << 20), (t, d, v)
    L, = layouts([backward(2048, 128, 50257, 2048, F32)])
    assert not L["cached"]


def test_where_dw_is_written_through_the_caches(layouts):
    """Rows of dW that are not whole 128-byte lines, of few tokens, as long as the caches hold dW."""
    sizes = [(*c, True) for c in narrow.SPLIT_LINES] + [(16, 1024, 32000, False), (100, 4096, 32000, False),
                                                       (96, 2760, 32000, False), (200, 1112, 50257, False),
                                                       (256, 1288, 32000, False), (300, 1000, 32000, False)]
    for (t, d, v, cached), L in zip(sizes, layouts([backward(t, d, v, t) for t, d, v, _ in sizes])):
        assert (L["dw_tp"], L["dw_tq"], L["dw_splits"]) == (256, 256, 1), (t, d, v)  # (whose kernel it is for)
        assert L["dw_cached"] == cached, (t, d, v)
    L, = layouts([backward(16, 1000, 32000, 16, F32)])
    assert not L["dw_cached"]
