"""GPU parity of the output-head losses where calls are large: 256-wide tiles of
every product, more tiles than workgroups (each then takes several, the next
one's loads behind the epilogue), several pieces of the vocabulary with a partial
last one, sums over the tokens in splits of wide tiles.  tests/test_head_layout.py
holds that CASES reach all of these, by the library's own rule.

The oracle is the definitions in fp64 on the device; tests/head_device.py has it
and the bounds.
"""

import sys

import pytest
import torch

import head_device as dev

BF16, F32 = torch.bfloat16, torch.float32

# (tokens, hidden, vocab, K) -- K 0: cross entropy
CASES = {
    "wide tiles, two pieces": (1500, 1024, 100003, 0),
    "packed rows, two pieces": (700, 300, 300007, 0),
    "long token sums": (8192, 256, 30001, 0),
    "long token sums, two pieces": (20000, 300, 15001, 0),
    "token sums, narrower tiles": (3000, 256, 15001, 0),
    "one slab a tile": (4100, 64, 40003, 0),
    "many tiles of dH": (16500, 1100, 8003, 0),
    "stream, wide": (250, 264, 100100, 0),
    "stream, few tokens": (120, 264, 40100, 0),
    "stream, several pieces": (384, 640, 300007, 0),
    "two parts of ds, two pieces": (100, 64, 600011, 0),
    "two parts of ds, stream, two pieces": (100, 70, 600011, 0),
    "distillation, two pieces": (1500, 512, 100003, 12),
    "distillation, packed rows": (1100, 264, 100003, 5),
    "distillation, long token sums": (8192, 256, 30001, 3),
    "distillation, stream, several pieces": (384, 136, 300007, 8),
    "distillation, two parts of ds": (90, 64, 600011, 20),
}


def edges(v):
    """Rows next to every border that a piece (of either type) may have: pieces are
    multiples of 256; the first and last rows, and the borders of equal parts."""
    e = {0, 255, 256, v - 1, v // 256 * 256 - 1, v // 256 * 256}
    padded = (v + 255) // 256 * 256
    for parts in range(2, 9):
        step = (-(-padded // parts) + 255) // 256 * 256
        for x in range(step, v, step):
            e.update((x - 1, x))
    return sorted(x for x in e if 0 <= x < v)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", list(CASES))
def test_large_calls(case, dtype):
    t, d, v, k = CASES[case]
    print(f"case {case} {CASES[case]} {dtype}", flush=True)
    sys.stdout.flush()
    if k == 0:
        h, w, y, up = dev.inputs(t, d, v, dtype, 900 + t, edges(v), dead=0.1)
        gl = torch.where(y != dev.IGN, 0.3 / t, float("nan")).float()
        args = dict(y=y, gl=gl)
    else:
        h, w, _, up = dev.inputs(t, d, v, dtype, 900 + t, edges(v))
        ids, z = dev.teacher(t, k, v, 950 + t, edges(v))
        h[~(ids >= 0).any(1)] = float("nan")
        args = dict(ids=ids, z=z, tau=2.0)
    got = dev.run(h, w, up, **args)
    dev.check(case, got, h, w, up, **args)
