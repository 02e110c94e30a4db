"""The output-head losses at the ends of their ranges: offsets that pass 2^31
elements in every large array, the most tokens, the largest vocabulary, the
longest rows.  Checked like the large cases (tests/head_device.py)."""

import pytest
import torch

import head_device as dev

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32

# (tokens, hidden, vocab, K, tokens a block of the check)
CASES = {
    "tokens x vocab past 2^31": (4000000, 64, 700, 0, 65536),
    "tokens x hidden past 2^31": (1000000, 2304, 300, 0, 65536),
    "vocab x hidden past 2^31": (70, 2560, 1048577, 0, 70),
    "the most tokens": ((1 << 24) - 1, 8, 200, 0, 262144),
    "many pieces": (300, 136, 4200000, 0, 100),
    "the longest rows": (400, 65536, 500, 0, 400),
    "the longest rows, few tokens": (70, 65536, 500, 0, 70),
    "distillation, the largest vocabulary": (3, 8, (1 << 27) - 1, 1024, 3),
    "distillation, tokens x entries past 2^31": (2200000, 64, 300, 1000, 16384),
}


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", list(CASES))
def test_ends_of_the_ranges(case, dtype):
    t, d, v, k, block = CASES[case]
    print(f"case {case} {CASES[case]} {dtype}", flush=True)
    torch.cuda.empty_cache()
    edges = [x for x in (0, 255, 256, v - 1) if x < v]
    if k == 0:
        h, w, y, up = dev.inputs(t, d, v, dtype, 700 + d, edges, dead=0.1 if t > 100 else 0.0)
        args = dict(y=y)
    else:
        h, w, _, up = dev.inputs(t, d, v, dtype, 700 + d, edges)
        ids, z = dev.teacher(t, k, v, 750 + d, edges)
        h[~(ids >= 0).any(1)] = float("nan")
        args = dict(ids=ids, z=z, tau=2.0)
    got = dev.run(h, w, up, **args)
    dev.check(case, got, h, w, up, block=block, **args)
    del got, h, w, args
    torch.cuda.empty_cache()
