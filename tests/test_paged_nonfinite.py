"""Infinities and NaN in the queries, keys and values of paged attention: what a row sees reaches it, whether its unit
is split over the GPU or not, and what it does not see leaves no trace, to the bit.
"""
import math

import pytest
import torch

import paged_ref
from test_paged_attention import make, run

gpu = pytest.mark.gpu

# type, heads, head size, new tokens of a sequence: one for each kernel (any type, and odd heads; 16 rows; 64 rows;
# two query tiles; one query tile)
PATHS = {"any": ("f32", 8, 2, 128, 3), "odd": ("bf16", 6, 2, 33, 3), "few": ("bf16", 8, 2, 128, 1),
         "few wide": ("f16", 16, 2, 256, 1), "more": ("bf16", 8, 2, 128, 9), "many": ("bf16", 8, 2, 128, 40),
         "many wide": ("f16", 8, 2, 256, 40)}


@gpu
@pytest.mark.parametrize("keys", [60, 9000])  # within one part of a unit; over many parts
@pytest.mark.parametrize("path", PATHS)
def test_nan_in_queries_and_keys(path, keys):
    dt, hq, hk, D, new = PATHS[path]
    # the first sequence has NaN in one query row, in the second every key holds NaN, in the third a run of keys that
    # fills parts of its own; the last is clean
    c = make(dt, hq, hk, D, 16, [(keys, new), (keys, new), (keys, new), (keys - 9, new)], seed=31)
    c["q"][new - 1, :, 0] = math.nan
    for b, first, behind in ((1, 0, keys), (2, keys // 4, keys // 2)):
        for j in range(first, min(behind, keys)):
            c["k"][int(c["table"][b, j // 16]) * 16 + j % 16, :, 0] = math.nan
    out, lse = run(c)
    torch.cuda.synchronize()
    ref, tol, rl, lt = paged_ref.attention(c["q"], c["k"], c["v"], c["table"], c["lens"], c["starts"], 16, D ** -0.5)
    gone = torch.isnan(rl)
    assert gone[new - 1:3 * new].all() and not gone[:new - 1].any() and not gone[3 * new:].any()
    assert torch.isnan(out.cpu()[gone]).all(), "a row of NaN scores became finite"
    assert torch.isnan(lse.cpu()[gone]).all()
    paged_ref.check_rows(out, ref, tol, c["q"].dtype)
    assert ((lse.cpu().double() - rl).abs() <= lt)[~gone].all()
