"""Infinities and NaN in the queries, keys and values of paged attention: what a row sees reaches it, whether its unit
is split over the GPU or not, and what it does not see leaves no trace, to the bit.
"""
import math

import pytest
import torch

import paged_ref
from memory_bound_decode_qk_gb300 import edge_ops
from test_paged_attention import make, run

gpu = pytest.mark.gpu

# type, heads, head size, new tokens of a sequence, tokens of a page: one for each kernel (any type, and odd heads;
# 16 rows; 64 rows; two query tiles; one query tile)
PATHS = {"any": ("f32", 8, 2, 128, 3, 16), "odd": ("bf16", 6, 2, 33, 3, 16), "few": ("bf16", 8, 2, 128, 1, 16),
         "few wide": ("f16", 16, 2, 256, 1, 16), "more": ("bf16", 8, 2, 128, 13, 13),
         "more wide": ("f16", 8, 2, 256, 20, 12), "many": ("bf16", 8, 2, 128, 40, 16),
         "many few": ("bf16", 8, 2, 128, 9, 16), "many wide": ("f16", 8, 2, 256, 40, 16)}


@gpu
@pytest.mark.parametrize("keys", [60, 9000])  # within one part of a unit; over many parts
@pytest.mark.parametrize("path", PATHS)
def test_nan_in_queries_and_keys(path, keys):
    dt, hq, hk, D, new, page = PATHS[path]
    # the first sequence has NaN in one query row, in the second every key holds NaN, in the third a run of keys that
    # fills parts of its own; the last is clean
    c = make(dt, hq, hk, D, page, [(keys, new), (keys, new), (keys, new), (keys - 9, new)], seed=31)
    c["q"][new - 1, :, 0] = math.nan
    for b, first, behind in ((1, 0, keys), (2, keys // 4, keys // 2)):
        for j in range(first, min(behind, keys)):
            c["k"][int(c["table"][b, j // page]) * page + j % page, :, 0] = math.nan
    out, lse = run(c)
    torch.cuda.synchronize()
    ref, tol, rl, lt = paged_ref.attention(c["q"], c["k"], c["v"], c["table"], c["lens"], c["starts"], page, D ** -0.5)
    gone = torch.isnan(rl)
    assert gone[new - 1:3 * new].all() and not gone[:new - 1].any() and not gone[3 * new:].any()
    assert torch.isnan(out.cpu()[gone]).all(), "a row of NaN scores became finite"
    assert torch.isnan(lse.cpu()[gone]).all()
    paged_ref.check_rows(out, ref, tol, c["q"].dtype)
    assert ((lse.cpu().double() - rl).abs() <= lt)[~gone].all()


def poison(c, b, j, value, what="v"):
    c[what][int(c["table"][b, j // c["page"]]) * c["page"] + j % c["page"]] = value


WIDE = [(8, 2, 128), (4, 4, 64), (2, 1, 80), (8, 2, 256), (3, 1, 192)]


@gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hk,D", WIDE)
@pytest.mark.parametrize("window", [0, 150])
def test_unseen_values_change_no_bit(dt, hq, hk, D, window):
    # prompts and a late chunk.  With two query tiles the first ends keys before the second; the values that only
    # the second sees must not change how the first is summed
    c = make(dt, hq, hk, D, 16, [(700, 600), (257, 257), (1900, 300)], seed=32)
    want, lse = run(c, window=window)
    marks = [(0, 131, math.inf), (0, 400, math.nan), (1, 120, -math.inf), (1, 255, math.nan), (2, 1700, math.inf)]
    for b, j, bad in marks:
        poison(c, b, j, bad)
    sees = torch.zeros(want.shape[0], dtype=torch.bool)
    for b, j, _ in marks:
        first, n, at = int(c["starts"][b]), int(c["starts"][b + 1] - c["starts"][b]), int(c["lens"][b])
        pos = torch.arange(at - n, at)
        sees[first:first + n] |= (pos >= j) & ((pos - j < window) if window else True)
    for _ in range(10):
        out, stats = run(c, window=window)
        assert torch.equal(out[~sees], want[~sees]) and torch.equal(stats, lse)
        assert not torch.isfinite(out[sees]).any(), "what a row sees reaches it"


@gpu
@pytest.mark.parametrize("hq,hk,D", [(8, 2, 128), (8, 2, 256)])
def test_unseen_values_of_a_long_context(hq, hk, D):
    # infinities that only the last tokens of a chunk see, 32 thousand keys before them: the sum must neither run
    # into the kernel's limit of two seconds for a wait nor take much longer than without
    c = make("bf16", hq, hk, D, 64, [(32768, 300), (32768, 300)], seed=33)
    d = {n: x.cuda() for n, x in c.items() if n != "page"}

    def go():
        out = edge_ops.paged_attention(d["q"], d["k"], d["v"], d["table"], d["lens"], page_size=64, q_starts=d["starts"])
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        edge_ops.paged_attention(d["q"], d["k"], d["v"], d["table"], d["lens"], page_size=64, q_starts=d["starts"], out=out)
        end.record()
        end.synchronize()
        return out, start.elapsed_time(end)

    want, clean_ms = go()
    for b, j in ((0, 32700), (0, 32560), (1, 32767)):
        poison(c, b, j, math.inf)
    d["v"] = c["v"].cuda()
    out, ms = go()
    print(f"{ms:.3f} ms, {clean_ms:.3f} ms without infinities")
    sees = torch.zeros(600, dtype=torch.bool)
    sees[32560 - 32468:300] = True
    sees[599] = True
    assert torch.equal(out[~sees], want[~sees])
    assert (out[sees] == math.inf).all()
    assert ms < 50, "the row sums of a context of 32768 keys take 70 ms and more one by one"


@gpu
@pytest.mark.parametrize("hq,hk,D", [(128, 32, 64), (64, 16, 256)])
def test_unseen_values_before_many_units_without_an_edge(hq, hk, D):
    # chunks with infinities and NaN in their last keys, each followed by sequences of one token over whole tiles of
    # keys: hundreds of units that have no edge, through which the search of the edges runs ahead of the sums
    shape = []
    for i in range(12):
        shape += [(300 + i, 300 + i)] + [(128 + 128 * (k % 2), 1) for k in range(12)]
    c = make("bf16", hq, hk, D, 16, shape, seed=34)
    rows = c["q"].shape[0] * (hq // hk) / len(shape)
    assert rows > 64, "the call is one for the kernel of wide chunks"
    want, lse = run(c)
    sees = torch.zeros(want.shape[0], dtype=torch.bool)
    for i in range(12):
        b = 13 * i
        n = shape[b][0]
        poison(c, b, n - 1, math.nan)
        poison(c, b, n - 3, math.inf)
        sees[int(c["starts"][b]) + n - 3:int(c["starts"][b]) + n] = True
    for _ in range(20):
        out, stats = run(c)
        assert torch.equal(out[~sees], want[~sees]) and torch.equal(stats, lse)
        assert not torch.isfinite(out[sees]).any()


@gpu
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("path", PATHS)
def test_a_value_whose_weight_underflows_is_seen(path, value):
    # a weight is small, never nothing: e^-500 of an infinity is one, and NaN stays NaN
    dt, hq, hk, D, new, page = PATHS[path]
    c = make(dt, hq, hk, D, page, [(200, new), (90, new)], seed=35)
    c["q"][:] = 1.0
    for b, j in ((0, 198), (1, 89)):
        poison(c, b, j, value)
        poison(c, b, j, -500.0 / D ** 0.5, "k")
    out, _ = run(c)
    sees = torch.zeros(2 * new, dtype=torch.bool)
    sees[max(0, new - 2):new] = True
    sees[2 * new - 1] = True
    out = out.cpu()
    assert not torch.isfinite(out[sees]).any(), "a value that the row sees was passed over"
    assert torch.isfinite(out[~sees]).all()
