"""Attention of sequences with at most 8 rows per key head, 16-bit: the weights keep two 16-bit parts.

Bound.  With half steps h of the type, the first part of a weight is off by at most h relative to it, so the second is
at most that and off by h of itself: h^2 of the weight (2^-16, 2^-22), and for fp16 at least half a step of its
subnormals, 2^-25, of a row whose largest weight is 1 or more.  Weights sum to 1 over the row's sum, so with m keys of
values up to X the row is off by at most (h^2 + m 2^-25) X more than an fp32 call's bound, before its one rounding.
"""
import math

import pytest
import torch

import paged_ref
from test_paged_attention import make, run

gpu = pytest.mark.gpu


def check(c, starts=True, **kw):
    out, lse = run(c, starts=starts, **kw)
    torch.cuda.synchronize()
    dt, D = c["q"].dtype, c["q"].shape[2]
    ref, tol, rl, lt = paged_ref.attention(c["q"].float(), c["k"].float(), c["v"].float(), c["table"], c["lens"],
                                           c["starts"] if starts else None, c["page"], D ** -0.5, **kw)
    X = c["v"].double().nan_to_num(0).abs().max()
    m = int(c["lens"].max())
    tol = tol + (paged_ref.HALF[dt] ** 2 + (m * 2.0 ** -25 if dt == torch.float16 else 0.0)) * X
    paged_ref.check_rows(out, ref, tol, dt)
    got = lse.cpu().double()  # -inf where a row sees nothing
    assert ((got == rl) | ((got - rl).abs() <= lt)).all()


@gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hk,D", [(4, 2, 64), (8, 2, 128), (16, 2, 256), (24, 4, 256), (5, 1, 80), (3, 3, 128),
                                     (6, 2, 192), (8, 1, 8)])
def test_one_rounding_of_decode_rows(dt, hq, hk, D):
    check(make(dt, hq, hk, D, 16, [(n, 1) for n in (1, 2, 15, 16, 17, 33, 64, 65, 127, 300)], seed=40 + D), starts=False)


@gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("window", [0, 20])
def test_one_rounding_of_small_chunks(dt, window):
    # a chunk of up to 8 rows per key head; 8, 6, 2 and 0 rows, and sequences split over the GPU
    check(make(dt, 4, 2, 128, 16, [(40, 4), (33, 3), (17, 1), (9, 0), (2, 4), (5000, 3)], seed=41), window=window)


@gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("new", [1, 3])
def test_infinite_values_that_a_row_sees(dt, new):
    # the second part of a weight has either sign, and may be zero: an infinity stays what the formula has
    c = make(dt, 4, 2, 128, 16, [(50, new), (40, new), (9000, new)], seed=42)
    for b, j, bad in ((0, 20, math.inf), (1, 39, -math.inf), (2, 100, -math.inf)):
        c["v"][int(c["table"][b, j // 16]) * 16 + j % 16] = bad
    out, _ = run(c)
    out = out.cpu()
    assert (out[:new] == math.inf).all()
    assert (out[2 * new - 1] == -math.inf).all() and torch.isfinite(out[new:2 * new - 1]).all()
    assert (out[2 * new:] == -math.inf).all()
