"""Every cut that the 8-bit product chooses is computed and compared: tiles of 16, 32 and 64 tokens by one CTA, whole and
over clusters, and pairs, each of them also with several tiles for a CTA one after the other; rows that do not start on
16 bytes, whole and over clusters.

The cuts come from a model of the times.  So that a change of the model cannot leave one without a test, the library's
host code says here, on the CPU, how 60,000 drawn calls and the compared ones are cut."""
import math
import random

import pytest

import q8_cuts
import test_q8_matmul as product

# tokens, channels, sum: cuts that the sizes of test_q8_matmul.py do not reach
SHAPES = [(38, 19973, 96), (1, 5269, 5568), (151, 19811, 32), (1576, 31, 3952), (1127, 17, 3744), (855, 17, 3936),
          (462, 19, 7744), (4955, 21, 16), (3662, 21, 8128), (2452, 17, 5392), (2036, 21, 5552), (1370, 17, 6880),
          (43, 1549, 57072), (81, 12553, 1360), (51, 19929, 1824), (171, 19483, 912), (485, 13989, 688),
          (926, 15725, 80), (2730, 4243, 16), (17, 19579, 32), (1, 6527, 2592), (752, 17, 3280), (20, 1609, 5152),
          (441, 21, 4032), (35, 1589, 15296), (287, 12133, 272), (2940, 12223, 16),
          # rows that do not start on 16 bytes, over clusters of 3 and 6
          (130, 70, 750), (65, 131, 1613)]


def kinds(cuts):
    """(int8, kernel, tokens of a tile, CTAs that share one, whether a CTA has several)"""
    return [(c.int8, c.kernel, c.tokens, c.split, c.rounds > 1) for c in cuts]


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    return q8_cuts.build(str(tmp_path_factory.mktemp("cuts")))


@pytest.fixture(scope="module")
def compared(program):
    shapes = product.SHAPES + SHAPES
    return set(kinds(q8_cuts.cuts(program, [(*s, int8) for s in shapes for int8 in (False, True)])))


def test_no_call_has_a_cut_that_is_not_compared(program, compared):
    rng = random.Random(12)

    def span(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    calls = [(span(1, 5000), span(16, 20000), 16 * span(1, 608), rng.random() < 0.5) for _ in range(40000)]
    calls += [(span(20, 70), span(16, 20000), 16 * span(100, 8191), rng.random() < 0.5) for _ in range(10000)]
    calls += [(span(1, 5000), span(16, 20000), 16 * span(1, 608) + 1, rng.random() < 0.5) for _ in range(10000)]
    missing = {}
    for call, kind in zip(calls, kinds(q8_cuts.cuts(program, calls))):
        if kind not in compared:
            missing.setdefault(kind, call)
    assert not missing, missing


def test_every_tile_and_every_form_is_compared(compared):
    for int8 in (False, True):
        for tokens in (16, 32, 64):
            assert (int8, "one", tokens, 1, False) in compared and (int8, "one", tokens, 1, True) in compared
            assert {2, 3, 4, 5, 6, 8} <= {c[3] for c in compared if c[:3] == (int8, "one", tokens)}
        for tokens in range(96, 193 if int8 else 257, 32):
            assert (int8, "pair", tokens, 1, False) in compared and (int8, "pair", tokens, 1, True) in compared
        assert set(range(1, 9)) == {c[3] for c in compared if c[:2] == (int8, "any")}
        assert (int8, "few", 8, 1, False) in compared


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("t,n,k", SHAPES)
def test_sizes(t, n, k, fp8):
    product.test_sizes(t, n, k, fp8)
