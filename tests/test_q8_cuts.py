"""How calls of the 8-bit product are cut, on the CPU: which kernel serves a call, and what it falls back on."""
import pytest

import q8_cuts


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    return q8_cuts.build(str(tmp_path_factory.mktemp("cuts")))


MANY = [(1201, 5120, 2048), (4096, 19456, 2560), (130, 19456, 9728), (677, 5029, 928), (5000, 3840, 9728)]


@pytest.mark.parametrize("int8", [False, True])
def test_pairs_serve_many_tokens(program, int8):
    for cut in q8_cuts.cuts(program, [(*c, int8) for c in MANY]):
        assert cut.status == 0 and cut.int8 == int8 and cut.kernel == "pair", cut


@pytest.mark.parametrize("int8", [False, True])
def test_without_room_for_pairs_single_ctas_serve_every_call(program, int8):
    """The occupancy calculator fails, or the launch of pairs finds no room."""
    calls = [(*c, int8) for c in MANY]
    for cut in q8_cuts.cuts(program, calls, "c"):
        assert cut.status == 0 and cut.kernel == "one" and cut.split == 1, cut
    for cut in q8_cuts.cuts(program, [c + (2, 0, 1) for c in calls]):
        assert cut.status == 0 and cut.kernel == "one", cut


def test_a_kernel_whose_registers_nobody_knows_is_not_launched(program):
    """int8 warps ask for registers, and would wait for ever if there were too few."""
    for cut in q8_cuts.cuts(program, [(64, 2560, 9728, True), (4096, 2560, 9728, True)], "r"):
        assert cut.status == 7 and cut.kernel == "none", cut


def test_a_call_that_fails_leaves_no_error_for_the_next(program):
    """A launch that the runtime refuses, then the same calls again."""
    calls = [(1, 2560, 2560, True), (64, 2560, 9728, False), (5, 33, 47, True), (64, 2560, 9728, True)]
    for call in calls:
        bad, good, other = q8_cuts.cuts(program, [call + (2, 0, 1), call, calls[0]])
        assert bad.status == 7 and bad.kernel == "none"
        assert good.status == 0 and other.status == 0, (call, good, other)
    bad, good = q8_cuts.cuts(program, [(64, 2560, 9728, True), (1, 2560, 2560, True)], "r")
    assert bad.status == 7 and good.status == 0
