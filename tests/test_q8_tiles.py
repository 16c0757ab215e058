"""The 8-bit product where a CTA computes many tiles one after the other: each tile's scales, sums and barriers are
the next one's."""
import pytest
import torch

from memory_bound_decode_qk_gb300 import edge_ops
from test_q8_matmul import check, operands

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
# odd numbers of channels: every store form but the plain one orders the lanes of a warp by itself.  Ragged last
# tiles of channels, of which some lanes store nothing; scales that differ by powers of two from token to token
@pytest.mark.parametrize("t,n,k", [(16, 100001, 64), (31, 60007, 80), (64, 60005, 64), (2049, 6007, 48), (4099, 2563, 64),
                                   (1100, 12001, 1040)])
def test_every_tile_has_its_own_scales(t, n, k, dtype, fp8):
    a, w, sa, sw, bias = operands(t, n, k, fp8, 31)
    sa = sa * torch.exp2((torch.arange(t, device="cuda") * 7 % 13).float())
    first = edge_ops.matmul_q8(a, w, sa, sw, bias=bias.to(dtype), dtype=dtype)
    check(first, a, w, sa, sw, bias.to(dtype), dtype, fp8)
    for _ in range(5):
        assert torch.equal(edge_ops.matmul_q8(a, w, sa, sw, bias=bias.to(dtype), dtype=dtype), first)


@pytest.mark.parametrize("fp8", [False, True])
# sums cut over a cluster: 1 to 63 channels or tokens more than a tile, so that some lanes and warps store nothing
@pytest.mark.parametrize("t,n,k", [(9, 1, 2592), (9, 65, 1968), (17, 131, 3872), (33, 129, 9728), (64, 193, 9728), (2, 70, 321),
                                   (9, 201, 9727), (65, 65, 2049), (20, 131, 579)])
def test_ragged_ends_of_a_cut_sum(t, n, k, fp8):
    a, w, sa, sw, bias = operands(t, n, k, fp8, 32)
    for dtype in (torch.float32, torch.bfloat16):
        first = edge_ops.matmul_q8(a, w, sa, sw, bias=bias.to(dtype), dtype=dtype)
        check(first, a, w, sa, sw, bias.to(dtype), dtype, fp8)
        for _ in range(20):
            assert torch.equal(edge_ops.matmul_q8(a, w, sa, sw, bias=bias.to(dtype), dtype=dtype), first)
