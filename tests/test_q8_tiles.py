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
