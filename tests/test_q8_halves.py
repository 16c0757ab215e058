"""int8 codes of values halfway between two codes: the even one, as the definition round(p Q / m) has it.

Why no tolerance is needed.  Quantized rows of 16-bit types: p = P 2^a, m = M 2^b with whole P, M of 11 bits (or 8)
each.  A quotient y = 127 p / m that is not halfway, n + 1/2, differs from it by |254 p - (2 n + 1) m| / (2 m), at
least 2^min(a - b, 0) / (2 M).  For y in [2^e, 2^(e + 1)), 2^(a - b) is more than 2^(e - 8), so that is more than
2^(e - 20), and the rounding of y to fp32 moves it by 2^(e - 24) at most (the kernel's y is one rounding of a number
that is right to 2^-46).  Halfway quotients are fp32 numbers themselves.  So the codes are those of the definition,
every one."""
import pytest
import torch

import q8_ref as ref
from memory_bound_decode_qk_gb300 import edge_ops

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CALLS = {
    "quantize": lambda x: edge_ops.quantize_q8(x),
    "norm": lambda x: edge_ops.rmsnorm_q8(x),
    "norm with a weight": lambda x: edge_ops.rmsnorm_q8(x, torch.zeros_like(x[0]), weight_offset=1),
    "add norm": lambda x: edge_ops.add_rmsnorm_q8(x, torch.zeros_like(x)),
}


def maxima(dt):
    """Every significand of a 16-bit type, 4096 of fp32."""
    if dt == "fp32":
        return 1.0 + torch.rand(4096, generator=torch.Generator().manual_seed(3))
    n = 128 if dt == "bf16" else 1024
    return 1.0 + torch.arange(n) / n


def definition(x):
    """round(127 p / m) in 64 bits.  (127 p is exact there, and a quotient that is halfway too.)"""
    p = x.double()
    return (p * 127.0 / p.abs().amax(-1, keepdim=True)).round().to(torch.int8)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_the_proof_on_every_pair_of_significands(dt):
    """The plain codes against whole numbers: 127 p / m is rounded in integers, for all m and 61 p of each."""
    top = 128 if dt == "bf16" else 1024
    M = torch.arange(top, 2 * top, dtype=torch.int64)
    g = torch.Generator().manual_seed(5)
    P = torch.randint(1, 2 * top, (top, 61), generator=g)
    P = torch.cat([M[:, None], torch.minimum(P, M[:, None]), M[:, None]], 1)
    P[:, 1:31] = P[:, 1:31] // 2 * 2  # more even ones: halves of others
    q, r = (127 * P) // M[:, None], (127 * P) % M[:, None]
    want = q + ((2 * r > M[:, None]) | ((2 * r == M[:, None]) & (q % 2 == 1))).long()
    x = (P.double() / top).float().to(DT[dt])
    assert torch.equal(x.double(), P.double() / top)
    assert torch.equal(ref.plain_codes(x.float(), False).long(), want)
    assert torch.equal(definition(x).long(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("n", [64, 37, 9000])
@pytest.mark.parametrize("power", [0, -3, 9])
def test_half_of_the_maximum(power, n, dt, call):
    m = maxima(dt)
    x = torch.zeros(len(m), n, dtype=torch.float64)
    x[:, 0], x[:, 3], x[:, n - 1] = m, m / 2, -m / 2
    x = (x * 2.0 ** power).to(DT[dt])
    codes, _ = CALLS[call](x.cuda())
    want = torch.zeros(len(m), n, dtype=torch.int8)
    want[:, 0], want[:, 3], want[:, n - 1] = 127, 64, -64
    assert torch.equal(codes.cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("dt", ["fp16", "fp32"])
@pytest.mark.parametrize("unit", [1.0, 1.25, 1.5, 1.75, 3.0, 5.0, 7.0])
@pytest.mark.parametrize("n", [256, 255])
def test_every_half(n, unit, dt, call):
    """A maximum of 127 units, and all odd multiples of half of one."""
    halves = (torch.arange(-127, 127, dtype=torch.float64) + 0.5) * unit
    x = torch.zeros(3, n, dtype=torch.float64)
    x[:, :254], x[:, 254] = halves, 127 * unit
    typed = x.to(DT[dt])
    assert torch.equal(typed.double(), x)
    codes, _ = CALLS[call](typed.cuda())
    assert torch.equal(codes.cpu(), (x / unit).round().to(torch.int8))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,n", [(1024, 4096), (300, 2561), (33, 40000)])
def test_quantized_rows_are_the_definition(rows, n, dt):
    x = torch.randn(rows, n, generator=torch.Generator().manual_seed(rows)).to(DT[dt])
    codes, _ = edge_ops.quantize_q8(x.cuda())
    assert torch.equal(codes.cpu(), definition(x))


@pytest.mark.gpu
@pytest.mark.parametrize("most", [3.4e38, 2.0 ** 127, 1.5 * 2.0 ** 126, 2.0 ** 104, 2.0 ** -110, 1.3 * 2.0 ** -118])
@pytest.mark.parametrize("n", [64, 33])
def test_the_largest_and_smallest_maxima(n, most):
    """Where the rest of the inverse is subnormal, and next to the smallest step."""
    x = torch.zeros(2, n)
    x[:, 1] = most
    x[:, 2], x[1, 3] = x[0, 1] / 2, -x[0, 1] / 2
    codes, scales = edge_ops.quantize_q8(x.cuda())
    want = torch.zeros(2, n, dtype=torch.int8)
    want[:, 1], want[:, 2], want[1, 3] = 127, 64, -64
    assert torch.equal(codes.cpu(), want) and scales.isfinite().all()
