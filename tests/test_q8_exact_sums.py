"""E4M3 products whose sums fp32 holds exactly: bit for bit.

The bound of test_q8_matmul.py is a worst case over all terms, which an accumulator of fewer bits could meet too.  Here
operands are whole numbers up to 16 in size (E4M3 has all of them), so products are whole numbers up to 256, and with k up
to 65,520 terms every partial sum, in any order, is a whole number below 2^24: an accumulator of fp32's 24 bits makes no
error at all, rounding or cutting, and one that holds fewer loses the ones below."""
import pytest
import torch

from memory_bound_decode_qk_gb300 import edge_ops

pytestmark = pytest.mark.gpu

# the stream of weights (up to 8 tokens), one CTA whole and over clusters, pairs with one tile and several, rows off 16
# bytes whole and over clusters
SHAPES = [(1, 64, 9728), (5, 200, 65520), (12, 640, 65520), (20, 130, 9728), (40, 640, 65520), (64, 2560, 65520),
          (64, 60005, 2048), (300, 700, 65520), (700, 2560, 65520), (1201, 5120, 2048), (4099, 2563, 1040), (3, 70, 65519),
          (64, 640, 9725), (700, 1500, 515)]


def codes(x):
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def product(a, w):
    t, n = a.shape[0], w.shape[0]
    one = torch.ones(max(t, n), device="cuda")
    return edge_ops.matmul_q8(codes(a), codes(w), one[:t], one[:n], dtype=torch.float32)


@pytest.mark.parametrize("signed", [False, True])
@pytest.mark.parametrize("t,n,k", SHAPES)
def test_whole_numbers(t, n, k, signed):
    g = torch.Generator(device="cuda").manual_seed(t + n + k)
    a = torch.randint(-16 if signed else 0, 17, (t, k), generator=g, device="cuda").float()
    w = torch.randint(-16 if signed else 0, 17, (n, k), generator=g, device="cuda").float()
    assert torch.equal(product(a, w).double(), a.double() @ w.double().T)


@pytest.mark.parametrize("t,n,k", SHAPES)
def test_ones_behind_a_large_sum(t, n, k):
    """256 in every term but the last seven, which are 1."""
    a, w = torch.full((t, k), 16.0, device="cuda"), torch.full((n, k), 16.0, device="cuda")
    a[:, -7:] = 1.0
    w[:, -7:] = 1.0
    w[::2, -1] = 0.0
    want = torch.full((t, n), 256.0 * (k - 7) + 7, device="cuda", dtype=torch.float64)
    want[:, ::2] -= 1
    assert torch.equal(product(a, w).double(), want)
