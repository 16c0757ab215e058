"""Plain forms of the 8-bit linear operators, and the bounds their results are held to.

Rows.  p are a row's products, m the largest in size, Q = 127 or 448, step = max(m / Q, 2^-126).  The kernels form
p in fp32 (at most two roundings), inv = Q / m (one) and p * inv (one), so a code is the rounding of
y (1 + e), y = p / step, |e| <= 5 u with u = 2^-24 (the 64-bit step has none).  An int8 code is then within 1/2 + 127 * 5 u of
y, an E4M3 code within half its spacing at y, plus 5 u |y|.  A gate's value has an error of its own
(gate_error below), its row's maximum the same, so both count.

Scales.  step: the rounding of m and of the division.  r of a norm: a thread sums at most 64 terms in fp32 one
after another (an error of 64 u at most), 5 more sums in the warp and 16 over warps; half of that passes the root;
the reciprocal root has 2 ulp (4 u), the mean and its scale 3 u, the last product 1 u: 56 u in all.
"""
import torch

U = 2.0 ** -24
TOP = {False: 127.0, True: 448.0}
SCALE_BOUND = 56 * U
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def values(codes, fp8):
    """The numbers that the codes stand for, without their scale."""
    return codes.view(torch.float8_e4m3fn).double() if fp8 else codes.double()


def e4m3_half(y):
    """Half the spacing of E4M3 at y (normals from 2^-6)."""
    e = torch.frexp(y.abs().clamp(min=2.0 ** -6)).exponent.double() - 1
    return torch.exp2(e - 4)


def steps(p, fp8):
    """(p in steps, step of each row) in 64 bits."""
    step = (p.abs().amax(-1) / TOP[fp8]).clamp(min=2.0 ** -126)
    return p / step[..., None], step


def norm_products(s, w, offset):
    return s.double() * (1.0 if w is None else w.double() + offset)


def norm_factor(s, eps):
    return 1.0 / (s.double().square().mean(-1) + eps).sqrt()


def gate_products(x, act):
    g, u = x.double().chunk(2, -1)
    v = g if act == "silu" else 2.0 * (2.0 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3)
    return torch.sigmoid(v) * g * u, v


def gate_error(v):
    """The relative error of a gate: its exponential (2^-22), the argument's roundings (5 of them, each |v| u) and
    the products and quotients (8)."""
    return (4 + 5 * v.abs() + 8) * U


def check_codes(codes, y, fp8, err=0.0):
    """codes against y = p / step in 64 bits, p having a relative error of `err` beyond the roundings above."""
    got = values(codes, fp8)
    slack = (5 * U + err) * y.abs()
    half = e4m3_half(y.abs() + slack) if fp8 else 0.5
    assert (got.abs() <= TOP[fp8]).all()
    off = (got - y).abs() - half - slack
    assert (off <= 0).all(), (off.max().item(), (off > 0).sum().item())


def plain_codes(p, fp8):
    """The codes of fp32 products p on the CPU, by the formula with IEEE operations: what the kernels have to give bit
    for bit.  int8: p Q / m rounded to fp32 and then to the nearest even code, the quotient in 64 bits (p Q is exact
    there)."""
    m = p.abs().amax(-1, keepdim=True)
    inv = torch.minimum(torch.full_like(m, TOP[fp8]) / m, torch.tensor(2.0 ** 126))
    if not fp8:
        y = torch.where(inv < 2.0 ** 126, p.double() * TOP[fp8] / m.double(), p.double() * 2.0 ** 126)
        return y.float().round().to(torch.int8)
    return (p * inv).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def product_sums(a, w, fp8):
    """(sums, sums of absolute values) of a w^T in 64 bits; exact for int8."""
    x, y = values(a, fp8), values(w, fp8)
    return x @ y.T, x.abs() @ y.abs().T


def product_exact(sums, sa, sw, bias, dtype):
    """What the kernels have to give for an exactly known sum: fp32 operations in the stated order, one rounding."""
    y = sums.float() * sa[:, None] * sw
    return (y if bias is None else y + bias.float()).to(dtype)


def product_bound(mags, k, sa, sw, bias, want, dtype):
    """How far an E4M3 product may be off: the matrix instructions add 32 products at a time to an fp32 sum, aligned
    to the largest and cut (a step of the sum, 2^-23, for each of the k/32 additions, and as much for the products
    inside one); parts of a split sum are joined in fp32 (at most 32 more); three roundings and the bias's follow, and the output's."""
    sums = mags * sa.double()[:, None] * sw.double() * ((2 * (k // 32 + 1) + 32) * 2.0 ** -23)
    last = want.abs() + (0.0 if bias is None else bias.double().abs())
    return sums + last * (4 * U + HALF[dtype]) + TINY[dtype]
