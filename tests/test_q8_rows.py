"""Rows in 8 bits with a scale each: norm, residual and norm, gate, quantization, against their formulas."""
import pytest
import torch

import q8_ref as ref
from memory_bound_decode_qk_gb300 import edge_ops

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# rows x codes: single values, odd lengths, a vector more or less than a warp or a CTA holds, the longest row in
# registers (16-bit types: 32,768) and one that is longer
SHAPES = [(1, 1), (3, 7), (5, 48), (2, 100), (1, 2560), (67, 2048), (9, 2056), (700, 128), (400, 1152), (310, 4096),
          (2, 9728), (305, 9728), (2, 32768), (3, 32776), (2, 40001),
          # an element per load: one and two groups of 8 held, the rest computed again, rows for a second round
          (300, 511), (65, 2561), (9, 4095), (3, 8193), (5, 10239), (5000, 33)]


def rows_of(dt, rows, n, seed=0, spread=12.0):
    g = torch.Generator().manual_seed(seed * 1000003 + rows * 977 + n)
    x = torch.randn(rows, n, generator=g)
    x[:, ::61] *= spread
    return x.to(DT[dt])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows,n", SHAPES)
def test_quantize(rows, n, dt, fp8):
    x = rows_of(dt, rows, n)
    codes, scales = edge_ops.quantize_q8(x.cuda(), fp8=fp8)
    assert codes.shape == x.shape and scales.shape == (rows,)
    y, step = ref.steps(x.double(), fp8)
    ref.check_codes(codes.cpu(), y, fp8)
    assert ((scales.cpu().double() - step).abs() <= 2 * ref.U * step).all()
    assert torch.equal(codes.cpu(), ref.plain_codes(x.float(), fp8))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("weight", [None, 0, 1])
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows,n", SHAPES)
def test_norm(rows, n, dt, weight, add, fp8):
    if add and weight is None and n > 4096:
        pytest.skip("covered by the other forms")
    x = rows_of(dt, rows, n, 1)
    w = None if weight is None else (0.1 * rows_of(dt, 1, n, 2, 1.0)[0].float() + 1 - weight).to(DT[dt])
    wd = None if w is None else w.cuda()
    s = x
    if add:
        r = (4 * rows_of(dt, rows, n, 3).float()).to(DT[dt])
        s = (x.float() + r.float()).to(DT[dt])
        rd = r.cuda()
        codes, scales = edge_ops.add_rmsnorm_q8(x.cuda(), rd, wd, weight_offset=weight or 0, fp8=fp8)
        assert torch.equal(rd.cpu(), s)
    else:
        codes, scales = edge_ops.rmsnorm_q8(x.cuda(), wd, weight_offset=weight or 0, fp8=fp8)
    y, step = ref.steps(ref.norm_products(s, w, weight or 0), fp8)
    ref.check_codes(codes.cpu(), y, fp8)
    want = step * ref.norm_factor(s, 1e-6)
    assert ((scales.cpu().double() - want).abs() <= ref.SCALE_BOUND * want).all()
    p = s.float() if w is None else s.float() * (w.float() + weight)
    assert torch.equal(codes.cpu(), ref.plain_codes(p, fp8))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows,n", SHAPES)
def test_gate(rows, n, dt, act, fp8):
    x = rows_of(dt, rows, 2 * n, 4, 3.0)
    codes, scales = edge_ops.glu_act_q8(x.cuda(), act, fp8=fp8)
    p, v = ref.gate_products(x, act)
    y, step = ref.steps(p, fp8)
    err = ref.gate_error(v)
    # the maximum may be that of any product near it: the largest error among those
    top = torch.where(p.abs() * (1 + 2 * err) >= p.abs().amax(-1, keepdim=True), err, torch.zeros_like(err)).amax(-1)
    ref.check_codes(codes.cpu(), y, fp8, err + 2 * top[:, None])
    assert ((scales.cpu().double() - step).abs() <= (2 * ref.U + 2 * top) * step).all()


CALLS = {
    "quantize": lambda x, **k: edge_ops.quantize_q8(x, **k),
    "norm": lambda x, **k: edge_ops.rmsnorm_q8(x, torch.ones_like(x[0]), **k),
    "add norm": lambda x, **k: edge_ops.add_rmsnorm_q8(x, torch.zeros_like(x), **k),
    "gate": lambda x, **k: edge_ops.glu_act_q8(torch.cat([torch.full_like(x, 100.0), x], -1), **k),
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("n", [64, 2560, 33, 33000])
def test_rows_of_nothing_and_of_extremes(n, call, fp8):
    """Zeros, one value among zeros, the smallest and the largest values."""
    x = torch.zeros(6, n)
    x[1, n // 2] = -3.0
    x[2] = 2.0 ** -140
    x[2, 0] = 2.0 ** -132
    x[3] = 2.0 ** -120
    x[4] = 1e18
    x[5, -1], x[5, 0] = 1e-30, 1.0
    codes, scales = CALLS[call](x.cuda(), fp8=fp8)
    got = ref.values(codes.cpu(), fp8)
    assert not scales.isnan().any() and not got.isnan().any()
    assert (got[0] == 0).all()
    top = ref.TOP[fp8]
    one = torch.zeros(n, dtype=torch.float64)
    one[n // 2] = -top
    assert torch.equal(got[1], one)
    # below the smallest step (2^-126) values keep an absolute precision of half of it; a row there is rounded to
    # a step or two
    assert (got[2].abs() <= 2).all()
    # 2^-120 is below both 127 * 2^-126 and 448 * 2^-126, so it is 64 of the smallest steps; a hundred times that is not
    assert (got[3] == (top if call == "gate" else 64.0)).all()
    assert (got[4] == top).all()
    assert got[5, 0] == top and (got[5, 1:] == 0).all()
    if call == "quantize":
        assert scales[0].item() == 2.0 ** -126 and scales[4].item() == torch.tensor(1e18).div(torch.tensor(top)).item()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("n", [256, 37])
def test_nan_and_infinities_stay_in_their_row(n, call, bad, dt, fp8):
    x = rows_of(dt, 5, n, 5).cuda()
    clean, clean_scales = CALLS[call](x.clone(), fp8=fp8)
    x[2, n // 3] = bad
    codes, scales = CALLS[call](x, fp8=fp8)
    keep = torch.tensor([0, 1, 3, 4])
    assert torch.equal(codes[keep], clean[keep]) and torch.equal(scales[keep], clean_scales[keep])
    if bad != bad or "norm" in call:
        assert scales[2].isnan()
    else:
        assert not scales[2].isfinite()


def test_a_nan_weight_reaches_every_row():
    w = torch.ones(128, device="cuda")
    w[5] = float("nan")
    _, scales = edge_ops.rmsnorm_q8(torch.randn(4, 128, device="cuda"), w)
    assert scales.isnan().all()


@pytest.mark.parametrize("off", [1, 4, 8])
def test_addresses_off_the_vector_and_neighbours_left_alone(off):
    rows, n = 5, 192
    x = rows_of("bf16", rows + 1, n, 6).cuda().flatten()[off:off + rows * n].view(rows, n)
    room = torch.full((rows * n + 64,), 77, dtype=torch.int8, device="cuda")
    marks = torch.full((rows + 2,), 7.0, device="cuda")
    out = room[off:off + rows * n].view(rows, n)
    edge_ops.quantize_q8(x, out=out, scales=marks[1:-1])
    assert torch.equal(out.cpu(), ref.plain_codes(x.float().cpu(), False))
    assert (room[:off] == 77).all() and (room[off + rows * n:] == 77).all()
    assert marks[0] == 7.0 and marks[-1] == 7.0


def test_leading_dimensions_float8_results_and_empty_batches():
    x = torch.randn(2, 3, 64, device="cuda", dtype=torch.float16)
    out = torch.empty(2, 3, 64, device="cuda", dtype=torch.float8_e4m3fn)
    codes, scales = edge_ops.rmsnorm_q8(x, fp8=True, out=out)
    assert codes is out and scales.shape == (2, 3)
    flat, flat_scales = edge_ops.rmsnorm_q8(x.view(6, 64), fp8=True)
    assert torch.equal(flat.view(2, 3, 64), out.view(torch.uint8)) and torch.equal(flat_scales, scales.flatten())
    for call in (edge_ops.quantize_q8, edge_ops.rmsnorm_q8, edge_ops.glu_act_q8):
        codes, scales = call(x[:0])
        assert codes.shape[0] == 0 and scales.shape == (0, 3)
    codes, scales = edge_ops.add_rmsnorm_q8(x[:0], x[:0].clone())
    assert codes.shape == (0, 3, 64)


def test_many_rows_and_a_row_of_the_longest_length():
    x = torch.randn(70000, 64, device="cuda")
    codes, _ = edge_ops.quantize_q8(x)
    assert torch.equal(codes.cpu(), ref.plain_codes(x.cpu(), False))
    x = torch.randn(1, 2 ** 24, device="cuda", dtype=torch.bfloat16)
    codes, scales = edge_ops.rmsnorm_q8(x)
    assert torch.equal(codes.cpu(), ref.plain_codes(x.float().cpu(), False))
    want = ref.steps(x.cpu().double(), False)[1] * ref.norm_factor(x.cpu(), 1e-6)
    assert ((scales.cpu().double() - want).abs() <= ref.SCALE_BOUND * want).all()


def test_rows_past_32_bits():
    """Offsets of the input past 2^32 bytes, of the codes past 2^31."""
    rows, n = 530000, 4096
    x = torch.zeros(rows, n, device="cuda", dtype=torch.bfloat16)
    x[-1] = torch.linspace(-1, 1, n).to(torch.bfloat16)
    codes, scales = edge_ops.quantize_q8(x)
    assert torch.equal(codes[-1:].cpu(), ref.plain_codes(x[-1:].float().cpu(), False))
    assert (codes[:-1] == 0).all()
