"""The 8-bit matrix product: int8 bit for bit against exact sums, E4M3 against 64 bits within the derived bound."""
import os
import subprocess
import sys

import pytest
import torch

import q8_ref as ref
from memory_bound_decode_qk_gb300 import edge_ops

pytestmark = pytest.mark.gpu

# tokens, channels, summed length: single values, lengths that suit no vector, every limit between the paths and
# the sizes around a tile, sums longer than 1024 terms (int8 accumulators are emptied there) and ragged ends
SHAPES = [(1, 1, 1), (3, 5, 7), (2, 33, 20), (65, 70, 33), (130, 129, 100), (17, 300, 1028),
          (1, 16, 16), (1, 2560, 2560), (2, 4100, 1040), (4, 512, 9728), (7, 1000, 48), (8, 128, 128),
          (9, 640, 2048), (16, 272, 4096), (17, 128, 1024), (33, 2560, 9728), (64, 1152, 1040), (65, 384, 144),
          (100, 257, 2064), (128, 130, 1024), (129, 512, 1200), (200, 6144, 2560), (256, 128, 4112), (257, 640, 512),
          (1000, 1024, 1040), (1201, 5120, 2048), (300, 131, 16), (2048, 2304, 1536),
          # the cuts of the tensor-memory kernel: 16, 32 and 64 tokens by one CTA, unsplit and over clusters of 2 to
          # 8, and pairs with 32 to 256 tokens in steps of 32
          (1243, 131, 144), (546, 5450, 32), (17, 3661, 3872), (9, 64, 1488), (9, 69, 1968), (9, 64, 2592),
          (9, 74, 2960), (9, 66, 3856), (9, 68, 4000), (609, 138, 3824), (246, 131, 4672), (862, 132, 4752),
          (1248, 135, 2992), (834, 132, 2592), (65, 3853, 4736), (1230, 136, 3968), (1242, 391, 1568), (1409, 5014, 32),
          (588, 2592, 528), (985, 5335, 144), (500, 4957, 672), (582, 5635, 544), (677, 5029, 928), (1424, 5915, 32),
          (521, 4906, 272), (197, 4923, 32), (296, 4891, 32), (392, 4872, 32), (418, 5545, 32), (587, 4907, 32),
          (676, 4871, 32), (975, 133, 2480), (429, 132, 1936), (679, 69, 3472), (319, 136, 3520), (514, 65, 2480),
          (1000, 141, 3376),
          # rows that do not start on 16 bytes: whole, and cut over clusters of 2 to 8
          (1, 2560, 9725), (2, 70, 321), (9, 201, 9727), (20, 130, 579), (64, 2560, 4862), (65, 1200, 2049), (90, 333, 1023),
          (130, 640, 1544), (300, 700, 4097), (512, 2570, 1031), (1201, 130, 2044), (700, 1500, 515)]


def operands(t, n, k, fp8, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + t * 31 + n * 17 + k)

    def codes(rows):
        if fp8:
            x = torch.randn(rows, k, generator=g, device="cuda") * 40
            return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return torch.randint(-128, 128, (rows, k), generator=g, device="cuda", dtype=torch.int8)

    return (codes(t), codes(n), torch.rand(t, generator=g, device="cuda") * 1e-3 + 1e-5,
            torch.rand(n, generator=g, device="cuda") * 1e-3 + 1e-5, torch.randn(n, generator=g, device="cuda"))


def check(out, a, w, sa, sw, bias, dtype, fp8):
    sums, mags = ref.product_sums(a, w, fp8)
    if not fp8:
        want = ref.product_exact(sums, sa, sw, bias, dtype)
        assert torch.equal(out, want), ((out != want).sum().item(), (out.double() - want.double()).abs().max().item())
        return
    want = sums * sa.double()[:, None] * sw.double()
    if bias is not None:
        want = want + bias.double()
    far = (out.double() - want).abs() - ref.product_bound(mags, a.shape[1], sa, sw, bias, want, dtype)
    assert (far <= 0).all(), (far.max().item(), (far > 0).sum().item())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("t,n,k", SHAPES)
def test_sizes(t, n, k, fp8):
    a, w, sa, sw, bias = operands(t, n, k, fp8)
    for dtype, b in ((torch.bfloat16, None), (torch.float32, bias), (torch.float16, bias.half())):
        out = edge_ops.matmul_q8(a, w, sa, sw, bias=b, dtype=dtype)
        assert out.dtype is dtype and out.shape == (t, n)
        check(out, a, w, sa, sw, b, dtype, fp8)


@pytest.mark.parametrize("t,n,k", [(1, 48, 131056), (3, 130, 131071), (70, 130, 131056), (300, 40, 131056),
                                   (1300, 2560, 131056)])
@pytest.mark.parametrize("value", [(-128, -128), (-128, 127), (127, 127)])
def test_the_largest_int8_sums(t, n, k, value):
    a = torch.full((t, k), value[0], dtype=torch.int8, device="cuda")
    w = torch.full((n, k), value[1], dtype=torch.int8, device="cuda")
    # channel j drops its last j terms, so that sums differ in their low bits
    for j in range(7):
        w[j::7, k - j:] = 0
    one_t, one_n = torch.ones(t, device="cuda"), torch.ones(n, device="cuda")
    out = edge_ops.matmul_q8(a, w, one_t, one_n, dtype=torch.float32)
    terms = torch.tensor([k - j % 7 for j in range(n)], dtype=torch.float64)
    want = (terms * value[0] * value[1]).float().cuda().expand(t, n)
    assert torch.equal(out, want)


@pytest.mark.parametrize("t,n", [(1, 200), (5, 200), (40, 200), (90, 200), (300, 200), (677, 5029)])
def test_e4m3_extremes_and_nan(t, n):
    k = 512
    a, w, sa, sw, _ = operands(t, n, k, True, 3)
    a[:, ::2] = 0x7E   # 448
    w[:, ::2] = 0xFE   # -448
    a[0, 1::2] = 0x01  # the smallest subnormal
    out = edge_ops.matmul_q8(a, w, sa, sw, dtype=torch.float32)
    check(out, a, w, sa, sw, None, torch.float32, True)
    w[7, 3] = 0x7F     # NaN
    a[-1, 5] = 0xFF
    got = edge_ops.matmul_q8(a, w, sa, sw, dtype=torch.float32)
    nan = torch.zeros(t, n, dtype=torch.bool, device="cuda")
    nan[:, 7] = True
    nan[-1] = True
    assert torch.equal(got.isnan(), nan) and torch.equal(got[~nan], out[~nan])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("t,n", [(1, 70), (3, 70), (30, 70), (150, 70), (677, 5029)])
def test_scales_of_nothing_infinities_and_nan(t, n, fp8):
    a, w, sa, sw, _ = operands(t, n, 64, fp8, 4)
    sums, _ = ref.product_sums(a, w, fp8)
    sa[0], sw[1], sw[2] = 0.0, float("inf"), float("nan")
    out = edge_ops.matmul_q8(a, w, sa, sw, dtype=torch.float32)
    want = ref.product_exact(sums, sa, sw, None, torch.float32)
    assert torch.equal(out.isnan(), want.isnan())
    assert torch.equal(out.isinf(), want.isinf())
    if not fp8:
        assert torch.equal(out.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("t,n", [(1, 136), (6, 136), (40, 136), (300, 136), (677, 5030), (677, 5032)])
@pytest.mark.parametrize("off", [1, 2, 4, 16])
def test_addresses_and_neighbours(t, n, off, fp8):
    """Operands that start off the vector; values behind and before the output stay as they were."""
    k = 176
    a, w, sa, sw, _ = operands(t, n, k, fp8, 5)
    at = torch.zeros(t * k + 32, dtype=a.dtype, device="cuda")[off:off + t * k].view(t, k).copy_(a)
    wt = torch.zeros(n * k + 32, dtype=a.dtype, device="cuda")[off:off + n * k].view(n, k).copy_(w)
    room = torch.full((t * n + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
    out = room[off:off + t * n].view(t, n)
    edge_ops.matmul_q8(at, wt, sa, sw, out=out)
    check(out, a, w, sa, sw, None, torch.bfloat16, fp8)
    assert (room[:off] == 5.0).all() and (room[off + t * n:] == 5.0).all()


@pytest.mark.parametrize("t,n,k", [(1, 70, 131071), (5, 90, 300), (40, 130, 1031), (100, 70, 37), (64, 128, 2560), (3, 2, 1)])
@pytest.mark.parametrize("off", [0, 1, 7, 15])
def test_rows_that_start_anywhere_read_nothing_else(t, n, k, off):
    """NaN around the operands, and in the rows next to each other, stays out of the sums."""
    a, w, sa, sw, _ = operands(t, n, k, True, 10)
    around = torch.full((max(t, n) * k + 64,), 0x7F, dtype=torch.uint8, device="cuda")
    at, wt = around.clone()[off:off + t * k].view(t, k), around[off:off + n * k].view(n, k)
    at.copy_(a)
    wt.copy_(w)
    out = edge_ops.matmul_q8(at, wt, sa, sw, dtype=torch.float32)
    check(out, a, w, sa, sw, None, torch.float32, True)
    wt[1::2] = 0x7F
    got = edge_ops.matmul_q8(at, wt, sa, sw, dtype=torch.float32)
    assert got[:, 1::2].isnan().all() and torch.equal(got[:, ::2], out[:, ::2])
    wt.copy_(w)
    at[1::2] = 0xFF
    got = edge_ops.matmul_q8(at, wt, sa, sw, dtype=torch.float32)
    assert got[1::2].isnan().all() and torch.equal(got[::2], out[::2])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("t,n,k", [(3, 2560, 2047), (70, 640, 4098), (1, 2560, 9728), (12, 640, 4096), (48, 512, 9728), (128, 256, 9728),
                                   (700, 1024, 2048)])
def test_runs_streams_and_graphs_give_the_same_bits(t, n, k, fp8):
    a, w, sa, sw, _ = operands(t, n, k, fp8, 6)
    first = edge_ops.matmul_q8(a, w, sa, sw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(first) for _ in range(3)]
    edge_ops.matmul_q8(a, w, sa, sw, out=outs[0], stream=side)
    edge_ops.matmul_q8(a, w, sa, sw, out=outs[1])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        edge_ops.matmul_q8(a, w, sa, sw, out=outs[2])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out, first)
    b = operands(t, n, k, fp8, 7)[0]
    a.copy_(b)  # the graph reads its operands when it runs
    graph.replay()
    assert torch.equal(outs[2], edge_ops.matmul_q8(b, w, sa, sw))


@pytest.mark.parametrize("fp8", [False, True])
def test_two_streams_at_once(fp8):
    """Calls that share the GPU: pairs of CTAs, clusters and streams of weights beside each other."""
    calls = [operands(t, n, k, fp8, 20) for t, n, k in ((700, 2560, 2048), (48, 512, 9728), (4, 2560, 2560), (200, 6144, 1024))]
    want = [edge_ops.matmul_q8(*c[:4]) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for _ in range(20):
        for i, (c, s) in enumerate(zip(calls, streams)):
            got[i].append(edge_ops.matmul_q8(*c[:4], stream=s))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)


def test_first_calls_of_a_process_in_a_graph():
    """What a call asks of the runtime once (shared memory, resident clusters) can be asked during a capture."""
    code = """
import sys
sys.path[:0] = [{root!r}, {here!r}]
import torch, test_q8_matmul as m
from memory_bound_decode_qk_gb300 import edge_ops
sets = [m.operands(t, n, k, q, 21) for t, n, k in ((4, 640, 512), (48, 512, 9728), (700, 2560, 2048), (5, 90, 2047)) for q in (True, False)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    outs = [edge_ops.matmul_q8(*s[:4]) for s in sets]
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(o, edge_ops.matmul_q8(*s[:4])) for o, s in zip(outs, sets))
print("same")
"""
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", code.format(root=os.path.dirname(here), here=here)], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


def test_leading_dimensions_and_empty_batches():
    a, w, sa, sw, _ = operands(6, 40, 64, False, 8)
    out = edge_ops.matmul_q8(a.view(2, 3, 64), w, sa.view(2, 3), sw, dtype=torch.float32)
    assert torch.equal(out.view(6, 40), edge_ops.matmul_q8(a, w, sa, sw, dtype=torch.float32))
    assert edge_ops.matmul_q8(a[:0], w, sa[:0], sw).shape == (0, 40)
    f8 = a.view(torch.float8_e4m3fn)
    assert torch.equal(edge_ops.matmul_q8(f8, w.view(torch.uint8), sa, sw).view(torch.int16),
                       edge_ops.matmul_q8(a.view(torch.uint8), w.view(torch.uint8), sa, sw).view(torch.int16))


@pytest.mark.parametrize("fp8", [False, True])
def test_outputs_past_32_bits(fp8):
    """The last row of an output of more than 2^32 bytes."""
    t, n, k = 140000, 16000, 32
    a, w, sa, sw, _ = operands(t, n, k, fp8, 9)
    out = edge_ops.matmul_q8(a, w, sa, sw)
    rows = torch.tensor([0, 65535, 134217, t - 1], device="cuda")
    check(out[rows], a[rows], w, sa[rows], sw, None, torch.bfloat16, fp8)
