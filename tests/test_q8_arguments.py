"""Calls of the 8-bit linear operators that are refused: by the C ABI (no GPU: nothing is launched) and by the
binding."""
import pytest
import torch

from memory_bound_decode_qk_gb300 import _build, edge_ops

OK, NULL, DTYPE, SHAPE, ALIGN, ALIAS, UNSUP, CUDA, VALUE = range(9)
F32, F16, BF16, FP8, INT8 = range(5)
X, R, W, O, S, B = 0x10000000, 0x20000000, 0x30000000, 0x40000000, 0x50000000, 0x60000000


@pytest.fixture(scope="module")
def L():
    _build.build()
    return edge_ops.lib()


def rms(L, out=O, q=INT8, s=S, x=X, w=W, dt=BF16, rows=4, n=64, eps=1e-6, off=0):
    return L.edge_rmsnorm_q8(out, q, s, x, w, dt, rows, n, eps, off, None)


def add(L, out=O, q=INT8, s=S, x=X, r=R, w=W, dt=BF16, rows=4, n=64, eps=1e-6, off=0):
    return L.edge_add_rmsnorm_q8(out, q, s, x, r, w, dt, rows, n, eps, off, None)


def glu(L, out=O, q=INT8, s=S, x=X, dt=BF16, rows=4, n=64, act=0):
    return L.edge_glu_act_q8(out, q, s, x, dt, rows, n, act, None)


def quant(L, out=O, q=INT8, s=S, x=X, dt=BF16, rows=4, n=64):
    return L.edge_quantize_q8(out, q, s, x, dt, rows, n, None)


def mm(L, out=O, dt=BF16, a=X, w=W, q=INT8, sa=S, sw=R, bias=B, t=4, n=64, k=128):
    return L.edge_matmul_q8(out, dt, a, w, q, sa, sw, bias, t, n, k, None)


def test_empty_calls_launch_nothing(L):
    assert rms(L, rows=0) == OK and add(L, rows=0) == OK and glu(L, rows=0) == OK
    assert quant(L, rows=0) == OK and mm(L, t=0) == OK
    assert L.edge_last_cuda_error() == 0


@pytest.mark.parametrize("call", [rms, add, glu, quant])
def test_row_calls_refuse(L, call):
    assert call(L, out=None) == NULL and call(L, s=None) == NULL and call(L, x=None) == NULL
    assert call(L, q=BF16) == DTYPE and call(L, q=7) == DTYPE and call(L, dt=INT8) == DTYPE
    assert call(L, dt=FP8) == DTYPE
    assert call(L, rows=-1) == SHAPE and call(L, n=0) == SHAPE and call(L, rows=2 ** 62, n=2 ** 10) == SHAPE
    assert call(L, n=2 ** 24 + 1, rows=1) == UNSUP
    assert call(L, x=X + 1) == ALIGN and call(L, s=S + 2) == ALIGN
    assert call(L, out=X + 64) == ALIAS and call(L, out=X) == ALIAS and call(L, s=X + 4) == ALIAS
    assert call(L, s=O + 16) == ALIAS


def test_norms_and_gate_refuse(L):
    for call in (rms, add):
        assert call(L, eps=-1.0) == VALUE and call(L, eps=float("nan")) == VALUE and call(L, off=2) == VALUE
        assert call(L, w=W + 1) == ALIGN
        assert call(L, out=W - 4) == ALIAS and call(L, s=W + 120) == ALIAS
    assert add(L, r=None) == NULL and add(L, r=X) == ALIAS and add(L, r=W - 8) == ALIAS
    assert add(L, out=R + 10) == ALIAS and add(L, s=R) == ALIAS and add(L, r=R + 1) == ALIGN
    assert glu(L, act=2) == VALUE and glu(L, act=-1) == VALUE


def test_matmul_refuses(L):
    for name in ("out", "a", "w", "sa", "sw"):
        assert mm(L, **{name: None}) == NULL
    assert mm(L, dt=FP8) == DTYPE and mm(L, dt=INT8) == DTYPE and mm(L, q=BF16) == DTYPE and mm(L, q=9) == DTYPE
    assert mm(L, t=-1) == SHAPE and mm(L, n=0) == SHAPE and mm(L, k=0) == SHAPE
    assert mm(L, k=131072) == UNSUP and mm(L, t=2 ** 24 + 1) == UNSUP and mm(L, n=2 ** 24 + 1) == UNSUP
    assert mm(L, out=O + 1) == ALIGN and mm(L, bias=B + 1) == ALIGN and mm(L, sa=S + 1) == ALIGN
    assert mm(L, sw=R + 2) == ALIGN and mm(L, dt=F32, out=O + 2) == ALIGN
    assert mm(L, out=X) == ALIAS and mm(L, out=W + 128 * 64 - 2) == ALIAS and mm(L, out=S + 8) == ALIAS
    assert mm(L, out=R) == ALIAS and mm(L, out=B + 2) == ALIAS


def test_other_calls_do_not_take_int8(L):
    assert L.edge_rmsnorm(O, INT8, X, W, BF16, 4, 64, 1e-6, 0, 1.0, None) == DTYPE
    assert L.edge_quantize_fp8(O, X, INT8, 16, 1.0, None) == DTYPE


def test_host_tensors_are_refused():
    x = torch.zeros(4, 64)
    codes, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    for call in (lambda: edge_ops.quantize_q8(x), lambda: edge_ops.rmsnorm_q8(x), lambda: edge_ops.glu_act_q8(x),
                 lambda: edge_ops.add_rmsnorm_q8(x, x), lambda: edge_ops.matmul_q8(codes, codes, s, s)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.gpu
def test_binding_refuses():
    dev = dict(device="cuda")
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16, **dev), torch.zeros(64, dtype=torch.bfloat16, **dev)
    i8, u8 = torch.zeros(4, 64, dtype=torch.int8, **dev), torch.zeros(4, 64, dtype=torch.uint8, **dev)
    s = torch.zeros(4, **dev)
    other = torch.cuda.Stream()
    for call, error in [
            (lambda: edge_ops.quantize_q8(x.t()), ValueError),
            (lambda: edge_ops.quantize_q8(x, out=u8), TypeError),
            (lambda: edge_ops.quantize_q8(x, fp8=True, out=i8), TypeError),
            (lambda: edge_ops.quantize_q8(x, out=i8[:2]), ValueError),
            (lambda: edge_ops.quantize_q8(x, scales=s[:3]), ValueError),
            (lambda: edge_ops.quantize_q8(x, scales=s.double()), TypeError),
            (lambda: edge_ops.quantize_q8(x[:, :0]), ValueError),
            (lambda: edge_ops.quantize_q8(x.double()), TypeError),
            (lambda: edge_ops.quantize_q8(i8), TypeError),
            (lambda: edge_ops.rmsnorm_q8(x, w[:32]), ValueError),
            (lambda: edge_ops.rmsnorm_q8(x, w.float()), TypeError),
            (lambda: edge_ops.rmsnorm_q8(x, w.cpu()), ValueError),
            (lambda: edge_ops.add_rmsnorm_q8(x, x[:2]), ValueError),
            (lambda: edge_ops.add_rmsnorm_q8(x, x.float()), TypeError),
            (lambda: edge_ops.add_rmsnorm_q8(x, x), edge_ops.EdgeError),
            (lambda: edge_ops.glu_act_q8(x[:, :63].contiguous()), ValueError),
            (lambda: edge_ops.glu_act_q8(x, "relu"), KeyError),
            (lambda: edge_ops.matmul_q8(x, i8, s, s), TypeError),
            (lambda: edge_ops.matmul_q8(i8, u8, s, s), TypeError),
            (lambda: edge_ops.matmul_q8(i8, i8[:, :32].contiguous(), s, s), ValueError),
            (lambda: edge_ops.matmul_q8(i8, i8.cpu(), s, s), ValueError),
            (lambda: edge_ops.matmul_q8(i8, i8, s[:3], s), ValueError),
            (lambda: edge_ops.matmul_q8(i8, i8, s, s.double()), TypeError),
            (lambda: edge_ops.matmul_q8(i8, i8, s, s, bias=s), TypeError),
            (lambda: edge_ops.matmul_q8(i8, i8, s, s, dtype=torch.float64), TypeError),
            (lambda: edge_ops.matmul_q8(i8, i8, s, s, out=x), ValueError),
            (lambda: edge_ops.matmul_q8(i8.t(), i8, s, s), ValueError),
            (lambda: edge_ops.matmul_q8(i8, i8[0], s, s), ValueError)]:
        with pytest.raises(error):
            call()

    class Elsewhere:
        cuda_stream = 0
        device = torch.device("cuda", 63)

    for call in (lambda: edge_ops.quantize_q8(x, stream=Elsewhere()), lambda: edge_ops.rmsnorm_q8(x, stream=Elsewhere()),
                 lambda: edge_ops.add_rmsnorm_q8(x, x.clone(), stream=Elsewhere()),
                 lambda: edge_ops.glu_act_q8(x, stream=Elsewhere()),
                 lambda: edge_ops.matmul_q8(i8, i8, s, s, stream=Elsewhere())):
        with pytest.raises(ValueError, match="cuda:63"):
            call()
    codes, _ = edge_ops.quantize_q8(x, stream=other)
    other.synchronize()
    assert (codes == 0).all()
