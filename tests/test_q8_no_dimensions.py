"""Tensors without dimensions or channels are refused by the 8-bit calls, and say so."""
import pytest
import torch

from memory_bound_decode_qk_gb300 import edge_ops


def calls(device):
    x = torch.tensor(1.0, device=device)
    code, codes = torch.tensor(1, dtype=torch.int8, device=device), torch.zeros(4, 64, dtype=torch.int8, device=device)
    s = torch.zeros(4, device=device)
    return [lambda: edge_ops.quantize_q8(x), lambda: edge_ops.rmsnorm_q8(x), lambda: edge_ops.add_rmsnorm_q8(x, x.clone()),
            lambda: edge_ops.glu_act_q8(x), lambda: edge_ops.matmul_q8(code, codes, s, s),
            lambda: edge_ops.matmul_q8(codes, code, s, s), lambda: edge_ops.matmul_q8(codes, codes[:0], s, s[:0])]


@pytest.mark.parametrize("i", range(7))
def test_on_the_host(i):
    with pytest.raises(ValueError, match="CUDA"):
        calls("cpu")[i]()


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(7))
def test_on_the_device(i):
    with pytest.raises(ValueError, match="at least"):
        calls("cuda")[i]()
