"""Waits of the tcgen05 kernels that run out: a kernel of its own waits, with a limit of 20 ms, for barriers that nothing
arrives on, and every flag that must be set is."""
import ctypes
import os
import subprocess

import pytest
import torch

from memory_bound_decode_qk_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))
LIMIT = 20_000_000  # ns


@pytest.fixture(scope="module")
def waits(tmp_path_factory):
    path = str(tmp_path_factory.mktemp("waits") / "waits.so")
    r = subprocess.run([_build.nvcc()] + _build.NVCC_FLAGS + ["-I", _build.CSRC, "-shared", "-o", path,
                                                              os.path.join(HERE, "wait_limits.cu")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(path)
    lib.pair.argtypes = [ctypes.c_int, ctypes.c_uint64, ctypes.c_void_p]
    lib.one.argtypes = [ctypes.c_uint64, ctypes.c_void_p]
    return lib


def test_the_waits_compile(waits):
    assert waits.pair and waits.one


@pytest.mark.gpu
@pytest.mark.parametrize("who", [0, 1])
def test_a_wait_of_either_cta_fails_the_pair(waits, who):
    out = torch.full((64,), 7, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert waits.pair(who, LIMIT, out.data_ptr()) == 0
    assert (out == 1).all(), out.tolist()


@pytest.mark.gpu
def test_a_wait_that_ends_fails_nobody(waits):
    out = torch.full((64,), 7, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert waits.pair(2, LIMIT, out.data_ptr()) == 0
    assert (out == 0).all(), out.tolist()


@pytest.mark.gpu
def test_later_waits_of_a_failed_cta_end_at_once(waits):
    out = torch.full((64,), 7, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert waits.one(LIMIT, out.data_ptr()) == 0
    assert (out[:32] == 1).all() and (out[32:] < 1000).all(), out.tolist()
