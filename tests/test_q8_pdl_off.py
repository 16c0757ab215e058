"""The 8-bit linear operators with programmatic dependent launch switched off (EDGE_OPS_PDL=0).

The library reads the variable once per process, so a child pytest runs a cross-section of the cases with it set: every
kernel family, launched without the programmatic-serialization attribute.
"""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))

FILES = ["test_q8_rows.py", "test_q8_matmul.py", "test_q8_layer.py"]
SELECT = " or ".join([
    "test_quantize and (67-2048 or 2-40001)",
    "test_norm and 310-4096 and bf16",
    "test_gate and 305-9728",
    "test_sizes and (3-5-7 or 1-2560-2560 or 16-272-4096 or 1201-5120-2048 or 9-66-3856 or 521-4906-272)",
    "test_runs_streams_and_graphs_give_the_same_bits",
    "test_step_in_a_graph_and_on_another_stream",
])


def test_q8_cases_with_dependent_launch_off():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    env = dict(os.environ, EDGE_OPS_PDL="0")
    env.pop("EDGE_OPS_REPORT_STATS", None)
    r = subprocess.run([sys.executable, "-m", "pytest", *[os.path.join(HERE, f) for f in FILES], "-q", "-x", "-p",
                        "no:cacheprovider", "-m", "gpu", "-k", SELECT],
                       env=env, capture_output=True, text=True, timeout=1200)
    tail = r.stdout[-3000:] + r.stderr[-2000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and " deselected" in r.stdout, tail
