"""The paged-cache operators with programmatic dependent launch switched off (EDGE_OPS_PDL=0).

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

FILES = ["test_paged_attention.py", "test_rope_axes.py", "test_pages.py", "test_paged_serving.py"]
SELECT = " or ".join([
    "test_decode and (8-2-128 or 16-2-256)",
    "test_chunks and 13 and 8-2-128",
    "test_page_sizes and bf16",
    "test_wide_chunks_cross_and_bad_pages",
    "test_wide_chunk_on_another_stream_and_in_a_graph",
    "test_long_sequences_split_over_the_gpu",
    "test_prologue and (text256 or many_d128)",
    "test_qkv_write and (d128 or generic)",
    "test_random_histories",
    "test_on_another_stream_and_in_a_graph",
    "test_prompts_forks_steps_and_compaction",
])


def test_paged_cases_with_dependent_launch_off():
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
