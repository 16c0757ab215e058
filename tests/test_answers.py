"""What the library keeps of the runtime's answers: the host code with a runtime whose questions fail at first, on the
CPU."""
import os
import subprocess

import pytest

from memory_bound_decode_qk_gb300 import _build

KEPT = r"""
#include <cstdio>
#include "answers.h"

int asked = 0;
int main() {
    static edge::Answers<3> answers;
    int a, b;
    auto says = [](int v) { return [v] { ++asked; return v; }; };
    // a question that fails is asked again, and its answer kept once there is one
    bool ok = answers.get(&a, 2, 0, says(-1)) == -1 && answers.get(&a, 2, 0, says(-1)) == -1 && asked == 2;
    ok = ok && answers.get(&a, 2, 0, says(76)) == 76 && answers.get(&a, 2, 0, says(5)) == 76 && asked == 3;
    // none at all is an answer; kernel, size and device are told apart
    ok = ok && answers.get(&a, 8, 0, says(0)) == 0 && answers.get(&a, 8, 0, says(5)) == 0 && asked == 4;
    ok = ok && answers.get(&a, 2, 1, says(70)) == 70 && answers.get(&a, 2, 0, says(5)) == 76 && asked == 5;
    // a full table asks every time
    ok = ok && answers.get(&b, 2, 0, says(9)) == 9 && answers.get(&b, 2, 0, says(8)) == 8 && asked == 7;
    std::puts(ok ? "right" : "wrong");
    return !ok;
}
"""

# the runtime calls that edge_ops.cu makes here, in place of the runtime's
FAKES = r"""
#include <cstdio>
#include "launch.h"

int device = 0, asked = 0;
bool broken = true;
extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t*) {
    ++asked;
    *n = 76;
    return broken ? cudaErrorUnknown : cudaSuccess;
}
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* f, const void*) {
    ++asked;
    f->numRegs = 80;
    return broken ? cudaErrorUnknown : cudaSuccess;
}
}
"""
CLUSTERS = FAKES + r"""
int main() {
    cudaLaunchConfig_t cfg = {};
    auto clusters = [&] { return edge::resident_clusters(&device, cfg, 2); };
    bool ok = clusters() == 0 && clusters() == 0 && asked == 2;  // (both fail)
    broken = false;
    ok = ok && clusters() == 76 && clusters() == 76 && asked == 3;
    device = 1;
    ok = ok && clusters() == 76 && asked == 4;
    std::puts(ok ? "right" : "wrong");
    return !ok;
}
"""
REGISTERS = FAKES + r"""
int main() {
    int n = 0;
    auto fails = [&] { return edge::kernel_registers(&device, &n) == cudaErrorUnknown; };
    auto says = [&] { n = 0; return edge::kernel_registers(&device, &n) == cudaSuccess && n == 80; };
    bool ok = fails() && fails() && asked == 2;
    broken = false;
    ok = ok && says() && says() && asked == 3;
    device = 1;  // devices are told apart
    ok = ok && says() && asked == 4;
    std::puts(ok ? "right" : "wrong");
    return !ok;
}
"""


def run(tmp_path, source, *objects):
    src, exe = tmp_path / "main.cpp", tmp_path / "main"
    src.write_text(source)
    cuda = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())), "include")
    cmd = ["g++", "-std=c++17", "-I", _build.CSRC, "-I", cuda, "-x", "c++", str(src), *objects, "-o", str(exe), "-pthread",
           "-Wl,--unresolved-symbols=ignore-all"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "right\n", r.stdout + r.stderr


def test_the_table(tmp_path):
    run(tmp_path, KEPT)


@pytest.mark.parametrize("source", [CLUSTERS, REGISTERS], ids=["clusters", "registers"])
def test_failed_questions_are_asked_again(tmp_path, source):
    run(tmp_path, source, os.path.join(_build.CSRC, "edge_ops.cu"))
