"""The 8-bit product's choice of kernel, tile and cut, as the library's own host code takes it: its objects linked with a
fake runtime (fake_runtime.h) that notes launches instead of making them."""
import collections
import os
import subprocess

from memory_bound_decode_qk_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))

# kernel: few, one (CTA), pair or any; rounds: tiles of the CTA (or cluster) that has most
Cut = collections.namedtuple("Cut", "status kernel tokens split rounds int8")

MAIN = r"""
#include "fake_runtime.h"
#include "../include/edge_ops.h"

// the first parameter of the kernels: what a call multiplies, and the tensor-memory kernel's tiles
struct Args {
    const void *a, *w, *sa, *sw, *bias;
    void* out;
    int tokens, n, k, out_dt;
    int nt, tiles_n, tiles_t, split, pairs, whole;
};
static_assert(sizeof(Args) == 88, "");

int main(int argc, char** argv) {
    fake::no_clusters = argc > 1 && std::strchr(argv[1], 'c');
    fake::no_registers = argc > 1 && std::strchr(argv[1], 'r');
    long t, n, k;
    int int8, dt, off, refuse;
    while (std::scanf("%ld %ld %ld %d %d %d %d", &t, &n, &k, &int8, &dt, &off, &refuse) == 7) {
        // addresses that nothing reads, far from each other
        char* at = (char*)(1ull << 44);
        const long far = 1l << 40;
        fake::launches = 0;
        fake::refuse = refuse;
        const int st = edge_matmul_q8(at, (edge_dtype)dt, at + far + off, at + 2 * far + off, int8 ? EDGE_INT8 : EDGE_FP8_E4M3,
                                      (float*)(at + 3 * far), (float*)(at + 4 * far), nullptr, t, n, k, nullptr);
        if (st != 0 || fake::launches != 1) {
            std::printf("%d none 0 0 0 0\n", st);
            continue;
        }
        const fake::Launch& l = fake::last;
        Args p;
        std::memcpy(&p, l.args, sizeof p);
        const bool tc = l.kernel.find("matmul_tc_kernel") != std::string::npos;
        const bool i8 = l.kernel.find("_kernelILb1E") != std::string::npos;
        if (p.tokens != t || p.n != n || p.k != k || (tc && p.tiles_t != (t + p.nt - 1) / p.nt)) return 3;
        if (tc) {
            const bool pair = l.kernel.find("ELb1EEEv") != std::string::npos;
            const long tiles = (long)p.tiles_n * p.tiles_t, ctas = l.grid / l.cluster;
            std::printf("%d %s %d %d %ld %d\n", st, pair ? "pair" : "one", p.nt, pair ? 1 : (int)l.cluster, (tiles + ctas - 1) / ctas, i8);
        } else {
            const bool any = l.kernel.find("matmul_any_kernel") != std::string::npos;
            std::printf("%d %s %d %u 1 %d\n", st, any ? "any" : "few", any ? 64 : 8, l.cluster, i8);
        }
    }
}
"""


def build(folder):
    """The program, in `folder`; returns its path."""
    obj = os.path.join(_build.LIB_DIR, "obj")
    names = ("edge_ops", "matmul_q8", "matmul_q8_few", "matmul_q8_tc")
    _build.build(force=not all(os.path.exists(os.path.join(obj, n + ".cu.o")) for n in names))
    src, exe = os.path.join(folder, "cuts.cpp"), os.path.join(folder, "cuts")
    with open(src, "w") as f:
        f.write(MAIN)
    cuda = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())), "include")
    r = subprocess.run(["g++", "-std=c++17", "-I", HERE, "-I", cuda, "-iquote", HERE, src,
                        *(os.path.join(obj, n + ".cu.o") for n in names), "-o", exe, "-pthread", "-no-pie",
                        "-Wl,--unresolved-symbols=ignore-all"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


def cuts(exe, calls, broken=""):
    """The Cut of each call (tokens, channels, sum, int8[, output dtype[, bytes off the alignment[, refused launches]]])."""
    lines = "\n".join(" ".join(str(int(x)) for x in (tuple(c) + (2, 0, 0)[len(c) - 4:])) for c in calls)
    r = subprocess.run([exe, broken or "-"], input=lines, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr)
    out = []
    for line in r.stdout.splitlines():
        s, kernel, tokens, split, rounds, int8 = line.split()
        out.append(Cut(int(s), kernel, int(tokens), int(split), int(rounds), bool(int(int8))))
    assert len(out) == len(calls)
    return out
