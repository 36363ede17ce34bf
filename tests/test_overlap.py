"""The check that two buffers of a call share no memory, against every pair of bytes."""
import os
import subprocess

from mixture_experts_layer_22_b200 import build as mbuild

MAIN = r"""
#include "overlap.cuh"
#include <cstdio>
#include <random>
using namespace moe;
int main()
{
    std::mt19937 r(1);
    auto u = [&](int a, int b) { return a + static_cast<int>(r() % (b - a + 1)); };
    long wrong = 0, yes = 0, tries = 400000;
    for (long t = 0; t < tries; ++t) {
        // steps alike two times in three, empty buffers, pieces side by side
        const int sa = u(1, 30), sb = u(0, 2) ? sa : u(1, 30), la = u(1, sa), lb = u(1, sb), na = u(0, 6), nb = u(0, 6);
        const int pa = u(1, 200), pb = u(1, 200);
        const Extent a(reinterpret_cast<void *>(static_cast<uintptr_t>(pa)), la, sa, na);
        const Extent b(reinterpret_cast<void *>(static_cast<uintptr_t>(pb)), lb, sb, nb);
        bool want = false;
        for (int i = 0; i < na; ++i)
            for (int j = 0; j < nb; ++j) want |= pa + i * sa < pb + j * sb + lb && pb + j * sb < pa + i * sa + la;
        yes += want;
        wrong += want != overlap(a, b);
        wrong += want != overlap(b, a);
    }
    wrong += overlap(Extent(nullptr, 100), Extent(reinterpret_cast<void *>(50), 4));
    std::printf("%ld %ld\n", wrong, yes);
}
"""


def test_overlap_against_every_pair_of_pieces(tmp_path):
    src, exe = tmp_path / "main.cc", tmp_path / "main"
    src.write_text(MAIN)
    subprocess.run(["g++", "-O2", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", mbuild.CSRC, str(src), "-o", str(exe)],
                   check=True, env={**os.environ, "LC_ALL": "C"})
    wrong, yes = map(int, subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split())
    assert wrong == 0 and 50000 < yes < 350000
