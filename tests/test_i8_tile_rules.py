"""Which kernel an 8-bit product runs (CPU only): the host's rules, compiled as
they stand, over the sizes that the GPU tests run for each kernel."""
import os
import subprocess

import pytest

import i8_kernel_cases as cases

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include <cstdio>
#include <cstring>
#include "gemm_i8_tiles.hpp"
int main(int argc, char**)
{
    if (argc > 1) {
        for (const auto& t : mg::kI8Tiles) std::printf("i8 %s\n", t.name);
        for (const auto& t : mg::kGradTiles) std::printf("grad %s\n", t.name);
        return 0;
    }
    char kind[16];
    int vec, wide, split;
    long long M, N, K;
    while (std::scanf("%15s %d %d %d %lld %lld %lld", kind, &vec, &wide, &split, &M, &N, &K) == 7) {
        const mg::I8Shape s = {!!vec, M, N, K};
        const mg::GradShape g = {!!vec, !!wide, !!split, M, N, K};
        if (!std::strcmp(kind, "edges")) {
            const mg::I8Edges e = mg::i8_edges(s);
            std::printf("%d %d\n", (int)e.rows, (int)e.cols);
            continue;
        }
        const mg::Tile& t = std::strcmp(kind, "i8") ? mg::kGradTiles[(int)mg::grad_tile(g)] : mg::kI8Tiles[(int)mg::i8_tile(s)];
        std::printf("%s\n", t.name);
    }
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    d = tmp_path_factory.mktemp("rules8")
    (d / "rules.cpp").write_text(SOURCE)
    exe = str(d / "rules")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "dense_gemm_engineering_run_amd", "csrc"),
                    str(d / "rules.cpp"), "-o", exe], check=True)

    def run(lines=None):
        if lines is None:
            return subprocess.run([exe, "names"], check=True, capture_output=True, text=True).stdout.splitlines()
        text = "\n".join(" ".join(str(int(x) if isinstance(x, bool) else x) for x in line) for line in lines)
        return subprocess.run([exe], input=text, check=True, capture_output=True, text=True).stdout.splitlines()

    return run


def test_the_tests_of_each_kernel_reach_it(ask):
    lines, want, reached = [], [], set()
    for aligned, table in ((True, cases.PRODUCTS), (False, cases.PRODUCTS_UNALIGNED)):
        for name, M, N in table:
            lines.append(("i8", aligned, False, False, M, N, 64))
            want.append(name)
            reached.add("i8 " + name)
    for wide, split_a in ((False, False), (True, False), (True, True)):
        for aligned in (True, False):
            for name, M, N in cases.gradients(wide, split_a, aligned):
                lines.append(("grad", aligned, wide, split_a, M, N, 64))
                want.append(name)
                reached.add("grad " + name)
    assert ask(lines) == want
    assert reached == set(ask())          # and no kernel is left out


def test_no_size_runs_out_of_rules(ask):
    sizes = [1, 15, 16, 33, 64, 100, 257, 1000, 4096, 30000, 1 << 20]
    lines = [(kind, vec, wide, split, M, N, 64) for kind in ("i8", "grad") for vec in (False, True)
             for wide, split in ((False, False), (True, False), (True, True)) for M in sizes for N in sizes]
    known = {n.split(" ", 1)[1] for n in ask()}
    assert set(ask(lines)) <= known


def test_the_tests_of_thin_edges_have_them(ask):
    got = ask([("edges", aligned, False, False, M, N, K) for aligned, M, N, K, _, _ in cases.EDGES])
    assert got == [f"{rows} {cols}" for _, _, _, _, rows, cols in cases.EDGES]


def test_edges_are_never_the_whole(ask):
    sizes = [1, 16, 100, 128, 129, 144, 257, 1000, 4097, 30000]
    lines = [("edges", vec, False, False, M, N, K) for vec in (False, True) for M in sizes for N in sizes for K in (0, 1, 4096, 131071)]
    for (_, _, _, _, M, N, _), line in zip(lines, ask(lines)):
        rows, cols = map(int, line.split())
        assert 0 <= rows <= 16 and 0 <= cols <= 16 and rows < M and cols < N
