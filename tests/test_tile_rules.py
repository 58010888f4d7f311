"""Which kernel a grouped or adapter call runs (CPU only): the host's rules,
compiled as they stand, over the sizes that the GPU tests run for each kernel,
and the grids that no launch can have."""
import os
import subprocess

import pytest

import dense_gemm_engineering_run_amd as g
import row_kernel_cases as cases
from dense_gemm_engineering_run_amd import _binding as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include <cstdio>
#include <cstring>
#include "gemm_tiles.hpp"
int main(int argc, char** argv)
{
    if (argc > 1) {
        for (const auto& t : mg::kRaggedTiles) std::printf("grouped %s\n", t.name);
        for (const auto& t : mg::kLoraTiles) std::printf("lora %s\n", t.name);
        return 0;
    }
    char kind[16];
    int f32, vec, bk;
    long long M, N, groups;
    while (std::scanf("%15s %d %d %d %lld %lld %lld", kind, &f32, &vec, &bk, &M, &N, &groups) == 7) {
        if (!std::strcmp(kind, "lora"))
            std::printf("%s\n", mg::tile_of(mg::lora_tile({!!f32, !!vec, !!bk, M, N})).name);
        else
            std::printf("%s\n", mg::tile_of(mg::ragged_tile({!!f32, !std::strcmp(kind, "rows"), !!vec, !!bk, M, N, groups})).name);
    }
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    d = tmp_path_factory.mktemp("rules")
    (d / "rules.cpp").write_text(SOURCE)
    exe = str(d / "rules")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "dense_gemm_engineering_run_amd", "csrc"),
                    str(d / "rules.cpp"), "-o", exe], check=True)

    def ask(lines=None):
        if lines is None:
            return subprocess.run([exe, "names"], check=True, capture_output=True, text=True).stdout.splitlines()
        text = "\n".join(" ".join(str(int(x) if isinstance(x, bool) else x) for x in line) for line in lines)
        return subprocess.run([exe], input=text, check=True, capture_output=True, text=True).stdout.splitlines()

    return ask


def test_the_tests_of_each_kernel_reach_it(rules):
    lines, want, left = [], [], 3
    for f32 in (False, True):
        for pad in (0, 1):
            by_rows, by_k = cases.grouped(f32, pad)
            for name, lens, N, majors in by_rows:
                for major in majors:
                    lines.append(("rows", f32, not pad, major == "k", sum(lens) + left, N, len(lens)))
                    want.append("grouped " + name)
            for name, lens, M, N in by_k:
                for m, n in ((M, N), (N, M)):          # C n-major and m-major
                    lines.append(("k", f32, not pad, 0, m, n, len(lens)))
                    want.append("grouped " + name)
            for name, M, N, majors in cases.lora(f32, pad):
                for major in majors:
                    lines.append(("lora", f32, not pad, major == "k", M, N, 0))
                    want.append("lora " + name)
    got = [("lora " if line[0] == "lora" else "grouped ") + name for line, name in zip(lines, rules(lines))]
    assert got == want, [(x, y, z) for x, y, z in zip(lines, got, want) if y != z]
    assert set(want) == set(rules())


def test_the_tests_of_values_reach_every_kernel(rules):
    seen = set()
    for (f32, pad), sizes in cases.LORA_VALUES.items():
        got = rules([("lora", f32, not pad, 1, M, N, 0) for M, N in sizes])
        assert got == list(sizes.values())
        seen |= set(got)
    # (of 16-bit inputs; 16x32 has B n-major)
    assert seen | {"16x32"} == {name for pad in (0, 1) for name, *_ in cases.lora(False, pad)}


def test_grids_that_no_launch_can_have_are_refused():
    """A launch has less than 2^32 threads along an axis.  (The addresses are
    not looked at: every call here is refused.)"""
    P = 1 << 45
    # 65535 groups of one row, 4096 tiles of 64 columns, 256 threads
    rows = lambda M, N, groups, dtype=0: g.gemm_run_grouped(M, N, 8, "k", "k", "n", dtype, P, 2 * P, 3 * P, 8, 8, N,
                                                            groups, 0, 4 * P)
    for dtype in range(5):
        assert rows(65535, 1 << 18, 65535, dtype) == b.GEMM_ERR_BAD_SHAPE
        assert rows(1 << 22, 1 << 20, 1, dtype) == b.GEMM_ERR_BAD_SHAPE
    by_k = lambda M, N, dtype: g.gemm_run_grouped_k(M, N, 8, "m", "n", "n", dtype, P, 2 * P, 3 * P, M, N, N, 1, 0, 4 * P, 0)
    for dtype in range(5):
        assert by_k(1 << 21, 1 << 21, dtype) == b.GEMM_ERR_BAD_SHAPE
    # 2^28 rows in the first kernel's 16-row tiles of 256 threads
    lora = b.Lora(adapters=1, rank=8, down=4 * P, up=5 * P, ld_down=8, ld_up=8, stride_down=64, stride_up=128, ids=6 * P)
    call = lambda M, dtype, A: g.gemm_run_lora(M, 16, 8, "k", "k", "n", dtype, A, 2 * P, 3 * P, 8, 8, 16, lora, 7 * P, 1 << 50)
    assert call(1 << 28, 0, P) == b.GEMM_ERR_BAD_SHAPE
    assert call(1 << 28, 2, P + 2) == b.GEMM_ERR_BAD_SHAPE          # unaligned
    assert g.gemm_run_lora(1 << 24, 1 << 18, 8, "k", "k", "n", 2, P, 2 * P, 3 * P, 8, 8, 1 << 18, None, 0, 0) == b.GEMM_ERR_BAD_SHAPE
