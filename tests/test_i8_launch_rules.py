"""What the 8-bit calls launch (CPU only): the host's rules, compiled as they
stand."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include <cstdio>
#include <cstring>
#include "gemm_i8_tiles.hpp"
int grad()
{
    int vec, wide, split, kmajor;
    long long M, N, K;
    while (std::scanf("%d %d %d %d %lld %lld %lld", &vec, &wide, &split, &kmajor, &M, &N, &K) == 7) {
        const mg::GradTile t = mg::grad_tile({!!vec, !!wide, !!split, M, N, K, !!kmajor});
        std::printf("%s%s\n", mg::kGradTiles[(int)t].name, mg::has_kernel(t, vec, wide, split, kmajor) ? "" : " (none)");
    }
    return 0;
}
int main(int argc, char** argv)
{
    if (argc > 1 && !std::strcmp(argv[1], "grad")) return grad();
    int vec;
    long long M, N, K;
    while (argc > 1 && std::scanf("%d %lld %lld %lld", &vec, &M, &N, &K) == 4)
        std::printf("%s\n", mg::kI8Tiles[(int)mg::i8_tile({!!vec, M, N, K})].name);
    while (std::scanf("%d %lld %lld %lld", &vec, &M, &N, &K) == 4) {
        const mg::I8Edges e = mg::i8_edges({!!vec, M, N, K});
        std::printf("%d %d", (int)e.rows, (int)e.cols);
        // Threads of the parts: what is left, the rows at the end, the columns at the end.
        const long long parts[3][2] = {{M - e.rows, N - e.cols}, {e.rows, N}, {M - e.rows, e.cols}};
        for (const auto& p : parts) {
            const mg::I8Shape s = {!!vec, p[0], p[1], K};
            const mg::Tile& t = mg::kI8Tiles[(int)mg::i8_tile(s)];
            std::printf(" %lld", p[0] && p[1] ? (long long)mg::i8_grid(s, t) * t.threads : 0);
        }
        std::printf(" %d", std::strncmp(mg::kI8Tiles[(int)mg::i8_tile({!!vec, M, N, K})].name, "unaligned", 9) != 0);
        std::printf("\n");
    }
}
"""


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    d = tmp_path_factory.mktemp("launches8")
    (d / "rules.cpp").write_text(SOURCE)
    exe = str(d / "rules")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "dense_gemm_engineering_run_amd", "csrc"),
                    str(d / "rules.cpp"), "-o", exe], check=True)
    return exe


@pytest.fixture(scope="module")
def edges(exe):
    def run(shapes):
        """Per (aligned, M, N, K): rows, columns cut off, the parts' threads, and
        whether the whole would run a kernel for aligned operands."""
        text = "\n".join(f"{int(a)} {M} {N} {K}" for a, M, N, K in shapes)
        out = subprocess.run([exe], input=text, check=True, capture_output=True, text=True).stdout
        got = [tuple(map(int, line.split())) for line in out.splitlines()]
        assert len(got) == len(shapes)
        return got

    return run


@pytest.fixture(scope="module")
def grad(exe):
    def run(calls):
        """Per (aligned, fp32 C, terms of A, A k-major, M, N, K): the tile's name."""
        text = "\n".join(" ".join(str(int(x)) for x in c) for c in calls)
        got = subprocess.run([exe, "grad"], input=text, check=True, capture_output=True, text=True).stdout.splitlines()
        assert len(got) == len(calls)
        return got

    return run


def test_the_parts_of_a_launch_that_fits_fit(edges):
    """What has no cut is refused by the entry point where it is too large."""
    long = [1 << 30, (1 << 30) - 126, (1 << 29) + 130, (1 << 23) + 5]
    shapes = [(vec, *s, K) for vec in (True, False) for n in (130, 144, 258, 1026) for m in long for s in ((m, n), (n, m))
              for K in (1, 16, 4096, 131071)]
    for s, got in zip(shapes, edges(shapes)):
        if got[0] or got[1]:
            assert max(got[2:5]) < 1 << 32, (s, got)


SIZES = [1, 15, 16, 31, 33, 64, 65, 100, 128, 130, 257, 400, 1000, 1950, 2304, 4096, 10000, 30000, 65536, 1 << 20]


def test_every_product_has_a_kernel_for_its_operands(edges):
    shapes = [(vec, M, N, K) for vec in (True, False) for M in SIZES for N in SIZES for K in (1, 100, 4096)]
    assert all(bool(got[5]) == s[0] for s, got in zip(shapes, edges(shapes)))


def test_every_gradient_has_a_kernel(grad):
    """16-bit C: A's terms; fp32 C: A's or Q's."""
    calls = [(vec, wide, split, kmajor, M, N, K) for vec in (True, False) for wide, split in ((False, True), (True, True), (True, False))
             for kmajor in (True, False) for M in SIZES for N in SIZES for K in (1, 100, 129, 4096)]
    names = grad(calls)
    assert not [c for c, name in zip(calls, names) if "none" in name]
    # ... and every tile runs for some call.
    assert len(set(names)) == 10


def test_edges_of_long_products_are_priced_by_their_length(edges):
    """Sizes measured with and without the cut, the faster one by 10 % and more
    (K in a multiple of 16 bytes, or at any byte)."""
    whole = [(True, 65536, 130, 2048), (True, 65536, 144, 2048), (True, 130, 65536, 2048), (True, 144, 32768, 4096),
             (True, 32768, 260, 2048), (True, 260, 8192, 4096), (True, 65536, 272, 512), (True, 16384, 130, 4096),
             (False, 130, 65536, 2048), (False, 65536, 260, 2048), (False, 16384, 130, 4096), (False, 130, 16384, 2048),
             (False, 8192, 272, 2048), (False, 260, 8192, 4096)]
    assert [got[:2] for got in edges(whole)] == [(0, 0)] * len(whole)
    cut = [(True, 8193, 4096, 4096, 1, 0), (True, 2049, 4096, 4096, 1, 0), (True, 4100, 4104, 2048, 4, 8),
           (True, 16384, 1030, 1024, 0, 6), (True, 2053, 4096, 2048, 5, 0), (False, 2049, 4096, 4096, 1, 0),
           (False, 4095, 2049, 1028, 0, 1), (False, 2048, 4112, 2048, 0, 16), (False, 8193, 4096, 4096, 1, 0)]
    assert [got[:2] for got in edges([s[:4] for s in cut])] == [s[4:] for s in cut]


# Gradients into a thin fp32 C: M, N, K, and where the tile that many tiles of it
# would take is 10 % and more behind, the fastest: bf16 A (Q's terms), others (A's)
THIN = [(64, 65536, 2048, "64x128", "64x128"), (16, 65536, 2048, "64x128", "64x128"), (100, 65536, 1024, "128x128", None),
        (65536, 64, 2048, None, "64x64"), (65536, 16, 2048, None, "64x64"), (65536, 128, 1024, None, "128x128, deep")]


def test_thin_fp32_gradients_run_tiles_that_fit_them(grad):
    calls, want = [], []
    for M, N, K, q, a in THIN:
        for split, name in ((False, q), (True, a)):
            for kmajor in (False, True) if name else ():
                calls.append((True, True, split, kmajor, M, N, K))
                want.append(name)
    assert grad(calls) == want


def test_inputs_gradients_of_a_tile_for_most_cus(grad):
    """A k-major, 129 to 160 tiles of 128 x 256: 64x128 tiles take 5 to 27 % longer."""
    assert grad([(True, True, True, True, *s) for s in ((2304, 1952, 2048), (20000, 256, 1000), (8192, 528, 2048), (1104, 4000, 1024))]) \
        == ["128x256"] * 4


def test_unaligned_wide_tiles_by_their_last_round(exe):
    """128x256 tiles beside 128x128 ones, two of which share a CU: measured 10 to 16 %
    slower with a last round of 1 to 128 tiles, 5 to 10 % faster with 160 and more."""
    shapes = [(128 * (n // 8), 2048, K) for K in (2500, 4096) for n in (264, 320, 384, 416, 448, 512, 640, 672, 928)]
    text = "\n".join(f"0 {M} {N} {K}" for M, N, K in shapes)
    got = subprocess.run([exe, "product"], input=text, check=True, capture_output=True, text=True).stdout.splitlines()
    n = "unaligned 128x128"
    w = "unaligned 128x256"
    assert got == [n, n, n, w, w, w, n, w, w] * 2
