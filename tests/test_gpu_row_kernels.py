"""Every kernel of the grouped and adapter products, at widths that are no
multiple of its tile: whole and partial last k-tiles, ragged groups, ranks of
any size, an unaligned C.  (tests/test_tile_rules.py holds the sizes to the
rules that pick the kernels.)  Tolerances are those of the modules whose
helpers run here."""
import pytest
import torch

import row_kernel_cases as cases
from test_gpu_grouped import run_k, run_rows
from test_gpu_lora import TYPES, Case, run, say

pytestmark = pytest.mark.gpu


def table(pick):
    """(type, padding, case) of every type."""
    out = []
    for dtype in TYPES:
        for pad in (0, 1):
            for case in pick(dtype == "f32", pad):
                out.append(pytest.param(dtype, pad, case, id=f"{dtype}-{pad}-{case[0]}".replace(" ", "-")))
    return out


@pytest.mark.parametrize("dtype,pad,case", table(lambda f32, pad: cases.grouped(f32, pad)[0]))
def test_grouped_by_rows(dtype, pad, case):
    _, lens, N, majors = case
    for b_major in majors:
        for K in (8, 64, 328):
            run_rows(lens, N, K, dtype, b_major, left=3, pad=pad)
        run_rows(lens, N, 200, dtype, b_major, left=3, pad=pad, kind="int5")
        if not pad:
            run_rows(lens, N, 136, dtype, b_major, left=3, c_pad=1)


@pytest.mark.parametrize("dtype,pad,case", table(lambda f32, pad: cases.grouped(f32, pad)[1]))
def test_grouped_by_k(dtype, pad, case):
    _, lens, M, N = case
    for c_major, m, n in (("n", M, N), ("m", N, M)):       # C m-major runs exchanged
        for accumulate in (False, True):
            run_k(lens, m, n, dtype, c_major, left=3, pad=pad, accumulate=accumulate)
            run_k(lens, m, n, dtype, c_major, left=3, pad=pad, accumulate=accumulate, kind="int5")


@pytest.mark.parametrize("dtype,pad,case", table(cases.lora))
def test_adapters(dtype, pad, case):
    _, M, N, majors = case
    ids = "packed" if M > 1000 else "mixed"
    for b_major in majors:
        # ranks: aligned up, past 64 columns of v, rows of up that are not aligned
        for K, R, mixed in ((40, 40, False), (64, 24, True), (72, 100, True), (328, 12, False), (264, 136, True)):
            run(M, N, K, 7, R, dtype, ids=ids, b_major=b_major, pad=pad, mixed=mixed)
        run(M, N, 104, 5, 72, dtype, ids=ids, b_major=b_major, pad=pad, kind="int5")
        run(M, N, 104, 5, 1, dtype, ids="distinct", b_major=b_major, pad=pad, kind="int5")
        if not pad:
            run(M, N + 1 if b_major == "k" else N, 264, 5, 16, dtype, ids="packed", b_major=b_major)   # C unaligned


@pytest.mark.parametrize("dtype,pad,case", table(cases.lora))
def test_adapters_without_ranks_scales_or_rows(dtype, pad, case):
    _, M, N, majors = case
    for b_major in majors:
        run(M, N, 200, 3, 32, dtype, ids="one", b_major=b_major, pad=pad, mixed=False, scales=False)
        run(M, N, 200, 3, 32, dtype, ids="none", b_major=b_major, pad=pad)


@pytest.mark.parametrize("dtype,pad,case", table(cases.lora))
def test_requests_do_not_see_each_other(dtype, pad, case):
    """A NaN in one slot's down, an infinity in another's up, both past a
    third's rank: rows of no or another slot keep their values."""
    _, M, N, majors = case
    for b_major in majors:
        for R in (24, 27):
            say(dtype, pad, M, N, b_major, R)
            x = Case(M, N, 200, 6, R, dtype, ids="distinct", b_major=b_major, pad=pad, mixed=False)
            x.ranks = torch.tensor([R, 10, R, 0, R, 3], dtype=torch.int32, device="cuda")
            x.down[2, 3, 5] = float("nan")
            x.up[4, 1] = float("inf")
            x.up[1, :, 10:] = float("nan")
            x.down[1, 10:] = float("inf")
            x.up[3] = float("nan")
            x.up[5, :, 3:] = float("inf")
            x.run()
            torch.cuda.synchronize()
            assert x.c[x.ids == 2].isnan().all()
            four = x.c[x.ids == 4]
            assert not four[:, 1].isfinite().any() and four[:, 2:].isfinite().all() and four[:, 0].isfinite().all()
            x.down[1, 10:], x.up[1, :, 10:], x.up[5, :, 3:], x.up[3] = 0, 0, 0, 0
            x.check((x.ids != 2) & (x.ids != 4))
