"""The grouped entry points without a GPU: every refusal, in the documented
order, before any HIP call, and the calls that launch nothing."""
import pytest

import dense_gemm_engineering_run_amd as g
from dense_gemm_engineering_run_amd import _binding as b

P = 1 << 24          # fake, 16-byte aligned device addresses (never dereferenced)


def rows(M=64, N=64, K=64, a="k", bm="k", c="n", dtype=0, A=P, B=2 * P, C=3 * P, lda=None, ldb=None, ldc=None,
         groups=4, stride=None, ends=4 * P):
    lda = max(1, K) if lda is None else lda
    ldb = max(1, K if bm in "kK" else N) if ldb is None else ldb
    ldc = max(1, N) if ldc is None else ldc
    stride = N * K if stride is None else stride
    return g.gemm_run_grouped(M, N, K, a, bm, c, dtype, A, B, C, lda, ldb, ldc, groups, stride, ends)


def by_k(M=64, N=64, K=64, a="m", bm="n", c="n", dtype=0, A=P, B=2 * P, C=3 * P, lda=None, ldb=None, ldc=None,
         groups=4, stride=None, ends=4 * P, accumulate=0):
    lda = max(1, M) if lda is None else lda
    ldb = max(1, N) if ldb is None else ldb
    ldc = max(1, N if c in "nN" else M) if ldc is None else ldc
    stride = M * N if stride is None else stride
    return g.gemm_run_grouped_k(M, N, K, a, bm, c, dtype, A, B, C, lda, ldb, ldc, groups, stride, ends, accumulate)


@pytest.mark.parametrize("call", [rows, by_k])
def test_refusals_shared_by_both(call):
    for kw in (dict(M=-1), dict(N=-1), dict(K=-1), dict(groups=-1), dict(groups=65536), dict(M=(1 << 30) + 1)):
        assert call(**kw) == b.GEMM_ERR_BAD_SHAPE, kw
    assert call(dtype=5) == b.GEMM_ERR_BAD_DTYPE
    assert call(dtype=-1) == b.GEMM_ERR_BAD_DTYPE
    for kw in (dict(lda=63), dict(ldb=63), dict(ldc=63), dict(stride=-1), dict(stride=1 << 60), dict(lda=1 << 62),
               dict(ldc=(1 << 63) - 1)):
        assert call(**kw) == b.GEMM_ERR_BAD_LD, kw
    for kw in (dict(A=0), dict(B=0), dict(C=0), dict(ends=0)):
        assert call(**kw) == b.GEMM_ERR_NULL_PTR, kw
    for kw in (dict(A=P + 2), dict(B=2 * P + 1), dict(C=3 * P + 2), dict(ends=4 * P + 2), dict(A=P + 1, dtype=2)):
        assert call(**kw) == b.GEMM_ERR_MISALIGNED, kw
    for kw in (dict(C=P + 16), dict(C=2 * P + 1024), dict(ends=3 * P + 64)):
        assert call(**kw) == b.GEMM_ERR_ALIAS, kw
    # the checks run in the header's order
    assert call(M=-1, a="x", dtype=9) == b.GEMM_ERR_BAD_SHAPE
    assert call(a="x", dtype=9, lda=0) == b.GEMM_ERR_BAD_MAJOR
    assert call(dtype=9, lda=0) == b.GEMM_ERR_BAD_DTYPE
    assert call(lda=0, A=0) == b.GEMM_ERR_BAD_LD
    assert call(A=0, C=3 * P + 1) == b.GEMM_ERR_NULL_PTR
    assert call(A=P + 1, C=P) == b.GEMM_ERR_MISALIGNED
    # a leading dimension whose tile offsets would pass 32 bits
    assert call(lda=1 << 24, A=1 << 44) == b.GEMM_ERR_BAD_SHAPE


def test_majors():
    for kw in (dict(a="m"), dict(c="m"), dict(bm="m"), dict(bm="x")):
        assert rows(**kw) == b.GEMM_ERR_BAD_MAJOR, kw
    for kw in (dict(a="k"), dict(bm="k"), dict(c="k")):
        assert by_k(**kw) == b.GEMM_ERR_BAD_MAJOR, kw


def test_matrices_of_the_groups_may_share_a_b_but_not_a_c():
    assert by_k(stride=64 * 64 - 1) == b.GEMM_ERR_BAD_LD
    assert by_k(stride=0) == b.GEMM_ERR_BAD_LD
    assert by_k(stride=0, groups=1, A=0) == b.GEMM_ERR_NULL_PTR      # one group: the stride is not used
    assert rows(stride=0, A=0) == b.GEMM_ERR_NULL_PTR                # passes the stride check


def test_calls_that_launch_nothing():
    for call in (rows, by_k):
        assert call(M=0, A=0, B=0, C=0, ends=0) == b.GEMM_OK
        assert call(N=0, A=0, B=0, C=0, ends=0) == b.GEMM_OK
        assert call(groups=0, A=0, B=0, C=0, ends=0) == b.GEMM_OK
    assert by_k(K=0, A=0, B=0, accumulate=1) == b.GEMM_OK
    # K == 0 still writes C: it needs C and the ends, not A and B
    assert rows(K=0, A=0, B=0, C=0) == b.GEMM_ERR_NULL_PTR
    assert by_k(K=0, A=0, B=0, ends=0) == b.GEMM_ERR_NULL_PTR


def test_torch_entry_points_refuse_what_is_not_on_a_gpu():
    import torch
    a, w, c = torch.zeros(4, 8), torch.zeros(2, 6, 8), torch.zeros(4, 6)
    ends = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        g.grouped_gemm(a, w, ends, c)
    with pytest.raises(ValueError):
        g.grouped_gemm_k(a.t(), c.t(), ends, torch.zeros(2, 8, 6))


def test_leading_dimension_of_views():
    import torch
    t = torch.zeros(4, 8)
    assert b._ld(t.shape, t.stride(), 0, 1) == 8 and b._ld(t.shape, t.stride(), 1, 0) is None
    assert b._ld(t.t().shape, t.t().stride(), 1, 0) == 8
    v = torch.zeros(4, 12)[:, :8]
    assert b._ld(v.shape, v.stride(), 0, 1) == 12
    one = torch.zeros(1, 5)
    assert b._ld(one.shape, one.stride(), 0, 1) == 16          # a single row: any
    col = torch.zeros(5, 1)
    assert b._ld(col.shape, col.stride(), 0, 1) == 1
    assert b._ld((3, 8), (0, 1), 0, 1) is None                  # rows that overlap
