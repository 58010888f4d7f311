"""The 8-bit entry points without a GPU: every refusal before any HIP call and
the calls that launch nothing."""
import pytest
import torch

import dense_gemm_engineering_run_amd as g
from dense_gemm_engineering_run_amd import _binding as b

P = 1 << 32          # fake, 16-byte aligned device addresses (never dereferenced)


def product(M=64, N=64, K=64, a="k", bm="k", c="n", type=0, A=P, B=2 * P, C=3 * P, lda=None, ldb=None, ldc=None,
            sa=4 * P, sb=5 * P, epi=None):
    return g.gemm_run_i8(M, N, K, a, bm, c, type, A, B, C, max(1, K) if lda is None else lda,
                         max(1, K) if ldb is None else ldb, max(1, N) if ldc is None else ldc, sa, sb, epi)


def grad(M=64, N=64, K=64, a="m", bm="n", c="n", dtype=0, A=P, Q=2 * P, C=3 * P, lda=None, ldq=None, ldc=None, s=4 * P,
         accumulate=0):
    lda = max(1, M if a in "mM" else K) if lda is None else lda
    return g.gemm_run_i8_grad(M, N, K, a, bm, c, dtype, A, Q, C, lda, max(1, N) if ldq is None else ldq,
                              max(1, N) if ldc is None else ldc, s, accumulate)


def quantize(M=64, K=64, type=0, X=P, Q=2 * P, s=3 * P, ldx=None, ldq=None):
    return g.gemm_quantize_rows(M, K, type, X, Q, s, max(1, K) if ldx is None else ldx, max(1, K) if ldq is None else ldq)


def restore(M=64, K=64, type=0, Q=P, s=3 * P, X=2 * P, ldq=None, ldx=None):
    return g.gemm_dequantize_rows(M, K, type, Q, s, X, max(1, K) if ldq is None else ldq, max(1, K) if ldx is None else ldx)


def expect(call, status, *cases):
    for kw in cases:
        assert call(**kw) == status, kw


def test_product_refusals():
    expect(product, b.GEMM_ERR_BAD_SHAPE, dict(M=-1), dict(N=-1), dict(K=-1), dict(M=(1 << 30) + 1), dict(K=1 << 17))
    expect(product, b.GEMM_ERR_BAD_MAJOR, dict(a="m"), dict(bm="n"), dict(c="m"), dict(a="x"))
    expect(product, b.GEMM_ERR_BAD_DTYPE, dict(type=3), dict(type=-1))
    expect(product, b.GEMM_ERR_BAD_LD, dict(lda=63), dict(ldb=63), dict(ldc=63), dict(lda=1 << 62))
    expect(product, b.GEMM_ERR_NULL_PTR, dict(A=0), dict(B=0), dict(C=0))
    expect(product, b.GEMM_ERR_MISALIGNED, dict(C=3 * P + 2), dict(C=3 * P + 1, type=1), dict(sa=4 * P + 2), dict(sb=5 * P + 1),
           dict(epi=b.Epilogue(1, 0, 6 * P + 2, 0)))
    expect(product, b.GEMM_ERR_ALIAS, dict(C=P), dict(C=2 * P + 64), dict(sa=3 * P), dict(sb=3 * P + 16384 - 4),
           dict(epi=b.Epilogue(1, 0, 3 * P + 64, 0)))
    expect(product, b.GEMM_ERR_BAD_SHAPE, dict(lda=1 << 23, A=1 << 45),
           dict(M=1 << 24, N=1 << 22, K=0, type=1, A=0, B=0, sa=0, sb=0, C=1 << 20))       # a grid no launch can have
    expect(product, b.GEMM_ERR_BAD_EPILOGUE, dict(epi=b.Epilogue(1, 0, 0, 3)), dict(epi=b.Epilogue(1, 0, 0, -1)))


def test_gradient_refusals():
    expect(grad, b.GEMM_ERR_BAD_SHAPE, dict(M=-1), dict(N=-1), dict(K=-1), dict(K=(1 << 30) + 1))
    expect(grad, b.GEMM_ERR_BAD_MAJOR, dict(a="n"), dict(bm="k"), dict(c="m"))
    expect(grad, b.GEMM_ERR_BAD_DTYPE, dict(dtype=5), dict(dtype=-1))
    expect(grad, b.GEMM_ERR_BAD_LD, dict(lda=63), dict(lda=63, a="k"), dict(ldq=63), dict(ldc=63))
    expect(grad, b.GEMM_ERR_NULL_PTR, dict(A=0), dict(Q=0), dict(C=0), dict(s=0))
    expect(grad, b.GEMM_ERR_MISALIGNED, dict(A=P + 2), dict(A=P + 1, dtype=2), dict(C=3 * P + 2), dict(s=4 * P + 2))
    expect(grad, b.GEMM_ERR_ALIAS, dict(C=P), dict(C=2 * P + 64), dict(s=3 * P + 64), dict(C=P, accumulate=1))
    expect(grad, b.GEMM_ERR_BAD_SHAPE, dict(lda=1 << 22, A=1 << 45), dict(ldq=1 << 23, Q=1 << 45),
           dict(M=1 << 24, N=1 << 22, K=0, dtype=2, A=0, Q=0, s=0, C=1 << 20))


def test_row_refusals():
    for call, read, write in ((quantize, "X", "Q"), (restore, "Q", "X")):
        expect(call, b.GEMM_ERR_BAD_SHAPE, dict(M=-1), dict(K=-1), dict(M=(1 << 30) + 1))
        expect(call, b.GEMM_ERR_BAD_DTYPE, dict(type=3), dict(type=-1))
        expect(call, b.GEMM_ERR_BAD_LD, dict(ldx=63), dict(ldq=63), dict(ldx=1 << 62))
        expect(call, b.GEMM_ERR_NULL_PTR, dict(X=0), dict(Q=0), dict(s=0))
        expect(call, b.GEMM_ERR_MISALIGNED, dict(X=8 * P + 2), dict(X=8 * P + 1, type=2), dict(s=3 * P + 2))
        expect(call, b.GEMM_ERR_ALIAS, {write: P, read: P}, {write: 3 * P}, {write: 3 * P + 252})
    assert quantize(s=P) == b.GEMM_ERR_ALIAS                             # the scales are written
    # grids no launch can have
    assert quantize(M=1 << 30, K=8, type=2, X=1 << 40, Q=1 << 44, s=1 << 45) == b.GEMM_ERR_BAD_SHAPE
    assert restore(M=1 << 30, K=8, type=2, X=1 << 40, Q=1 << 44, s=1 << 45) == b.GEMM_ERR_BAD_SHAPE


def test_calls_that_launch_nothing():
    assert product(M=0, A=0, B=0, C=0, sa=0, sb=0) == b.GEMM_OK
    assert product(N=0, A=0, B=0, C=0) == b.GEMM_OK
    assert grad(M=0, A=0, Q=0, C=0, s=0) == b.GEMM_OK
    assert grad(N=0, A=0, Q=0, C=0, s=0) == b.GEMM_OK
    assert grad(K=0, A=0, Q=0, s=0, accumulate=1) == b.GEMM_OK
    assert quantize(M=0, X=0, Q=0, s=0) == b.GEMM_OK
    assert restore(K=0, X=0, Q=0, s=0) == b.GEMM_OK


def test_torch_entry_points_refuse_what_is_not_on_a_gpu():
    z, q, s = torch.zeros(2, 8), torch.zeros(2, 8, dtype=torch.int8), torch.zeros(2)
    for call in (lambda: g.quantize_rows(z, q, s), lambda: g.dequantize_rows(q, s, z), lambda: g.gemm_i8(q, q, s, s, torch.zeros(2, 2)),
                 lambda: g.gemm_i8_grad(z.t(), q.t(), s, torch.zeros(8, 8))):
        with pytest.raises(ValueError):
            call()
