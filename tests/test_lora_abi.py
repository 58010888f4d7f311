"""The adapter entry points without a GPU: every refusal before any HIP call,
the calls that launch nothing, and the workspace's size."""
import pytest

import dense_gemm_engineering_run_amd as g
from dense_gemm_engineering_run_amd import _binding as b

P = 1 << 32          # fake, 16-byte aligned device addresses (never dereferenced)


def run(M=64, N=64, K=64, a="k", bm="k", c="n", dtype=0, A=P, B=2 * P, C=3 * P, lda=None, ldb=None, ldc=None,
        ws=8 * P, ws_bytes=1 << 30, none=False, **lora):
    lda = max(1, K) if lda is None else lda
    ldb = max(1, K if bm in "kK" else N) if ldb is None else ldb
    ldc = max(1, N) if ldc is None else ldc
    f = dict(adapters=4, rank=16, down=4 * P, up=5 * P, ids=6 * P, ranks=7 * P, scales=7 * P + 4096)
    f.update(lora)
    f.setdefault("ld_down", max(1, K))
    f.setdefault("ld_up", max(1, f["rank"]))
    f.setdefault("stride_down", max(0, f["rank"]) * K)
    f.setdefault("stride_up", N * max(0, f["rank"]))
    return g.gemm_run_lora(M, N, K, a, bm, c, dtype, A, B, C, lda, ldb, ldc, None if none else b.Lora(**f), ws, ws_bytes)


def test_refusals():
    for kw in (dict(M=-1), dict(N=-1), dict(K=-1), dict(rank=-1), dict(rank=4097), dict(adapters=-1),
               dict(adapters=(1 << 20) + 1), dict(M=(1 << 30) + 1)):
        assert run(**kw) == b.GEMM_ERR_BAD_SHAPE, kw
    for kw in (dict(a="m"), dict(c="m"), dict(bm="m"), dict(a="x")):
        assert run(**kw) == b.GEMM_ERR_BAD_MAJOR, kw
    assert run(dtype=5) == b.GEMM_ERR_BAD_DTYPE
    for kw in (dict(lda=63), dict(ldb=63), dict(ldc=63), dict(ld_down=63), dict(ld_up=15), dict(stride_down=-1),
               dict(stride_up=1 << 60), dict(ld_up=1 << 62)):
        assert run(**kw) == b.GEMM_ERR_BAD_LD, kw
    for kw in (dict(A=0), dict(B=0), dict(C=0), dict(down=0), dict(up=0), dict(ids=0)):
        assert run(**kw) == b.GEMM_ERR_NULL_PTR, kw
    for kw in (dict(A=P + 2), dict(C=3 * P + 1), dict(down=4 * P + 2), dict(up=5 * P + 1, dtype=2), dict(ids=6 * P + 2),
               dict(ranks=7 * P + 1), dict(scales=7 * P + 2), dict(ws=8 * P + 8)):
        assert run(**kw) == b.GEMM_ERR_MISALIGNED, kw
    for kw in (dict(C=P), dict(C=2 * P + 64), dict(down=3 * P), dict(up=3 * P + 16), dict(ids=3 * P + 64),
               dict(ranks=3 * P), dict(scales=3 * P + 128), dict(ws=3 * P), dict(ws=P), dict(ws=4 * P), dict(ws=6 * P)):
        assert run(**kw) == b.GEMM_ERR_ALIAS, kw
    assert run(lda=1 << 24, A=1 << 45) == b.GEMM_ERR_BAD_SHAPE          # tile offsets past 32 bits
    assert run(ld_down=1 << 24, down=1 << 45, stride_down=1 << 28) == b.GEMM_ERR_BAD_SHAPE


def test_workspace_is_checked_and_sized():
    need = g.gemm_lora_workspace_size(64, 64, 64, 0, 16)
    assert need >= 64 * 16 * 4
    assert run(ws=0, ws_bytes=0) == b.GEMM_ERR_WORKSPACE
    assert run(ws_bytes=need - 1) == b.GEMM_ERR_WORKSPACE
    assert g.gemm_lora_workspace_size(64, 64, 64, 0, 0) == 0
    assert g.gemm_lora_workspace_size(0, 64, 64, 0, 16) == 0
    # a workspace sized for more rows serves fewer
    last = 0
    for m in list(range(1, 1500)) + list(range(1500, 20000, 97)):
        size = g.gemm_lora_workspace_size(m, 4096, 4096, 2, 64)
        assert size >= last and size >= m * 64 * 4
        last = size
    for bad in (lambda: g.gemm_lora_workspace_size(-1, 1, 1, 0, 1), lambda: g.gemm_lora_workspace_size(1, 1, 1, 9, 1),
                lambda: g.gemm_lora_workspace_size(1, 1, 1, 0, 5000)):
        with pytest.raises(g.GemmError):
            bad()


def test_calls_that_launch_nothing():
    assert run(M=0, A=0, B=0, C=0, ids=0, ws=0, ws_bytes=0) == b.GEMM_OK
    assert run(N=0, A=0, B=0, C=0, up=0, ws=0, ws_bytes=0) == b.GEMM_OK
    assert run(M=0, none=True) == b.GEMM_OK


def test_torch_entry_point_refuses_what_is_not_on_a_gpu():
    import torch
    z = torch.zeros
    with pytest.raises(ValueError):
        g.gemm_lora(z(2, 8), z(4, 8), z(2, 4), z(3, 2, 8), z(3, 4, 2), z(2, dtype=torch.int32), z(64))
