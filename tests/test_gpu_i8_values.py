"""What the factors of the 8-bit layer's gradients hold, on the GPU.

Into 16-bit C, scales[k] * A[m][k] enters in two bf16 terms: rounded to fp32 (2^-24
of itself), its first 8 bits cut off (the rest is less than 2^-7 of it), the rest
rounded to 8 bits (2^-9 of that): 2^-24 + 2^-16 of itself.  The sum has 2 K fp32
terms.  With S = sum_k |A| |scales Q|,
    E = (2 K + 1) 2^-24 S + 2^-16 S,    then the rounding to C: eps(C) / 2 (|ref| + E)
(2^-25 more for fp16's subnormals).  Into fp32 C three terms hold the product whole:
(3 K + 2) 2^-24 S.  Of a term, bits below bf16's smallest subnormal are lost: 2^-133
times the other factor more for every k (and fp32's own, a few 2^-149 for every
addition).
"""
import pytest
import torch

import dense_gemm_engineering_run_amd as g
import i8_kernel_cases as cases
from test_gpu_i8 import F16, Gradient, ints, say

pytestmark = pytest.mark.gpu

NARROW = {"bf16_bf16": 2.0 ** -9, "f16_f16": 2.0 ** -12}      # half a step of the type at 1
KERNELS = [pytest.param(aligned, M, N, id=f"{name}-{M}x{N}-{'aligned' if aligned else 'not'}".replace(" ", "_"))
           for aligned in (True, False) for name, M, N in cases.gradients(False, False, aligned)]


def tolerance(x):
    a, v = x.a.double(), x.s.double()[:, None] * x.q.t().double()
    S, K = a.abs() @ v.abs(), a.shape[1]
    return a @ v, ((2 * K + 1) * 2.0 ** -24 + 2.0 ** -16) * S


def check(x):
    ref, E = tolerance(x)
    g.gemm_i8_grad(x.a, x.q, x.s, x.c)
    tol = E + torch.finfo(x.tout).eps / 2 * (ref.abs() + E) + (2.0 ** -25 if x.tout == F16 else 0)
    diff = (x.c.double() - ref).abs()
    bad = ~(diff <= tol)
    assert not bad.any(), (int(bad.sum()), float((diff / tol).max()), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("dtype", NARROW)
@pytest.mark.parametrize("a_major", "mk")
@pytest.mark.parametrize("aligned,M,N", KERNELS)
def test_bits_that_a_rounded_factor_would_lose(dtype, a_major, aligned, M, N):
    """Pairs of k with the same Q, opposite A, and scales 1 + half a step and 1:
    what is left is the half step's.  Exact: sums stay below 2^12, in steps of 2^-12."""
    K, half = 130, NARROW[dtype]
    x = Gradient(M, N, K, dtype, a_major, *((None, 0) if aligned else (1, 3)))
    twice = lambda t: t.repeat_interleave(2, 1)
    a = twice(ints((M, K // 2), 1, -2, 2).float())
    a[:, 1::2] *= -1
    q = twice(ints((N, K // 2), 2, -8, 8))
    x.a.copy_(a)
    x.q.copy_(q)
    x.s[0::2], x.s[1::2] = 1 + half, 1
    g.gemm_i8_grad(x.a, x.q, x.s, x.c)
    want = (a[:, 0::2].double().cuda() @ q[:, 0::2].double().t().cuda() * half).to(x.tout)
    assert torch.equal(x.c, want), (int((x.c != want).sum()), (x.c != want).nonzero()[0].tolist())


@pytest.mark.parametrize("dtype", NARROW)
@pytest.mark.parametrize("a_major", "mk")
@pytest.mark.parametrize("aligned,M,N", KERNELS)
def test_16_bit_outputs_are_off_by_their_own_rounding(dtype, a_major, aligned, M, N):
    for K in (8, 64, 131):
        say(dtype, a_major, aligned, M, N, K)
        check(Gradient(M, N, K, dtype, a_major, *((None, 0) if aligned else (1, 3)), seed=K))


@pytest.mark.parametrize("a_major", "mk")
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("size_a,size_s", [(2.0 ** -11, 2.0 ** 11), (2.0 ** 11, 2.0 ** -18)])
def test_restored_values_outside_fp16s_range(a_major, aligned, size_a, size_s):
    """Outputs within it: 2^11 * Q is past fp16's largest number, 2^-18 * Q mostly
    below its smallest normal one."""
    for M, N, K in ((40, 50, 64), (520, 610, 64), (1000, 1000, 40), (2304, 1950, 33)):
        x = Gradient(M, N, K, "f16_f16", a_major, *((None, 0) if aligned else (1, 3)))
        x.a.copy_(torch.randn((M, K), generator=torch.Generator().manual_seed(3)).clamp(-4, 4) * size_a)
        x.s.copy_((1 + ints((K,), 4, 0, 1023).float() / 1024) * size_s)
        check(x)
        assert torch.isfinite(x.c).all()


@pytest.mark.parametrize("dtype", NARROW)
@pytest.mark.parametrize("a_major", "mk")
@pytest.mark.parametrize("aligned,M,N", [(True, 48, 64), (False, 48, 50), (True, 1000, 1000), (True, 2304, 1950), (True, 3300, 3100)])
def test_an_infinity_of_a_keeps_its_sign(dtype, a_major, aligned, M, N):
    """inf * (scales Q) for whatever Q is not 0, also where the factor has so few
    bits that its second term would be 0."""
    K = 96
    x = Gradient(M, N, K, dtype, a_major, *((None, 0) if aligned else (1, 3)))
    x.s[10], x.s[20] = 0.5, 0.375
    x.a[3, 10], x.a[7, 20] = float("inf"), -float("inf")
    g.gemm_i8_grad(x.a, x.q, x.s, x.c)
    for m, k in ((3, 10), (7, 20)):
        want = x.a[m, k].double() * x.q[:, k].double()
        assert torch.equal(x.c[m].double().nan_to_num(7.0, 1e9, -1e9), want.nan_to_num(7.0, 1e9, -1e9)), (m, k)
    rest = torch.ones(M, dtype=torch.bool)
    rest[[3, 7]] = False
    assert torch.isfinite(x.c[rest.cuda()]).all()


@pytest.mark.parametrize("dtype", ["f32", "f16_f32", "bf16_f32"])
@pytest.mark.parametrize("a_major", "mk")
@pytest.mark.parametrize("aligned", [True, False])
def test_thin_fp32_outputs(dtype, a_major, aligned):
    for i, (M, N, K) in enumerate(((64, 40000, 70), (20, 33000, 33), (100, 50000, 130), (40000, 60, 64), (40000, 100, 131), (2304, 1950, 40))):
        say(dtype, a_major, aligned, M, N, K)
        at = (None, 0) if aligned else (1, 3)
        Gradient(M, N, K, dtype, a_major, *at, seed=i).run(accumulate=i % 2 == 1)
        Gradient(M, N, K, dtype, a_major, *at, "int", seed=i).run(accumulate=i % 2 == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16_f32", "bf16_bf16"])
@pytest.mark.parametrize("a_major", "mk")
@pytest.mark.parametrize("exponent", [-105, -110, -114, -118, -122, -127, -131])
def test_factors_near_the_end_of_the_range(dtype, a_major, exponent):
    """scales near 2^exponent, A near 1: what is lost is no more than the bits below 2^-133."""
    for M, N, K in ((40, 48, 64), (300, 600, 40), (2048, 2048, 64)):
        x = Gradient(M, N, K, dtype, a_major, None)
        a = torch.randn((M, K), generator=torch.Generator().manual_seed(1)).clamp(-4, 4)
        x.a.copy_(a)
        x.s.copy_(((1 + ints((K,), 2, 0, 1023).double() / 1024) * 2.0 ** exponent).float())
        A, Q, s = x.a.double(), x.q.double(), x.s.double()
        ref, S = A @ (s[:, None] * Q.t()), A.abs() @ (s[:, None] * Q.t().abs())
        other = A.abs().sum(1, keepdim=True) if dtype == "bf16_f32" else Q.abs().sum(1)
        E = (3 * K + 2) * 2.0 ** -24 * S + 2.0 ** -133 * other + 3 * K * 2.0 ** -149
        if dtype == "bf16_bf16":
            E = E + 2.0 ** -16 * S + torch.finfo(x.tout).eps / 2 * (ref.abs() + E) + 2.0 ** -134
        g.gemm_i8_grad(x.a, x.q, x.s, x.c)
        diff = (x.c.double() - ref).abs()
        assert bool((diff <= E).all()), float((diff / E).max())


@pytest.mark.parametrize("dtype", NARROW)
@pytest.mark.parametrize("a_major", "mk")
@pytest.mark.parametrize("aligned", [True, False])
def test_thin_16_bit_outputs_and_short_sums(dtype, a_major, aligned):
    for i, (M, N, K) in enumerate(((64, 40000, 70), (20, 33000, 33), (100, 40000, 128), (40000, 60, 64), (40000, 100, 131), (2304, 1950, 128),
                                   (2304, 1950, 129), (3000, 2816, 40))):
        say(dtype, a_major, aligned, M, N, K)
        at = (None, 0) if aligned else (1, 3)
        check(Gradient(M, N, K, dtype, a_major, *at, seed=i))
        Gradient(M, N, K, dtype, a_major, *at, "int", seed=i).run(accumulate=True)
