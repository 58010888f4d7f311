"""Infinities, NaN and the last bits of adapters, in every kernel.

The inputs are integers whose sums every step of the operator holds exactly,
so what comes out is the definition's value, bit for bit: an infinity where
the definition has one, of its sign, and NaN only where it has that.
"""
import pytest
import torch

from row_kernel_cases import LORA_VALUES
from test_gpu_lora import TYPES, Case, say

pytestmark = pytest.mark.gpu

# Rows, columns and padding (1: operands that are not 16-byte aligned): every
# kernel of the product.
KERNELS = [(M, N, pad) for (_, pad), sizes in LORA_VALUES.items() for M, N in sizes]


def definition(x):
    """C of integer inputs, infinities and NaN among them, in 64 bits."""
    ref = x.a.double() @ x.b.double().t()
    L, R, _ = x.down.shape
    for i in sorted(set(x.ids.tolist())):
        if not 0 <= i < L:
            continue
        m = (x.ids == i).nonzero().flatten()
        r = R if x.ranks is None else min(max(int(x.ranks[i]), 0), R)
        s = 1.0 if x.scales is None else float(x.scales[i])
        v, u = x.a[m].double() @ x.down[i, :r].double().t(), x.up[i, :, :r].double()
        total = torch.zeros((len(m), u.shape[0]), dtype=torch.float64, device="cuda")
        for k in range(r):
            total += v[:, k:k + 1] * u[:, k]
        ref[m] += s * total
    return ref


def same(x):
    want = definition(x).float().to(x.tout)
    wrong = ~((x.c == want) | (x.c.isnan() & want.isnan()))
    if wrong.any():
        m, n = wrong.nonzero()[0].tolist()
        raise AssertionError((int(wrong.sum()), (m, n), float(x.c[m, n]), float(want[m, n])))


def inner(M):
    return 64 if M > 1000 else 104


@pytest.mark.parametrize("M,N,pad", KERNELS)
@pytest.mark.parametrize("dtype", TYPES)
def test_one_infinity_of_an_adapter_keeps_its_sign(dtype, M, N, pad):
    """v_r up[n][r] of a finite v_r and an infinite up is an infinity of the
    product's sign (NaN for v_r = 0), whatever v_r's bits."""
    for b_major in "kn":
        say(dtype, M, N, pad, b_major)
        x = Case(M, N, inner(M), 3, 24, dtype, ids="distinct" if M < 300 else "packed", b_major=b_major, kind="int5", pad=pad,
                 mixed=False)
        if M > 1:
            x.ids[M // 2] = -1
        x.up[0, 3, 5] = float("inf")
        x.up[0, N - 1, 23] = -float("inf")
        x.up[1, 0, 0] = float("inf")
        x.up[1, 0, 9] = float("inf")          # two: NaN where their signs differ
        x.up[1, 40, 11] = float("nan")
        x.run()
        torch.cuda.synchronize()
        same(x)


@pytest.mark.parametrize("M,N,pad", KERNELS)
@pytest.mark.parametrize("dtype", TYPES)
def test_infinite_rows_meet_infinite_adapters(dtype, M, N, pad):
    """v = +inf in every column and up positive, here and there infinite: +inf."""
    say(dtype, M, N, pad)
    x = Case(M, N, inner(M), 2, 24, dtype, ids="one", kind="int5", pad=pad, mixed=False)
    x.up.copy_(x.up.abs() + 1)
    x.a[:, 7] = float("inf")
    x.b[:, 7], x.down[:, :, 7] = 1, 1
    x.up[1, 3, 5] = x.up[1, 3, 6] = x.up[1, 40, 23] = float("inf")
    x.run()
    torch.cuda.synchronize()
    assert (x.c == float("inf")).all(), (x.c != float("inf")).nonzero()[0].tolist()


@pytest.mark.parametrize("M,N,pad", KERNELS)
@pytest.mark.parametrize("dtype", ["f16_f16", "f16_f32"])
def test_small_v_meets_an_infinite_adapter(dtype, M, N, pad):
    """v_1 is below 2^-40 of v_0, which the finite part of fp16's two terms
    cannot hold beside it, but its product with an infinity is one."""
    say(dtype, M, N, pad)
    x = Case(M, N, inner(M), 2, 16, dtype, ids="one", kind="int5", pad=pad, mixed=False, scales=False)
    x.a.fill_(1)
    x.down.zero_()
    x.up.zero_()
    x.down[1, 0] = 2.0 ** 15
    x.down[1, 1, 3] = 2.0 ** -24
    x.up[1, :, 1] = float("inf")
    x.up[1, 1::2, 1] = -float("inf")
    x.run()
    torch.cuda.synchronize()
    sign = 1 - 2 * (torch.arange(N, device="cuda") % 2)
    assert (x.c == sign * float("inf")).all(), (x.c != sign * float("inf")).nonzero()[0].tolist()


@pytest.mark.parametrize("M,N,pad", KERNELS)
def test_an_infinity_counts_before_the_rounding(M, N, pad):
    """The shared product is past fp16's largest value, the adapter's term an
    infinity of the other sign: the sum is that infinity.  (An infinite shared
    product makes it NaN.)"""
    say(M, N, pad)
    for b_major in "kn":
        x = Case(M, N, inner(M), 2, 16, "f16_f16", ids="one", b_major=b_major, kind="int5", pad=pad, mixed=False, scales=False)
        x.a.fill_(50)
        x.b.fill_(-50)                        # -2500 inner(M) < -65504
        x.down.fill_(1)
        x.up.zero_()
        x.up[1, 40:, 3] = float("inf")
        x.b[50] = -float("inf")
        x.run()
        torch.cuda.synchronize()
        want = torch.full((N,), -float("inf"), device="cuda")
        want[40:] = float("inf")
        want[50] = float("nan")
        got = x.c.float()
        assert ((got == want) | (got.isnan() & want.isnan())).all()


@pytest.mark.parametrize("M,N,pad", KERNELS)
def test_fp32_outputs_hold_all_bits_of_v(M, N, pad):
    """bf16 inputs and an fp32 output: v reaches 2^22 as a sum of products of
    8-bit integers, exact in fp32, and up picks its columns one by one."""
    say(M, N, pad)
    for R in (40, 100):
        x = Case(M, N, 64, 3, R, "bf16_f32", ids="distinct" if M < 300 else "packed", kind="int5", pad=pad, mixed=False,
                 scales=False)
        gen = torch.Generator().manual_seed(M + R)
        for t in (x.a, x.down):
            t.copy_(torch.randint(-255, 256, t.shape, generator=gen).to(t.dtype))
        x.b.zero_()
        x.up.copy_((torch.arange(N)[:, None] % R == torch.arange(R)).to(x.up.dtype))
        x.run()
        torch.cuda.synchronize()
        same(x)
        assert x.c.abs().max() > 2 ** 17 and (M == 1 or (x.c.abs() % 2 == 1).any())


@pytest.mark.parametrize("M,N,pad", KERNELS)
def test_small_v_beside_a_large_one_in_fp16(M, N, pad):
    """One component of v is 2^15 and meets up = 0, the others are 2^11 to 2^29
    times smaller and make up all of the adapter's term.  fp16 scales a row by
    one power of two, so they are off by 2^-22 of themselves or by 2^-38 of the
    row's largest (half of fp16's smallest step, 2^-25, where that is 2^13 or
    more), whichever is more.  v is one product, so it is exact; up picks its
    components one by one, so adding the two terms is the only other rounding."""
    say(M, N, pad)
    R = 24
    x = Case(M, N, 64, 2, R, "f16_f32", ids="one", pad=pad, mixed=False, scales=False)
    gen = torch.Generator().manual_seed(M)
    x.a.zero_()
    x.b.zero_()
    x.a[:, 7] = 1
    v = torch.rand(R, generator=gen) * 18 - 14
    v = (2.0 ** v * torch.where(torch.rand(R, generator=gen) < 0.5, -1.0, 1.0)).half()
    v[0] = 2.0 ** 15
    x.down[1, :, 7] = v.cuda()
    x.up.copy_((torch.arange(N)[:, None] % (R - 1) + 1 == torch.arange(R)).to(x.up.dtype))
    x.run()
    torch.cuda.synchronize()
    v, u = v.double().cuda(), x.up[1].double()
    step = torch.maximum(2.0 ** -22 * v.abs(), torch.full_like(v, 2.0 ** -38 * 2.0 ** 15))
    tol = u @ (step + 2.0 ** -24 * v.abs())
    bad = ~((x.c.double() - u @ v).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((x.c.double() - u @ v).abs() / tol).max()))
