"""The 8-bit linear layer on the GPU: rows to 8 bits and back, integer products,
gradients from 8-bit checkpoints, against their definitions.

Rows to 8 bits and back, and integer products without an epilogue, are exact up
to roundings that the definition names, so they are compared bit for bit.

Products with an epilogue: v = fl(fl(fl(sum) sa) sb) as without; then alpha v,
beta C_old and the bias are added in at most three roundings of 2^-24 of
    S = |alpha v| + |beta C_old| + |bias|
each, so t is off by 3 2^-24 S.  ReLU adds nothing.  GELU has a slope of at
most 1.13, its erf is off by 1.5e-7 (of |t| / 2) and its own four roundings by
2^-24 |t| each: 1.13 * 3 2^-24 S + (0.75e-7 + 4 2^-24) |t|.  Last the rounding
to C's type, eps / 2 (2^-25 for fp16 subnormals).

Gradients, with S = sum_k |A| |scales Q|: a sum of n fp32 terms is off by
n 2^-24 S; a product with a scale, in fp32, by 2^-24 of itself, and
    16-bit C: rounded to A's type, by eps(A) / 2 of itself (fp16: 2^-25 where that
              is more); n = K
    fp32 C:   held whole by three terms; n = 3 K
E = (n + 2) 2^-24 S + eps(A) / 2 S + 2^-25 sum_k |A| (fp16), then eps(C) / 2 (|ref| + E).
Small integers with scales that are powers of two come out exactly.
"""
import math
import random

import pytest
import torch

import dense_gemm_engineering_run_amd as g
import i8_kernel_cases as cases

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
WIDE = {"f32": F32, "f16": F16, "bf16": BF16}
PAIRS = {"f32": (F32, F32), "f16_f32": (F16, F32), "bf16_bf16": (BF16, BF16), "f16_f16": (F16, F16), "bf16_f32": (BF16, F32)}
SENTINEL = 77


def say(*a):
    print(*a, flush=True)


def randn(shape, seed, std=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std


def ints(shape, seed, lo=-128, hi=127):
    return torch.randint(lo, hi + 1, shape, generator=torch.Generator().manual_seed(seed))


def place(t, pad=0, offset=0, fill=SENTINEL):
    """The matrix t on the GPU with `pad` more elements a row (None: up to 32, as
    many as make rows of 16-byte multiples), `offset` elements behind an aligned
    address; everything around it holds `fill`."""
    rows, cols = t.shape
    pad = 16 + -cols % 16 if pad is None else pad
    flat = torch.full((rows * (cols + pad) + offset + 16,), fill, dtype=t.dtype, device="cuda")
    v = flat[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(t)
    return v


def around(v):
    """What surrounds a placed matrix (the whole allocation, the matrix masked)."""
    base = v._base if v._base is not None else v
    flat = base.view(-1).clone()
    at = flat.as_strided(v.shape, v.stride(), v.storage_offset())
    at.zero_()
    return flat


def same(a, b):
    """Equal bit for bit, NaN equal to NaN."""
    return bool((((a == b) | (a.isnan() & b.isnan()))).all()) if a.is_floating_point() else torch.equal(a, b)


# ---------------------------------------------------------------- rows to 8 bits and back

def quantized(x):
    """The definition: the quotient of a 31-bit and a 24-bit number in 53 bits
    never reaches a half that it is not."""
    x = x.double()
    top = x.abs().amax(1, keepdim=True) if x.shape[1] else x.new_zeros((x.shape[0], 1))
    bad = ~torch.isfinite(x).all(1, keepdim=True)
    q = torch.round(127.0 * x / torch.where((top > 0) & ~bad, top, 1.0))
    q = torch.where(bad, 0.0, q)
    scales = torch.where(bad, float("nan"), top / 127.0).float()[:, 0]
    return q.to(torch.int8), scales


def check_rows(x, pad=0, offset=0):
    """Quantise x (CPU) and restore it, both bit for bit, nothing around touched."""
    M, K = x.shape
    xd = place(x, pad, offset, float("nan"))
    q = place(torch.full((M, K), SENTINEL, dtype=torch.int8), pad, offset)
    s = torch.full((M + 2,), 7.0, device="cuda")
    edge = around(q)
    g.quantize_rows(xd, q, s[1:M + 1])
    want_q, want_s = quantized(x.cuda())
    torch.cuda.synchronize()
    bad = (q != want_q).nonzero()
    assert not len(bad), (len(bad), bad[0].tolist(), q[tuple(bad[0])], want_q[tuple(bad[0])])
    assert same(s[1:M + 1], want_s) and s[0] == 7 and s[M + 1] == 7
    assert torch.equal(edge, around(q))
    y = place(torch.full((M, K), SENTINEL).to(x.dtype), pad, offset)
    edge = around(y)
    g.dequantize_rows(q, s[1:M + 1], y)
    assert same(y, (want_q.float() * want_s[:, None]).to(x.dtype))
    assert torch.equal(edge, around(y))


WIDTHS = [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 63, 64, 65, 127, 128, 255, 257, 511, 512, 513, 1000, 1023, 1025, 2047, 2049,
          4095, 4096, 4097, 8191, 8192, 8200, 16383, 16384, 16385, 32768, 32776, 40001]


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (1, 0), (0, 1), (3, 5)])
def test_rows_of_every_width(dtype, pad, offset):
    for K in WIDTHS:
        M = 3 if K > 4096 else 5
        say(dtype, K, pad, offset)
        check_rows((randn((M, K), K) * torch.exp(2 * randn((M, 1), K + 1))).to(WIDE[dtype]), pad, offset)


@pytest.mark.parametrize("dtype", WIDE)
def test_many_rows(dtype):
    for M, K in ((1, 4096), (2049, 1000), (4096, 520), (5000, 33), (2050, 4096), (2051, 2040), (70000, 8)):
        say(dtype, M, K)
        check_rows(randn((M, K), M).to(WIDE[dtype]))


@pytest.mark.parametrize("dtype", WIDE)
def test_ties_go_to_even(dtype):
    """127 x / 254 = x / 2: every odd x is a tie; the same at other powers of two."""
    for e in (-130, -100, -62, -61, -14, 0, 3, 7, 60, 99, 100, 101, 119):
        if dtype == "f16" and not -14 <= e <= 7 or dtype != "f16" and e == -14:
            continue
        x = torch.cat([torch.full((4, 1), 254.0), ints((4, 509), e + 500, -254, 254).float()], 1).double() * 2.0 ** e
        say(dtype, e)
        check_rows(x.to(WIDE[dtype]))
        check_rows(x.to(WIDE[dtype]), 1)


def test_fp32_next_to_a_tie():
    gen = random.Random(5)
    for trial in range(40):
        top = math.ldexp(gen.uniform(1, 2), gen.choice([-140, -126, -61, -3, 0, 5, 100, 126]))
        top = float(torch.tensor(top, dtype=F32))
        half = (ints((1, 600), trial, 0, 126).double() + 0.5) * top / 127.0
        x = half.float().view(torch.int32) + ints((1, 600), trial + 99, -3, 3).int()
        x = x.view(F32) * (1 - 2 * ints((1, 600), trial + 7, 0, 1)).float()
        x = torch.where(x.abs() <= top, x, 0.0)
        check_rows(torch.cat([x, torch.tensor([[top]])], 1))


@pytest.mark.parametrize("dtype", WIDE)
def test_rows_of_every_kind(dtype):
    t = WIDE[dtype]
    big, tiny = torch.finfo(t).max, torch.finfo(t).smallest_normal * torch.finfo(t).eps
    for K in (24, 1000, 33):
        x = randn((14, K), 3).to(t)
        x[1] = 0
        x[2] = -0.0
        x[3, K // 2] = float("inf")
        x[4, 0] = -float("inf")
        x[5, K - 1] = float("nan")
        x[6] = x[6].sign() * big
        x[7] = x[7].sign() * tiny
        x[8] = 0
        x[8, K - 2] = -tiny
        x[9] = (x[9].double() * tiny * 40).to(t)
        x[10, 3] = big
        x[11] = 0
        x[11, 1] = big
        x[12, :] = float("nan")
        x[13] = (x[13].double() * big / 8).to(t)
        for pad in (0, 1):
            check_rows(x, pad)


@pytest.mark.parametrize("dtype", WIDE)
def test_restoring_with_any_scale(dtype):
    q = ints((9, 777), 4).to(torch.int8).cuda()
    s = torch.tensor([1.0, -2.5, 0.0, float("inf"), float("nan"), 1e-30, 3e38, 600.0, 2.0 ** -149], device="cuda")
    y = torch.empty((9, 777), dtype=WIDE[dtype], device="cuda")
    g.dequantize_rows(q, s, y)
    assert same(y, (q.float() * s[:, None]).to(WIDE[dtype]))


def test_a_row_of_no_values():
    s = torch.full((3,), 7.0, device="cuda")
    g.quantize_rows(torch.empty((3, 0), device="cuda"), torch.empty((3, 0), dtype=torch.int8, device="cuda"), s)
    assert s.tolist() == [0, 0, 0]


# ---------------------------------------------------------------- products

def gelu(t):
    return 0.5 * t * (1.0 + torch.erf(t / math.sqrt(2.0)))


class Product:
    def __init__(self, M, N, K, dtype, pad=0, offset=0, seed=0, lo=-128, scaled=True, c_pad=0):
        self.t = WIDE[dtype]
        self.a, self.b = place(ints((M, K), seed + 1, lo).to(torch.int8), pad, offset), \
            place(ints((N, K), seed + 2, lo).to(torch.int8), pad, offset)
        # fp16 outputs stay in range
        size = (127.0 * math.sqrt(max(K, 1))) ** -0.5
        self.sa = (torch.exp(randn((M,), seed + 3)) * size).cuda() if scaled else None
        self.sb = (torch.exp(randn((N,), seed + 4)) * size / 30).cuda() if scaled else None
        self.c = place(randn((M, N), seed + 5).to(self.t), pad if pad is None else pad + c_pad, offset)

    def sums(self):
        return self.a.double() @ self.b.double().t()

    def value(self):
        v = self.sums().float()
        return v if self.sa is None else v * self.sa[:, None] * self.sb

    def run(self):
        edge = around(self.c)
        assert g.gemm_i8(self.a, self.b, self.sa, self.sb, self.c) is self.c
        torch.cuda.synchronize()
        assert torch.equal(edge, around(self.c))
        want = self.value().to(self.t)
        bad = ~((self.c == want) | (self.c.isnan() & want.isnan()))
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), self.c[tuple(bad.nonzero()[0])],
                               want[tuple(bad.nonzero()[0])])

    def run_epilogue(self, alpha, beta, bias, act):
        old = self.c.clone()
        (M, N), K = self.c.shape, self.a.shape[1]
        bias_t = randn((N,), 9).cuda() if bias else None
        epi = g.Epilogue(alpha, beta, bias_t.data_ptr() if bias else None, act)
        ld = lambda t: t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)
        zero = lambda t: t.data_ptr() if t is not None else 0
        st = g.gemm_run_i8(M, N, K, "k", "K", "n", {F32: 0, F16: 1, BF16: 2}[self.t], self.a.data_ptr(), self.b.data_ptr(),
                           self.c.data_ptr(), ld(self.a), ld(self.b), ld(self.c), zero(self.sa), zero(self.sb), epi,
                           torch.cuda.current_stream().cuda_stream)
        assert st == 0, g.gemm_status_str(st)
        v = self.value().double()
        o = old.double() if beta else torch.zeros_like(v)
        t = alpha * v + beta * o
        S = (alpha * v).abs() + (beta * o).abs()
        if bias:
            t, S = t + bias_t.double(), S + bias_t.double().abs()
        E = 3 * 2.0 ** -24 * S
        if act == g.GEMM_ACT_RELU:
            t = t.clamp(min=0)
        elif act == g.GEMM_ACT_GELU:
            E = 1.13 * E + (0.75e-7 + 4 * 2.0 ** -24) * (t.abs() + E)
            t = gelu(t)
        tol = E + torch.finfo(self.t).eps / 2 * (t.abs() + E) + (2.0 ** -25 if self.t == F16 else 0)
        diff = (self.c.double() - t).abs()
        assert bool((diff <= tol).all()), float((diff / tol).max())


PRODUCTS = [(1, 1, 1), (1, 16, 16), (2, 3, 5), (1, 300, 64), (16, 16, 128), (17, 33, 129), (5, 260, 1000), (32, 128, 96),
            (31, 500, 2048), (33, 100, 77), (48, 129, 256), (64, 64, 64), (65, 65, 65), (100, 90, 1028), (128, 256, 384),
            (129, 127, 255), (200, 1000, 130), (256, 256, 512), (257, 300, 1027), (300, 200, 136), (515, 520, 200), (1000, 70, 333)]


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("pad,offset", [(0, 0), (16, 0), (1, 0), (0, 3), (6, 2)])
def test_products(dtype, pad, offset):
    for i, (M, N, K) in enumerate(PRODUCTS):
        say(dtype, pad, offset, M, N, K)
        k16 = (K + 15) // 16 * 16 - K
        Product(M, N, K, dtype, pad + k16 if pad == 16 else pad, offset, seed=10 * i).run()


@pytest.mark.parametrize("dtype", WIDE)
def test_product_without_scales_and_with_an_unaligned_output(dtype):
    for M, N, K in ((3, 40, 64), (70, 50, 256), (300, 260, 512)):
        Product(M, N, K, dtype, scaled=False, lo=-1).run()
        x = Product(M, N, K, dtype)
        x.c = place(torch.zeros((M, N), dtype=x.t), 1, 1)
        x.run()


def test_longest_sum():
    """K = 131071 of -128 * -128: the largest sum, and none."""
    K = 131071
    for M, N in ((2, 3), (40, 20), (130, 200)):
        a, b = torch.full((M, K), -128, dtype=torch.int8, device="cuda"), torch.full((N, K), -128, dtype=torch.int8, device="cuda")
        a[1] = 127
        c = torch.zeros((M, N), device="cuda")
        g.gemm_i8(a, b, None, None, c)
        want = torch.full((M, N), 16384.0 * K, device="cuda", dtype=torch.float64)
        want[1] = -16256.0 * K
        assert torch.equal(c, want.float())


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("pad", [0, 1])
def test_product_epilogues(dtype, pad):
    for M, N, K in ((1, 300, 64), (20, 48, 512), (65, 40, 300), (150, 264, 130), (300, 280, 256)):
        for alpha, beta, bias, act in ((1, 0, True, 0), (1, 0, True, 1), (1, 0, True, 2), (0.5, 0, False, 0), (-1.5, 0.75, True, 2),
                                       (1, 1, False, 0), (0, 0, True, 1)):
            say(dtype, pad, M, N, K, alpha, beta, bias, act)
            Product(M, N, K, dtype, pad).run_epilogue(alpha, beta, bias, act)


@pytest.mark.parametrize("dtype", WIDE)
def test_product_of_no_values(dtype):
    c = torch.full((5, 7), 3.0, dtype=WIDE[dtype], device="cuda")
    z = torch.zeros((7, 0), dtype=torch.int8, device="cuda")
    g.gemm_i8(z[:5], z, None, None, c)
    assert bool((c == 0).all())
    bias = torch.arange(7.0, device="cuda") - 3
    g.gemm_i8(z[:5], z, None, None, c, bias=bias, activation=g.GEMM_ACT_RELU)
    assert torch.equal(c, bias.clamp(min=0).to(c.dtype).expand(5, 7))


def test_scales_that_are_not_numbers_reach_their_row_and_column_only():
    x = Product(40, 50, 96, "f32")
    x.sa[3], x.sa[5] = float("nan"), float("inf")
    x.sb[7] = float("nan")
    x.run()
    assert x.c[3].isnan().all() and x.c[:, 7].isnan().all() and int(x.c.isnan().sum()) == 50 + 40 - 1


# ---------------------------------------------------------------- gradients

class Gradient:
    def __init__(self, M, N, K, dtype, a_major, pad=0, offset=0, kind="normal", seed=0, c_pad=0):
        self.tin, self.tout = PAIRS[dtype]
        self.exact = kind == "int"
        nan = float("nan")
        shape = (K, M) if a_major == "m" else (M, K)
        a = ints(shape, seed + 1, -4, 4).float() if self.exact else randn(shape, seed + 1) * torch.exp(randn((shape[0], 1), seed + 7))
        a = place(a.to(self.tin), pad, offset, nan)
        self.a = a.t() if a_major == "m" else a
        q = ints((K, N), seed + 2, -4 if self.exact else -128, 4 if self.exact else 127)
        self.q = place(q.to(torch.int8), pad, offset).t()
        s = 2.0 ** ints((K,), seed + 3, -1, 1).float() if self.exact else torch.exp(randn((K,), seed + 3)) / 100
        self.s = s.cuda()
        self.c = place(ints((M, N), seed + 4, -9, 9).to(self.tout), pad if pad is None else pad + c_pad, offset)

    def reference(self, accumulate):
        a, x = self.a.double(), (self.s.double()[:, None] * self.q.t().double())
        ref, S, K = a @ x, a.abs() @ x.abs(), a.shape[1]
        narrow = self.tout != F32
        E = ((K if narrow else 3 * K) + 2) * 2.0 ** -24 * S
        if narrow:
            E = E + torch.finfo(self.tin).eps / 2 * S
            if self.tin == F16:
                E = E + 2.0 ** -25 * a.abs().sum(1, keepdim=True)
        if accumulate:
            ref = ref + self.c.double()
            E = E + 2.0 ** -24 * (S + self.c.double().abs())
        return ref, E

    def run(self, accumulate=False):
        ref, E = self.reference(accumulate)
        edge = around(self.c)
        assert g.gemm_i8_grad(self.a, self.q, self.s, self.c, accumulate=accumulate) is self.c
        torch.cuda.synchronize()
        assert torch.equal(edge, around(self.c))
        if self.exact:
            want = ref.float().to(self.tout)
            assert torch.equal(self.c, want), ((self.c != want).sum(), (self.c != want).nonzero()[0].tolist())
            return
        tol = E + torch.finfo(self.tout).eps / 2 * (ref.abs() + E) + (2.0 ** -25 if self.tout == F16 else 0)
        diff = (self.c.double() - ref).abs()
        bad = ~(diff <= tol)
        assert not bad.any(), (int(bad.sum()), float((diff / tol).max()), bad.nonzero()[0].tolist())


GRADIENTS = [(1, 1, 1), (2, 3, 5), (16, 16, 32), (17, 33, 40), (64, 64, 64), (1, 130, 100), (65, 66, 67), (128, 128, 128),
             (130, 250, 31), (40, 300, 1000), (129, 257, 515), (256, 256, 64), (257, 300, 200), (520, 264, 1100)]


@pytest.mark.parametrize("dtype", PAIRS)
@pytest.mark.parametrize("a_major", "mk")
@pytest.mark.parametrize("pad,offset", [(0, 0), (16, 0), (1, 0), (0, 3), (6, 2)])
def test_gradients(dtype, a_major, pad, offset):
    for i, (M, N, K) in enumerate(GRADIENTS):
        if pad == 16:           # aligned rows with room for whole chunks
            M, N, K = -(-M // 16) * 16, -(-N // 16) * 16, (K if a_major == "m" else -(-K // 16) * 16)
        say(dtype, a_major, pad, offset, M, N, K)
        Gradient(M, N, K, dtype, a_major, pad, offset, seed=10 * i).run(accumulate=i % 2 == 1)
        Gradient(M, N, K, dtype, a_major, pad, offset, "int", seed=10 * i).run(accumulate=i % 2 == 0)


@pytest.mark.parametrize("dtype", PAIRS)
@pytest.mark.parametrize("a_major", "mk")
def test_gradient_with_an_unaligned_output(dtype, a_major):
    for M, N, K in ((64, 80, 96), (272, 304, 256)):
        x = Gradient(M, N, K, dtype, a_major)
        x.c = place(x.c.cpu(), 1, 1)
        x.run()
        x.run(accumulate=True)


@pytest.mark.parametrize("dtype", PAIRS)
@pytest.mark.parametrize("a_major", "mk")
def test_gradient_of_no_values(dtype, a_major):
    x = Gradient(40, 50, 0, dtype, a_major)
    old = x.c.clone()
    g.gemm_i8_grad(x.a, x.q, x.s, x.c, accumulate=True)
    assert torch.equal(x.c, old)
    g.gemm_i8_grad(x.a, x.q, x.s, x.c)
    assert bool((x.c == 0).all())


@pytest.mark.parametrize("dtype", PAIRS)
@pytest.mark.parametrize("a_major", "mk")
def test_what_is_not_a_number_stays_where_it_belongs(dtype, a_major):
    """A NaN of A reaches its row, a NaN scale everything; past K and past the
    rows' ends nothing counts."""
    for M, N, K in ((48, 40, 50), (288, 272, 129)):
        x = Gradient(M, N, K, dtype, a_major, pad=7)
        y = Gradient(M, N, K, dtype, a_major, pad=7)
        x.a[5, K - 1] = float("nan")
        x.a[7, 2] = float("inf")
        y.run()
        g.gemm_i8_grad(x.a, x.q, x.s, x.c)
        rest = [m for m in range(M) if m not in (5, 7)]
        assert x.c[5].isnan().all() and not torch.isfinite(x.c[7]).any() and torch.equal(x.c[rest], y.c[rest])
        y.s[K // 2] = float("nan")
        g.gemm_i8_grad(y.a, y.q, y.s, y.c)
        assert y.c.isnan().all()


# ---------------------------------------------------------------- every kernel

@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("name,M,N", cases.PRODUCTS + cases.PRODUCTS_UNALIGNED)
def test_every_product_kernel(dtype, name, M, N):
    aligned = not name.startswith("unaligned")
    for i, K in enumerate((1, 16, 100, 128, 255, 256, 257, 1041)):       # K odd and even, k-tiles whole and not
        say(name, M, N, K)
        Product(M, N, K, dtype, *((None, 0) if aligned else (1, 3)), seed=i).run()
    if aligned:
        Product(M, N, 384, dtype, None).run_epilogue(0.5, 0.25, True, g.GEMM_ACT_GELU)
        x = Product(M, N, 160, dtype, None)
        x.c = place(x.c.cpu(), 1, 1)                                        # C at any element
        x.run()
    else:
        Product(M, N, 384, dtype, 1, 3).run_epilogue(0.5, 0.25, True, g.GEMM_ACT_GELU)


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("aligned,M,N,K,rows,cols", cases.EDGES)
def test_thin_edges(dtype, aligned, M, N, K, rows, cols):
    at = (None, 0) if aligned else (1, 3)
    Product(M, N, K, dtype, *at).run()
    Product(M, N, K, dtype, *at, scaled=False, lo=-1).run()
    Product(M, N, K, dtype, *at).run_epilogue(0.5, 0.25, True, g.GEMM_ACT_GELU)


def _gradient_kernels():
    out = []
    for dtype in PAIRS:
        tin, tout = PAIRS[dtype]
        for aligned in (True, False):
            for name, M, N in cases.gradients(tout == F32, tout == F32 and tin != BF16, aligned):
                out.append(pytest.param(dtype, aligned, M, N, id=f"{dtype}-{name}-{'aligned' if aligned else 'not'}".replace(" ", "_")))
    return out


@pytest.mark.parametrize("dtype,aligned,M,N", _gradient_kernels())
@pytest.mark.parametrize("a_major", "mk")
def test_every_gradient_kernel(dtype, aligned, M, N, a_major):
    for i, K in enumerate((1, 32, 64, 131, 256, 520)):
        say(dtype, aligned, a_major, M, N, K)
        at = (None, 0) if aligned else (1, 3)
        Gradient(M, N, K, dtype, a_major, *at, seed=i).run(accumulate=i % 2 == 1)
        if i in (3, 5):
            Gradient(M, N, K, dtype, a_major, *at, "int", seed=i).run(accumulate=i == 3)
    if aligned:
        x = Gradient(M, N, 200, dtype, a_major, None)
        x.c = place(x.c.cpu(), 1, 1)
        x.run()
        x.run(accumulate=True)


# ---------------------------------------------------------------- together

def layer(dtype, out, T=200, IN=264, OUT=136, seed=0):
    """A layer's step: tokens and weights to 8 bits, the output, both gradients."""
    t = WIDE[dtype]
    x, w, dy = (randn(s, seed + i).to(t).cuda() for i, s in enumerate(((T, IN), (OUT, IN), (T, OUT))))
    q8 = lambda z: (torch.empty(z.shape, dtype=torch.int8, device="cuda"), torch.empty(z.shape[0], device="cuda"))
    s = dict(x=x, w=w, dy=dy, xq=q8(x), wq=q8(w), y=torch.empty((T, OUT), dtype=t, device="cuda"),
             dw=torch.empty((OUT, IN), dtype=WIDE[out], device="cuda"), dx=torch.empty((T, IN), dtype=t, device="cuda"),
             back=torch.empty_like(x))

    def step(stream=None):
        (xq, xs), (wq, ws) = s["xq"], s["wq"]
        g.quantize_rows(s["x"], xq, xs, stream=stream)
        g.quantize_rows(s["w"], wq, ws, stream=stream)
        g.gemm_i8(xq, wq, xs, ws, s["y"], stream=stream)
        g.gemm_i8_grad(s["dy"].t(), xq.t(), xs, s["dw"], stream=stream)
        g.gemm_i8_grad(s["dy"], wq.t(), ws, s["dx"], stream=stream)
        g.dequantize_rows(xq, xs, s["back"], stream=stream)

    s["step"] = step
    return s


OUTPUTS = ("y", "dw", "dx", "back")


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")])
def test_a_layers_step(dtype, out):
    """Values against the quantised layer's, gradients against differences of it."""
    s = layer(dtype, out)
    s["step"]()
    xq, xs = quantized(s["x"])
    wq, ws = quantized(s["w"])
    x, w, dy = xq.double() * xs.double()[:, None], wq.double() * ws.double()[:, None], s["dy"].double()
    eps = torch.finfo(WIDE[dtype]).eps
    assert torch.equal(s["xq"][0], xq) and torch.equal(s["wq"][0], wq)
    for got, want, bound in ((s["y"], x @ w.t(), x.abs() @ w.abs().t()), (s["dw"], dy.t() @ x, dy.abs().t() @ x.abs()),
                             (s["dx"], dy @ w, dy.abs() @ w.abs()), (s["back"], x, x.abs())):
        # at most a rounding of a factor, of the output, and 800 of the sum
        assert bool(((got.double() - want).abs() <= (1.01 * eps + 800 * 2.0 ** -24) * bound).all())
    # The layer's output is linear in the restored x and w: a difference along a
    # direction is the gradient's product with it.
    loss = lambda x, w: float(((x @ w.t()) * dy).sum())
    for name, z, f, bound in (("dx", x, lambda d: loss(x + d, w) - loss(x - d, w), dy.abs() @ w.abs()),
                              ("dw", w, lambda d: loss(x, w + d) - loss(x, w - d), dy.abs().t() @ x.abs())):
        d = randn(tuple(z.shape), 77).double().cuda()
        off = abs(f(d) / 2 - float((s[name].double() * d).sum()))
        assert off <= (1.01 * eps + 800 * 2.0 ** -24) * float((bound * d.abs()).sum())


@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
def test_captured_and_replayed(dtype, out):
    s, e = layer(dtype, out), layer(dtype, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s["step"]()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s["step"]()
    for i in range(4):
        for name in ("x", "w", "dy"):
            v = (randn(tuple(s[name].shape), 100 * i + len(name)) * (i + 1)).to(s[name].dtype).cuda()
            s[name].copy_(v)
            e[name].copy_(v)
        for name in OUTPUTS:
            s[name].fill_(7)
        graph.replay()
        e["step"]()
        torch.cuda.synchronize()
        for name in OUTPUTS:
            assert torch.equal(s[name], e[name]), (i, name)


def test_offsets_past_32_bits():
    """Rows far apart: 700 of them span 4.9 GB."""
    ld, M, K, N = 7_000_000, 700, 130, 48
    far = torch.empty(ld * M, dtype=torch.int8, device="cuda").as_strided((M, K), (ld, 1))
    wide = torch.empty(ld * M // 2, dtype=BF16, device="cuda").as_strided((M, K), (ld // 2, 1))
    x = randn((M, K), 1).to(BF16).cuda()
    wide.copy_(x)
    s = torch.empty(M, device="cuda")
    g.quantize_rows(wide, far, s)
    q, scales = quantized(x)
    assert torch.equal(far, q) and torch.equal(s, scales)
    wide.zero_()
    g.dequantize_rows(far, s, wide)
    assert torch.equal(wide, (q.float() * scales[:, None]).to(BF16))
    w, ws = quantized(randn((N, K), 2).cuda())
    c = torch.empty((M, N), device="cuda")
    g.gemm_i8(far, w, s, ws, c)
    assert torch.equal(c, (q.double() @ w.double().t()).float() * s[:, None] * ws)
    dy = ints((M, N), 3, -3, 3).to(BF16).cuda()
    near, away = torch.empty((N, K), device="cuda"), torch.empty((N, K), device="cuda")
    g.gemm_i8_grad(dy.t(), q.t(), s, near)
    g.gemm_i8_grad(dy.t(), far.t(), s, away)
    assert torch.equal(near, away)
    big = torch.empty(ld * M // 2, dtype=BF16, device="cuda").as_strided((M, N), (ld // 2, 1))
    big.copy_(dy)
    g.gemm_i8_grad(big.t(), q.t(), s, away)
    assert torch.equal(near, away)
    g.gemm_i8_grad(dy, w.t(), ws, wide)               # C far apart
    dx = torch.empty((M, K), dtype=BF16, device="cuda")
    g.gemm_i8_grad(dy, w.t(), ws, dx)
    assert torch.equal(wide, dx)


def test_on_another_stream():
    s, e = layer("bf16", "f32"), layer("bf16", "f32")
    e["step"]()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s["step"](stream=side)
    side.synchronize()
    assert all(torch.equal(s[n], e[n]) for n in OUTPUTS)


def test_refusals():
    z8 = lambda *s: torch.zeros(s, dtype=torch.int8, device="cuda")
    z = lambda *s, t=F32: torch.zeros(s, dtype=t, device="cuda")
    bad = [lambda: g.quantize_rows(z(4, 8), z8(4, 9), z(4)), lambda: g.quantize_rows(z(4, 8), z(4, 8), z(4)),
           lambda: g.quantize_rows(z(4, 8), z8(4, 8), z(3)), lambda: g.quantize_rows(z(4, 8, t=torch.float64), z8(4, 8), z(4)),
           lambda: g.quantize_rows(z(8, 4).t(), z8(4, 8), z(4)), lambda: g.quantize_rows(z(4, 8), z8(4, 8), z(8)[::2]),
           lambda: g.dequantize_rows(z8(4, 8), z(4, t=F16), z(4, 8)), lambda: g.dequantize_rows(z8(8, 4).t(), z(4), z(4, 8)),
           lambda: g.gemm_i8(z8(4, 8), z8(5, 9), z(4), z(5), z(4, 5)), lambda: g.gemm_i8(z8(4, 8), z(5, 8), z(4), z(5), z(4, 5)),
           lambda: g.gemm_i8(z8(4, 8), z8(5, 8), z(5), z(5), z(4, 5)), lambda: g.gemm_i8(z8(4, 8), z8(5, 8), z(4), z(5), z8(4, 5)),
           lambda: g.gemm_i8(z8(8, 4).t(), z8(5, 8), z(4), z(5), z(4, 5)), lambda: g.gemm_i8(z8(4, 8), z8(5, 8), z(4), z(5), z(5, 4).t()),
           lambda: g.gemm_i8(z8(4, 8), z8(5, 8), z(4), z(5), z(4, 5), bias=z(4)),
           lambda: g.gemm_i8_grad(z(4, 8), z8(5, 8), z(8), z(4, 5)), lambda: g.gemm_i8_grad(z(4, 8), z8(8, 5).t(), z(5), z(4, 5)),
           lambda: g.gemm_i8_grad(z(4, 8), z8(8, 5).t(), z(8), z(4, 5, t=BF16)),
           lambda: g.gemm_i8_grad(z(4, 8), z8(8, 5).t(), z(8), z(5, 4).t()), lambda: g.gemm_i8_grad(z(4, 8), z(8, 5).t(), z(8), z(4, 5)),
           lambda: g.gemm_i8(z8(4, 8), z8(5, 8), z(4), z(5), z(4, 5).cpu())]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            say("accepted", i)
    with pytest.raises(g.GemmError):
        g.gemm_i8(z8(4, 8), z8(5, 8), z(4), z(5), z(4, 5), activation=9)
    with pytest.raises(g.GemmError):
        g.gemm_i8(z8(1, 131072), z8(1, 131072), None, None, z(1, 1))
