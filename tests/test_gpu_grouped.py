"""Grouped products on the GPU against their definition in 64 bits.

Tolerance, element by element.  The products of 16-bit inputs are exact in
fp32, those of fp32 inputs off by 2^-24 of themselves; a sum of K terms in any
order is off by at most K 2^-24 of the sum of their magnitudes (to first
order), the last rounding by half a step of the output type.  With
S = sum_k |a| |b|: (K + 2) 2^-24 S + eps(out) / 2 (|ref| + (K + 2) 2^-24 S).
fp16 results may be subnormal: half their step, 2^-25, is added.
Integer inputs of at most 5 in magnitude have one result in every order, and
it has to come out bit for bit.
"""
import numpy as np
import pytest
import torch

import dense_gemm_engineering_run_amd as g

pytestmark = pytest.mark.gpu

TYPES = {"f32": (torch.float32, torch.float32), "f16_f32": (torch.float16, torch.float32),
         "bf16_bf16": (torch.bfloat16, torch.bfloat16), "f16_f16": (torch.float16, torch.float16),
         "bf16_f32": (torch.bfloat16, torch.float32)}
SENTINEL = 77.0


def say(*a):
    print(*a, flush=True)


def ends_of(lens):
    return torch.tensor(np.cumsum(lens), dtype=torch.int32, device="cuda")


def ranges(ends, rows):
    """[start, end) of every group: the running maximum of the clamped ends."""
    out, top = [], 0
    for e in ends.tolist():
        e = max(top, min(max(e, 0), rows))
        out.append((top, e))
        top = e
    return out


def values(shape, dtype, seed, kind="normal"):
    gen = torch.Generator().manual_seed(seed)
    if kind == "int5":
        t = torch.randint(-5, 6, shape, generator=gen).float()
    else:
        t = torch.randn(shape, generator=gen)
    return t.to(dtype).cuda()


def padded(t, pad, fill, offset=0):
    """The same matrix (or matrices) with `pad` more elements per row holding
    `fill`, starting `offset` elements into its allocation."""
    shape = list(t.shape)
    shape[-1] += pad
    n = int(np.prod(shape))
    flat = torch.full((n + offset,), fill, dtype=t.dtype, device=t.device)
    v = flat[offset:].view(shape)[..., :t.shape[-1]]
    v.copy_(t)
    return v


def tolerance(S, ref, K, out):
    acc = (K + 2) * 2.0 ** -24 * S
    return acc + torch.finfo(out).eps / 2 * (ref.abs() + acc) + (2.0 ** -25 if out == torch.float16 else 0)


def check(got, ref, S, K, exact):
    out = got.dtype
    if exact:
        want = ref.to(torch.float32).to(out)
        assert torch.equal(got, want), int((got != want).sum())
        return
    diff = (got.double() - ref).abs()
    tol = tolerance(S, ref, K, out)
    bad = ~(diff <= tol)
    assert not bad.any(), (int(bad.sum()), float(diff.max()), bad.nonzero()[0].tolist())


def check_rows(a, b, ends, c, before, exact):
    """All of c: the groups' rows against the definition, the others unchanged."""
    K = a.shape[1]
    top = 0
    for i, (s, e) in enumerate(ranges(ends, a.shape[0])):
        if e > s:
            x, w = a[s:e].double(), b[i].double()
            check(c[s:e], x @ w.t(), x.abs() @ w.abs().t(), K, exact)
        top = e
    assert torch.equal(c[top:], before[top:])


def check_k(a, b, ends, c, before, accumulate, exact):
    K = a.shape[1]
    for i, (s, e) in enumerate(ranges(ends, K)):
        x, w = a[:, s:e].double(), b[:, s:e].double()
        ref, S = x @ w.t(), x.abs() @ w.abs().t()
        if accumulate:
            ref, S = ref + before[i].double(), S + before[i].double().abs()
        check(c[i], ref, S, e - s + 1, exact)


def rows_case(lens, N, K, dtype, b_major, kind="normal", left=0, pad=0, offset=0, seed=0, c_pad=None):
    tin, tout = TYPES[dtype]
    M, G = sum(lens) + left, len(lens)
    a = padded(values((M, K), tin, seed, kind), pad, float("nan"), offset)
    b = values((G, N, K), tin, seed + 1, kind)
    if b_major == "n":
        b = padded(b.transpose(1, 2).contiguous(), pad, float("nan"), offset).transpose(1, 2)
    else:
        b = padded(b, pad, float("nan"), offset)
    c = padded(torch.full((M, N), SENTINEL, dtype=tout, device="cuda"), pad if c_pad is None else c_pad, SENTINEL, offset)
    return a, b, ends_of(lens), c


def k_case(lens, M, N, dtype, c_major, kind="normal", left=0, pad=0, offset=0, seed=0):
    tin, tout = TYPES[dtype]
    K, G = sum(lens) + left, len(lens)
    a = padded(values((K, M), tin, seed, kind), pad, float("nan"), offset).t()
    b = padded(values((K, N), tin, seed + 1, kind), pad, float("nan"), offset).t()
    c = values((G, M, N) if c_major == "n" else (G, N, M), tout, seed + 2, "int5")
    c = padded(c, pad, SENTINEL, offset)
    return a, b, ends_of(lens), c if c_major == "n" else c.transpose(1, 2)


def run_rows(lens, N, K, dtype, b_major, **kw):
    kind = kw.get("kind", "normal")
    say("rows", lens if len(lens) < 20 else f"{len(lens)} groups of {sum(lens)}", N, K, dtype, b_major, kw)
    a, b, ends, c = rows_case(lens, N, K, dtype, b_major, **kw)
    before = c.clone()
    whole = c._base if c._base is not None else c
    padding = whole.clone()
    assert g.grouped_gemm(a, b, ends, c) is c
    torch.cuda.synchronize()
    check_rows(a, b, ends, c, before, kind == "int5")
    c.copy_(before)
    assert torch.equal(whole, padding), "written outside C"


def run_k(lens, M, N, dtype, c_major, accumulate=False, **kw):
    kind = kw.get("kind", "normal")
    say("k", lens if len(lens) < 20 else f"{len(lens)} groups of {sum(lens)}", M, N, dtype, c_major, accumulate, kw)
    a, b, ends, c = k_case(lens, M, N, dtype, c_major, **kw)
    before = c.clone()
    whole = c._base if c._base is not None else c
    padding = whole.clone()
    assert g.grouped_gemm_k(a, b, ends, c, accumulate=accumulate) is c
    torch.cuda.synchronize()
    check_k(a, b, ends, c, before, accumulate, kind == "int5")
    c.copy_(before)
    assert torch.equal(whole, padding), "written outside C"


LENS = {
    "one": [1],
    "ones": [1, 1, 0, 1, 0, 0, 2],
    "edges": [63, 64, 65, 0, 127, 128, 129, 1, 15, 16, 17],
    "wide": [255, 0, 256, 257, 3],
    "none": [0, 0, 0],
}


@pytest.mark.parametrize("lens", LENS, ids=list(LENS))
@pytest.mark.parametrize("b_major", "kn")
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_lengths(dtype, b_major, lens):
    run_rows(LENS[lens], 136, 200, dtype, b_major, left=5)


@pytest.mark.parametrize("lens", LENS, ids=list(LENS))
@pytest.mark.parametrize("c_major", "nm")
@pytest.mark.parametrize("dtype", TYPES)
def test_k_lengths(dtype, c_major, lens):
    run_k(LENS[lens], 136, 200, dtype, c_major, left=5)
    run_k(LENS[lens], 136, 200, dtype, c_major, left=5, accumulate=True)


@pytest.mark.parametrize("N,K", [(1, 1), (1, 64), (7, 3), (64, 8), (65, 31), (129, 33), (257, 129), (300, 520)])
@pytest.mark.parametrize("b_major", "kn")
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_odd_widths(dtype, b_major, N, K):
    run_rows([3, 40, 0, 70], N, K, dtype, b_major, kind="int5")


@pytest.mark.parametrize("M,N", [(1, 1), (1, 64), (7, 3), (64, 8), (65, 31), (129, 33), (257, 129), (300, 520)])
@pytest.mark.parametrize("c_major", "nm")
@pytest.mark.parametrize("dtype", TYPES)
def test_k_odd_widths(dtype, c_major, M, N):
    run_k([3, 40, 0, 70], M, N, dtype, c_major, kind="int5")
    run_k([3, 40, 0, 70], M, N, dtype, c_major, kind="int5", accumulate=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (1, 0), (3, 1), (8, 1)])
def test_padded_and_unaligned(dtype, pad, offset):
    for b_major in "kn":
        run_rows([20, 0, 100, 33], 72, 104, dtype, b_major, pad=pad, offset=offset, left=2)
    for c_major in "nm":
        run_k([20, 0, 100, 33], 72, 104, dtype, c_major, pad=pad, offset=offset, left=2)


@pytest.mark.parametrize("dtype", TYPES)
def test_aligned_operands_with_an_unaligned_c(dtype):
    run_rows([300, 0, 40], 264, 136, dtype, "k", c_pad=1)
    run_rows([700, 600], 520, 136, dtype, "n", c_pad=1)


@pytest.mark.parametrize("dtype", TYPES)
def test_largest_tiles_with_an_unaligned_c(dtype):
    say("unaligned c", dtype)
    run_rows([700, 0, 1, 900, 511], 5400, 136, dtype, "k", c_pad=1, left=3)
    for accumulate in (False, True):
        a, b, ends, c = k_case([300, 0, 65], 2104, 2600, dtype, "n", left=3)
        c = padded(c, 1, SENTINEL, 1)
        before, whole = c.clone(), c._base
        padding = whole.clone()
        g.grouped_gemm_k(a, b, ends, c, accumulate=accumulate)
        torch.cuda.synchronize()
        check_k(a, b, ends, c, before, accumulate, False)
        c.copy_(before)
        assert torch.equal(whole, padding), "written outside C"


@pytest.mark.parametrize("dtype", TYPES)
def test_more_groups_than_a_wave(dtype):
    rng = np.random.default_rng(7)
    lens = [int(x) for x in rng.integers(0, 9, size=200)]
    lens[64] = lens[127] = lens[128] = 0
    run_rows(lens, 72, 64, dtype, "k", left=3)
    run_k(lens, 40, 72, dtype, "n", left=3)


@pytest.mark.parametrize("dtype", ["bf16_bf16", "f16_f32", "f32"])
@pytest.mark.parametrize("lens", [[700, 0, 1, 900, 511], [2100], [128] * 16, [40] * 48])
def test_large_tiles(dtype, lens):
    """Enough rows and columns for the largest tiles, whole and partial."""
    for b_major in "kn":
        run_rows(lens, 1100, 328, dtype, b_major, left=9)
        run_rows(lens, 1024, 1024, dtype, b_major, kind="int5")
    run_k(lens, 1100, 776, dtype, "n", left=9)
    run_k(lens, 1024, 1024, dtype, "m", kind="int5")
    run_k(lens, 1024, 1024, dtype, "n", kind="int5", accumulate=True)


@pytest.mark.parametrize("dtype", ["bf16_bf16", "f16_f32", "f16_f16", "f32"])
@pytest.mark.parametrize("K", [40, 64, 72, 192, 328])
def test_wide_outputs(dtype, K):
    """Enough columns for the largest tile whatever the groups' lengths, with
    every kind of last k-tile."""
    for b_major in "kn":
        run_rows([700, 0, 1, 900, 511], 5400, K, dtype, b_major, left=3)      # 256x256
        run_rows([150, 0, 97, 128, 129] * 4, 2100, K, dtype, b_major, left=3)  # 128x256
        run_rows([40] * 48, 1100, K, dtype, b_major, left=3)                   # 64x128
        run_rows([600, 0, 300], 520, K, dtype, b_major, left=3)                # 128x128
    run_k([K, 0, 3, 2 * K, 65], 1100, 2104, dtype, "n", left=3)
    run_k([K, 0, 3, 2 * K, 65], 1100, 2104, dtype, "m", left=3, accumulate=True)


@pytest.mark.parametrize("lens,N", [([48], 1000), ([20] * 100, 300), ([48] * 70, 300), ([100] * 4, 1500),
                                    ([128] * 32, 500), ([100, 156] * 30, 500), ([300] * 16, 700)])
@pytest.mark.parametrize("dtype", TYPES)
def test_every_height_of_tile(dtype, lens, N):
    """Few and many tiles of each height: 32x64, 64x128, 128x64, 128x128, 128x256."""
    for b_major in "kn":
        run_rows(lens, N, 200, dtype, b_major, left=3)
        run_rows([n // 2 for n in lens] + lens, N, 72, dtype, b_major, kind="int5")
        run_rows(lens, N + 1, 201, dtype, b_major, left=3)


@pytest.mark.parametrize("M,N", [(129, 255), (301, 1023)])
@pytest.mark.parametrize("dtype", TYPES)
def test_unaligned_gradients_of_matrices(dtype, M, N):
    for c_major in "nm":
        run_k([65, 0, 1, 300, 129], M, N, dtype, c_major, left=3)
        run_k([64, 128, 63], M, N, dtype, c_major, kind="int5", accumulate=True, pad=2)


@pytest.mark.parametrize("ends", [[50, 20, 90], [-5, 30, 30], [1000, 40, 99], [100, 100, 100], [-1, -1, -1],
                                  [2 ** 31 - 1, -2 ** 31, 5]])
def test_ends_that_do_not_ascend_stay_in_bounds(ends):
    for dtype in ("bf16_bf16", "f32"):
        tin, tout = TYPES[dtype]
        a, b = values((100, 64), tin, 1), values((3, 72, 64), tin, 2)
        c = torch.full((120, 72), SENTINEL, dtype=tout, device="cuda")
        e = torch.tensor(ends, dtype=torch.int32, device="cuda")
        before = c.clone()
        g.grouped_gemm(a, b, e, c[:100])
        check_rows(a, b, e, c[:100], before[:100], False)
        assert torch.equal(c[100:], before[100:])
        cg = torch.full((3, 64, 72), SENTINEL, dtype=tout, device="cuda")
        y = values((100, 72), tin, 3)
        g.grouped_gemm_k(a.t(), y.t(), e, cg)
        check_k(a.t(), y.t(), e, cg, cg, False, False)


@pytest.mark.parametrize("N,K", [(136, 200), (1040, 264)])
@pytest.mark.parametrize("dtype", ["f16_f16", "bf16_f32", "f32"])
def test_groups_do_not_see_each_other(dtype, N, K):
    """NaN and infinities in one group's rows or matrix stay in that group."""
    lens = [40, 3, 0, 300, 130]
    for b_major in "kn":
        a, b, ends, c = rows_case(lens, N, K, dtype, b_major, left=4)
        a[sum(lens):] = float("nan")          # rows past the last end
        b[2] = float("inf")                   # a group without rows
        b[1, 0, 0] = float("nan")
        a[50, 1] = float("inf")               # in the fourth group
        before = c.clone()
        g.grouped_gemm(a, b, ends, c)
        ok = torch.ones(len(c), dtype=torch.bool, device="cuda")
        ok[40:43] = ok[50] = False
        assert torch.isfinite(c[ok]).all()
        assert torch.isnan(c[40:43, 0]).all() and not torch.isfinite(c[50]).any()
        assert torch.equal(c[sum(lens):], before[sum(lens):])
    a, b, ends, c = k_case(lens, N, 136, dtype, "n", left=4)
    a[:, sum(lens):] = float("nan")
    b[:, sum(lens):] = float("nan")
    b[:, 41] = float("nan")                   # in the second group
    g.grouped_gemm_k(a, b, ends, c)
    assert torch.isfinite(c[[0, 2, 3, 4]]).all() and torch.isnan(c[1]).all()


def test_no_k_writes_zeros():
    a, b = torch.zeros((6, 0), device="cuda"), torch.zeros((2, 5, 0), device="cuda")
    c = torch.full((6, 5), SENTINEL, device="cuda")
    g.grouped_gemm(a, b, ends_of([2, 3]), c)
    assert (c[:5] == 0).all() and (c[5:] == SENTINEL).all()
    cg = torch.full((2, 6, 5), SENTINEL, device="cuda")
    g.grouped_gemm_k(a, torch.zeros((5, 0), device="cuda"), ends_of([0, 0]), cg, accumulate=True)
    assert (cg == SENTINEL).all()
    g.grouped_gemm_k(a, torch.zeros((5, 0), device="cuda"), ends_of([0, 0]), cg)
    assert (cg == 0).all()


def test_one_matrix_for_all_groups():
    a = values((90, 64), torch.bfloat16, 1)
    w = values((72, 64), torch.bfloat16, 2)
    c = torch.zeros((90, 72), dtype=torch.bfloat16, device="cuda")
    ends = ends_of([30, 20, 40])
    g.grouped_gemm(a, w.expand(3, 72, 64), ends, c)
    check_rows(a, w.expand(3, 72, 64), ends, c, c, False)


@pytest.mark.parametrize("dtype", ["bf16_bf16", "f32"])
def test_repeated_calls_give_the_same_bits(dtype):
    a, b, ends, c = rows_case([300, 5, 0, 700], 520, 392, dtype, "k")
    g.grouped_gemm(a, b, ends, c)
    first = c.clone()
    ga, gb, _, gc = k_case([300, 5, 0, 700], 520, 392, dtype, "n")
    g.grouped_gemm_k(ga, gb, ends, gc)
    kfirst = gc.clone()
    for _ in range(4):
        g.grouped_gemm(a, b, ends, c)
        g.grouped_gemm_k(ga, gb, ends, gc)
        assert torch.equal(c, first) and torch.equal(gc, kfirst)


def test_on_another_stream():
    a, b, ends, c = rows_case([30, 0, 90], 136, 200, "bf16_bf16", "k")
    before = c.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g.grouped_gemm(a, b, ends, c, stream=s)
    s.synchronize()
    check_rows(a, b, ends, c, before, False)


def test_graph_takes_the_ends_of_each_replay():
    """One capture, replayed with other ends and other tokens."""
    lens = [30, 0, 90, 200]
    a, b, ends, c = rows_case(lens, 136, 200, "bf16_bf16", "k")
    dw = torch.zeros((4, 136, 200), dtype=torch.float32, device="cuda")
    dx = torch.zeros_like(a)
    dy = values(c.shape, torch.bfloat16, 9)

    def step():
        g.grouped_gemm(a, b, ends, c)
        g.grouped_gemm(dy, b.transpose(1, 2), ends, dx)
        g.grouped_gemm_k(dy.t(), a.t(), ends, dw)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i, l in enumerate([lens, [320, 0, 0, 0], [1, 2, 3, 4], [0, 0, 0, 0], [80, 80, 80, 80]]):
        ends.copy_(ends_of(l))
        a.copy_(values(a.shape, torch.bfloat16, 20 + i))
        for t in (c, dx, dw):
            t.fill_(SENTINEL)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (c, dx, dw)]
        for t in (c, dx, dw):
            t.fill_(SENTINEL)
        before = c.clone()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, (c, dx, dw))), l
        check_rows(a, b, ends, c, before, False)
        check_k(dy.t(), a.t(), ends, dw, dw, False, False)


def test_offsets_past_32_bits():
    """Rows and k over 4 GiB into A, and over 4 GiB into C."""
    K, M = 4096, 700_000
    base = values((997, K), torch.bfloat16, 3, "int5")
    a = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    for s in range(0, M, 997):
        a[s:s + 997] = base[:min(997, M - s)]
    lens = [10, M - 500, 0, 300]
    ends = ends_of(lens)
    b = values((4, 24, K), torch.bfloat16, 4, "int5")
    c = torch.full((M, 24), SENTINEL, dtype=torch.float32, device="cuda")
    g.grouped_gemm(a, b, ends, c)
    for i, (s, e) in enumerate(ranges(ends, M)):
        for lo, hi in ((s, min(e, s + 997)), (max(s, e - 997), e)):
            assert torch.equal(c[lo:hi].double(), a[lo:hi].double() @ b[i].double().t())
    assert (c[sum(lens):] == SENTINEL).all()
    # the same tokens as the summed index: 300 of them at the far end
    y = torch.zeros((M, 16), dtype=torch.bfloat16, device="cuda")
    y[-700:] = values((700, 16), torch.bfloat16, 5, "int5")
    ends2 = ends_of([M - 600, 300, 0, 300])
    cg = torch.zeros((4, 16, K), dtype=torch.float32, device="cuda")
    g.grouped_gemm_k(y.t(), a.t(), ends2, cg)
    for i, (s, e) in enumerate(ranges(ends2, M)):
        s = max(s, M - 700)
        assert torch.equal(cg[i].double(), y[s:e].double().t() @ a[s:e].double())
    # C over 4 GiB: 700,000 x 4096 of fp32
    w = values((2, K, 16), torch.bfloat16, 6, "int5")
    out = torch.empty((M, K), dtype=torch.float32, device="cuda")
    g.grouped_gemm(y, w, ends_of([M - 600, 600]), out)
    assert torch.equal(out[-600:].double(), y[-600:].double() @ w[1].double().t())
    assert torch.equal(out[-700:-600].double(), y[-700:-600].double() @ w[0].double().t())
    assert (out[:1000] == 0).all()


def test_mixture_of_experts_layer_and_its_gradients():
    """Two grouped products with an activation between, their gradients by the
    same entry points, against autograd of the same layer in 64 bits and
    against a difference quotient of the 64-bit loss."""
    T, E, H, F = 96, 5, 64, 136
    lens = [20, 0, 41, 5, 30]
    ends = ends_of(lens)
    x, w1, w2 = (values(s, torch.float32, i) * k for i, (s, k) in enumerate(
        [((T, H), 1.0), ((E, F, H), H ** -0.5), ((E, H, F), F ** -0.5)]))
    dy = values((T, H), torch.float32, 5)
    h = torch.empty((T, F), device="cuda")
    y = torch.empty((T, H), device="cuda")
    g.grouped_gemm(x, w1, ends, h)
    act = torch.relu(h)
    g.grouped_gemm(act, w2, ends, y)
    dact, dx = torch.empty_like(h), torch.empty_like(x)
    g.grouped_gemm(dy, w2.transpose(1, 2), ends, dact)
    dw2 = g.grouped_gemm_k(dy.t(), act.t(), ends, torch.empty_like(w2))
    dh = dact * (h > 0)
    g.grouped_gemm(dh, w1.transpose(1, 2), ends, dx)
    dw1 = g.grouped_gemm_k(dh.t(), x.t(), ends, torch.empty_like(w1))

    def loss(x, w1, w2):
        total = 0
        for i, (s, e) in enumerate(ranges(ends, T)):
            total = total + ((torch.relu(x[s:e] @ w1[i].t()) @ w2[i].t()) * dy[s:e].double()).sum()
        return total

    ref = [t.double().requires_grad_() for t in (x, w1, w2)]
    loss(*ref).backward()
    for got, want in zip((dx, dw1, dw2), (t.grad for t in ref)):
        # sums of at most H + F + T products over two layers, each within 2^-24:
        # (136 + 136) 2^-24 of magnitudes a few times the norm
        assert float((got.double() - want).norm()) <= 272 * 2.0 ** -24 * 4 * float(want.norm())
    # the directional difference quotient: the loss is piecewise linear in each
    # argument, so away from the kinks the central difference is its slope
    for k, got in enumerate((dx, dw1, dw2)):
        d = values(got.shape, torch.float64, 30 + k)
        plus, minus = [t.detach().clone() for t in ref], [t.detach().clone() for t in ref]
        step = 1e-7
        plus[k] += step * d
        minus[k] -= step * d
        slope = float(loss(*plus) - loss(*minus)) / (2 * step)
        along = float((got.double() * d).sum())
        assert abs(slope - along) <= 1e-3 * float(got.double().norm() * d.norm()), k


def test_torch_entry_points_refuse():
    a, b, ends, c = rows_case([4, 4], 16, 32, "bf16_bf16", "k")
    for bad in (lambda: g.grouped_gemm(a, b.float(), ends, c), lambda: g.grouped_gemm(a, b, ends.long(), c),
                lambda: g.grouped_gemm(a, b, ends[:1], c), lambda: g.grouped_gemm(a, b, ends, c[:4]),
                lambda: g.grouped_gemm(a.t().contiguous().t(), b, ends, c),
                lambda: g.grouped_gemm(a, b, ends.cpu(), c), lambda: g.grouped_gemm(a, b, ends, c.half()),
                lambda: g.grouped_gemm(a[:, ::2], b[:, :, ::2], ends, c),
                lambda: g.grouped_gemm_k(a, a, ends, torch.zeros(2, 8, 8, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(g.GemmError) as e:
        g.grouped_gemm(a, b, ends, a[:, :16])
    assert e.value.status == g.GEMM_ERR_ALIAS
