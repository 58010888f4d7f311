"""A shared projection with an adapter per row, on the GPU, against its
definition in 64 bits.

Tolerance, element by element, with S1 = sum_k |a||b|, V_r = sum_k |a||down_r|
and S2 = |scale| sum_r V_r |up_r|: every sum of n terms is off by at most
(n + 2) 2^-24 of its magnitudes.  v enters the second product split in two
terms of the input type: off by 2^-22 of itself for fp16 (two roundings of
2^-11), 2^-16 for bf16 (two of 2^-8), not split in fp32; fp16 scales v by row, where the smaller term's
smallest step is 2^-24 against a row's largest value of 2^13, 2^-37 of the
row's largest V times sum |up|.  With 2R terms in the second sum, a rounding
for the scale (of the sum, or of v before it is split) and one for adding:
    E = (K + 2) 2^-24 S1 + ((K + 2) + (2R + 6)) 2^-24 S2 + split S2
and eps(out) / 2 (|ref| + E) for the last rounding (2^-25 for fp16 subnormals).
Integer inputs of at most 5 give integers that every step holds exactly.
"""
import random

import pytest
import torch

import dense_gemm_engineering_run_amd as g

pytestmark = pytest.mark.gpu

TYPES = {"f32": (torch.float32, torch.float32), "f16_f32": (torch.float16, torch.float32),
         "bf16_bf16": (torch.bfloat16, torch.bfloat16), "f16_f16": (torch.float16, torch.float16),
         "bf16_f32": (torch.bfloat16, torch.float32)}
SPLIT = {torch.float32: 0.0, torch.float16: 2.0 ** -22, torch.bfloat16: 2.0 ** -16}
SENTINEL = 77.0


def say(*a):
    print(*a, flush=True)


def values(shape, dtype, seed, kind="normal", std=1.0):
    gen = torch.Generator().manual_seed(seed)
    t = torch.randint(-5, 6, shape, generator=gen).float() if kind == "int5" else torch.randn(shape, generator=gen) * std
    return t.to(dtype).cuda()


def padded(t, pad, fill, offset=0):
    shape = list(t.shape)
    shape[-1] += pad
    n = 1
    for s in shape:
        n *= s
    flat = torch.full((n + offset,), fill, dtype=t.dtype, device=t.device)
    v = flat[offset:].view(shape)[..., :t.shape[-1]]
    v.copy_(t)
    return v


def ids_of(pattern, M, L, seed=0):
    rng = random.Random(seed)
    if pattern == "one":
        ids = [L - 1] * M
    elif pattern == "none":
        ids = [-1] * M
    elif pattern == "distinct":
        ids = [m % L for m in range(M)]
    elif pattern == "packed":
        ids = sorted(rng.randrange(-1, L) for _ in range(M))
    else:
        ids = [rng.choice([-1, L, 2 ** 31 - 1, -2 ** 31] + list(range(L)) * 3) for _ in range(M)]
    return torch.tensor(ids, dtype=torch.int32, device="cuda")


class Case:
    def __init__(self, M, N, K, L, R, dtype, ids="mixed", b_major="k", kind="normal", pad=0, offset=0, mixed=True,
                 scales=True, seed=0):
        self.tin, self.tout = TYPES[dtype]
        nan = float("nan")
        mk = lambda shape, s, std: padded(values(shape, self.tin, seed + s, kind, std), pad, nan, offset)
        self.a = mk((M, K), 1, 1.0)
        self.b = mk((N, K), 2, 0.3) if b_major == "k" else mk((K, N), 2, 0.3).t()
        self.down, self.up = mk((L, R, K), 3, 0.3), mk((L, N, R), 4, 0.3)
        self.c = padded(torch.full((M, N), SENTINEL, dtype=self.tout, device="cuda"), pad, SENTINEL, offset)
        self.ids = ids_of(ids, M, L, seed) if isinstance(ids, str) else torch.tensor(ids, dtype=torch.int32, device="cuda")
        rng = random.Random(seed)
        self.ranks = torch.tensor([rng.choice([R, R, R // 2, 1, 0, R + 9, -3]) if mixed else R for _ in range(L)],
                                  dtype=torch.int32, device="cuda") if mixed else None
        self.scales = torch.tensor([2.0 ** rng.randrange(-1, 3) for _ in range(L)], device="cuda") if scales else None
        self.dtype, self.exact = dtype, kind == "int5"
        need = g.gemm_lora_workspace_size(M, N, K, g.dtype_code(self.tin, self.tout), R)
        self.need = need
        # NaN all over: what the first kernel does not write must not count
        self.ws = torch.full((need // 4 + 16,), nan, device="cuda")

    def run(self, stream=None):
        return g.gemm_lora(self.a, self.b, self.c, self.down, self.up, self.ids, self.ws[:self.need // 4],
                           ranks=self.ranks, scales=self.scales, stream=stream)

    def reference(self):
        a, b = self.a.double(), self.b.double()
        ref, S1 = a @ b.t(), a.abs() @ b.abs().t()
        L, R, K = self.down.shape
        S2, fine = torch.zeros_like(ref), torch.zeros_like(ref)
        for i in sorted(set(self.ids.tolist())):
            if not 0 <= i < L:
                continue
            m = self.ids == i
            r = R if self.ranks is None else min(max(int(self.ranks[i]), 0), R)
            s = 1.0 if self.scales is None else float(self.scales[i])
            d, u = self.down[i, :r].double(), self.up[i, :, :r].double()
            ref[m] += s * ((a[m] @ d.t()) @ u.t())
            V = a[m].abs() @ d.abs().t()
            S2[m] += abs(s) * (V @ u.abs().t())
            if r:
                fine[m] += abs(s) * V.amax(1, keepdim=True) * u.abs().sum(1)
        E = (K + 2) * 2.0 ** -24 * S1 + (K + 2 + 2 * R + 6) * 2.0 ** -24 * S2 + SPLIT[self.tin] * S2
        if self.tin == torch.float16:
            E = E + 2.0 ** -37 * fine
        return ref, E

    def check(self, rows=None):
        ref, E = self.reference()
        got = self.c
        if rows is not None:
            ref, E, got = ref[rows], E[rows], got[rows]
        if self.exact:
            want = ref.float().to(self.tout)
            assert torch.equal(got, want), (int((got != want).sum()), (got != want).nonzero()[0].tolist())
            return
        out = self.tout
        tol = E + torch.finfo(out).eps / 2 * (ref.abs() + E) + (2.0 ** -25 if out == torch.float16 else 0)
        diff = (got.double() - ref).abs()
        bad = ~(diff <= tol)
        assert not bad.any(), (int(bad.sum()), float((diff / tol).max()), bad.nonzero()[0].tolist())


def run(*args, **kw):
    say(args, kw)
    x = Case(*args, **kw)
    before = x.c.clone()
    whole = x.c._base if x.c._base is not None else x.c
    padding, ws_end = whole.clone(), x.ws[x.need // 4:].clone()
    assert x.run() is x.c
    torch.cuda.synchronize()
    x.check()
    x.c.copy_(before)
    assert torch.equal(whole, padding), "written outside C"
    assert torch.equal(x.ws[x.need // 4:].isnan(), ws_end.isnan()), "written outside the workspace"


@pytest.mark.parametrize("ids", ["one", "none", "distinct", "packed", "mixed"])
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 130, 300])
@pytest.mark.parametrize("dtype", TYPES)
def test_rows(dtype, M, ids):
    run(M, 136, 264, 9, 24, dtype, ids=ids)


@pytest.mark.parametrize("K", [31, 32, 300, 1100])
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("dtype", TYPES)
def test_few_rows(dtype, pad, K):
    """The streaming kernels: every number of rows, order of B and last k-tile."""
    for M in (1, 12, 16, 24, 32, 50, 90):
        for b_major in "kn":
            run(M, 200, K, 5, 40, dtype, b_major=b_major, pad=pad)
            run(M, 33, K, 5, 136, dtype, b_major=b_major, pad=pad, ids="distinct", kind="int5")


@pytest.mark.parametrize("R", [1, 3, 8, 16, 31, 32, 33, 64, 65, 100, 128, 200])
@pytest.mark.parametrize("dtype", TYPES)
def test_ranks(dtype, R):
    run(70, 72, 200, 5, R, dtype, kind="int5")
    run(20, 72, 520, 5, R, dtype, b_major="n")


@pytest.mark.parametrize("N,K", [(1, 1), (1, 64), (7, 3), (64, 8), (65, 31), (129, 33), (257, 129), (300, 520)])
@pytest.mark.parametrize("b_major", "kn")
@pytest.mark.parametrize("dtype", TYPES)
def test_odd_widths(dtype, b_major, N, K):
    run(37, N, K, 6, 8, dtype, b_major=b_major, kind="int5")
    run(150, N, K, 6, 16, dtype, b_major=b_major, ids="packed")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (1, 0), (3, 1), (8, 1)])
def test_padded_and_unaligned(dtype, pad, offset):
    for b_major in "kn":
        run(40, 72, 104, 5, 16, dtype, b_major=b_major, pad=pad, offset=offset)
        run(200, 72, 104, 5, 24, dtype, b_major=b_major, pad=pad, offset=offset)


@pytest.mark.parametrize("dtype", ["bf16_bf16", "f16_f16", "f16_f32", "f32"])
@pytest.mark.parametrize("K", [40, 64, 72, 328])
def test_large_tiles(dtype, K):
    """Enough rows and columns for every tile, with every kind of last k-tile."""
    for b_major in "kn":
        run(2100, 2600, K, 5, 40, dtype, b_major=b_major, ids="packed", mixed=False)
        run(700, 1100, K, 7, 64, dtype, b_major=b_major, ids="mixed", kind="int5")
        run(300, 700, K, 7, 16, dtype, b_major=b_major, ids="packed")
        run(4000, 2601, K + 1, 5, 40, dtype, b_major=b_major, ids="packed", mixed=False)
        run(1500, 1501, K + 1, 7, 24, dtype, b_major=b_major, ids="mixed")
        run(300, 701, K + 1, 7, 16, dtype, b_major=b_major, ids="packed")


@pytest.mark.parametrize("R", [1, 4, 12, 100])
@pytest.mark.parametrize("dtype", TYPES)
def test_unaligned_up_beside_aligned_operands(dtype, R):
    """Rows of up of few columns, in every kernel of the aligned product."""
    for M, N in ((1, 72), (24, 72), (40, 136), (140, 136), (300, 520), (1500, 1504), (2100, 2600)):
        run(M, N, 264, 5, R, dtype, ids="mixed" if M < 1000 else "packed", mixed=R > 4)
    run(300, 520, 72, 5, R, dtype, b_major="n", kind="int5")


@pytest.mark.parametrize("dtype", TYPES)
def test_unaligned_c_beside_aligned_operands(dtype):
    for M, N in ((20, 73), (140, 137), (300, 521), (1500, 1501), (2100, 2601)):
        run(M, N, 264, 5, 16, dtype, ids="packed")


@pytest.mark.parametrize("M", [1, 48, 600])
@pytest.mark.parametrize("dtype", ["bf16_bf16", "f16_f16", "f32"])
def test_ranks_and_scales_may_be_left_out(dtype, M):
    run(M, 264, 264, 5, 32, dtype, mixed=False, scales=False)
    run(M, 264, 264, 5, 32, dtype, mixed=True, scales=False)


@pytest.mark.parametrize("R", [24, 27])
@pytest.mark.parametrize("M,N", [(40, 136), (300, 136), (2048, 2304)])
@pytest.mark.parametrize("dtype", TYPES)
def test_requests_do_not_see_each_other(dtype, M, N, R):
    """Infinities and NaN of one slot, of a row, and past a slot's rank."""
    x = Case(M, N, 200, 6, R, dtype, ids="mixed", mixed=False)
    x.ranks = torch.tensor([R, 10, R, 0, R, 3], dtype=torch.int32, device="cuda")
    x.down[2, 3, 5] = float("nan")
    x.up[4, 1] = float("inf")
    x.up[1, :, 10:] = float("nan")
    x.down[1, 10:] = float("inf")
    x.up[3] = float("nan")
    x.down[5, 3:] = float("nan")
    x.up[5, :, 3:] = float("inf")
    x.a[7] = float("inf")
    x.run()
    torch.cuda.synchronize()
    ok = (x.ids != 2) & (x.ids != 4)
    ok[7] = False
    assert ok.any() and (x.ids == 2).any() and (x.ids == 4).any()
    assert torch.isfinite(x.c[ok]).all()
    assert torch.isnan(x.c[x.ids == 2]).all()
    four = x.ids == 4
    four[7] = False
    assert not torch.isfinite(x.c[four][:, 1]).any() and torch.isfinite(x.c[four][:, 2:]).all()
    # past the rank nothing counts: the same values as with those columns cleared
    x.down[1, 10:], x.up[1, :, 10:], x.down[5, 3:], x.up[5, :, 3:], x.up[3] = 0, 0, 0, 0, 0
    x.check(ok)


def test_fp16_adapters_far_from_one():
    """v far above and below what fp16 holds: it is scaled row by row."""
    for up, down in ((1e-4, 200.0), (100.0, 3e-6), (1.0, 1e-3)):
        x = Case(50, 72, 264, 4, 16, "f16_f32", mixed=False, scales=False)
        x.down.copy_(x.down * down)
        x.a.copy_(x.a * 30)
        x.up.copy_(x.up * up)
        x.b.zero_()
        x.run()
        torch.cuda.synchronize()
        x.check()
        assert (x.c[(x.ids >= 0) & (x.ids < 4)] != 0).any()


def test_the_same_adapter_in_every_slot():
    x = Case(30, 72, 104, 1, 16, "bf16_bf16", ids=[0] * 30, mixed=False, scales=False)
    x.run()
    first = x.c.clone()
    x.down, x.up = x.down.expand(8, 16, 104), x.up.expand(8, 72, 16)
    x.ids = ids_of("distinct", 30, 8)
    x.run()
    assert torch.equal(first, x.c)


def test_no_adapters_is_the_plain_product():
    for L, R in ((0, 8), (3, 0)):
        x = Case(40, 72, 104, L, R, "bf16_f32", ids=[0] * 40, mixed=False, scales=False)
        x.run()
        x.check()
    x = Case(40, 72, 104, 2, 8, "bf16_f32", ids="mixed")
    code = g.dtype_code(x.tin, x.tout)
    assert g.gemm_run_lora(40, 72, 104, "k", "k", "n", code, x.a.data_ptr(), x.b.data_ptr(), x.c.data_ptr(), 104, 104,
                           72, None, 0, 0, torch.cuda.current_stream().cuda_stream) == 0
    x.ids.fill_(-1)
    torch.cuda.synchronize()
    x.check()
    a, b, c = torch.zeros((4, 0), device="cuda"), torch.zeros((5, 0), device="cuda"), torch.ones((4, 5), device="cuda")
    g.gemm_lora(a, b, c, torch.zeros((2, 3, 0), device="cuda"), torch.ones((2, 5, 3), device="cuda"),
                torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda"))
    assert (c == 0).all()


@pytest.mark.parametrize("M", [1, 64, 500])
def test_repeated_calls_give_the_same_bits(M):
    x = Case(M, 1032, 520, 9, 64, "bf16_bf16")
    x.run()
    first = x.c.clone()
    for _ in range(4):
        x.ws.fill_(float("nan"))
        x.run()
        assert torch.equal(x.c, first)


def test_a_row_does_not_depend_on_its_neighbours():
    """The same request alone and in a batch of others: within the tolerance
    of both, and bit for bit when only the others' adapters change."""
    x = Case(48, 264, 520, 6, 32, "bf16_f32", ids="distinct", mixed=False)
    x.run()
    first = x.c.clone()
    x.ids[1:] = 5 - x.ids[1:]
    x.down[1:] *= 2
    x.run()
    assert torch.equal(first[0], x.c[0])


def test_two_streams_with_workspaces_of_their_own():
    xs = [Case(200, 520, 264, 5, 32, "bf16_bf16", seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in xs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for x, s in zip(xs, streams):
            x.run(stream=s)
    torch.cuda.synchronize()
    for x in xs:
        x.check()


def test_graph_takes_the_ids_of_each_replay():
    x = Case(80, 264, 264, 7, 32, "bf16_bf16", mixed=True)
    x.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.run()
    for i, pattern in enumerate(["one", "none", "distinct", "packed", "mixed"]):
        x.ids.copy_(ids_of(pattern, 80, 7, i))
        x.a.copy_(values(x.a.shape, x.tin, 50 + i))
        x.ws.fill_(float("nan"))
        x.c.fill_(SENTINEL)
        graph.replay()
        torch.cuda.synchronize()
        got = x.c.clone()
        x.check()
        x.run()
        torch.cuda.synchronize()
        assert torch.equal(got, x.c), pattern


def test_slots_past_32_bits():
    """Slots over 4 GiB apart, and rows of A over 4 GiB into it."""
    L, R, K, N = 600, 64, 65536, 40
    down = torch.zeros((L, R, K), dtype=torch.bfloat16, device="cuda")
    up = torch.zeros((L, N, R), dtype=torch.bfloat16, device="cuda")
    for i in (0, 3, 599):
        down[i] = values((R, K), torch.bfloat16, i, "int5") * (torch.arange(K, device="cuda") % 64 == 0)
        up[i] = values((N, R), torch.bfloat16, i + 1, "int5")
    M = 40000
    a = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    a[-20:] = values((20, K), torch.bfloat16, 9, "int5") * (torch.arange(K, device="cuda") % 64 == 0)
    b = values((N, K), torch.bfloat16, 10, "int5")
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    ids[-20:] = torch.tensor([599, 0, 3, 599] * 5, dtype=torch.int32, device="cuda")
    c = torch.full((M, N), SENTINEL, device="cuda")
    ws = torch.empty(g.gemm_lora_workspace_size(M, N, K, g.DTYPE_BF16_F32, R), dtype=torch.uint8, device="cuda")
    g.gemm_lora(a, b, c, down, up, ids, ws)
    x = a[-20:].double()
    ref = x @ b.double().t()
    for m in range(20):
        i = int(ids[M - 20 + m])
        ref[m] += up[i].double() @ (down[i].double() @ x[m])
    # v reaches 25 * 1024 < 2^16, the sums 25 * 1024 * (5 * 64 + 1) < 2^24
    assert torch.equal(c[-20:].double(), ref) and (c[:-20] == 0).all()


def test_adapted_attention_projections_of_a_batch():
    """Three adapted projections as a decoder uses them (a prompt and single
    tokens in one batch, one workspace for all), then the plain product on the
    result, against 64 bits."""
    T, H = 90, 128
    ids = torch.tensor([0] * 40 + [-1] * 20 + [2] * 28 + [1, 3], dtype=torch.int32, device="cuda")
    x = values((T, H), torch.float32, 1)
    ws = torch.empty(g.gemm_lora_workspace_size(T, H, H, g.DTYPE_F32, 16), dtype=torch.uint8, device="cuda")
    outs, refs = [], []
    for s in range(3):
        w, down, up = values((H, H), torch.float32, 10 + s, std=H ** -0.5), values((4, 16, H), torch.float32, 20 + s, std=H ** -0.5), \
            values((4, H, 16), torch.float32, 30 + s, std=0.25)
        outs.append(g.gemm_lora(x, w, torch.empty((T, H), device="cuda"), down, up, ids, ws))
        ref = x.double() @ w.double().t()
        for m in range(T):
            if ids[m] >= 0:
                i = int(ids[m])
                ref[m] += up[i].double() @ (down[i].double() @ x[m].double())
        refs.append(ref)
    scores = g.gemm(outs[0], outs[1], torch.empty((T, T), device="cuda"))
    y = g.gemm(torch.softmax(scores / H ** 0.5, 1), outs[2].t(), torch.empty((T, H), device="cuda"))
    want = torch.softmax(refs[0] @ refs[1].t() / H ** 0.5, 1) @ refs[2]
    # five products of at most 160 terms each on values of order one, carried
    # through a softmax whose arguments are of order sqrt(H) <= 16: 5 * 160 * 16 * 2^-24
    assert float((y.double() - want).norm()) <= 5 * 160 * 16 * 2.0 ** -24 * float(want.norm())


def test_torch_entry_point_refuses():
    x = Case(8, 16, 32, 3, 8, "bf16_bf16")
    call = lambda **kw: g.gemm_lora(**{**dict(a=x.a, b=x.b, c=x.c, down=x.down, up=x.up, ids=x.ids, workspace=x.ws,
                                              ranks=x.ranks, scales=x.scales), **kw})
    for kw in (dict(b=x.b.float()), dict(up=x.up.float()), dict(ids=x.ids.long()), dict(ids=x.ids[:4]),
               dict(ranks=x.ranks[:1]), dict(scales=x.scales.double()), dict(scales=x.scales[:2]), dict(c=x.c[:4]),
               dict(up=x.up[:2]), dict(down=x.down[:, :4]), dict(a=x.a.t().contiguous().t()), dict(ids=x.ids.cpu()),
               dict(workspace=x.ws[::2]), dict(down=x.down.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(g.GemmError) as e:
        call(workspace=x.ws[:1])
    assert e.value.status == g.GEMM_ERR_WORKSPACE
