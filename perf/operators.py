"""The grouped and low-rank-adapter products: cases, inputs, plain forms, exact values.

Three operators stand beside the dense product C = A * B^T:

  grouped    rows of A sorted by group (the tokens of a mixture of experts,
             sorted by expert); group g's rows times its own matrix B_g:
                 C[m][n] = sum_k A[m][k] B_g[n][k],   ends[g-1] <= m < ends[g]
             The forward product has B_g k-major (weights N x K); the gradient
             of the tokens is the same call with the weights read n-major.
  grouped_k  the gradient of the weights: the summed index is what is grouped,
                 C_g[m][n] = sum over the k of group g of A[m][k] B[n][k]
             with A and B the m/n-major views of two row-major token matrices.
  lora       a projection shared by all rows plus the low-rank adapter of each
             row's request:
                 C[m][n] = sum_k A[m][k] B[n][k]
                         + scale_i sum_r (sum_k A[m][k] down_i[r][k]) up_i[n][r],   i = ids[m]

With `own` false, run() computes them in elementary torch operations in fp32,
rounded once at the end; with `own` true it calls this repository's package.
"""
import math
import random

import torch

own = False

TYPES = {"f32": (torch.float32, torch.float32), "f16_f32": (torch.float16, torch.float32),
         "bf16_bf16": (torch.bfloat16, torch.bfloat16), "f16_f16": (torch.float16, torch.float16),
         "bf16_f32": (torch.bfloat16, torch.float32)}


def listed():
    return [
        # One decoding step of a few requests: 16 (token, expert) rows over 8
        # experts, mostly one to four rows each; the weights are the traffic.
        dict(name="grouped_decode_16x4096x4096_g8_bf16", op="grouped", M=16, N=4096, K=4096, G=8, b_major="k",
             dtype="bf16_bf16", skew=0.5, pad=0, route=1),
        # A small prompt over many small experts, some of them empty, rows left
        # over at the end of a padded buffer.
        dict(name="grouped_prompt_1000x1024x2048_g64_f16", op="grouped", M=1000, N=1024, K=2048, G=64, b_major="k",
             dtype="f16_f16", skew=1.0, pad=24, route=2),
        # A prefill or training batch, forward.
        dict(name="grouped_fwd_8192x4096x2048_g16_bf16", op="grouped", M=8192, N=4096, K=2048, G=16, b_major="k",
             dtype="bf16_bf16", skew=0.7, pad=0, route=3),
        # The largest: a long training batch over 8 experts.
        dict(name="grouped_fwd_32768x4096x4096_g8_bf16", op="grouped", M=32768, N=4096, K=4096, G=8, b_major="k",
             dtype="bf16_bf16", skew=0.3, pad=0, route=4),
        # The tokens' gradient: the same weights (4096 x 2048 each) read n-major.
        dict(name="grouped_dgrad_8192x2048x4096_g16_bf16", op="grouped", M=8192, N=2048, K=4096, G=16, b_major="n",
             dtype="bf16_bf16", skew=0.7, pad=0, route=3),
        # Single precision at odd sizes.
        dict(name="grouped_ragged_4095x2049x1028_g6_f32", op="grouped", M=4095, N=2049, K=1028, G=6, b_major="k",
             dtype="f32", skew=0.5, pad=0, route=5),
        # The weights' gradient of the forward case above, into fp32 gradients.
        dict(name="grouped_wgrad_4096x2048_t8192_g16_bf16_f32", op="grouped_k", M=4096, N=2048, K=8192, G=16,
             c_major="n", dtype="bf16_f32", skew=0.7, pad=0, route=3),
        # The weights' gradient of a small model with many experts and a short batch.
        dict(name="grouped_wgrad_512x256_t1000_g32_bf16", op="grouped_k", M=512, N=256, K=1000, G=32, c_major="n",
             dtype="bf16_bf16", skew=1.0, pad=0, route=6),
        # One request's next token through an adapted projection: latency.
        dict(name="lora_decode_1x4096x4096_r16_bf16", op="lora", M=1, N=4096, K=4096, L=8, R=16, rows="single",
             mixed=False, dtype="bf16_bf16", route=7),
        # A decoding batch of 64 requests, each with an adapter of its own rank
        # (some with none).
        dict(name="lora_decode_64x4096x4096_r64_f16", op="lora", M=64, N=4096, K=4096, L=48, R=64, rows="single",
             mixed=True, dtype="f16_f16", route=8),
        # Prompts of eight requests packed one behind the other.
        dict(name="lora_prefill_4096x4096x4096_r64_bf16", op="lora", M=4096, N=4096, K=4096, L=8, R=64, rows="packed",
             mixed=False, dtype="bf16_bf16", route=9),
        # A mixed batch (prompts and single tokens) at odd sizes, fp32 outputs.
        dict(name="lora_mixed_515x2056x1032_r24_f16_f32", op="lora", M=515, N=2056, K=1032, L=12, R=24, rows="mixed",
             mixed=True, dtype="f16_f32", route=10),
    ]


def _size(rng, lo, hi, step=1):
    """A size spread over the logarithm of [lo, hi], a multiple of `step`."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(step, v // step * step)


def draw(rng):
    op = rng.choice(["grouped", "grouped", "grouped_k", "lora", "lora"])
    # Widths are mostly multiples of 8 (one 16-byte load of 16-bit elements),
    # some are odd.
    step = rng.choice([8, 8, 64, 64, 1])
    route = rng.randrange(1 << 30)
    dtype = rng.choice(["bf16_bf16", "bf16_bf16", "f16_f16", "bf16_f32", "f16_f32", "f32"])
    N, K = _size(rng, 128, 8192, step), _size(rng, 128, 8192, step)
    # Weights of all groups stay below 2^29 elements and the flops below the
    # largest listed case's.
    G = min(_size(rng, 1, 128), max(1, (1 << 29) // (N * K)))
    M = _size(rng, 1, min(32768, max(1, (1 << 39) // (N * K * (8 if dtype == "f32" else 1)))))
    if op == "grouped":
        return dict(op=op, M=M, N=N, K=K, G=G, b_major=rng.choice("kkn"), dtype=dtype, skew=rng.uniform(0, 1.2),
                    pad=rng.choice([0, 0, 0, M // 10]), route=route)
    if op == "grouped_k":
        return dict(op=op, M=N, N=K, K=M, G=G, c_major=rng.choice("nnm"), dtype=dtype, skew=rng.uniform(0, 1.2),
                    pad=rng.choice([0, 0, 0, M // 10]), route=route)
    R = rng.choice([4, 8, 16, 16, 32, 64, 64, 128])
    return dict(op=op, M=M, N=N, K=K, L=_size(rng, 1, 64), R=R, rows=rng.choice(["single", "packed", "packed", "mixed"]),
                mixed=rng.choice([False, True]), dtype=dtype, route=route)


# ---------------------------------------------------------------- lengths and ids (host)

def group_ends(case):
    """Ends of the groups: `rows - pad` rows dealt out with log-normal weights."""
    rng = random.Random(case["route"])
    rows = (case["K"] if case["op"] == "grouped_k" else case["M"]) - case["pad"]
    w = [math.exp(case["skew"] * rng.gauss(0, 1)) for _ in range(case["G"])]
    counts = [0] * case["G"]
    if rows <= 2048:
        for g in rng.choices(range(case["G"]), weights=w, k=rows):
            counts[g] += 1
    else:
        total = sum(w)
        counts = [int(rows * x / total) for x in w]
        counts[rng.randrange(case["G"])] += rows - sum(counts)
    ends, e = [], 0
    for c in counts:
        e += c
        ends.append(e)
    return ends


def row_ids(case):
    """Adapter of each row (-1: none): a row per request, or packed prompts."""
    rng = random.Random(case["route"])
    M, L = case["M"], case["L"]

    def adapter():
        return -1 if rng.random() < 0.1 and M > 1 else rng.randrange(L)

    if case["rows"] == "single":
        return [adapter() for _ in range(M)]
    singles = M // 8 if case["rows"] == "mixed" else 0
    ids = [adapter() for _ in range(singles)]
    parts = min(8, M - singles)
    cuts = sorted(rng.sample(range(1, M - singles), parts - 1)) if parts > 1 else []
    for a, b in zip([0] + cuts, cuts + [M - singles]):
        ids += [adapter()] * (b - a)
    return ids


def adapter_ranks(case):
    rng = random.Random(case["route"] + 1)
    R = case["R"]
    return [max(1, R >> rng.randrange(3)) if case["mixed"] else R for _ in range(case["L"])]


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, std, dtype, g):
    """Normal values, made in pieces so that no fp32 copy of the whole is held."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    flat = t.view(-1)
    for i in range(0, flat.numel(), 1 << 27):
        n = min(1 << 27, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device="cuda") * std
    return t


def prepare(case, seed):
    g = _gen(seed)
    tin, tout = TYPES[case["dtype"]]
    M, N, K = case["M"], case["N"], case["K"]
    s = dict(case=case)
    if case["op"] == "lora":
        # Tokens of unit size, weights that keep it, adapters of a tenth of it.
        s["a"] = _normal((M, K), 1.0, tin, g)
        s["b"] = _normal((N, K), K ** -0.5, tin, g)
        s["down"] = _normal((case["L"], case["R"], K), K ** -0.5, tin, g)
        s["up"] = _normal((case["L"], N, case["R"]), 0.1 * case["R"] ** -0.5, tin, g)
        ids, ranks = row_ids(case), adapter_ranks(case)
        s["ids"] = torch.tensor(ids, dtype=torch.int32, device="cuda")
        s["ranks"] = torch.tensor(ranks, dtype=torch.int32, device="cuda")
        scales = [2.0 ** (i % 3) for i in range(case["L"])]
        s["scales"] = torch.tensor(scales, dtype=torch.float32, device="cuda")
        s["c"] = torch.zeros((M, N), dtype=tout, device="cuda")
        rows = {}
        for m, i in enumerate(ids):
            if i >= 0:
                rows.setdefault(i, []).append(m)
        s["by_adapter"] = [(i, ranks[i], scales[i], torch.tensor(r, device="cuda")) for i, r in sorted(rows.items())]
        if own:
            import dense_gemm_engineering_run_amd as gemm
            need = gemm.gemm_lora_workspace_size(M, N, K, gemm.dtype_code(tin, tout), case["R"])
            s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        return s
    ends = group_ends(case)
    s["ends_host"] = ends
    s["ends"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    if case["op"] == "grouped":
        s["a"] = _normal((M, K), 1.0, tin, g)
        shape = (case["G"], N, K) if case["b_major"] == "k" else (case["G"], K, N)
        b = _normal(shape, K ** -0.5, tin, g)
        s["b"] = b if case["b_major"] == "k" else b.transpose(1, 2)
        s["c"] = torch.zeros((M, N), dtype=tout, device="cuda")
    else:
        # Token-major matrices: gradients of the outputs and the layer's inputs.
        s["a"] = _normal((K, M), 0.02, tin, g).t()
        s["b"] = _normal((K, N), 1.0, tin, g).t()
        shape = (case["G"], M, N) if case["c_major"] == "n" else (case["G"], N, M)
        c = torch.zeros(shape, dtype=tout, device="cuda")
        s["c"] = c if case["c_major"] == "n" else c.transpose(1, 2)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import dense_gemm_engineering_run_amd as gemm
    op = s["case"]["op"]
    if op == "grouped":
        return gemm.grouped_gemm(s["a"], s["b"], s["ends"], s["c"])
    if op == "grouped_k":
        return gemm.grouped_gemm_k(s["a"], s["b"], s["ends"], s["c"])
    return gemm.gemm_lora(s["a"], s["b"], s["c"], s["down"], s["up"], s["ids"], s["workspace"],
                          ranks=s["ranks"], scales=s["scales"])


def _run_plain(s):
    op, c = s["case"]["op"], s["c"]
    if op == "grouped":
        out = torch.zeros(c.shape, dtype=c.dtype, device=c.device)
        start = 0
        for g, end in enumerate(s["ends_host"]):
            if end > start:
                out[start:end] = s["a"][start:end].float() @ s["b"][g].float().t()
            start = end
        return out
    if op == "grouped_k":
        out = torch.zeros(c.shape, dtype=c.dtype, device=c.device)
        start = 0
        for g, end in enumerate(s["ends_host"]):
            if end > start:
                out[g] = s["a"][:, start:end].float() @ s["b"][:, start:end].float().t()
            start = end
        return out
    x = s["a"].float()
    y = x @ s["b"].float().t()
    for i, rank, scale, rows in s["by_adapter"]:
        v = x[rows] @ s["down"][i, :rank].float().t()
        y[rows] += scale * (v @ s["up"][i, :, :rank].float().t())
    return y.to(c.dtype)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    tin, tout = TYPES[case["dtype"]]
    ei, eo = tin.itemsize, tout.itemsize
    M, N, K = case["M"], case["N"], case["K"]
    if case["op"] == "lora":
        ids, ranks = row_ids(case), adapter_ranks(case)
        b = (M * K + N * K) * ei + M * N * eo + 4 * M
        b += sum(ranks[i] * (K + N) * ei + 8 for i in set(ids) if i >= 0)
        f = 2 * M * N * K + sum(2 * ranks[i] * (K + N) for i in ids if i >= 0)
        return {"bytes": b, "flops": f}
    ends = group_ends(case)
    lens = [e - s for s, e in zip([0] + ends, ends)]
    rows = ends[-1]
    if case["op"] == "grouped":
        used = sum(1 for x in lens if x)
        return {"bytes": (rows * K + used * N * K) * ei + rows * N * eo + 4 * case["G"], "flops": 2 * rows * N * K}
    return {"bytes": rows * (M + N) * ei + case["G"] * M * N * eo + 4 * case["G"], "flops": 2 * rows * M * N}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    a, b = s["a"].double(), s["b"]
    c = s["c"]
    if case["op"] == "lora":
        # Row by row of adapters: every adapter's update of all rows, kept for its own.
        y = torch.mm(a, b.double().transpose(0, 1))
        ids = s["ids"].long()
        for i in range(case["L"]):
            mine = (ids == i).nonzero().flatten()
            if mine.numel() == 0:
                continue
            r = int(s["ranks"][i])
            delta = torch.mm(s["down"][i, :r].double(), a[mine].transpose(0, 1))         # r x rows
            delta = torch.mm(s["up"][i, :, :r].double(), delta).transpose(0, 1)           # rows x N
            y.index_add_(0, mine, delta * s["scales"][i].double())
        return y
    rows = case["M"] if case["op"] == "grouped" else case["K"]
    group = torch.bucketize(torch.arange(rows, device="cuda"), s["ends"].long(), right=True)   # G: past the last
    out = torch.zeros(c.shape, dtype=torch.float64, device="cuda")
    for g in range(case["G"]):
        mine = (group == g).nonzero().flatten()
        if mine.numel() == 0:
            continue
        if case["op"] == "grouped":
            out[mine] = torch.mm(b[g].double(), a[mine].transpose(0, 1)).transpose(0, 1)
        else:
            out[g] = torch.mm(b[:, mine].double(), a[:, mine].transpose(0, 1)).transpose(0, 1)
    return out
