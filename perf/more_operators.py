"""The 8-bit linear layer: cases, inputs, plain forms, exact values.

A linear layer's tokens and weights are held as 8-bit integers with one fp32
scale a row (a token of the activations, an output channel of the weights):

  checkpoint  tokens to 8 bits and back: each row's largest magnitude stands for
              127,
                  scale_m = max_k |x[m][k]| / 127,   q[m][k] = round(127 x[m][k] / max_k |x[m][k]|)
              (ties to even), and the values they stand for, q[m][k] * scale_m,
              in the type of x: what a training step keeps of an activation and
              reads back in its backward pass.
  i8          the layer's output from the integers,
                  C[m][n] = act(scale_a[m] scale_b[n] sum_k A[m][k] B[n][k] + bias[n])
  grad        its gradients from 8-bit checkpoints, whose scales lie along the
              summed index,
                  C[m][n] = sum_k A[m][k] scales[k] Q[n][k]
              The weights' gradient sums over tokens: A the gradient of the
              outputs, Q the layer's inputs, both read token by token (A
              m-major).  The inputs' gradient sums over output channels: A the
              same gradient, k-major, Q the weights.

With `own` false, run() computes them in elementary torch operations in fp32
(the rounding to integers, a value next to a border, in fp64), rounded once at
the end; with `own` true it calls this repository's package.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # One token of a decoding step: latency.
        dict(name="checkpoint_1x4096_bf16", op="checkpoint", M=1, K=4096, dtype="bf16"),
        # The activations of a training batch.
        dict(name="checkpoint_8192x4096_bf16", op="checkpoint", M=8192, K=4096, dtype="bf16"),
        # Single precision at odd sizes: rows that start at any byte.
        dict(name="checkpoint_4095x2049_f32", op="checkpoint", M=4095, K=2049, dtype="f32"),
        # One token's projection: the weights are the traffic.
        dict(name="i8_decode_1x4096x4096_bf16", op="i8", M=1, N=4096, K=4096, dtype="bf16", bias=False, act="none"),
        # A decoding batch through the first layer of a feed-forward block.
        dict(name="i8_decode_64x8192x2048_f16", op="i8", M=64, N=8192, K=2048, dtype="f16", bias=True, act="gelu"),
        # A prompt.
        dict(name="i8_prompt_1000x1024x2048_bf16", op="i8", M=1000, N=1024, K=2048, dtype="bf16", bias=True, act="relu"),
        # A prefill or training batch: the largest.
        dict(name="i8_fwd_8192x4096x4096_bf16", op="i8", M=8192, N=4096, K=4096, dtype="bf16", bias=False, act="none"),
        # Odd sizes, single-precision outputs; rows of 1028 bytes.
        dict(name="i8_ragged_4095x2049x1028_f32", op="i8", M=4095, N=2049, K=1028, dtype="f32", bias=True, act="none"),
        # The weights' gradient of the training batch, into fp32 gradients.
        dict(name="grad_weights_4096x4096_t8192_bf16_f32", op="grad", M=4096, N=4096, K=8192, a_major="m", dtype="bf16",
             out="f32"),
        # The inputs' gradient of the same layer.
        dict(name="grad_inputs_8192x4096x4096_bf16", op="grad", M=8192, N=4096, K=4096, a_major="k", dtype="bf16",
             out="bf16"),
        # The weights' gradient of a small layer and a short batch.
        dict(name="grad_weights_512x256_t1000_f16", op="grad", M=512, N=256, K=1000, a_major="m", dtype="f16", out="f16"),
        # Single precision at odd sizes.
        dict(name="grad_weights_2049x1028_t4095_f32", op="grad", M=2049, N=1028, K=4095, a_major="m", dtype="f32",
             out="f32"),
    ]


def _size(rng, lo, hi, step=1):
    """A size spread over the logarithm of [lo, hi], a multiple of `step`."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(step, v // step * step)


def draw(rng):
    op = rng.choice(["checkpoint", "i8", "i8", "grad", "grad"])
    # Widths are mostly multiples of 16 (one load of 8-bit values), some are odd.
    step = rng.choice([16, 16, 64, 64, 8, 1])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    N, K = _size(rng, 128, 8192, step), _size(rng, 128, 8192, step)
    if op == "checkpoint":
        # No more bytes than the listed batch.
        return dict(op=op, M=_size(rng, 1, min(32768, (1 << 26) // (K * TYPES[dtype].itemsize))), K=K, dtype=dtype)
    # Tokens: no more products than the largest listed case, outputs of at most 2^26.
    M = _size(rng, 1, min(32768, (1 << 37) // (N * K), (1 << 26) // max(N, K)))
    if op == "i8":
        return dict(op=op, M=M, N=N, K=K, dtype=dtype, bias=rng.choice([False, True]),
                    act=rng.choice(["none", "none", "relu", "gelu"]))
    out = rng.choice([dtype, "f32"])
    if rng.random() < 0.5:
        return dict(op=op, M=N, N=K, K=M, a_major="m", dtype=dtype, out=out)
    return dict(op=op, M=M, N=N, K=K, a_major="k", dtype=dtype, out=out)


# ---------------------------------------------------------------- inputs

def _normal(shape, std, g):
    return torch.randn(shape, generator=g, device="cuda") * std


def _tokens(rows, width, g):
    """Activations in fp32: tokens of different size, a few wide channels, and
    padding tokens of zeros in longer batches."""
    x = _normal((rows, width), 1.0, g) * torch.exp(0.5 * _normal((rows, 1), 1.0, g))
    x[:, torch.randint(0, width, (max(1, width // 512),), generator=g, device="cuda")] *= 8.0
    if rows > 64:
        x[torch.randint(0, rows, (rows // 64,), generator=g, device="cuda")] = 0.0
    return x


def _to8(x):
    """Rows as a user holds them: 8-bit integers and a scale each."""
    s = x.abs().amax(1) / 127.0
    return torch.round(x / torch.where(s > 0, s, 1.0)[:, None]).to(torch.int8), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    M, K, t = case["M"], case["K"], TYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "checkpoint":
        s["x"] = _tokens(M, K, g).to(t)
        s["q"] = torch.zeros((M, K), dtype=torch.int8, device="cuda")
        s["scales"] = torch.zeros(M, device="cuda")
        s["restored"] = torch.zeros((M, K), dtype=t, device="cuda")
        return s
    N = case["N"]
    if case["op"] == "i8":
        s["a"], s["scale_a"] = _to8(_tokens(M, K, g))
        s["b"], s["scale_b"] = _to8(_normal((N, K), K ** -0.5, g))
        s["bias"] = _normal((N,), 0.1, g) if case["bias"] else None
        s["c"] = torch.zeros((M, N), dtype=t, device="cuda")
        return s
    if case["a_major"] == "m":          # K tokens: gradients of the outputs and the layer's inputs
        s["a"] = _normal((K, M), 0.02, g).to(t).t()
        q, s["scales"] = _to8(_tokens(K, N, g))
    else:                               # K output channels of the weights
        s["a"] = _normal((M, K), 0.02, g).to(t)
        q, s["scales"] = _to8(_normal((K, N), N ** -0.5, g))
    s["q"] = q.t()
    s["c"] = torch.zeros((M, N), dtype=TYPES[case["out"]], device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import dense_gemm_engineering_run_amd as gemm
    case = s["case"]
    if case["op"] == "checkpoint":
        gemm.quantize_rows(s["x"], s["q"], s["scales"])
        return gemm.dequantize_rows(s["q"], s["scales"], s["restored"]), s["scales"]
    if case["op"] == "i8":
        return gemm.gemm_i8(s["a"], s["b"], s["scale_a"], s["scale_b"], s["c"], bias=s["bias"],
                            activation=getattr(gemm, "GEMM_ACT_" + case["act"].upper()))
    return gemm.gemm_i8_grad(s["a"], s["q"], s["scales"], s["c"])


def _run_plain(s):
    case = s["case"]
    if case["op"] == "checkpoint":
        x = s["x"].double()
        top = x.abs().amax(1, keepdim=True)
        q = torch.round(127.0 * x / torch.where(top > 0, top, 1.0)).float()
        scales = (top / 127.0).float()
        return (q * scales).to(s["x"].dtype), scales[:, 0]
    if case["op"] == "i8":
        y = s["a"].float() @ s["b"].float().t()
        y = y * s["scale_a"][:, None] * s["scale_b"][None, :]
        if s["bias"] is not None:
            y = y + s["bias"]
        if case["act"] == "relu":
            y = torch.where(y < 0, 0.0, y)
        elif case["act"] == "gelu":
            y = 0.5 * y * (1.0 + torch.erf(y * 0.5 ** 0.5))
        return y.to(s["c"].dtype)
    values = s["q"].float() * s["scales"]
    return (s["a"].float() @ values.t()).to(s["c"].dtype)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    M, K, e = case["M"], case["K"], TYPES[case["dtype"]].itemsize
    if case["op"] == "checkpoint":
        # x read, q written and read, the restored values written, the scales.
        return {"bytes": M * K * (2 * e + 2) + 4 * M, "flops": 4 * M * K}
    N = case["N"]
    if case["op"] == "i8":
        return {"bytes": (M + N) * (K + 4) + M * N * e + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    return {"bytes": M * K * e + N * K + 4 * K + M * N * TYPES[case["out"]].itemsize, "flops": 2 * M * N * K}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "checkpoint":
        x = s["x"].double()
        step = x.abs().max(dim=1).values / 127
        # |x| in units of the step, half of it added, rounded down; an exact half to the even one.
        n = (x.abs() * 127) / x.abs().max(dim=1).values.clamp(min=1e-300)[:, None]
        low = n.floor()
        odd = low - 2 * (low / 2).floor()
        up = (n - low > 0.5) | ((n - low == 0.5) & (odd == 1))
        return (low + up) * x.sign() * step[:, None], step
    if case["op"] == "i8":
        y = torch.mm(s["b"].double() * s["scale_b"].double()[:, None], s["a"].double().transpose(0, 1)).transpose(0, 1)
        y = y * s["scale_a"].double()[:, None]
        if s["bias"] is not None:
            y = y + s["bias"].double()
        if case["act"] == "relu":
            y = y.clamp(min=0)
        elif case["act"] == "gelu":
            y = y / 2 * torch.special.erfc(-y / math.sqrt(2.0))
        return y
    scaled = s["a"].double() * s["scales"].double()
    return torch.mm(s["q"].double(), scaled.transpose(0, 1)).transpose(0, 1)
