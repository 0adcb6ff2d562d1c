"""The operators of a dense gated feed-forward layer, in 8-bit integers for
serving and in 16 bits with gradients for training, as cases that can be timed
and compared.

Five operators, by the case's ``op``:

``quantize``   activations or weights to 8-bit integers with one scale a row
``dense``      C = A . B^T over 8-bit integers, a scale for each token (row of
               A) and each channel (row of B)
``gated_int8`` h = silu(g) * u with (g, u) the halves of the columns of such a
               product, W's rows: the gate's, then the up projection's
``gated``      the same over bf16 or fp16 operands
``train``      a training step's part of it: forward, and from the gradient of
               h those of x and W

``own`` selects what ``run`` computes: the plain formulas in elementary torch
operations (False), or the package's operators (True).
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # between the two products of a layer, sixty-four sequences in decode
        dict(name="quantize_decode", op="quantize", M=64, K=14336, x="bf16"),
        # the input of a linear layer in prefill
        dict(name="quantize_prefill", op="quantize", M=8192, K=8192, x="bf16"),
        # one sequence through an attention-out layer: one pass over the weights
        dict(name="dense_decode", op="dense", M=1, N=8192, K=8192, out="bf16"),
        # an odd batch through a fused QKV layer, K that ends inside a step
        dict(name="dense_ragged", op="dense", M=777, N=10240, K=4104, out="f32"),
        # a prefill chunk through a fused QKV layer
        dict(name="dense_prefill", op="dense", M=8192, N=10240, K=8192, out="bf16"),
        # sixteen sequences in decode
        dict(name="gated_int8_decode", op="gated_int8", M=16, F=14336, K=4096, out="bf16"),
        # a prefill chunk
        dict(name="gated_int8_prefill", op="gated_int8", M=8192, F=14336, K=4096, out="bf16"),
        # one sequence in decode
        dict(name="gated_decode", op="gated", M=1, F=14336, K=4096, type="bf16"),
        # an odd batch, odd widths
        dict(name="gated_ragged", op="gated", M=777, F=5001, K=2055, type="f16"),
        # a prefill chunk
        dict(name="gated_prefill", op="gated", M=4096, F=14336, K=4096, type="bf16"),
        # a small model's layer, a short and odd batch of tokens
        dict(name="train_small", op="train", M=1000, F=1365, K=520, type="f16"),
        # a large model's layer, a long sequence
        dict(name="train_large", op="train", M=8192, F=14336, K=4096, type="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "dense", "dense", "gated_int8", "gated", "train", "train"])
    if op == "quantize":
        return dict(op=op, M=_log(rng, 1, 8192), K=_log(rng, 64, 14336),
                    x=rng.choice(["bf16", "f16", "f32"]))
    if op == "dense":
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 256, 10240), K=_log(rng, 128, 8192),
                    out=rng.choice(["bf16", "f16", "f32"]))
    if op == "gated_int8":
        return dict(op=op, M=_log(rng, 1, 8192), F=_log(rng, 256, 14336), K=_log(rng, 128, 4096),
                    out=rng.choice(["bf16", "f16"]))
    return dict(op=op, M=_log(rng, 1, 4096 if op == "gated" else 8192), F=_log(rng, 256, 14336),
                K=_log(rng, 128, 4096), type=rng.choice(["bf16", "f16"]))


def _rows(shape, dtype, unit):
    """An empty tensor whose rows are padded to `unit` elements, as the
    products ask for."""
    *lead, K = shape
    return torch.empty((*lead, -(-K // unit) * unit), device="cuda", dtype=dtype)[..., :K]


def _normal(g, shape, dtype, sigma):
    t = _rows(shape, dtype, 8)
    t.copy_(torch.randn(shape, device="cuda", generator=g).mul_(sigma))
    return t


def _codes(g, shape):
    """8-bit integers as a quantiser leaves normal values: a row's largest is
    about four deviations."""
    t = _rows(shape, torch.int8, 16)
    v = torch.randn(shape, device="cuda", generator=g).mul_(32)
    t.copy_(v.round_().clamp_(-127, 127))
    return t


def _scales(g, n, centre):
    return centre * torch.exp(0.5 * torch.randn(n, device="cuda", generator=g))


def prepare(case, seed):
    g, op = torch.Generator(device="cuda").manual_seed(seed), case["op"]
    s, M, K = dict(case), case["M"], case["K"]
    if op == "quantize":
        x = torch.randn((M, K), device="cuda", generator=g)
        x *= torch.exp(0.7 * torch.randn((1, K), device="cuda", generator=g))  # outlier channels
        s["in"] = x.to(TYPES[case["x"]])
        return s
    if op in ("dense", "gated_int8"):
        N = case["N"] if op == "dense" else 2 * case["F"]
        s["A"], s["B"] = _codes(g, (M, K)), _codes(g, (N, K))
        s["SA"] = _scales(g, M, 1 / 32)
        s["SB"] = _scales(g, N, 1 / (32 * math.sqrt(K)))
        return s
    dtype = TYPES[case["type"]]
    s["A"] = _normal(g, (M, K), dtype, 1.0)
    s["B"] = _normal(g, (2 * case["F"], K), dtype, 1 / math.sqrt(K))
    if op == "train":
        s["dh"] = _normal(g, (M, case["F"]), dtype, 0.1)
    return s


# ------------------------------------------------------------------ the plain forms

def _quantize(s):
    x = s["in"].float()
    most = x.abs().amax(1, keepdim=True).clamp_(min=2.0 ** -100)
    return (x * (127.0 / most)).round_().to(torch.int8), (most / 127.0)[:, 0]


def _integer_product(A, B):
    """Exact sums of products of 8-bit integers: 1024 of them stay below 2^24,
    where fp32 is exact; the parts' sums are 32-bit integers."""
    total = 0
    for k in range(0, A.shape[1], 1024):
        total = total + (A[:, k:k + 1024].float() @ B[:, k:k + 1024].float().t()).int()
    return total


def _dense(s):
    sums = _integer_product(s["A"], s["B"]).float()
    return (sums * s["SA"][:, None] * s["SB"][None, :]).to(TYPES[s["out"]])


def _gated_int8(s):
    F = s["F"]
    sums = _integer_product(s["A"], s["B"]).float() * s["SA"][:, None] * s["SB"][None, :]
    g, u = sums[:, :F], sums[:, F:]
    return (g / (1 + torch.exp(-g)) * u).to(TYPES[s["out"]])


def _gated(s):
    F, x, W = s["F"], s["A"].float(), s["B"].float()
    g, u = x @ W[:F].t(), x @ W[F:].t()
    return (g / (1 + torch.exp(-g)) * u).to(s["A"].dtype)


def _train(s):
    F, t, x, W, dh = s["F"], s["A"].dtype, s["A"].float(), s["B"].float(), s["dh"].float()
    g, u = x @ W[:F].t(), x @ W[F:].t()
    sig = 1 / (1 + torch.exp(-g))
    silu = g * sig
    dg = dh * u * (sig + silu * (1 - sig))
    du = dh * silu
    dx = dg @ W[:F] + du @ W[F:]
    dW = torch.cat([dg.t() @ x, du.t() @ x])
    return (silu * u).to(t), dx.to(t), dW.to(t)


PLAIN = dict(quantize=_quantize, dense=_dense, gated_int8=_gated_int8, gated=_gated, train=_train)


def run(state):
    s = state
    if not own:
        return PLAIN[s["op"]](s)
    import dense_gemm_bf16_amd as g
    if s["op"] == "quantize":
        return g.quantize_int8(s["in"])
    if s["op"] == "dense":
        return g.matmul_int8(s["A"], s["SA"], s["B"], s["SB"], out_dtype=TYPES[s["out"]])
    if s["op"] == "gated_int8":
        return g.gated_matmul_int8(s["A"], s["SA"], s["B"], s["SB"], out_dtype=TYPES[s["out"]])
    if s["op"] == "gated":
        return g.gated_matmul(s["A"], s["B"])
    h, gu = g.gated_matmul(s["A"], s["B"], save=True)
    return (h, *g.gated_matmul_backward(s["dh"], s["A"], s["B"], gu))


def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if op == "quantize":
        return {"bytes": M * K * (size[case["x"]] + 1) + 4 * M, "flops": 3 * M * K}
    if op == "dense":
        N = case["N"]
        return {"bytes": M * K + N * K + 4 * (M + N) + M * N * size[case["out"]],
                "flops": 2 * M * N * K}
    F = case["F"]
    if op == "gated_int8":
        return {"bytes": M * K + 2 * F * K + 4 * (M + 2 * F) + M * F * size[case["out"]],
                "flops": 4 * M * F * K}
    if op == "gated":
        return {"bytes": 2 * (M * K + 2 * F * K + M * F), "flops": 4 * M * F * K}
    # x, W and dh in; h, dx and dW out; three products of 2 F columns
    return {"bytes": 2 * (2 * M * K + 4 * F * K + 2 * M * F), "flops": 12 * M * F * K}


# ------------------------------------------------------------------ in 64 bits, from the definitions

def _exact_quantize(s):
    """The codes are defined by fp32 roundings: of 127 / amax and of its
    product with x, each of which 64 bits hold before it is rounded."""
    x = s["in"].double()
    most = torch.maximum(x.max(1).values, -x.min(1).values).clamp(min=2.0 ** -100)
    factor = (127 / most).float().double()
    q = torch.round((x * factor[:, None]).float().double())
    return q.to(torch.int8), most / 127


def _exact_sums(s):
    A = s["A"].double() * s["SA"].double().unsqueeze(1)
    B = s["B"].double() * s["SB"].double().unsqueeze(1)
    return torch.mm(A, B.t())


def _exact_gate(gu, F):
    return gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]


def _exact_train(s):
    F = s["F"]
    x, W, dh = (s[n].double() for n in ("A", "B", "dh"))
    gu = torch.mm(x, W.t())
    h = _exact_gate(gu, F)
    sig = torch.sigmoid(gu[:, :F])
    d = torch.empty_like(gu)
    d[:, :F] = dh * gu[:, F:] * sig * (1 + gu[:, :F] * (1 - sig))
    d[:, F:] = dh * gu[:, :F] * sig
    return h, torch.mm(d, W), torch.mm(d.t(), x)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quantize":
        return _exact_quantize(s)
    if op == "dense":
        return _exact_sums(s)
    if op == "gated_int8":
        return _exact_gate(_exact_sums(s), s["F"])
    if op == "gated":
        return _exact_gate(torch.mm(s["A"].double(), s["B"].double().t()), s["F"])
    return _exact_train(s)
