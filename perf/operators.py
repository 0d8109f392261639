"""The 8-bit product and the cross entropy, as they are measured.

Five operators: ``quantize_tokens`` (per-token int8 activations), ``matmul_int8``
(int8 tokens times int8 codes, scaled per token and channel), its input
gradient ``matmul_int8_grad``, and ``cross_entropy`` over a large vocabulary with
``cross_entropy_grad``. ``run`` computes them in plain torch operations, or with
``own`` through the package.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # one token of a 4096-wide layer while a model generates: latency only
        dict(name="quantize_1x4096_bf16", op="quantize", T=1, n=4096, type="bf16", channel=False),
        # the inputs of an MLP's down projection for 8192 calibration tokens,
        # with a layer's column scales folded in
        dict(name="quantize_8192x14336_f32", op="quantize", T=8192, n=14336, type="f32", channel=True),
        # one token through a square attention projection: the codes' bytes and latency
        dict(name="product_1x4096x4096_bf16", op="product", T=1, m=4096, n=4096, out="bf16", packed=True),
        # a batch of 37 generating sequences through an MLP's gate projection
        dict(name="product_37x14336x4096_f16", op="product", T=37, m=14336, n=4096, out="f16", packed=True),
        # a ragged prompt through a layer of odd sizes, rows neither padded nor aligned
        dict(name="product_777x1003x1531_f32", op="product", T=777, m=1003, n=1531, out="f32", packed=False),
        # 8192 tokens of prompts or of calibration through an MLP's gate projection
        dict(name="product_8192x14336x4096_bf16", op="product", T=8192, m=14336, n=4096, out="bf16", packed=True),
        # output gradients of one sequence through a small k/v projection, in the Grams' own type
        dict(name="product_grad_512x1024x2048_f32", op="product_grad", T=512, m=1024, n=2048, type="f32",
             channel=False),
        # output gradients of 8192 calibration tokens through an MLP's down projection
        dict(name="product_grad_8192x4096x14336_bf16", op="product_grad", T=8192, m=4096, n=14336, type="bf16",
             channel=False),
        # the surprise at one token, an odd vocabulary
        dict(name="entropy_1x2048x50257_f16", op="entropy", T=1, d=2048, V=50257, type="f16", masked=0.0),
        # the loss of 4096 tokens over a large vocabulary
        dict(name="entropy_4096x4096x128256_bf16", op="entropy", T=4096, d=4096, V=128256, type="bf16", masked=0.1),
        # gradients for a short padded batch of a small model, ragged, in the Grams' own type
        dict(name="entropy_grad_333x1000x10007_f32", op="entropy_grad", T=333, d=1000, V=10007, type="f32",
             masked=0.25),
        # gradients for 4096 tokens over a large vocabulary
        dict(name="entropy_grad_4096x4096x128256_bf16", op="entropy_grad", T=4096, d=4096, V=128256, type="bf16",
             masked=0.1),
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]: a multiple of 64, of 8, or any."""
    x = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    k = rng.choice((1, 8, 64))
    return min(hi, max(lo, x // k * k))


def draw(rng):
    op = rng.choice(("quantize", "product", "product", "product_grad", "entropy", "entropy_grad"))
    while True:
        if op == "quantize":
            c = dict(op=op, T=_size(rng, 1, 8192), n=_size(rng, 64, 14336), type=rng.choice(("f32", "bf16", "f16")),
                     channel=rng.random() < 0.3)
        elif op == "product":
            c = dict(op=op, T=_size(rng, 1, 8192), m=_size(rng, 64, 14336), n=_size(rng, 64, 14336),
                     out=rng.choice(("f32", "bf16", "f16")), packed=rng.random() < 0.8)
        elif op == "product_grad":
            c = dict(op=op, T=_size(rng, 1, 8192), m=_size(rng, 64, 14336), n=_size(rng, 64, 14336),
                     type=rng.choice(("f32", "bf16", "f16")), channel=rng.random() < 0.3)
        else:
            c = dict(op=op, T=_size(rng, 1, 4096), d=_size(rng, 64, 4096), V=_size(rng, 1000, 128256),
                     type=rng.choice(("f32", "bf16", "f16")), masked=rng.choice((0.0, 0.1, 0.5)))
        if op not in ("product", "product_grad") or c["T"] * c["m"] * c["n"] <= 8192 * 14336 * 4096:
            return c


def _rows(x, packed):
    """``x`` (int8) in a zeroed buffer whose rows start at multiples of 128 bytes,
    as a program that keeps it lays it out once; or as it is."""
    if not packed:
        return x
    buf = torch.zeros(x.size(0), (x.size(1) + 127) // 128 * 128, dtype=torch.int8, device=x.device)
    buf[:, :x.size(1)] = x
    return buf[:, :x.size(1)]


def _codes(m, n, g):
    """4-bit codes and row scales of a Gaussian weight matrix (absmax / 7)."""
    W = 0.02 * torch.randn(m, n, device=DEV, generator=g)
    s = W.abs().amax(1) / 7.0
    return (W / s[:, None]).round().clamp(-8, 7).to(torch.int8), s


def _activations(T, n, g):
    """Gaussian activations whose channels differ in size, one in a hundred by 20."""
    c = torch.exp(0.5 * torch.randn(n, device=DEV, generator=g))
    c = torch.where(torch.rand(n, device=DEV, generator=g) < 0.01, 20 * c, c)
    return torch.randn(T, n, device=DEV, generator=g) * c


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, s = case["op"], dict(case)
    if op == "quantize":
        s["X"] = _activations(case["T"], case["n"], g).to(TYPES[case["type"]])
        s["c"] = torch.exp(0.3 * torch.randn(case["n"], device=DEV, generator=g)) if case["channel"] else None
    elif op == "product":
        X = _activations(case["T"], case["n"], g)
        s["sx"] = X.abs().amax(1) / 127.0
        s["Xq"] = _rows((X / s["sx"][:, None]).round().clamp(-127, 127).to(torch.int8), case["packed"])
        Vq, s["sv"] = _codes(case["m"], case["n"], g)
        s["Vq"] = _rows(Vq, case["packed"])
    elif op == "product_grad":
        s["Vq"], s["sv"] = _codes(case["m"], case["n"], g)
        s["G"] = (1e-3 * torch.randn(case["T"], case["m"], device=DEV, generator=g)).to(TYPES[case["type"]])
        s["c"] = torch.exp(0.3 * torch.randn(case["n"], device=DEV, generator=g)) if case["channel"] else None
    else:
        T, d, V, t = case["T"], case["d"], case["V"], TYPES[case["type"]]
        # hidden states of unit size, and an output layer whose logits spread by about 2
        s["X"] = torch.randn(T, d, device=DEV, generator=g).to(t)
        W = torch.empty(V, d, device=DEV, dtype=t)
        for a in range(0, V, 32768):
            W[a:a + 32768] = torch.randn(min(32768, V - a), d, device=DEV, generator=g) * (2.0 / math.sqrt(d))
        s["W"] = W
        y = torch.randint(0, V, (T,), device=DEV, generator=g)
        s["y"] = torch.where(torch.rand(T, device=DEV, generator=g) < case["masked"], -100, y)
        if op == "entropy_grad":  # the mean over the rows that have a target, and the forward pass's lse
            n = (s["y"] >= 0).sum().clamp(min=1).float()
            s["g"] = torch.where(s["y"] >= 0, 1.0 / n, 0.0).float()
            s["lse"] = _plain_entropy(s)[1]
    return s


def _plain_entropy(s):
    z = s["X"].float() @ s["W"].float().t()
    top = z.amax(1, keepdim=True)
    lse = (top + (z - top).exp().sum(1, keepdim=True).log()).squeeze(1)
    has = (s["y"] >= 0) & (s["y"] < z.size(1))
    zy = z.gather(1, torch.where(has, s["y"], 0)[:, None]).squeeze(1)
    return torch.where(has, lse - zy, 0.0), lse


def _plain(s):
    op = s["op"]
    if op == "quantize":
        x = s["X"].float()
        if s["c"] is not None:
            x = x * s["c"]
        a = x.abs().amax(1)
        sx = torch.where(a == 0, torch.ones_like(a), a / torch.full_like(a, 127.0))
        return (x / sx[:, None]).round().clamp(-127, 127).to(torch.int8), sx
    if op == "product":
        y = s["Xq"].float() @ s["Vq"].float().t()
        return (y * s["sx"][:, None] * s["sv"]).to(TYPES[s["out"]])
    if op == "product_grad":
        y = (s["G"].float() * s["sv"]) @ s["Vq"].float()
        return (y if s["c"] is None else y * s["c"]).to(s["G"].dtype)
    if op == "entropy":
        return _plain_entropy(s)
    W, X, V = s["W"].float(), s["X"].float(), s["V"]
    has = (s["y"] >= 0) & (s["y"] < V)
    p = (X @ W.t()).sub_(s["lse"][:, None]).exp_()
    p.scatter_add_(1, torch.where(has, s["y"], 0)[:, None], torch.full_like(p[:, :1], -1.0))
    p.mul_(torch.where(has, s["g"], 0.0)[:, None])
    return (p @ W).to(s["W"].dtype), (p.t() @ X).to(s["W"].dtype)


def run(state):
    if not own:
        return _plain(state)
    import kronecker_factored_gptq_amd as bk
    op, s = state["op"], state
    if op == "quantize":
        return bk.quantize_tokens(s["X"], s["c"])
    if op == "product":
        return bk.matmul_int8(s["Xq"], s["sx"], s["Vq"], s["sv"], out_dtype=TYPES[s["out"]])
    if op == "product_grad":
        return bk.matmul_int8_grad(s["G"], s["Vq"], s["sv"], s["c"])
    if op == "entropy":
        return bk.cross_entropy(s["X"], s["W"], s["y"])
    return bk.cross_entropy_grad(s["X"], s["W"], s["y"], s["lse"], s["g"])


def work(case):
    op, T = case["op"], case["T"]
    if op == "quantize":
        n = case["n"]
        return dict(bytes=T * n * (BYTES[case["type"]] + 1) + 4 * T + 4 * n * case["channel"], flops=3 * T * n)
    if op == "product":
        m, n = case["m"], case["n"]
        return dict(bytes=T * n + m * n + 4 * (T + m) + T * m * BYTES[case["out"]], flops=2 * T * m * n)
    if op == "product_grad":
        m, n = case["m"], case["n"]
        return dict(bytes=T * (m + n) * BYTES[case["type"]] + m * n + 4 * m + 4 * n * case["channel"],
                    flops=2 * T * m * n)
    d, V, e = case["d"], case["V"], BYTES[case["type"]]
    if op == "entropy":
        return dict(bytes=(T + V) * d * e + 16 * T, flops=2 * T * V * d)
    return dict(bytes=2 * (T + V) * d * e + 16 * T, flops=6 * T * V * d)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["X"].double()
        if s["c"] is not None:
            x = (x * s["c"].double())
        a = x.abs().max(dim=1).values
        return None, torch.where(a > 0, a / 127, 1.0)  # whole codes: none is rounded here
    if op == "product":
        out = torch.mm(s["Xq"].double(), s["Vq"].double().t())
        return out.mul_(s["sv"].double()).mul_(s["sx"].double()[:, None])
    if op == "product_grad":
        W = s["Vq"].double() * s["sv"].double()[:, None]
        out = torch.mm(s["G"].double(), W)
        return out if s["c"] is None else out * s["c"].double()
    X, W, T, V = s["X"].double(), s["W"].double(), case["T"], case["V"]
    z = torch.mm(X, W.t())
    rows = (s["y"] >= 0).nonzero().squeeze(1)
    if op == "entropy":
        lse = torch.logsumexp(z, 1)
        loss = torch.zeros(T, dtype=torch.float64, device=DEV)
        loss[rows] = lse[rows] - z[rows, s["y"][rows]]
        return loss, lse
    p = torch.exp(z - s["lse"].double()[:, None])  # the lse that the call is given
    del z
    p[rows, s["y"][rows]] -= 1
    w = torch.zeros(T, dtype=torch.float64, device=DEV)
    w[rows] = s["g"].double()[rows]
    p *= w[:, None]
    return torch.mm(p, W), torch.mm(p.t(), X)
