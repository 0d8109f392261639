"""The product in 8-bit floating point and the tokens of experts, as they are measured.

``quantize_fp8`` (e4m3 codes with a scale for each block of 128), ``matmul_fp8`` (tokens
times a layer's weights, or times those of each token's experts), its input gradient
``matmul_fp8_grad``, ``sort_tokens`` and ``gather_tokens`` (tokens sorted by expert),
``combine_tokens`` (and back, weighted) and ``combine_tokens_grad``. ``run`` computes
them in plain torch operations, or with ``own`` through the package.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
FP8 = torch.float8_e4m3fn
BLOCK = 128


def listed():
    return [
        # one token's row to the 8 experts it was routed to, while a model generates: latency only
        dict(name="sort_1x8of64_2048_bf16", op="sort", T=1, k=8, E=64, n=2048, type="bf16", dropped=0.0),
        # the tokens of long prompts in the order of their experts, some of them padding
        dict(name="sort_8192x8of128_2048_bf16", op="sort", T=8192, k=8, E=128, n=2048, type="bf16", dropped=0.1),
        # the experts' results of long prompts, weighted, back at their tokens
        dict(name="combine_8192x8_2048_bf16", op="combine", T=8192, k=8, E=128, n=2048, type="bf16", dropped=0.1),
        # its gradient for a short padded batch of odd sizes, in the Grams' own type
        dict(name="combine_grad_777x6_1531_f32", op="combine_grad", T=777, k=6, E=60, n=1531, type="f32",
             dropped=0.25),
        # the inputs of an MLP's down projection for 8192 tokens
        dict(name="quantize_8192x14336_bf16", op="quantize", T=8192, n=14336, type="bf16", rows=1),
        # a layer's weights of odd sizes, once when a model is loaded
        dict(name="quantize_w_4003x11009_f32", op="quantize", T=4003, n=11009, type="f32", rows=BLOCK),
        # one token through a square attention projection: the codes' bytes and latency
        dict(name="product_1x4096x4096_bf16", op="product", T=1, m=4096, n=4096, type="bf16", padded=True),
        # 8192 tokens of prompts or of calibration through an MLP's gate projection
        dict(name="product_8192x14336x4096_bf16", op="product", T=8192, m=14336, n=4096, type="bf16", padded=True),
        # 32 generating sequences through their experts' first projection: the weights' bytes
        dict(name="experts_32x8of64_2048x4096_f16", op="experts", T=32, k=8, E=64, m=2048, n=4096, type="f16"),
        # prompts through their experts' first projection
        dict(name="experts_4096x8of64_2048x4096_bf16", op="experts", T=4096, k=8, E=64, m=2048, n=4096, type="bf16"),
        # output gradients of one ragged sequence through a layer of odd sizes, in the Grams' own type
        dict(name="product_grad_333x1000x1531_f32", op="product_grad", T=333, m=1000, n=1531, type="f32",
             padded=False),
        # output gradients of prompts through their experts' second projection
        dict(name="experts_grad_4096x4of32_4096x2048_bf16", op="experts_grad", T=4096, k=4, E=32, m=4096, n=2048,
             type="bf16"),
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]: a multiple of 128, of 16, or any."""
    x = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    k = rng.choice((1, 16, 128))
    return min(hi, max(lo, x // k * k))


def draw(rng):
    op = rng.choice(("sort", "combine", "combine_grad", "quantize", "quantize", "product", "product", "experts",
                     "experts", "product_grad", "experts_grad"))
    while True:
        c = dict(op=op, T=_size(rng, 1, 8192), type=rng.choice(("f32", "bf16", "f16")))
        if op in ("sort", "combine", "combine_grad"):
            c.update(E=_size(rng, 2, 256), n=_size(rng, 64, 8192), dropped=rng.choice((0.0, 0.1, 0.5)))
            c["k"] = rng.randint(1, min(8, c["E"]))
            if c["T"] * c["k"] * c["n"] * BYTES[c["type"]] <= 8192 * 8 * 2048 * 2:
                return c
        elif op == "quantize":
            c.update(n=_size(rng, 64, 14336), rows=rng.choice((1, 1, BLOCK)))
            return c
        elif op in ("product", "product_grad"):
            c.update(m=_size(rng, 64, 14336), n=_size(rng, 64, 14336), padded=rng.random() < 0.8)
            if c["T"] * c["m"] * c["n"] <= 4096 * 14336 * 4096:
                return c
        else:
            c.update(E=_size(rng, 2, 64), m=_size(rng, 64, 4096), n=_size(rng, 64, 4096))
            c["k"] = rng.randint(1, min(8, c["E"]))
            if c["E"] * c["m"] * c["n"] <= 64 * 2048 * 4096 and c["T"] * c["k"] * c["m"] * c["n"] <= 2 ** 37:
                return c


def _activations(T, n, g):
    """Gaussian activations whose channels differ in size, one in a hundred by 20."""
    c = torch.exp(0.5 * torch.randn(n, device=DEV, generator=g))
    c = torch.where(torch.rand(n, device=DEV, generator=g) < 0.01, 20 * c, c)
    return torch.randn(T, n, device=DEV, generator=g) * c


def _weights(batch, m, n, g):
    """Gaussian weights whose channels differ in size."""
    w = torch.randn(batch, m, n, device=DEV, generator=g)
    return w.mul_(0.02 * torch.exp(0.3 * torch.randn(batch, m, 1, device=DEV, generator=g)))


def _routes(case, g):
    """k experts of each token, int64, some more popular than others; -1 for a token that is dropped."""
    T, k, E = case["T"], case["k"], case["E"]
    score = torch.randn(T, E, device=DEV, generator=g) + 0.4 * torch.randn(E, device=DEV, generator=g)
    ids = score.topk(k, dim=1).indices
    out = torch.rand(T, device=DEV, generator=g).argsort() < int(T * case.get("dropped", 0.0))
    return torch.where(out[:, None], -1, ids)


def _rows(x, padded):
    """Codes in a zeroed buffer whose rows start at multiples of 128 bytes, as a
    program that keeps them lays them out once; or as they are."""
    if not padded:
        return x
    buf = torch.zeros(x.shape[:-1] + ((x.size(-1) + 127) // 128 * 128,), dtype=torch.uint8, device=x.device).view(FP8)
    buf.view(torch.uint8)[..., :x.size(-1)] = x.view(torch.uint8)
    return buf[..., :x.size(-1)]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, T, t, s = case["op"], case["T"], TYPES[case["type"]], dict(case)
    if "E" in case:
        s["ids"] = _routes(case, g)
        s["order"], s["slots"], s["offsets"] = _plain_sort(s["ids"], case["E"])
        s["R"] = int(s["offsets"][-1])  # the rows that have a token
        s["most"] = max(1, int((s["offsets"][1:] - s["offsets"][:-1]).max()))
    if op in ("combine", "combine_grad"):
        s["Ys"] = torch.randn(s["R"], case["n"], device=DEV, generator=g).to(t)
        s["w"] = torch.randn(T, case["k"], device=DEV, generator=g).softmax(1)
        s["G"] = (1e-3 * torch.randn(T, case["n"], device=DEV, generator=g)).to(t)
    elif op == "sort":
        s["X"] = _activations(T, case["n"], g).to(t)
    elif op == "quantize":
        s["X"] = (_activations(T, case["n"], g) if case["rows"] == 1 else _weights(1, T, case["n"], g)[0]).to(t)
    else:
        E, m, n = case.get("E"), case["m"], case["n"]
        q, sw = _plain_quantize(_weights(E or 1, m, n, g), BLOCK)
        q = _rows(q, case.get("padded", True))
        s["Wq"], s["sw"] = (q, sw) if E else (q[0], sw[0])
        if op in ("product", "experts"):
            q, sx = _plain_quantize(_activations(T, n, g), 1)
            s["sx"] = sx.t().contiguous().t()  # the tokens' scales of a block side by side, as quantize_fp8 has them
            s["Xq"] = _rows(q, case.get("padded", True))
            s["order"] = s["order"][:s["R"]] if E else None
        else:
            s["G"] = (1e-3 * torch.randn(s["R"] if E else T, m, device=DEV, generator=g)).to(t)
    return s


# ---- plain forms ------------------------------------------------------------
def _plain_sort(ids, E):
    flat = ids.reshape(-1)
    N = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    key, order = key.sort(stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=flat.device))
    at = torch.arange(N, device=flat.device)
    slots = torch.empty_like(order)
    slots[order] = torch.where(key < E, at, -1)
    order = torch.where(key < E, order, -1)
    return order.int(), slots.int().view(ids.shape), offsets.int()


def _plain_quantize(x, rows):
    """Codes and scales of blocks of rows x 128 of the last two dimensions."""
    x = x.float()
    a, n = x.shape[-2:]
    na, nb = -(-a // rows), -(-n // BLOCK)
    pad = torch.nn.functional.pad(x.abs(), (0, nb * BLOCK - n, 0, na * rows - a))
    top = pad.reshape(*x.shape[:-2], na, rows, nb, BLOCK).amax((-3, -1))
    del pad
    s = torch.where(top == 0, 1.0, (top / torch.full_like(top, 448.0)).clamp(min=2.0 ** -126))
    return (x / _spread(s, rows, a, n)).clamp_(-448, 448).to(FP8), s


def _spread(s, rows, a, n):
    """Each block's scale at all of its elements."""
    return s.repeat_interleave(rows, -2)[..., :a, :].repeat_interleave(BLOCK, -1)[..., :n]


def _values(q, s, rows):
    return q.float() * _spread(s, rows, q.size(-2), q.size(-1))


def _place(s):
    """Each sorted row's expert and its place among that expert's rows."""
    at = torch.arange(s["R"], device=DEV)
    e = torch.searchsorted(s["offsets"], at.int(), right=True) - 1
    return e, at - s["offsets"].long()[e]


def _plain(s):
    op, T = s["op"], s["T"]
    if op == "sort":
        order, slots, offsets = _plain_sort(s["ids"], s["E"])
        tok = order.long() // s["k"]
        return torch.where((order >= 0)[:, None], s["X"][tok.clamp(min=0)], 0), order, slots, offsets
    if op == "quantize":
        return _plain_quantize(s["X"], s["rows"])
    if op == "product":
        return (_values(s["Xq"], s["sx"], 1) @ _values(s["Wq"], s["sw"], BLOCK).t()).to(TYPES[s["type"]])
    if op == "product_grad":
        return (s["G"].float() @ _values(s["Wq"], s["sw"], BLOCK)).to(s["G"].dtype)
    if op == "experts":
        e, i = _place(s)
        X = torch.zeros(s["E"], s["most"], s["n"], device=DEV)
        X[e, i] = _values(s["Xq"], s["sx"], 1)[s["order"].long() // s["k"]]
        Y = torch.bmm(_values(s["Wq"], s["sw"], BLOCK), X.transpose(1, 2).contiguous())
        return Y.transpose(1, 2)[e, i].to(TYPES[s["type"]])
    if op == "experts_grad":
        e, i = _place(s)
        G = torch.zeros(s["E"], s["most"], s["m"], device=DEV)
        G[e, i] = s["G"].float()
        return torch.bmm(G, _values(s["Wq"], s["sw"], BLOCK))[e, i].to(s["G"].dtype)
    has, slot = s["slots"] >= 0, s["slots"].long().clamp(min=0)
    y = s["Ys"].float()[slot] * has[:, :, None]
    if op == "combine":
        return (y * s["w"][:, :, None]).sum(1).to(s["Ys"].dtype)
    G = s["G"].float()
    dw = (y * G[:, None]).sum(2)
    dYs = torch.empty(s["R"] + 1, s["n"], device=DEV)  # the last row for the dropped tokens
    dYs[torch.where(has, slot, s["R"])] = s["w"][:, :, None] * G[:, None]
    return dYs[:s["R"]].to(s["Ys"].dtype), dw


def run(state):
    if not own:
        return _plain(state)
    import kronecker_factored_gptq_amd as bk
    op, s = state["op"], state
    if op == "sort":
        order, slots, offsets = bk.sort_tokens(s["ids"], s["E"])
        return bk.gather_tokens(s["X"], order, s["k"]), order, slots, offsets
    if op == "combine":
        return bk.combine_tokens(s["Ys"], s["slots"], s["w"])
    if op == "combine_grad":
        return bk.combine_tokens_grad(s["G"], s["Ys"], s["slots"], s["w"])
    if op == "quantize":
        return bk.quantize_fp8(s["X"], block_rows=s["rows"])
    if op == "product":
        return bk.matmul_fp8(s["Xq"], s["sx"], s["Wq"], s["sw"], out_dtype=TYPES[s["type"]])
    if op == "experts":
        return bk.matmul_fp8(s["Xq"], s["sx"], s["Wq"], s["sw"], offsets=s["offsets"], order=s["order"],
                             per_token=s["k"], out_dtype=TYPES[s["type"]])
    if op == "product_grad":
        return bk.matmul_fp8_grad(s["G"], s["Wq"], s["sw"])
    return bk.matmul_fp8_grad(s["G"], s["Wq"], s["sw"], offsets=s["offsets"])


def work(case):
    op, T, e = case["op"], case["T"], BYTES[case["type"]]
    if op in ("sort", "combine", "combine_grad"):
        n, kept = case["n"], (1 - case["dropped"]) * T * case["k"]
        if op == "sort":  # every row of Xs is written, each token read once, 8 + 4 + 4 bytes of a route
            return dict(bytes=T * n * e + T * case["k"] * (n * e + 16) + 4 * case["E"] + 4, flops=T * case["k"])
        if op == "combine":
            return dict(bytes=(kept + T) * n * e + 8 * T * case["k"], flops=2 * kept * n)
        return dict(bytes=(2 * kept + T) * n * e + 12 * T * case["k"], flops=3 * kept * n)
    n = case["n"]
    nb = -(-n // BLOCK)
    if op == "quantize":
        return dict(bytes=T * n * (e + 1) + 4 * nb * -(-T // case["rows"]), flops=3 * T * n)
    m, k = case["m"], case.get("k", 1)
    layer = m * n + 4 * nb * -(-m // BLOCK)
    if "E" in case:
        layer *= min(case["E"], T * k)
    if op in ("product", "experts"):
        return dict(bytes=T * (n + 4 * nb) + layer + T * k * m * e, flops=2 * T * k * m * n)
    return dict(bytes=T * k * (m + n) * e + layer, flops=2 * T * k * m * n)


# ---- in 64 bits -------------------------------------------------------------
def _exact_values(q, s, rows):
    """q times its block's scale, block by block of columns."""
    out = q.float().double()
    for b in range(s.size(-1)):
        f = s[..., b].double().unsqueeze(-1)
        if rows > 1:
            f = f.repeat_interleave(rows, -2)[..., :q.size(-2), :]
        out[..., b * BLOCK:(b + 1) * BLOCK] *= f
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "sort":
        rows = [r for e in range(case["E"]) for r in (s["ids"] == e).nonzero()[:, 0].tolist()]
        out = torch.zeros(case["T"] * case["k"], case["n"], dtype=torch.float64, device=DEV)
        out[:len(rows)] = s["X"].double()[torch.tensor(rows, device=DEV)]
        return out, None, None, None  # whole numbers: none is rounded here
    if op == "quantize":
        x, r, n = s["X"].double(), case["rows"], case["n"]
        S = torch.empty(-(-x.size(0) // r), -(-n // BLOCK), dtype=torch.float64, device=DEV)
        for b in range(S.size(1)):
            cols = x[:, b * BLOCK:(b + 1) * BLOCK].abs().max(dim=1).values
            rows = torch.stack([p.max() for p in cols.split(r)]) if r > 1 else cols
            S[:, b] = torch.where(rows > 0, rows / 448, 1.0)
        for b in range(S.size(1)):
            f = S[:, b].repeat_interleave(r)[:x.size(0)] if r > 1 else S[:, b]
            x[:, b * BLOCK:(b + 1) * BLOCK] /= f[:, None]
        return x, S
    if op in ("product", "product_grad"):
        W = _exact_values(s["Wq"], s["sw"], BLOCK)
        return torch.mm(_exact_values(s["Xq"], s["sx"], 1), W.t()) if op == "product" else torch.mm(s["G"].double(), W)
    if op in ("experts", "experts_grad"):
        off = s["offsets"].tolist()
        X = _exact_values(s["Xq"], s["sx"], 1)[s["order"].long() // case["k"]] if op == "experts" else s["G"].double()
        out = torch.empty(s["R"], case["m"] if op == "experts" else case["n"], dtype=torch.float64, device=DEV)
        for e in range(case["E"]):
            if off[e] < off[e + 1]:
                W = _exact_values(s["Wq"][e], s["sw"][e], BLOCK)
                out[off[e]:off[e + 1]] = torch.mm(X[off[e]:off[e + 1]], W.t() if op == "experts" else W)
        return out
    Y, w, G, slots = s["Ys"].double(), s["w"].double(), s["G"].double(), s["slots"].long()
    if op == "combine":
        out = torch.zeros(case["T"], case["n"], dtype=torch.float64, device=DEV)
        for j in range(case["k"]):
            t = (slots[:, j] >= 0).nonzero().squeeze(1)
            out[t] += w[t, j, None] * Y[slots[t, j]]
        return out
    dY, dw = torch.zeros_like(Y), torch.zeros_like(w)
    for j in range(case["k"]):
        t = (slots[:, j] >= 0).nonzero().squeeze(1)
        dY[slots[t, j]] = w[t, j, None] * G[t]
        dw[t, j] = (G[t] * Y[slots[t, j]]).sum(1)
    return dY, dw
